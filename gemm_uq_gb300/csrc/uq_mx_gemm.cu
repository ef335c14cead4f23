// uq_mx_gemm.cu -- product of two microscaled 4-bit operands on the block-scaled tensor instructions (tcgen05,
// kind::mxf4 / kind::mxf4nvf4), dense or grouped by expert, optionally with the SiLU gate.
//
// The 128 lanes of the accumulator are rows of the weight, its columns are rows of x ("tokens"): a tile of few
// tokens then costs few columns, whatever the count, and a batch of one streams the weight at full tile height.
// Both operands come by TMA in the 128-byte-swizzled K-major layout, 256 k (128 bytes) of a row per step; the scale
// tiles come by plain bulk copies and go from shared to tensor memory by tcgen05.cp, in order before the MMAs.
// Nothing is unpacked: the instruction multiplies e2m1 codes and applies both scales.
//
// One persistent CTA per SM, 192 threads: warp 0 TMA producer, warp 1 tensor memory and MMA issue, warps 2..5 epilogue.
// The work is a list of tiles (a weight tile of 128 rows, or the gate and the up tile of the same 128 outputs, x a
// token tile of TN) of `steps` k steps each.  The ring of stages runs on across tiles, and two accumulators let the
// epilogue of one tile run under the next one's MMAs.  Many tiles: CTA c takes whole tiles c, c + P, ...  Few tiles
// (decode: the weights are streamed once and the time is the memory's): all steps in a row are cut into P equal
// ranges, so every SM streams the same bytes; a tile cut between CTAs leaves fp32 partial sums, and the last of its
// contributors adds them in CTA order, so that nobody waits and equal calls give equal bits.
// Every wait is bounded; on a timeout the roles stop, copies in flight are waited for (bounded), the tensor memory is
// freed, and the fault word tells.
#include <cuda.h>

#include "uq_mx.cuh"

namespace uq {

namespace {

constexpr int THREADS = 192;
constexpr int STEP_K = 256;                     // k per stage: 128 bytes of a row, four MMAs of 64
constexpr int MAX_STAGES = 12;
constexpr int HEAD = 1024;                      // barriers and flags before the stages

// ---- PTX wrappers ------------------------------------------------------------------------------
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(smem_u32(bar)) : "memory");
}
// K-major operand, 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return ((uint64_t)(addr & 0x3FFFFu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// scale tile: 32 rows of 16 bytes, unswizzled, 8-row groups 128 bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return ((uint64_t)(addr & 0x3FFFFu) >> 4) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}
// one 512-byte scale tile -> 4 tensor-memory columns, repeated in the four lane quarters
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}
template <int FMT>
__device__ __forceinline__ void mma_block_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                 uint32_t sfb, uint32_t accumulate) {
    if constexpr (FMT == UQ_MXFP4)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
// Instruction descriptor: A and B e2m1, both K-major, M = 128, N = n, scales ue8m0 (MXFP4) or ue4m3; the scale
// factor ids (which bytes of a scale column) are OR-ed in per instruction.
template <int FMT> __device__ __forceinline__ uint32_t block_idesc(int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (FMT == UQ_MXFP4 ? 1u << 23 : 0u) | (1u << 27);
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Tiles are numbered in groups of GROUP weight tiles, token tiles within a group, weight tiles fastest, so that CTAs
// running at the same time share both operands' tiles in L2.
constexpr int GROUP = 16;

struct Tile {
    int expert, nt;                             // weight tile nt of this expert
    int row0, rows, first;                      // token rows: first, count (<= TN), first - the expert's first
};
__device__ __forceinline__ int offset_of(const MxGemmArgs& a, int e) { return min(max(__ldg(a.offsets + e), 0), a.rows); }

// `before`: token tiles before each expert (shared memory, experts + 1 entries), unused when there is one weight
__device__ __forceinline__ Tile find_tile(const MxGemmArgs& a, const int* before, int tt_all, int tile) {
    Tile t;
    const int per = GROUP * tt_all, g = tile / per, in = tile - g * per;
    const int width = min(GROUP, a.NT - g * GROUP);
    const int tt = in / width;
    t.nt = g * GROUP + in - tt * width;
    int e = 0, r0 = 0, r1 = a.rows, lt = tt;
    if (a.offsets) {
        int hi = a.experts;
        while (hi - e > 1) {
            const int mid = (e + hi) >> 1;
            if (before[mid] <= tt) e = mid; else hi = mid;
        }
        r0 = offset_of(a, e);
        r1 = max(offset_of(a, e + 1), r0);
        lt = tt - before[e];
    }
    t.expert = e;
    t.first = lt * a.TN;
    t.row0 = r0 + t.first;
    t.rows = min(a.TN, r1 - t.row0);
    return t;
}

// The k steps [k0, k1) of a tile that a CTA takes next.
struct Segment {
    int tile, k0, k1;
};
struct Schedule {
    long long u, u1, units;                     // split: this CTA's range of all steps
    int tile, tiles, steps, ctas;
    bool split;
    __device__ __forceinline__ Schedule(const MxGemmArgs& a, int tt_all) {
        steps = a.steps;
        tiles = tt_all * a.NT;
        ctas = gridDim.x;
        const int waves = (tiles + ctas - 1) / ctas;
        // whole tiles unless they would leave over 12 % of the SMs' time idle
        split = (long long)tiles * 100 < (long long)waves * ctas * 88;
        units = (long long)tiles * steps;
        if (split && units < 2LL * ctas) ctas = units < 2 ? 1 : (int)(units / 2);
        tile = blockIdx.x;
        u = u1 = 0;
        if (split && (int)blockIdx.x < ctas) {
            u = begin(blockIdx.x);
            u1 = begin(blockIdx.x + 1);
        }
    }
    __device__ __forceinline__ long long begin(int c) const { return units * c / ctas; }
    __device__ __forceinline__ int owner(long long v) const { return (int)(((v + 1) * ctas - 1) / units); }
    __device__ __forceinline__ bool next(Segment& s) {
        if (!split) {
            if (tile >= tiles) return false;
            s.tile = tile;
            s.k0 = 0;
            s.k1 = steps;
            tile += ctas;
            return true;
        }
        if (u >= u1) return false;
        s.tile = (int)(u / steps);
        s.k0 = (int)(u - (long long)s.tile * steps);
        s.k1 = (int)min((long long)steps, s.k0 + (u1 - u));
        u += s.k1 - s.k0;
        return true;
    }
};

__device__ __forceinline__ void store_one(const MxGemmArgs& a, long long at, float v) {
    if (a.ytype == UQ_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    else if (a.ytype == UQ_FP16) static_cast<__half*>(a.y)[at] = __float2half_rn(v);
    else static_cast<float*>(a.y)[at] = v;
}

template <int FMT, int NA>
__global__ void __launch_bounds__(THREADS, 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap wmap_up,
               const __grid_constant__ CUtensorMap xmap, const MxGemmArgs a) {
    constexpr int TPS = STEP_K / mx_tile_k(FMT);                   // scale tiles per step and 128 rows
    constexpr int A_BYTES = 128 * 128, SF_BYTES = TPS * 512;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* head = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(head);            // [stages] operands and scales landed
    uint64_t* empty = full + MAX_STAGES;                           // [stages] consumed by the MMAs
    uint64_t* acc_full = empty + MAX_STAGES;                       // [2] accumulator complete
    uint64_t* acc_empty = acc_full + 2;                            // [2] accumulator read by the epilogue
    uint64_t* drain = acc_empty + 2;                               // after a timeout: the MMAs issued so far
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
    int* last_flag = reinterpret_cast<int*>(tmem_ptr + 2);
    uint8_t* ring = head + HEAD;
    const int TN = a.TN, AB = a.accs;
    const int b_bytes = TN * 128, stage_bytes = NA * A_BYTES + b_bytes + (NA + 1) * SF_BYTES;
    int* before = reinterpret_cast<int*>(ring + (size_t)a.stages * stage_bytes);   // [experts + 1]

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    // One stage = step kt of a tile: both operands' codes and scale tiles, counted in bytes on full[s].
    auto load_weights = [&](const Tile& t, int kt, int s) {
        uint8_t* st = ring + (size_t)s * stage_bytes;
        const int tiles = min(TPS, a.ktiles - kt * TPS), n = t.nt * 128;
        mbar_arrive_expect_tx(&full[s], (uint32_t)(NA * A_BYTES + b_bytes + (NA + 1) * tiles * 512));
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            tma_2d(st + i * A_BYTES, i ? &wmap_up : &wmap, kt * 128, t.expert * a.N + n, &full[s]);
            bulk_g2s(st + NA * A_BYTES + b_bytes + i * SF_BYTES,
                     (i ? a.wscales_up : a.wscales) + t.expert * a.wscale_stride + ((long long)t.nt * a.ktiles + kt * TPS) * 512,
                     tiles * 512, &full[s]);
        }
    };
    auto load_tokens = [&](const Tile& t, int kt, int s) {
        uint8_t* st = ring + (size_t)s * stage_bytes;
        const int tiles = min(TPS, a.ktiles - kt * TPS);
        const long long xtile = (a.offsets ? (long long)((t.row0 - t.first) >> 7) + t.expert : 0) + (t.first >> 7);
        tma_2d(st + NA * A_BYTES, &xmap, kt * 128, t.row0, &full[s]);
        bulk_g2s(st + NA * A_BYTES + b_bytes + NA * SF_BYTES, a.xscales + (xtile * a.ktiles + kt * TPS) * 512, tiles * 512,
                 &full[s]);
    };

    int pre = 0;                                                   // stages whose weights are requested already
    if (warp == 0) {
        if (a.offsets) {
            int run = 0;
            for (int e0 = 0; e0 < a.experts; e0 += 32) {
                const int e = e0 + lane;
                const int n = e < a.experts ? (max(offset_of(a, e + 1) - offset_of(a, e), 0) + TN - 1) / TN : 0;
                int incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                if (e < a.experts) before[e] = run + incl - n;
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) before[a.experts] = run;
            __syncwarp();
        }
        if (lane == 0) {
            for (int s = 0; s < a.stages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&acc_full[i], 1);
                mbar_init(&acc_empty[i], 4);
            }
            mbar_init(drain, 1);
            *abort_flag = 0;
            fence_barrier_init();
            fence_proxy_async_smem();
            // The first stages' weights do not depend on the kernel before: requested ahead of everything else.
            const int tt_all = a.offsets ? before[a.experts] : (a.rows + TN - 1) / TN;
            Schedule sch(a, tt_all);
            Segment g;
            while (pre < a.stages && sch.next(g)) {
                const Tile t = find_tile(a, before, tt_all, g.tile);
                for (int kt = g.k0; kt < g.k1 && pre < a.stages; ++kt) load_weights(t, kt, pre++);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_ptr)), "r"((uint32_t)a.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_ptr;
    const uint32_t sf_col = tmem + AB * NA * TN;                   // scale columns, per stage
    constexpr uint32_t SF_COLS = (NA + 1) * TPS * 4;
    const int tt_all = a.offsets ? before[a.experts] : (a.rows + TN - 1) / TN;
    Schedule sch(a, tt_all);
    Segment g;

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ producer
        if (a.wait) asm volatile("griddepcontrol.wait;" ::: "memory");
        int issued = 0, s = 0;
        uint32_t ph = 1;                                           // empty[] of the first round counts as free
        bool ok = true;
        while (ok && sch.next(g)) {
            const Tile t = find_tile(a, before, tt_all, g.tile);
            for (int kt = g.k0; kt < g.k1; ++kt) {
                if (issued >= pre) {
                    if (*abort_flag || !mbar_wait_bounded(&empty[s], ph, a.fault, FAULT_MX_WAIT)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    load_weights(t, kt, s);
                }
                load_tokens(t, kt, s);
                ++issued;
                if (++s == a.stages) { s = 0; ph ^= 1; }
            }
        }
        // let the last copies land before the CTA can leave
        for (int j = issued - 1; j >= 0 && j >= issued - a.stages; --j)
            mbar_wait_bounded(&full[j % a.stages], (uint32_t)((j / a.stages) & 1), a.fault, FAULT_MX_WAIT);
    } else if (warp == 1 && lane == 0) {
        // ------------------------------------------------------------ MMA issue
        const uint32_t ring0 = smem_u32(ring);
        int s = 0, n = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (; ok && sch.next(g); ++n) {
            const Tile t = find_tile(a, before, tt_all, g.tile);
            const uint32_t idesc = block_idesc<FMT>((t.rows + 15) / 16 * 16);
            const uint32_t xshift = (uint32_t)(t.first & 127) >> 5;   // first scale column of the tile inside its 128 rows
            const int buf = AB == 2 ? n & 1 : 0;
            const uint32_t acc = tmem + buf * NA * TN;
            // the epilogue has read this accumulator's tile before (its first use counts as read)
            const uint32_t aph = (uint32_t)((AB == 2 ? n >> 1 : n) & 1) ^ 1u;
            if (!mbar_wait_bounded(&acc_empty[buf], aph, a.fault, FAULT_MX_WAIT)) ok = false;
            fence_after();
            uint32_t on = 0;
            for (int kt = g.k0; ok && kt < g.k1; ++kt) {
                if (*abort_flag || !mbar_wait_bounded(&full[s], ph, a.fault, FAULT_MX_WAIT)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t st = ring0 + s * stage_bytes, sc = st + NA * A_BYTES + b_bytes;
                const uint32_t col = sf_col + s * SF_COLS;
                const int tiles = min(TPS, a.ktiles - kt * TPS);
#pragma unroll
                for (int j = 0; j < TPS; ++j) {
                    if (j >= tiles) break;
#pragma unroll
                    for (int i = 0; i <= NA; ++i)
                        cp_scales(col + (i * TPS + j) * 4, scale_desc(sc + i * SF_BYTES + j * 512));
                }
                const int mmas = min(4, (a.K - kt * STEP_K + 63) >> 6);
                const uint64_t bd = operand_desc(st + NA * A_BYTES);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= mmas) break;
                    // MXFP4: two instructions share a scale tile (bytes 0-1, then 2-3); NVFP4: one tile each
                    const int j = FMT == UQ_MXFP4 ? q >> 1 : q;
                    const uint32_t id = FMT == UQ_MXFP4 ? (uint32_t)(q & 1) * 2 : 0u;
                    const uint32_t desc = idesc | (id << 4) | (id << 29);
#pragma unroll
                    for (int i = 0; i < NA; ++i)
                        mma_block_scaled<FMT>(acc + i * TN, operand_desc(st + i * A_BYTES) + 2 * q, bd + 2 * q, desc,
                                              col + (i * TPS + j) * 4, col + (NA * TPS + j) * 4 + xshift, on);
                    on = 1;
                }
                commit(&empty[s]);
                if (++s == a.stages) { s = 0; ph ^= 1; }
            }
            commit(&acc_full[buf]);
        }
        if (!ok) {
            *abort_flag = 1;
            commit(drain);
            mbar_wait_bounded(drain, 0, a.fault, FAULT_MX_WAIT);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue: lane = row of the weight tile
        const int q = warp & 3, row = q * 32 + lane, et = threadIdx.x - 64;
        const int esize = a.ytype == UQ_FP32 ? 4 : 2;
        if (a.offsets) {
            // rows that belong to nobody
            uint8_t* y = static_cast<uint8_t*>(a.y);
            const long long b0 = (long long)offset_of(a, a.experts) * a.N * esize, b1 = (long long)a.rows * a.N * esize;
            const long long c0 = min((b0 + 15) & ~15ll, b1), c1 = max(b1 & ~15ll, c0);
            const long long at = blockIdx.x * 128LL + et, all = gridDim.x * 128LL;
            for (long long i = b0 + at * 2; i < c0; i += all * 2) *reinterpret_cast<uint16_t*>(y + i) = 0;
            for (long long i = c0 + at * 16; i < c1; i += all * 16) *reinterpret_cast<uint4*>(y + i) = make_uint4(0, 0, 0, 0);
            for (long long i = c1 + at * 2; i < b1; i += all * 2) *reinterpret_cast<uint16_t*>(y + i) = 0;
        }
        for (int n = 0; sch.next(g); ++n) {
            const Tile t = find_tile(a, before, tt_all, g.tile);
            const int buf = AB == 2 ? n & 1 : 0;
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * NA * TN;
            // after a timeout the segments are walked without waiting (the warps stay together at the barriers below)
            if (!*abort_flag &&
                !mbar_wait_bounded(&acc_full[buf], (uint32_t)((AB == 2 ? n >> 1 : n) & 1), a.fault, FAULT_MX_WAIT))
                *abort_flag = 1;
            __syncwarp();
            fence_after();
            const bool whole = g.k0 == 0 && g.k1 == a.steps;
            const int nn = t.nt * 128 + row;
            const float al = a.alpha * (a.alpha_e ? __ldg(a.alpha_e + t.expert) : 1.f);
            const float au = a.alpha * (a.alpha_up ? __ldg(a.alpha_up + t.expert) : 1.f);
            auto put = [&](int c, const float* v) {                // column c .. c + 15 of this lane's row, NA sums each
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float r = v[j] * al;
                    if constexpr (NA == 2) r = silu_mul(r, v[16 + j] * au);
                    if (nn < a.N && c + j < t.rows) store_one(a, (long long)(t.row0 + c + j) * a.N + nn, r);
                }
            };
            const long long slot_floats = (long long)NA * TN * 128;
            // the slot of a contributor's sums of this tile: its first tile, or its last
            auto slot = [&](int c) { return a.partials + (2LL * c + (sch.begin(c) / sch.steps == g.tile ? 0 : 1)) * slot_floats; };
            float* mine = whole ? nullptr : slot(blockIdx.x);
            for (int c = 0; c < t.rows; c += 16) {
                uint32_t r[NA * 16];
#pragma unroll
                for (int i = 0; i < NA; ++i) tmem_ld16(acc + i * TN + c, *reinterpret_cast<uint32_t(*)[16]>(r + 16 * i));
                tmem_ld_wait();
                if (c + 16 >= t.rows) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[buf]);
                }
                float v[NA * 16];
#pragma unroll
                for (int j = 0; j < NA * 16; ++j) v[j] = __uint_as_float(r[j]);
                if (whole) {
                    put(c, v);
                } else {
#pragma unroll
                    for (int j = 0; j < NA * 16; ++j) __stcg(mine + ((j >> 4) * TN + c + (j & 15)) * 128 + row, v[j]);
                }
            }
            if (whole) continue;
            // the last contributor to arrive adds all contributors' sums, in CTA order
            const long long v0 = (long long)g.tile * sch.steps;
            const int c0 = sch.owner(v0), c1 = sch.owner(v0 + sch.steps - 1);
            __threadfence();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (et == 0) {
                const unsigned int before_me = atomicAdd(a.tickets + g.tile, 1u);
                *last_flag = before_me == (unsigned)(c1 - c0);
                if (*last_flag) a.tickets[g.tile] = 0;             // ready for the next call
                __threadfence();
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (!*last_flag) continue;
            for (int c = 0; c < t.rows; c += 16) {
                float v[NA * 16] = {};
                for (int k = c0; k <= c1; ++k) {
                    const float* p = slot(k);
#pragma unroll
                    for (int j = 0; j < NA * 16; ++j) v[j] += __ldcg(p + ((j >> 4) * TN + c + (j & 15)) * 128 + row);
                }
                put(c, v);
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"((uint32_t)a.tmem_cols) : "memory");
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

// codes [rows][K/2] as bytes, boxes of 128 bytes x `box` rows, 128-byte swizzle
bool codes_map(CUtensorMap* m, const uint8_t* codes, long long rows, int K, int box) {
    cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    cuuint32_t b[2] = {128, (cuuint32_t)box};
    cuuint32_t es[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, b, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int NA>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& up, const CUtensorMap& x, const MxGemmArgs& a, cudaStream_t st) {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(mx_gemm_kernel<FMT, NA>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = a.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.wait ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<FMT, NA>, w, up, x, a);
}

}  // namespace

// Tiles, ring and grid of one product, and the workspace it needs.
void mx_gemm_plan(int fmt, bool gated, MxGemmArgs& a, int sms, size_t* partial_bytes, size_t* ticket_bytes) {
    const int tps = STEP_K / mx_tile_k(fmt), NA = gated ? 2 : 1;
    a.steps = (a.K + STEP_K - 1) / STEP_K;
    a.ktiles = mx_ktiles(a.K, fmt);
    a.wscale_stride = mx_row_tiles(a.N, 0) * a.ktiles * 512;
    // token tile: the rows an expert gets on average (all of them when there is one).  Under 64 only where no second
    // tile can follow: a tile's scale columns then always start at an even column.
    const int mean = a.offsets ? (a.rows + a.experts - 1) / a.experts : a.rows;
    a.TN = a.rows <= 16 ? 16 : (a.rows <= 32 ? 32 : (mean <= 64 ? 64 : 128));
    a.NT = (a.N + 127) / 128;
    const int stage_bytes = NA * 16384 + a.TN * 128 + (NA + 1) * tps * 512;
    const int table = a.offsets ? (a.experts + 1) * 4 : 0;
    // tensor memory: two accumulators where 512 columns hold them beside three stages of scales
    const int sf = (NA + 1) * tps * 4;
    a.accs = 2 * NA * a.TN + 3 * sf <= 512 ? 2 : 1;
    a.stages = min(min((222 * 1024 - HEAD - table) / stage_bytes, MAX_STAGES), (512 - a.accs * NA * a.TN) / sf);
    const int cols = a.accs * NA * a.TN + a.stages * sf;
    a.tmem_cols = cols <= 64 ? 64 : (cols <= 128 ? 128 : (cols <= 256 ? 256 : 512));
    a.smem = 1024 + HEAD + a.stages * stage_bytes + table;
    a.ctas = sms;
    *partial_bytes = (size_t)2 * sms * NA * a.TN * 128 * sizeof(float);
    // tiles are split only below 88 % of some number of waves, so below 9 waves of them
    *ticket_bytes = (size_t)9 * sms * sizeof(unsigned int);
}

cudaError_t launch_mx_gemm(int fmt, const uint8_t* xcodes, const uint8_t* wcodes, const uint8_t* wcodes_up,
                           const MxGemmArgs& a, cudaStream_t st) {
    if (!encode_fn()) return cudaErrorNotSupported;
    CUtensorMap w, up, x;
    if (!codes_map(&w, wcodes, (long long)a.experts * a.N, a.K, 128)) return cudaErrorInvalidValue;
    up = w;
    if (wcodes_up && !codes_map(&up, wcodes_up, (long long)a.experts * a.N, a.K, 128)) return cudaErrorInvalidValue;
    if (!codes_map(&x, xcodes, a.rows, a.K, a.TN)) return cudaErrorInvalidValue;
    if (fmt == UQ_MXFP4)
        return wcodes_up ? launch<UQ_MXFP4, 2>(w, up, x, a, st) : launch<UQ_MXFP4, 1>(w, up, x, a, st);
    return wcodes_up ? launch<UQ_NVFP4, 2>(w, up, x, a, st) : launch<UQ_NVFP4, 1>(w, up, x, a, st);
}

}  // namespace uq
