// uq_mx_gemm.cu -- product of two microscaled 4-bit operands on the block-scaled tensor instructions (tcgen05,
// kind::mxf4 / kind::mxf4nvf4), dense or grouped by expert, optionally with the SiLU gate.
//
// The 128 lanes of the accumulator are rows of the weight, its columns are rows of x ("tokens"): a tile of few
// tokens then costs few columns, whatever the count, and a batch of one streams the weight at full tile height.
// Both operands come by TMA in the 128-byte-swizzled K-major layout, 256 k (128 bytes) of a row per step; the scale
// tiles come by plain bulk copies and go from shared to tensor memory by tcgen05.cp, in order before the MMAs.
// Nothing is unpacked: the instruction multiplies e2m1 codes and applies both scales.
//
// A CTA owns NA weight tiles (two: 256 rows, or the gate and the up tile of the same 128 outputs) x one token tile
// of TN, and 1/S of K; the S CTAs of a cluster add their partial sums through distributed shared memory in rank
// order (few tiles: decode).  Roles (192 threads): warp 0 TMA producer, warp 1 tensor memory and MMA issue, warps
// 2..5 epilogue.  Every wait is bounded; on a timeout the roles stop, copies in flight are waited for (bounded), the
// tensor memory is freed, and the fault word tells.
#include <cuda.h>

#include "uq_mx.cuh"

namespace uq {

namespace {

constexpr int THREADS = 192;
constexpr int STEP_K = 256;                     // k per stage: 128 bytes of a row, four MMAs of 64
constexpr int MAX_STAGES = 10;
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
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The output tile a CTA works on.
struct Tile {
    int expert;                                 // -1: none
    int row0, rows;                             // its token rows: first, count (<= TN)
    int first;                                  // row0 - first row of the expert
    int nt;                                     // weight tile
};

// Tiles are numbered in groups of GROUP weight tiles, token tiles within a group, weight tiles fastest, so that CTAs
// running at the same time share both operands' tiles in L2.
constexpr int GROUP = 16;

__device__ __forceinline__ Tile find_tile(const MxGemmArgs& a, int tile) {
    Tile t;
    t.expert = -1;
    const int lane = threadIdx.x & 31;
    auto begin = [&](int e) { return min(max(__ldg(a.offsets + e), 0), a.rows); };
    int tt_all;                                 // token tiles of all experts
    if (!a.offsets) {
        tt_all = (a.rows + a.TN - 1) / a.TN;
    } else {
        int n = 0;
        for (int e = lane; e < a.experts; e += 32) n += (max(begin(e + 1) - begin(e), 0) + a.TN - 1) / a.TN;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        tt_all = n;
    }
    if (tile >= tt_all * a.NT) return t;
    const int per = GROUP * tt_all, g = tile / per;
    const int width = min(GROUP, a.NT - g * GROUP), in = tile - g * per;
    int tt = in / width;
    t.nt = g * GROUP + in % width;
    if (!a.offsets) {
        t.expert = 0;
        t.row0 = t.first = tt * a.TN;
        t.rows = min(a.TN, a.rows - t.row0);
        return t;
    }
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
        const int e = e0 + lane;
        const int r0 = e < a.experts ? begin(e) : 0, r1 = e < a.experts ? max(begin(e + 1), r0) : 0;
        const int n = (r1 - r0 + a.TN - 1) / a.TN;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, tt >= incl - n && tt < incl);
        if (hit) {
            const int src = __ffs(hit) - 1;
            t.expert = e0 + src;
            t.first = (tt - __shfl_sync(0xffffffffu, incl - n, src)) * a.TN;
            const int b0 = __shfl_sync(0xffffffffu, r0, src), b1 = __shfl_sync(0xffffffffu, r1, src);
            t.row0 = b0 + t.first;
            t.rows = min(a.TN, b1 - t.row0);
            return t;
        }
        tt -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return t;
}

template <class T> __device__ __forceinline__ void store8(T* p, const float (&v)[8], int n, bool vec) {
    if (vec) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) {
            Vec<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(v[h * V + i]);
            reinterpret_cast<Vec<T, V>*>(p)[h] = o;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
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
    uint64_t* done = empty + MAX_STAGES;                           // all MMAs of the tile complete
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
    uint8_t* ring = head + HEAD;

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int S = a.S, rank = blockIdx.x % S, TN = a.TN;
    const int b_bytes = TN * 128, stage_bytes = NA * A_BYTES + b_bytes + (NA + 1) * SF_BYTES;
    const Tile t = find_tile(a, blockIdx.x / S);
    const int esize = a.ytype == UQ_FP32 ? 4 : 2;

    // rows that belong to nobody
    if (a.offsets) {
        if (a.wait) asm volatile("griddepcontrol.wait;" ::: "memory");
        const long long kept = min(max(__ldg(a.offsets + a.experts), 0), a.rows);
        uint8_t* y = static_cast<uint8_t*>(a.y);
        const long long b0 = kept * a.N * esize, b1 = (long long)a.rows * a.N * esize;
        for (long long i = b0 + (blockIdx.x * (long long)THREADS + threadIdx.x) * 2; i < b1; i += gridDim.x * (long long)THREADS * 2)
            *reinterpret_cast<uint16_t*>(y + i) = 0;
    }
    if (t.expert < 0) return;                                      // the whole cluster: its CTAs share the tile

    // this CTA's steps of k
    const int k0 = (int)((long long)a.steps * rank / S), k1 = (int)((long long)a.steps * (rank + 1) / S);
    const int n0 = t.nt * (a.gated ? 128 : NA * 128);
    // the second weight tile of an odd count does not exist
    const int na = a.gated ? 2 : (NA == 2 && n0 + 128 < a.N ? 2 : 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_ptr)), "r"((uint32_t)a.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_ptr;
    const uint32_t sf_col = tmem + NA * TN;                        // scale columns, per stage
    constexpr uint32_t SF_COLS = (NA + 1) * TPS * 4;

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ producer
        auto weights = [&](int kt, int s) {
            uint8_t* st = ring + (size_t)s * stage_bytes;
            const int tiles = min(TPS, a.ktiles - kt * TPS);
            mbar_arrive_expect_tx(&full[s], (uint32_t)(na * A_BYTES + b_bytes + (na + 1) * tiles * 512));
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                if (i >= na) break;
                const bool up = a.gated && i == 1;
                const int n = n0 + (a.gated ? 0 : i * 128);
                tma_2d(st + i * A_BYTES, up ? &wmap_up : &wmap, kt * 128, t.expert * a.N + n, &full[s]);
                const uint8_t* sc = (up ? a.wscales_up : a.wscales) + (long long)t.expert * a.wscale_stride;
                bulk_g2s(st + NA * A_BYTES + b_bytes + i * SF_BYTES,
                         sc + ((long long)(n >> 7) * a.ktiles + kt * TPS) * 512, tiles * 512, &full[s]);
            }
        };
        const long long xtile = (a.offsets ? (long long)((t.row0 - t.first) >> 7) + t.expert : 0) + (t.first >> 7);
        auto tokens = [&](int kt, int s) {
            uint8_t* st = ring + (size_t)s * stage_bytes;
            const int tiles = min(TPS, a.ktiles - kt * TPS);
            tma_2d(st + NA * A_BYTES, &xmap, kt * 128, t.row0, &full[s]);
            bulk_g2s(st + NA * A_BYTES + b_bytes + NA * SF_BYTES, a.xscales + (xtile * a.ktiles + kt * TPS) * 512,
                     tiles * 512, &full[s]);
        };
        // the weights of the first stages do not depend on the kernel before: requested ahead of the wait for it
        const int pre = min(k1 - k0, a.stages);
        for (int i = 0; i < pre; ++i) weights(k0 + i, i);
        if (a.wait) asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int i = 0; i < pre; ++i) tokens(k0 + i, i);
        int issued = pre, s = 0;
        uint32_t ph = 0;
        for (int kt = k0 + pre; kt < k1 && !*abort_flag; ++kt, ++issued) {
            if (!mbar_wait_bounded(&empty[s], ph, a.fault, FAULT_MX_WAIT)) {
                *abort_flag = 1;
                break;
            }
            weights(kt, s);
            tokens(kt, s);
            if (++s == a.stages) { s = 0; ph ^= 1; }
        }
        // let the last copies land before the CTA can leave
        for (int j = issued - 1; j >= 0 && j >= issued - a.stages; --j)
            mbar_wait_bounded(&full[j % a.stages], (uint32_t)((j / a.stages) & 1), a.fault, FAULT_MX_WAIT);
    } else if (warp == 1 && lane == 0) {
        // ------------------------------------------------------------ MMA issue
        const uint32_t idesc = block_idesc<FMT>((t.rows + 15) / 16 * 16);
        const uint32_t ring0 = smem_u32(ring);
        const uint32_t xshift = (uint32_t)(t.first & 127) >> 5;    // first scale column of a tile inside its 128 rows
        int s = 0;
        uint32_t ph = 0, acc = 0;
        for (int kt = k0; kt < k1; ++kt) {
            if (*abort_flag || !mbar_wait_bounded(&full[s], ph, a.fault, FAULT_MX_WAIT)) {
                *abort_flag = 1;
                break;
            }
            fence_after();
            const uint32_t st = ring0 + s * stage_bytes, sc = st + NA * A_BYTES + b_bytes;
            const uint32_t col = sf_col + s * SF_COLS;
            const int tiles = min(TPS, a.ktiles - kt * TPS);
            for (int j = 0; j < tiles; ++j) {
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    if (i < na) cp_scales(col + (i * TPS + j) * 4, scale_desc(sc + i * SF_BYTES + j * 512));
                cp_scales(col + (NA * TPS + j) * 4, scale_desc(sc + NA * SF_BYTES + j * 512));
            }
            const int mmas = min(4, (a.K - kt * STEP_K + 63) >> 6);
            const uint64_t bd = operand_desc(st + NA * A_BYTES);
            for (int q = 0; q < mmas; ++q) {
                // MXFP4: two instructions share a scale tile (bytes 0-1, then 2-3); NVFP4: one tile each
                const int j = FMT == UQ_MXFP4 ? q >> 1 : q;
                const uint32_t id = FMT == UQ_MXFP4 ? (uint32_t)(q & 1) * 2 : 0u;
                const uint32_t desc = idesc | (id << 4) | (id << 29);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    if (i < na)
                        mma_block_scaled<FMT>(tmem + i * TN, operand_desc(st + i * A_BYTES) + 2 * q, bd + 2 * q, desc,
                                              col + (i * TPS + j) * 4, col + (NA * TPS + j) * 4 + xshift, acc);
                acc = 1;
            }
            commit(&empty[s]);
            if (++s == a.stages) { s = 0; ph ^= 1; }
        }
        commit(done);
    }
    __syncwarp();
    if (warp >= 2) {
        // ------------------------------------------------------------ accumulators -> shared memory [token][row], fp32
        if (!mbar_wait_bounded(done, 0, a.fault, FAULT_MX_WAIT)) *abort_flag = 1;
        __syncwarp();
        fence_after();
        float* stage = reinterpret_cast<float*>(ring);
        const int q = warp & 3, row = q * 32 + lane;
        for (int i = 0; i < na; ++i)
            for (int c = 0; c < t.rows; c += 16) {
                uint32_t r[16];
                tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + i * TN + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) stage[(c + j) * (NA * 128) + i * 128 + row] = __uint_as_float(r[j]);
            }
    }
    // Tensor memory is given back before the cluster waits for its CTAs: one that holds it waits for nobody, so CTAs
    // whose allocation waits for it always get it.
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"((uint32_t)a.tmem_cols) : "memory");
    if (S > 1) cluster_sync();
    if (!*abort_flag) {
        // ---------------------------------------------------------------- sum over the ranks, scale, gate, store
        const float al = a.alpha * (a.alpha_e ? __ldg(a.alpha_e + t.expert) : 1.f);
        const float au = a.alpha * (a.alpha_up ? __ldg(a.alpha_up + t.expert) : 1.f);
        const int groups = (a.gated ? 128 : na * 128) / 8;
        const int items = t.rows * groups;
        const uint32_t stage = smem_u32(ring);
        const bool vec = (long long)a.N * esize % 16 == 0;
        for (int it = rank * THREADS + threadIdx.x; it < items; it += S * THREADS) {
            const int c = it / groups, g = it % groups, n = n0 + g * 8;
            if (n >= a.N) continue;
            float v[8] = {}, u[8] = {};
            for (int r = 0; r < S; ++r) {
                const uint32_t src = (S > 1 ? cluster_addr(stage, r) : stage) + (c * (NA * 128) + g * 8) * 4;
                const float4 p = ld_cluster4(src), q = ld_cluster4(src + 16);
                v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
                v[4] += q.x; v[5] += q.y; v[6] += q.z; v[7] += q.w;
                if (NA == 2 && a.gated) {
                    const float4 x = ld_cluster4(src + 512), z = ld_cluster4(src + 528);
                    u[0] += x.x; u[1] += x.y; u[2] += x.z; u[3] += x.w;
                    u[4] += z.x; u[5] += z.y; u[6] += z.z; u[7] += z.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] *= al;
                if (NA == 2 && a.gated) v[i] = silu_mul(v[i], u[i] * au);
            }
            const long long at = (long long)(t.row0 + c) * a.N + n;
            const int count = min(8, a.N - n);
            const bool wide = vec && count == 8;
            if (a.ytype == UQ_BF16) store8(static_cast<__nv_bfloat16*>(a.y) + at, v, count, wide);
            else if (a.ytype == UQ_FP16) store8(static_cast<__half*>(a.y) + at, v, count, wide);
            else store8(static_cast<float*>(a.y) + at, v, count, wide);
        }
    }
    if (S > 1) cluster_sync();                                     // no CTA leaves while another reads its sums
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
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& up, const CUtensorMap& x, const MxGemmArgs& a, long long grid,
                   size_t smem, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(mx_gemm_kernel<FMT, NA>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = a.S;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
    if (a.wait) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<FMT, NA>, w, up, x, a);
}

}  // namespace

// Shapes, tiles and splits of one product; the pointers are filled in by the caller.
cudaError_t launch_mx_gemm(int fmt, const uint8_t* xcodes, const uint8_t* wcodes, const uint8_t* wcodes_up, MxGemmArgs a,
                           int sms, cudaStream_t st) {
    if (!encode_fn()) return cudaErrorNotSupported;
    const int tps = STEP_K / mx_tile_k(fmt);
    a.steps = (a.K + STEP_K - 1) / STEP_K;
    a.ktiles = mx_ktiles(a.K, fmt);
    a.wscale_stride = mx_row_tiles(a.N, 0) * a.ktiles * 512;
    a.gated = wcodes_up != nullptr;
    // token tile: the rows an expert gets on average (all of them when there is one).  32 only where no second tile
    // can follow: a tile's scale columns then always start at an even column.
    const int mean = a.offsets ? (a.rows + a.experts - 1) / a.experts : a.rows;
    a.TN = a.rows <= 32 ? 32 : (mean <= 64 ? 64 : 128);
    const int nt1 = (a.N + 127) / 128;
    const long long tt = a.offsets ? min((long long)a.rows, a.rows / a.TN + (long long)a.experts) : (a.rows + a.TN - 1) / a.TN;
    const int NA = a.gated || (a.TN == 128 && (nt1 + 1) / 2 * tt >= sms) ? 2 : 1;
    a.NT = a.gated || NA == 1 ? nt1 : (nt1 + 1) / 2;
    const long long tiles = a.NT * tt;
    a.S = 1;
    while (a.S < 8 && tiles * a.S * 2 <= 3LL * sms && a.steps >= 4 * a.S) a.S *= 2;
    const int stage_bytes = NA * 16384 + a.TN * 128 + (NA + 1) * tps * 512;
    const int most = (a.steps + a.S - 1) / a.S;
    a.stages = min(min((200 * 1024) / stage_bytes, MAX_STAGES), most);
    const int cols = NA * a.TN + a.stages * (NA + 1) * tps * 4;
    a.tmem_cols = cols <= 64 ? 64 : (cols <= 128 ? 128 : (cols <= 256 ? 256 : 512));
    while (NA * a.TN + a.stages * (NA + 1) * tps * 4 > 512) --a.stages;
    size_t body = (size_t)a.stages * stage_bytes;
    const size_t sums = (size_t)a.TN * NA * 512;
    if (body < sums) body = sums;
    const size_t smem = 1024 + HEAD + body;
    CUtensorMap w, up, x;
    if (!codes_map(&w, wcodes, (long long)a.experts * a.N, a.K, 128)) return cudaErrorInvalidValue;
    up = w;
    if (a.gated && !codes_map(&up, wcodes_up, (long long)a.experts * a.N, a.K, 128)) return cudaErrorInvalidValue;
    if (!codes_map(&x, xcodes, a.rows, a.K, a.TN)) return cudaErrorInvalidValue;
    const long long grid = tiles * a.S;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    if (fmt == UQ_MXFP4)
        return NA == 2 ? launch<UQ_MXFP4, 2>(w, up, x, a, grid, smem, st) : launch<UQ_MXFP4, 1>(w, up, x, a, grid, smem, st);
    return NA == 2 ? launch<UQ_NVFP4, 2>(w, up, x, a, grid, smem, st) : launch<UQ_NVFP4, 1>(w, up, x, a, grid, smem, st);
}

}  // namespace uq
