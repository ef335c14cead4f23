// uq_mx_gemm.cu -- product of two microscaled 4-bit operands on the block-scaled tensor instructions (tcgen05,
// kind::mxf4 / kind::mxf4nvf4), dense or grouped by expert, optionally with the SiLU gate.
//
// The 128 lanes of the accumulator are rows of the weight, its columns are rows of x ("tokens"): a tile of few
// tokens then costs few columns, whatever the count, and a batch of one streams the weight at full tile height.
// Both operands come by TMA in the 128-byte-swizzled K-major layout, 512 k of a row per step (two 128-byte columns in
// one box where K allows); the scale tiles come by TMA too and go from shared to tensor memory by tcgen05.cp, in order
// before the MMAs.
// Nothing is unpacked: the instruction multiplies e2m1 codes and applies both scales.
//
// One persistent CTA per SM, 224 threads: warp 0 loads the weights, warp 6 the tokens, warp 1 allocates tensor memory and
// issues the MMAs, warps 2..5 are the epilogue.
// The work is a list of tiles (a weight tile of 128 rows, or the gate and the up tile of the same 128 outputs, x a
// token tile of TN) of `steps` k steps each; CTA c takes tiles c, c + P, ...  The ring of stages runs on across tiles,
// and two accumulators let the epilogue of one tile run under the next one's MMAs.  Where tiles would fill at most half
// of the SMs and it saves time (split_of), a cluster of S CTAs shares each tile's k steps and adds the fp32 sums through
// distributed shared memory in rank order, so equal calls give equal bits.
// One GB300, graph replay, weights from DRAM, us with x quantized in the call / before: 1 x 14336 x 4096 MXFP4 9.0 / 8.8
// (6.9 / 6.4 where L2 keeps them), 37 x 4096 x 14336 NVFP4 13.7 / 11.9; 512 x 2048 x 2048 MXFP4 7.4 / 6.1; large products
// on pairs of CTAs (below) 8192^3 MXFP4 185 / 156 (7.0 PFLOP/s), NVFP4 201 / 167.  What bounds them: few tokens start and
// end of a kernel (3 us) and then memory; many the tensor cores (their pipe is active in 81 % of an 8192^3's cycles).
// Every wait is bounded; on a timeout the roles stop, copies in flight are waited for (bounded), the tensor memory is
// freed, and the fault word tells.
#include <algorithm>

#include "uq_mx_quant.cuh"
#include "uq_tcgen05.cuh"

namespace uq {

namespace {

constexpr int THREADS = 224;
constexpr int QUANT_WARPS = 4;                  // of the kernel that quantizes the tokens itself, in place of warp 6
constexpr int FUSED_THREADS = THREADS + (QUANT_WARPS - 1) * 32;
constexpr int FUSED_ROWS = 3;                   // its most tokens (rule at mx_gemm_quantizes)
constexpr int STEP_K = 512;                     // k per stage: two 128-byte columns of a row, eight MMAs of 64
// The tensor maps of a launch.
struct MxGemmMaps {
    CUtensorMap w, x, w_scales, x_scales, up, up_scales;
};

constexpr int MAX_SPLIT = 8;                    // CTAs of a cluster sharing a tile's steps
constexpr int MAX_STAGES = 12;
constexpr int HEAD = 1024;                      // barriers and flags before the stages

// ---- PTX wrappers ------------------------------------------------------------------------------
// The producer and the MMA warp run their loops as whole warps, so that every operand is a warp-uniform value, and the
// elected lane issues (one lane in a divergent branch issued a tcgen05 instruction every ~120 cycles).
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(UQ_ELECT "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];\n\t}"
                 :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
// (high word of a scale tile's descriptor: 32 rows of 16 bytes, unswizzled, 8-row groups 128 bytes apart)
#define UQ_SCALES_HI "0x00004008"

// The instructions that share a scale tile, issued by the elected lane of the converged warp: tcgen05.cp of the tile
// of each operand (512 bytes -> 4 tensor-memory columns, repeated in the four lane quarters), then the MMAs.  MXFP4: a
// tile's four blocks are 128 k, two MMAs (bytes 0-1 of the scale columns, then 2-3; the second one only if `two`);
// NVFP4: 64 k, one MMA.  The operand descriptors advance by 32 bytes (2) per MMA.
//   d accumulator, a / b low descriptor words, sa / sb the scale tiles', ca / cb the scale columns written, cu the scale
//   column of B that is used, on: add to the accumulator (the first MMA's; the second always does).
template <int FMT>
__device__ __forceinline__ void issue_tile(uint32_t d, uint32_t a, uint32_t b, uint32_t sa, uint32_t sb, uint32_t ca,
                                           uint32_t cb, uint32_t cu, uint32_t idesc, uint32_t on, uint32_t two) {
    if constexpr (FMT == UQ_MXFP4)
        asm volatile("{\n\t.reg .pred p, e, f, t;\n\t.reg .b64 da, db, sa, sb;\n\t.reg .b32 i2;\n\t"
                     "mov.b64 da, {%1, " UQ_OPERAND_HI "};\n\tmov.b64 db, {%2, " UQ_OPERAND_HI "};\n\t"
                     "mov.b64 sa, {%3, " UQ_SCALES_HI "};\n\tmov.b64 sb, {%4, " UQ_SCALES_HI "};\n\t"
                     "or.b32 i2, %8, 0x40000020;\n\tsetp.ne.b32 p, %9, 0;\n\tsetp.eq.b32 t, %8, %8;\n\t"
                     "elect.sync _|e, 0xffffffff;\n\tsetp.ne.and.b32 f, %10, 0, e;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%5], sa;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%6], sb;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %8, [%5], [%7], p;\n\t"
                     "add.s64 da, da, 2;\n\tadd.s64 db, db, 2;\n\t"
                     "@f tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, i2, [%5], [%7], t;\n\t}"
                     :: "r"(d), "r"(a), "r"(b), "r"(sa), "r"(sb), "r"(ca), "r"(cb), "r"(cu), "r"(idesc), "r"(on), "r"(two)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 da, db, sa, sb;\n\t"
                     "mov.b64 da, {%1, " UQ_OPERAND_HI "};\n\tmov.b64 db, {%2, " UQ_OPERAND_HI "};\n\t"
                     "mov.b64 sa, {%3, " UQ_SCALES_HI "};\n\tmov.b64 sb, {%4, " UQ_SCALES_HI "};\n\t"
                     "setp.ne.b32 p, %9, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%5], sa;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%6], sb;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], da, db, %8, [%5], [%7], p;\n\t}"
                     :: "r"(d), "r"(a), "r"(b), "r"(sa), "r"(sb), "r"(ca), "r"(cb), "r"(cu), "r"(idesc), "r"(on)
                     : "memory");
}
// the same for a second weight tile against the same tokens, whose scales are in place
template <int FMT>
__device__ __forceinline__ void issue_more(uint32_t d, uint32_t a, uint32_t b, uint32_t sa, uint32_t ca, uint32_t cu,
                                           uint32_t idesc, uint32_t on, uint32_t two) {
    if constexpr (FMT == UQ_MXFP4)
        asm volatile("{\n\t.reg .pred p, e, f, t;\n\t.reg .b64 da, db, sa;\n\t.reg .b32 i2;\n\t"
                     "mov.b64 da, {%1, " UQ_OPERAND_HI "};\n\tmov.b64 db, {%2, " UQ_OPERAND_HI "};\n\t"
                     "mov.b64 sa, {%3, " UQ_SCALES_HI "};\n\t"
                     "or.b32 i2, %6, 0x40000020;\n\tsetp.ne.b32 p, %7, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
                     "elect.sync _|e, 0xffffffff;\n\tsetp.ne.and.b32 f, %8, 0, e;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], sa;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %6, [%4], [%5], p;\n\t"
                     "add.s64 da, da, 2;\n\tadd.s64 db, db, 2;\n\t"
                     "@f tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, i2, [%4], [%5], t;\n\t}"
                     :: "r"(d), "r"(a), "r"(b), "r"(sa), "r"(ca), "r"(cu), "r"(idesc), "r"(on), "r"(two) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 da, db, sa;\n\t"
                     "mov.b64 da, {%1, " UQ_OPERAND_HI "};\n\tmov.b64 db, {%2, " UQ_OPERAND_HI "};\n\t"
                     "mov.b64 sa, {%3, " UQ_SCALES_HI "};\n\t"
                     "setp.ne.b32 p, %7, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], sa;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], da, db, %6, [%4], [%5], p;\n\t}"
                     :: "r"(d), "r"(a), "r"(b), "r"(sa), "r"(ca), "r"(cu), "r"(idesc), "r"(on) : "memory");
}
// Instruction descriptor: A and B e2m1, both K-major, M = 128, N = n, scales ue8m0 (MXFP4) or ue4m3; the scale
// factor ids (which bytes of a scale column) are OR-ed in per instruction.
template <int FMT> __device__ __forceinline__ uint32_t block_idesc(int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (FMT == UQ_MXFP4 ? 1u << 23 : 0u) | (1u << 27);
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// A whole warp's wait: false for all lanes once WAIT_LIMIT_NS have passed (the fault word then tells) or the CTA was
// told to stop.  Polls without a suspend hint: a warp put to sleep for up to a microsecond woke too late for a ring
// whose steps take a quarter of that.
// CLUSTER: arrivals of the pair's other CTA count on the barrier.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned int* fault, volatile int* abort_flag) {
    unsigned long long t0 = 0;
    for (unsigned int i = 0;; ++i) {
        uint32_t ok;
        if constexpr (CLUSTER)
            asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                         "selp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        else
            asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
        if (i % 32 == 0) {
            bool stop = *abort_flag != 0;
            if (!t0) t0 = global_ns();
            else if (global_ns() - t0 > WAIT_LIMIT_NS) {
                atomicOr(fault, FAULT_MX_WAIT);
                stop = true;
            }
            if (__any_sync(0xffffffffu, stop)) return false;
        }
    }
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Tiles are numbered in groups of a.group weight tiles, token tiles within a group, weight tiles fastest, so that CTAs
// running at the same time share both operands' tiles in L2.

struct Tile {
    int expert, nt;                             // weight tile nt of this expert
    int row0, rows, first;                      // token rows: first, count (<= TN), first - the expert's first
};
__device__ __forceinline__ int offset_of(const MxGemmArgs& a, int e) { return min(max(ld_written(a.offsets + e), 0), a.rows); }

// The table of the experts' token tiles (shared memory): tiles before each expert, then each expert's first row,
// experts + 1 entries both.
__host__ __device__ constexpr int table_bytes(int experts) { return 2 * (experts + 1) * 4; }

__device__ __forceinline__ Tile find_tile(const MxGemmArgs& a, const int* before, int tt_all, int tile) {
    Tile t;
    // divisions only where they are needed: they are a part of a short call's start
    int tt = 0;
    t.nt = tile;
    if (tt_all > 1) {
        const unsigned per = a.group * tt_all, g = a.NT > a.group ? (unsigned)tile / per : 0, in = tile - g * per;
        const unsigned width = min(a.group, a.NT - (int)g * a.group);
        tt = in / width;
        t.nt = g * a.group + in - tt * width;
    }
    int e = 0, r0 = 0, r1 = a.rows, lt = tt;
    if (a.offsets) {
        int hi = a.experts;
        while (hi - e > 1) {
            const int mid = (e + hi) >> 1;
            if (before[mid] <= tt) e = mid; else hi = mid;
        }
        const int* start = before + a.experts + 1;
        r0 = start[e];
        r1 = max(start[e + 1], r0);
        lt = tt - before[e];
    }
    t.expert = e;
    t.first = lt * a.TN;
    t.row0 = r0 + t.first;
    t.rows = min(a.TN, r1 - t.row0);
    return t;
}

// Fills the table (one warp).  128 experts at a time, all their offsets requested before the first is used.
__device__ __forceinline__ void token_tiles(const MxGemmArgs& a, int* before) {
    const int lane = threadIdx.x & 31;
    int* start = before + a.experts + 1;
    int run = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 128) {
        int o[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) o[j] = offset_of(a, min(e0 + lane * 4 + j, a.experts));
        int n[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[j] = (max(o[j + 1] - o[j], 0) + a.TN - 1) / a.TN;    // 0 past the last expert
            sum += n[j];
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        int at = run + incl - sum;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int e = e0 + lane * 4 + j;
            if (e < a.experts) {
                before[e] = at;
                start[e] = o[j];
            }
            at += n[j];
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
        before[a.experts] = run;
        start[a.experts] = offset_of(a, a.experts);
    }
    __syncwarp();
}

// Rows that belong to nobody are zero; thread `at` of `all`.
__device__ __forceinline__ void zero_tail(const MxGemmArgs& a, long long at, long long all) {
    const int esize = a.ytype == UQ_FP32 ? 4 : 2;
    uint8_t* y = static_cast<uint8_t*>(a.y);
    const long long b0 = (long long)offset_of(a, a.experts) * a.N * esize, b1 = (long long)a.rows * a.N * esize;
    const long long c0 = min((b0 + 15) & ~15ll, b1), c1 = max(b1 & ~15ll, c0);
    for (long long i = b0 + at * 2; i < c0; i += all * 2) *reinterpret_cast<uint16_t*>(y + i) = 0;
    for (long long i = c0 + at * 16; i < c1; i += all * 16) *reinterpret_cast<uint4*>(y + i) = make_uint4(0, 0, 0, 0);
    for (long long i = c1 + at * 2; i < b1; i += all * 2) *reinterpret_cast<uint16_t*>(y + i) = 0;
}

// With launch overlap (or behind the call's own quantizer) a kernel starts while the one before it on the stream still
// runs; this one's tokens and offsets may be its output, and y may be read by it.  The weights are requested before.
__device__ __forceinline__ void after_prior_work(const MxGemmArgs& a) {
    if (a.wait) asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Lets the next kernel's CTAs start as these leave their SMs.  Not before this kernel's own wait, since the next one may
// request weights that work before this kernel writes; and not before this CTA has its tensor memory: one that started
// before and took it would hold it until this kernel is done.
__device__ __forceinline__ void launch_dependents(const MxGemmArgs& a) {
    after_prior_work(a);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The tiles of a CTA and its k steps of them.
struct Schedule {
    int tile, tiles, stride, k0, k1;
    __device__ __forceinline__ Schedule(const MxGemmArgs& a, int tt_all) {
        tiles = tt_all * a.NT;
        if (a.S > 1) {                          // one tile per cluster
            const int rank = (int)cluster_rank();
            asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(tile));
            stride = tiles;
            k0 = a.share * rank + min(rank, a.extra);
            k1 = k0 + a.share + (rank < a.extra);
        } else {
            tile = blockIdx.x;
            stride = gridDim.x;
            k0 = 0;
            k1 = a.steps;
        }
    }
    __device__ __forceinline__ bool more() const { return tile < tiles; }
    __device__ __forceinline__ void advance() { tile += stride; }
};

// Up to four neighbouring outputs (count of them) at element `at`; the split tiles' path.
__device__ __forceinline__ void store4(const MxGemmArgs& a, long long at, int count, const float (&v)[4]) {
    auto go = [&](auto t) {
        using T = decltype(t);
        T* y = static_cast<T*>(a.y) + at;
        if (count >= 4 && a.N % 4 == 0) {
            Vec<T, 4> o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o.v[i] = from_f32<T>(v[i]);
            *reinterpret_cast<Vec<T, 4>*>(y) = o;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < count) y[i] = from_f32<T>(v[i]);
        }
    };
    if (a.ytype == UQ_BF16) go(__nv_bfloat16());
    else if (a.ytype == UQ_FP16) go(__half());
    else go(float());
}
// Writes 16 columns (tokens m0 .. m0 + count) of this lane's output nn; the warp's lanes hold 32 consecutive outputs.
// 16-bit types with an even N: neighbouring lanes exchange every other value and store pairs of outputs, so a store
// covers 64 bytes of each of two tokens, and conversions and stores are halved.
template <class T> __device__ __forceinline__ void put16(const MxGemmArgs& a, int m0, int count, int nn, const float (&v)[16]) {
    T* y = static_cast<T*>(a.y);
    if constexpr (sizeof(T) == 2) {
        if (!(a.N & 1)) {
            const int odd = threadIdx.x & 1;
            T* p = y + (long long)(m0 + odd) * a.N + (nn & ~1);
            const long long step = 2ll * a.N;
#pragma unroll
            for (int j = 0; j < 16; j += 2, p += step) {
                const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                const uint32_t w = pack2(T(), odd ? got : v[j], odd ? v[j + 1] : got);
                if (nn < a.N && j + odd < count) *reinterpret_cast<uint32_t*>(p) = w;
            }
            return;
        }
    }
    T* p = y + (long long)m0 * a.N + nn;
#pragma unroll
    for (int j = 0; j < 16; ++j, p += a.N)
        if (nn < a.N && j < count) *p = from_f32<T>(v[j]);
}
// silu(g) * u = g * u / (1 + e^-g) to 2^-20: e^-g = 2^t with t = -g log2(e) rounded, corrected to first order by what
// the rounding left (t alone would lose |t| 2^-24) wherever 2^t is finite and matters, |t| < 128, then an approximate
// reciprocal.  Below g = -88.72 e^-g exceeds fp32 and the result is zero.  A gated tile's epilogue is
// 128 of these per lane beside MMAs that may take only a few thousand cycles; with expf and a correctly rounded
// division it took longer than they did (16384 rows, 64 experts of 1408 x 2048 gated: 150 us; now 82 to 90, and 47 without
// the gate: the epilogue still outlasts the MMAs at such short k).
__device__ __forceinline__ float swiglu(float g, float u) {
    const float t = g * -1.4426950408889634f;
    const float left = fmaf(g, -1.4426950408889634f, -t) - g * 1.9259630e-8f;      // log2(e) = 1.44269502.. + 1.92596e-8
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    if (fabsf(t) < 128.f) e = fmaf(e * 0.6931471805599453f, left, e);
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return g * r * u;
}
// the sums r of 16 columns (gate and up: 2 x 16) -> output
template <int NA>
__device__ __forceinline__ void finish16(const MxGemmArgs& a, int m0, int count, int nn, const uint32_t* r, float al, float au) {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        v[j] = __uint_as_float(r[j]) * al;
        if constexpr (NA == 2) v[j] = swiglu(v[j], __uint_as_float(r[16 + j]) * au);
    }
    if (a.ytype == UQ_BF16) put16<__nv_bfloat16>(a, m0, count, nn, v);
    else if (a.ytype == UQ_FP16) put16<__half>(a, m0, count, nn, v);
    else put16<float>(a, m0, count, nn, v);
}

// Quantizes the tokens (at most FUSED_ROWS) of every step of this CTA straight into the ring, in the layouts TMA would
// have left.  A unit is 256 k of one row; a step has 2 * rows units, and warp w of the quantizers takes every fourth,
// eight lanes' values of four units requested ahead of the four being quantized.  Every CTA quantizes the same rows,
// which for few rows costs less than a launch of its own before (rule at mx_gemm_quantizes).
template <int FMT, class T>
__device__ __forceinline__ void quantize_tokens(const MxGemmArgs& a, Schedule sch, int w, uint32_t tokens0, int stage_bytes,
                                                uint32_t sf_off, uint32_t full0, uint32_t empty0, volatile int* abort_flag) {
    constexpr int TPS = STEP_K / mx_tile_k(FMT), AHEAD = 4;
    constexpr int LANES = mx_tile_k(FMT) / 8;                      // lanes of a scale tile
    const int lane = threadIdx.x & 31, per = 2 * a.rows;           // units of a step
    const T* x = static_cast<const T*>(a.xraw);
    const SixT six(a.tscale);
    int tiles = 0;
    for (; sch.more(); sch.advance()) ++tiles;
    const int steps = sch.k1 - sch.k0, total = (tiles * steps * per - w + QUANT_WARPS - 1) / QUANT_WARPS;
    int ls = w / per % steps, lu = w % per;                        // step and unit to be requested next
    Raw<T> cur[AHEAD] = {}, nxt[AHEAD] = {};
    auto request = [&](Raw<T> (&v)[AHEAD]) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int k = (sch.k0 + ls) * STEP_K + (lu & 1) * 256 + lane * 8;
            v[i] = Raw<T>{};
            if (k < a.K) v[i].load(x + (long long)(lu >> 1) * a.ldx + k);
            lu += QUANT_WARPS;
            while (lu >= per) {
                lu -= per;
                if (++ls == steps) ls = 0;
            }
        }
    };
    // the unit being quantized: its step's stage, how many steps have gone before, k step, unit of the step
    int n = w / per, s = n % a.stages, kt = sch.k0 + n % steps, un = w % per;
    uint32_t ph = 1u ^ (uint32_t)(n / a.stages & 1);
    after_prior_work(a);
    request(cur);
    for (int u = 0; u < total; u += AHEAD) {
        if (u + AHEAD < total) request(nxt);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (u + i >= total) break;
            if (n >= a.stages && !warp_wait(empty0 + s * 8, ph, a.fault, abort_flag)) {
                *abort_flag = 1;
                return;
            }
            const int r = un >> 1, h = un & 1;
            const uint32_t st = tokens0 + s * stage_bytes;
            uint32_t byte;
            const uint32_t q = quantize8<FMT>(cur[i], six, a.tscale, byte);
            if (kt * STEP_K + h * 256 + lane * 8 >= a.K) byte = 0; // (q is 0 there)
            const uint32_t word = scale_word<FMT>(byte, lane);
            // 128-byte column h of the row, 16-byte parts swizzled by the row
            asm volatile("st.shared.b32 [%0], %1;" :: "r"(st + h * (a.TN * 128) + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4), "r"(q) : "memory");
            if (lane % LANES == 0)
                asm volatile("st.shared.b32 [%0], %1;" :: "r"(st + sf_off + (h * (TPS / 2) + lane / LANES) * 512 + r * 16), "r"(word) : "memory");
            fence_proxy_async_smem();                              // the MMAs read through the async proxy
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(full0 + s * 8) : "memory");
            un += QUANT_WARPS;
            while (un >= per) {
                un -= per;
                ++n;
                if (++kt == sch.k1) kt = sch.k0;
                if (++s == a.stages) { s = 0; ph ^= 1; }
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) cur[i] = nxt[i];
    }
}

// FUSED: the tokens are quantized in the kernel
template <int FMT, int NA, bool FUSED>
__global__ void __launch_bounds__(FUSED ? FUSED_THREADS : THREADS, 1)
mx_gemm_kernel(const __grid_constant__ MxGemmMaps maps, const MxGemmArgs a) {
    constexpr int TPS = STEP_K / mx_tile_k(FMT);                   // scale tiles per step and 128 rows
    constexpr int A_BYTES = 128 * (STEP_K / 2), SF_BYTES = TPS * 512;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* head = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(head);            // [stages] operands and scales landed
    uint64_t* empty = full + MAX_STAGES;                           // [stages] consumed by the MMAs
    uint64_t* acc_full = empty + MAX_STAGES;                       // [2] accumulator complete
    uint64_t* acc_empty = acc_full + 2;                            // [2] accumulator read by the epilogue
    uint64_t* drain = acc_empty + 2;                               // after a timeout: the MMAs issued so far
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
    uint8_t* ring = head + HEAD;
    const int TN = a.TN, AB = a.accs;
    const int b_bytes = TN * (STEP_K / 2), stage_bytes = NA * A_BYTES + b_bytes + (NA + 1) * SF_BYTES;
    int* before = reinterpret_cast<int*>(ring + (size_t)a.stages * stage_bytes);   // the table, when rows are by expert

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    // One stage = step kt of a tile: both operands' codes and scale tiles, counted in bytes on full[s].  Columns and
    // scale tiles past K are filled with zeros.
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(full), empty0 = smem_u32(empty);
    auto load_codes = [&](uint32_t dst, const CUtensorMap* map, int row, int rows, int kt, uint32_t bar) {
        if (a.folded) {
            tma_3d(dst, map, 0, row, kt * 2, bar);
        } else {
            tma_2d(dst, map, kt * 256, row, bar);
            tma_2d(dst + rows * 128, map, kt * 256 + 128, row, bar);
        }
    };
    auto load_weights = [&](const Tile& t, int kt, int s) {
        const uint32_t st = ring0 + s * stage_bytes, bar = full0 + s * 8;
        expect_bytes(bar, NA * (A_BYTES + SF_BYTES));
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            load_codes(st + i * A_BYTES, i ? &maps.up : &maps.w, t.expert * a.N + t.nt * 128, 128, kt, bar);
            tma_3d(st + NA * A_BYTES + b_bytes + i * SF_BYTES, i ? &maps.up_scales : &maps.w_scales, 0, kt * TPS,
                   t.expert * a.row_tiles + t.nt, bar);
        }
    };
    auto load_tokens = [&](const Tile& t, int kt, int s) {
        const uint32_t st = ring0 + s * stage_bytes, bar = full0 + s * 8;
        expect_bytes(bar, b_bytes + SF_BYTES);
        load_codes(st + NA * A_BYTES, &maps.x, t.row0, TN, kt, bar);
        tma_3d(st + NA * A_BYTES + b_bytes + NA * SF_BYTES, &maps.x_scales, 0, kt * TPS,
               (a.offsets ? ((t.row0 - t.first) >> 7) + t.expert : 0) + (t.first >> 7), bar);
    };

    if (warp == 0) {
        if (lane < 6) asm volatile("prefetch.tensormap [%0];" :: "l"(&maps.w + lane) : "memory");
        if (a.offsets) {
            after_prior_work(a);
            token_tiles(a, before);
        }
        if (lane < a.stages) {
            mbar_init(&full[lane], FUSED ? 1 + 2 * a.rows : 2);
            mbar_init(&empty[lane], 1);
        } else if (lane >= 30) {
            mbar_init(&acc_full[lane - 30], 1);
            mbar_init(&acc_empty[lane - 30], 4);
        } else if (lane == 29) {
            mbar_init(drain, 1);
            *abort_flag = 0;
        }
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    __syncthreads();
    const int tt_all = a.offsets ? before[a.experts] : (a.rows + TN - 1) / TN;
    Schedule sch(a, tt_all);
    constexpr uint32_t SF_COLS = (NA + 1) * TPS * 4;               // scale columns of a stage
    constexpr int TMEM_WARPS = 1 + 4;                              // warps that use tensor memory
    uint32_t tmem = 0;
    if (warp >= 1 && warp <= 5) {
        if (warp == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         :: "r"(smem_u32(tmem_ptr)), "r"((uint32_t)a.tmem_cols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        fence_before();
        asm volatile("bar.sync 1, %0;" :: "n"(TMEM_WARPS * 32) : "memory");
        fence_after();
        tmem = (uint32_t)uniform((int)*tmem_ptr);
        if (warp == 1) launch_dependents(a);
    }

    if (warp == 0 || (!FUSED && warp == 6)) {
        // ------------------------------------------------------------ producers
        // The weights do not depend on the kernel before, the tokens may.
        const bool tokens = warp == 6;
        if (tokens) after_prior_work(a);
        int issued = 0, s = 0;
        uint32_t ph = 1;                                           // empty[] of the first round counts as free
        bool ok = true;
        for (; ok && sch.more(); sch.advance()) {
            Tile t = find_tile(a, before, tt_all, sch.tile);
            t.row0 = uniform(t.row0);
            t.expert = uniform(t.expert);
            for (int kt = sch.k0; kt < sch.k1; ++kt) {
                if (issued >= a.stages && !warp_wait(empty0 + s * 8, ph, a.fault, abort_flag)) {
                    ok = false;
                    break;
                }
                if (tokens) load_tokens(t, kt, s);
                else load_weights(t, kt, s);
                ++issued;
                if (++s == a.stages) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) *abort_flag = 1;
        // let the last copies land before the CTA can leave (bounded; after a timeout a stage may lack its other half)
        for (int j = issued - 1; j >= 0 && j >= issued - a.stages; --j)
            mbar_wait_bounded(&full[j % a.stages], (uint32_t)((j / a.stages) & 1), a.fault, FAULT_MX_WAIT);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        constexpr int PER = FMT == UQ_MXFP4 ? 2 : 1;               // MMAs per scale tile
        const uint32_t sf0 = tmem + AB * NA * TN;
        const int full_steps = a.K / STEP_K;
        int s = 0, n = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (; ok && sch.more(); sch.advance(), ++n) {
            const Tile t = find_tile(a, before, tt_all, sch.tile);
            const uint32_t idesc = block_idesc<FMT>((uniform(t.rows) + 15) / 16 * 16);
            const uint32_t xshift = (uint32_t)(uniform(t.first) & 127) >> 5;   // first scale column of the tile in its 128 rows
            const int buf = AB == 2 ? n & 1 : 0;
            const uint32_t acc = tmem + buf * NA * TN;
            // the epilogue has read this accumulator's tile before (its first use counts as read)
            const uint32_t aph = (uint32_t)((AB == 2 ? n >> 1 : n) & 1) ^ 1u;
            if (!warp_wait(smem_u32(&acc_empty[buf]), aph, a.fault, abort_flag)) ok = false;
            fence_after();
            uint32_t on = 0;
            for (int kt = sch.k0; ok && kt < sch.k1; ++kt) {
                if (!warp_wait(full0 + s * 8, ph, a.fault, abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t st = ring0 + s * stage_bytes;
                const uint32_t al = desc_lo(st), bl = al + NA * (A_BYTES >> 4), sl = bl + (b_bytes >> 4);
                const uint32_t col = sf0 + s * SF_COLS, cb = col + NA * TPS * 4, cu = cb + xshift;
                // scale tile j: its first MMA is 32-byte part q % 4 of the 128-byte column q / 4
                auto issue = [&](int j, uint32_t two) {
                    const int q = j * PER;
                    const uint32_t ao = (q >> 2) * (16384 >> 4) + 2 * (q & 3), bo = bl + (q >> 2) * (TN * 8) + 2 * (q & 3);
                    issue_tile<FMT>(acc, al + ao, bo, sl + j * 32, sl + NA * (SF_BYTES >> 4) + j * 32, col + j * 4, cb + j * 4,
                                    cu + j * 4, idesc, on, two);
                    if constexpr (NA == 2)
                        issue_more<FMT>(acc + TN, al + (A_BYTES >> 4) + ao, bo, sl + (SF_BYTES >> 4) + j * 32,
                                        col + (TPS + j) * 4, cu + j * 4, idesc, on, two);
                    on = 1;
                };
                if (kt < full_steps) {
#pragma unroll
                    for (int j = 0; j < TPS; ++j) issue(j, 1);
                } else {
                    const int mmas = (a.K - kt * STEP_K + 63) >> 6;                // K ends inside the step
                    for (int j = 0; j * PER < mmas; ++j) issue(j, j * PER + 1 < mmas);
                }
                commit(empty0 + s * 8);
                if (++s == a.stages) { s = 0; ph ^= 1; }
            }
            commit(smem_u32(&acc_full[buf]));
        }
        if (!ok) {
            *abort_flag = 1;
            __syncwarp();
            commit(smem_u32(drain));
            mbar_wait_bounded(drain, 0, a.fault, FAULT_MX_WAIT);
        }
    } else if (FUSED && warp >= 6) {
        // ------------------------------------------------------------ quantizers
        if constexpr (FUSED) {
            const uint32_t tokens0 = ring0 + NA * A_BYTES, sf_off = b_bytes + NA * SF_BYTES;
            if (a.xtype == UQ_BF16)
                quantize_tokens<FMT, __nv_bfloat16>(a, sch, warp - 6, tokens0, stage_bytes, sf_off, full0, empty0, abort_flag);
            else if (a.xtype == UQ_FP16)
                quantize_tokens<FMT, __half>(a, sch, warp - 6, tokens0, stage_bytes, sf_off, full0, empty0, abort_flag);
            else
                quantize_tokens<FMT, float>(a, sch, warp - 6, tokens0, stage_bytes, sf_off, full0, empty0, abort_flag);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue: lane = row of the weight tile
        const int q = warp & 3, row = q * 32 + lane, et = threadIdx.x - 64;
        if (a.offsets) {
            after_prior_work(a);
            zero_tail(a, blockIdx.x * 128LL + et, gridDim.x * 128LL);
        }
        for (int n = 0; sch.more(); sch.advance(), ++n) {
            const Tile t = find_tile(a, before, tt_all, sch.tile);
            const int buf = AB == 2 ? n & 1 : 0;
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * NA * TN;
            // after a timeout the tiles are walked without waiting
            if (!warp_wait(smem_u32(&acc_full[buf]), (uint32_t)((AB == 2 ? n >> 1 : n) & 1), a.fault, abort_flag)) *abort_flag = 1;
            __syncwarp();
            fence_after();
            const int nn = t.nt * 128 + row;
            const float al = a.alpha * (a.alpha_e ? ld_written(a.alpha_e + t.expert) : 1.f);
            const float au = a.alpha * (a.alpha_up ? ld_written(a.alpha_up + t.expert) : 1.f);
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
                if (a.S > 1) {
                    // the MMAs are done with the ring: the sums are left there, [token][weight tile][row]
                    float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
                    for (int j = 0; j < NA * 16; ++j)
                        if (c + (j & 15) < t.rows) sums[((c + (j & 15)) * NA + (j >> 4)) * 128 + row] = __uint_as_float(r[j]);
                } else {
                    finish16<NA>(a, t.row0 + c, t.rows - c, nn, r, al, au);
                }
            }
        }
    }
    __syncwarp();
    // Tensor memory is given back before the cluster waits for its CTAs: one that holds it waits for nobody, so CTAs
    // whose allocation waits for it always get it.
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"((uint32_t)a.tmem_cols) : "memory");
    if (a.S > 1) {
        cluster_sync();
        const Schedule mine(a, tt_all);
        if (mine.more()) {
            const Tile t = find_tile(a, before, tt_all, mine.tile);
            const float al = a.alpha * (a.alpha_e ? ld_written(a.alpha_e + t.expert) : 1.f);
            const float au = a.alpha * (a.alpha_up ? ld_written(a.alpha_up + t.expert) : 1.f);
            // a thread takes four neighbouring outputs of a token; the CTAs' sums are all requested before they are added
            for (int it = (int)cluster_rank() * (int)blockDim.x + threadIdx.x; it < t.rows * 32; it += a.S * (int)blockDim.x) {
                const int c = it >> 5, r = (it & 31) * 4, nn = t.nt * 128 + r;
                if (nn >= a.N) continue;
                float4 p[MAX_SPLIT * NA];
#pragma unroll
                for (int k = 0; k < MAX_SPLIT; ++k)
#pragma unroll
                    for (int h = 0; h < NA; ++h)
                        p[k * NA + h] = k < a.S ? ld_cluster4(ring0 + ((c * NA + h) * 128 + r) * 4, k) : make_float4(0.f, 0.f, 0.f, 0.f);
                float v[4] = {}, u[4] = {};
#pragma unroll
                for (int k = 0; k < MAX_SPLIT; ++k) {
                    const float4 x = p[k * NA];
                    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                    if constexpr (NA == 2) {
                        const float4 y = p[k * NA + 1];
                        u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] *= al;
                    if constexpr (NA == 2) v[i] = swiglu(v[i], u[i] * au);
                }
                store4(a, (long long)(t.row0 + c) * a.N + nn, a.N - nn, v);
            }
        }
        cluster_sync();                                            // no CTA leaves while another reads its sums
    }
}

// ------------------------------------------------------------------------------------------------
// Pairs of CTAs (cta_group::2) for many rows.  One MMA spans two SMs: 256 weight rows (128 in each SM's tensor memory) x
// up to 256 tokens, each SM holding half of the token rows in shared memory.  With one SM alone a 128 x 128 x 64 MMA
// reads 8 KB of shared memory in the 64 cycles it computes, all that shared memory delivers, beside the copies that
// refill it; the pair's 256 x 256 MMA reads 8 KB per SM in 128 cycles, and every byte loaded is used twice as often.
// The even CTA issues the scale copies and the MMAs for both; TMA loads of both count their bytes on its full[]
// barriers; commits arrive in both.  A tile's accumulator is 256 columns (tokens; or 128 gate + 128 up); two of them
// overlap in as many columns as the scales take (MXFP4 48, NVFP4 96, in two halves that alternate by step), and the
// epilogue reads those columns first, so the next tile's MMAs wait for a fifth to a third of an epilogue only.
constexpr int PAIR_STEP = 256;
template <int FMT, int NA> struct Pair {
    static constexpr int TN = 256 / NA;                            // tokens per tile
    static constexpr int TPS = PAIR_STEP / mx_tile_k(FMT);         // scale tiles per step and 128 rows
    static constexpr int XT = TN / 128;                            // row tiles of the tokens' scales
    static constexpr int A = NA * 128 * 128, B = TN / 2 * 128, SA = NA * TPS * 512, SB = XT * TPS * 512;
    static constexpr int STAGE = A + B + SA + SB;
    static constexpr int STAGES = 218 * 1024 / STAGE;
    static constexpr int SF = (NA + XT) * TPS * 4;                 // scale columns of a step
    static constexpr int OVER = 2 * SF;                            // columns the two accumulators share
    static_assert(STAGE % 1024 == 0 && STAGES <= MAX_STAGES, "stage layout");
};

__device__ __forceinline__ void pair_tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(UQ_ELECT "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];\n\t}"
                 :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
// The instructions that share a scale tile of the pair's operands: the copies of its three scale tiles (NA = 1: weights,
// tokens' first and second 128 rows; NA = 2: gate, up, tokens) to columns c0, c1, c2, in both CTAs from their own shared
// memory, then the MMAs as issue_tile issues them.  ca / cb: the scale columns of weights and tokens.
template <int FMT, int NA>
__device__ __forceinline__ void pair_tile(uint32_t d, uint32_t a, uint32_t b, uint32_t s0, uint32_t s1, uint32_t s2, uint32_t c0,
                                          uint32_t c1, uint32_t c2, uint32_t cb, uint32_t idesc, uint32_t on, uint32_t two) {
#define UQ_PAIR_HEAD \
    "{\n\t.reg .pred p, e, f, t;\n\t.reg .b64 da, db, dc, x, y, z;\n\t.reg .b32 i2, d1;\n\t" \
    "mov.b64 da, {%1, " UQ_OPERAND_HI "};\n\tmov.b64 db, {%2, " UQ_OPERAND_HI "};\n\t" \
    "mov.b64 x, {%3, " UQ_SCALES_HI "};\n\tmov.b64 y, {%4, " UQ_SCALES_HI "};\n\tmov.b64 z, {%5, " UQ_SCALES_HI "};\n\t" \
    "setp.ne.b32 p, %11, 0;\n\tsetp.eq.b32 t, %10, %10;\n\telect.sync _|e, 0xffffffff;\n\t" \
    "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%6], x;\n\t" \
    "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%7], y;\n\t" \
    "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%8], z;\n\t"
#define UQ_PAIR_ARGS \
    :: "r"(d), "r"(a), "r"(b), "r"(s0), "r"(s1), "r"(s2), "r"(c0), "r"(c1), "r"(c2), "r"(cb), "r"(idesc), "r"(on), "r"(two) \
    : "memory"
    if constexpr (FMT == UQ_MXFP4 && NA == 1)
        asm volatile(UQ_PAIR_HEAD "or.b32 i2, %10, 0x40000020;\n\tsetp.ne.and.b32 f, %12, 0, e;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %10, [%6], [%9], p;\n\t"
                     "add.s64 da, da, 2;\n\tadd.s64 db, db, 2;\n\t"
                     "@f tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, i2, [%6], [%9], t;\n\t}"
                     UQ_PAIR_ARGS);
    else if constexpr (FMT == UQ_MXFP4)                            // the up tile: 128 rows (16 KB) and 128 columns on
        asm volatile(UQ_PAIR_HEAD "or.b32 i2, %10, 0x40000020;\n\tsetp.ne.and.b32 f, %12, 0, e;\n\t"
                     "add.s32 d1, %0, 128;\n\tadd.s64 dc, da, 1024;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %10, [%6], [%9], p;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [d1], dc, db, %10, [%7], [%9], p;\n\t"
                     "add.s64 da, da, 2;\n\tadd.s64 db, db, 2;\n\tadd.s64 dc, dc, 2;\n\t"
                     "@f tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, i2, [%6], [%9], t;\n\t"
                     "@f tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [d1], dc, db, i2, [%7], [%9], t;\n\t}"
                     UQ_PAIR_ARGS);
    else if constexpr (NA == 1)
        asm volatile(UQ_PAIR_HEAD
                     "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], da, db, %10, [%6], [%9], p;\n\t}"
                     UQ_PAIR_ARGS);
    else
        asm volatile(UQ_PAIR_HEAD "add.s32 d1, %0, 128;\n\tadd.s64 dc, da, 1024;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], da, db, %10, [%6], [%9], p;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [d1], dc, db, %10, [%7], [%9], p;\n\t}"
                     UQ_PAIR_ARGS);
#undef UQ_PAIR_HEAD
#undef UQ_PAIR_ARGS
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(addr) : "memory");
}

template <int FMT, int NA>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
mx_gemm_pair_kernel(const __grid_constant__ MxGemmMaps maps, const MxGemmArgs a) {
    using P = Pair<FMT, NA>;
    constexpr int TN = P::TN, TPS = P::TPS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* head = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(head);            // [STAGES] both CTAs' loads landed (even CTA's)
    uint64_t* empty = full + MAX_STAGES;                           // [STAGES] consumed by the MMAs
    uint64_t* acc_full = empty + MAX_STAGES;                       // [2] accumulator complete
    uint64_t* acc_free = acc_full + 2;                             // the shared columns have been read (even CTA's)
    uint64_t* drain = acc_free + 1;
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_ptr + 1);
    uint8_t* ring = head + HEAD;
    int* before = reinterpret_cast<int*>(ring + P::STAGES * P::STAGE);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(full), empty0 = smem_u32(empty);

    if (warp == 0) {
        if (lane < 6) asm volatile("prefetch.tensormap [%0];" :: "l"(&maps.w + lane) : "memory");
        if (a.offsets) {
            after_prior_work(a);
            token_tiles(a, before);
        }
        if (lane == 0) {
            for (int s = 0; s < P::STAGES; ++s) {
                mbar_init(&full[s], 2);
                mbar_init(&empty[s], 1);
            }
            for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1);
            mbar_init(acc_free, 8);
            mbar_init(drain, 1);
            *abort_flag = 0;
            fence_barrier_init();
            fence_proxy_async_smem();
        }
        __syncwarp();
    }
    __syncthreads();
    cluster_sync();                                                // the other CTA's barriers are ready
    const int tt_all = a.offsets ? before[a.experts] : (a.rows + TN - 1) / TN;
    const int tiles = tt_all * a.NT, stride = gridDim.x >> 1;
    uint32_t tmem = 0;
    if (warp >= 1 && warp <= 5) {
        if (warp == 1) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(tmem_ptr)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
        fence_before();
        asm volatile("bar.sync 1, 160;" ::: "memory");
        fence_after();
        tmem = (uint32_t)uniform((int)*tmem_ptr);
        if (warp == 1) launch_dependents(a);
    }
    // the token columns a tile's MMAs use: a multiple of 16, half of the rows in each CTA
    auto columns = [&](const Tile& t) { return (uniform(t.rows) + 15) / 16 * 16; };

    if (warp == 0 || warp == 6) {
        // ------------------------------------------------------------ producers
        const bool tokens = warp == 6;
        if (tokens) after_prior_work(a);
        const uint32_t lead_full0 = cluster_addr(full0, 0);
        int issued = 0, s = 0;
        uint32_t ph = 1;                                           // empty[] of the first round counts as free
        bool ok = true;
        for (int tile = blockIdx.x >> 1; ok && tile < tiles; tile += stride) {
            const Tile t = find_tile(a, before, tt_all, tile);
            const int e = uniform(t.expert), n = t.nt * 256 + (int)rank * 128;
            const int row = uniform(t.row0) + (int)rank * (columns(t) >> 1);
            const int xtile = (a.offsets ? (uniform(t.row0 - t.first) >> 7) + e : 0) + (uniform(t.first) >> 7);
            for (int kt = 0; kt < a.steps; ++kt) {
                if (issued >= P::STAGES && !warp_wait<true>(empty0 + s * 8, ph, a.fault, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t st = ring0 + s * P::STAGE, bar = lead_full0 + s * 8;
                if (rank == 0) expect_bytes(full0 + s * 8, 2 * (tokens ? P::B + P::SB : P::A + P::SA));
                if (tokens) {
                    pair_tma_2d(st + P::A, &maps.x, kt * 128, row, bar);
                    pair_tma_3d(st + P::A + P::B + P::SA, &maps.x_scales, 0, kt * TPS, xtile, bar);
                } else {
#pragma unroll
                    for (int i = 0; i < NA; ++i) {
                        pair_tma_2d(st + i * (128 * 128), i ? &maps.up : &maps.w, kt * 128, e * a.N + n, bar);
                        pair_tma_3d(st + P::A + P::B + i * TPS * 512, i ? &maps.up_scales : &maps.w_scales, 0, kt * TPS,
                                    e * a.row_tiles + (n >> 7), bar);
                    }
                }
                ++issued;
                if (++s == P::STAGES) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) *abort_flag = 1;
        // Let the last copies land before the CTA can leave: both CTAs' are counted on the even one's barriers, and the
        // CTAs leave together.
        if (rank == 0)
            for (int j = issued - 1; j >= 0 && j >= issued - P::STAGES; --j)
                mbar_wait_bounded(&full[j % P::STAGES], (uint32_t)((j / P::STAGES) & 1), a.fault, FAULT_MX_WAIT);
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMA issue
        constexpr int PER = FMT == UQ_MXFP4 ? 2 : 1;               // MMAs per scale tile
        const int full_steps = a.K / PAIR_STEP;
        int s = 0, n = 0;
        uint32_t ph = 0, half = 0;
        bool ok = true;
        for (int tile = blockIdx.x >> 1; ok && tile < tiles; tile += stride, ++n) {
            const Tile t = find_tile(a, before, tt_all, tile);
            const uint32_t idesc = block_idesc<FMT>(columns(t)) + (1u << 27);      // M = 256
            const uint32_t acc = tmem + (n & 1) * (256 - P::OVER);
            // the epilogue of the tile before has read the shared columns
            if (n && !warp_wait<true>(smem_u32(acc_free), (uint32_t)(n - 1) & 1, a.fault, abort_flag)) ok = false;
            fence_after();
            uint32_t on = 0;
            for (int kt = 0; ok && kt < a.steps; ++kt) {
                if (!warp_wait<true>(full0 + s * 8, ph, a.fault, abort_flag)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint32_t al = desc_lo(ring0 + s * P::STAGE), bl = al + (P::A >> 4), sl = bl + (P::B >> 4);
                const uint32_t sx = sl + (P::SA >> 4), col = tmem + 512 - P::OVER + half * P::SF, cx = col + NA * TPS * 4;
                // scale tile j: its first MMA is 32-byte part j * PER of the column
                auto issue = [&](int j, uint32_t two) {
                    const uint32_t at = 2 * j * PER;
                    // the tokens' two row tiles of one scale tile lie together: 8 columns
                    if constexpr (NA == 1)
                        pair_tile<FMT, 1>(acc, al + at, bl + at, sl + j * 32, sx + j * 32, sx + (TPS + j) * 32, col + j * 4,
                                          cx + j * 8, cx + j * 8 + 4, cx + j * 8, idesc, on, two);
                    else
                        pair_tile<FMT, 2>(acc, al + at, bl + at, sl + j * 32, sl + (TPS + j) * 32, sx + j * 32, col + j * 4,
                                          col + (TPS + j) * 4, cx + j * 4, cx + j * 4, idesc, on, two);
                    on = 1;
                };
                if (kt < full_steps) {
#pragma unroll
                    for (int j = 0; j < TPS; ++j) issue(j, 1);
                } else {
                    const int mmas = (a.K - kt * PAIR_STEP + 63) >> 6;             // K ends inside the step
                    for (int j = 0; j * PER < mmas; ++j) issue(j, j * PER + 1 < mmas);
                }
                half ^= 1;
                pair_commit(empty0 + s * 8);
                if (++s == P::STAGES) { s = 0; ph ^= 1; }
            }
            pair_commit(smem_u32(&acc_full[n & 1]));
        }
        if (!ok) {
            *abort_flag = 1;
            __syncwarp();
            pair_commit(smem_u32(drain));
            mbar_wait_bounded(drain, 0, a.fault, FAULT_MX_WAIT);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue: lane = weight row
        const int q = warp & 3, row = q * 32 + lane;
        if (a.offsets) {
            after_prior_work(a);
            zero_tail(a, blockIdx.x * 128LL + threadIdx.x - 64, gridDim.x * 128LL);
        }
        const uint32_t lead_free = cluster_addr(smem_u32(acc_free), 0);
        int n = 0;
        for (int tile = blockIdx.x >> 1; tile < tiles; tile += stride, ++n) {
            const Tile t = find_tile(a, before, tt_all, tile);
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (n & 1) * (256 - P::OVER);
            // after a timeout the tiles are walked without waiting
            if (!warp_wait<true>(smem_u32(&acc_full[n & 1]), (uint32_t)(n >> 1) & 1, a.fault, abort_flag)) *abort_flag = 1;
            __syncwarp();
            fence_after();
            const int nn = t.nt * 256 + (int)rank * 128 + row;
            const float al = a.alpha * (a.alpha_e ? ld_written(a.alpha_e + t.expert) : 1.f);
            const float au = a.alpha * (a.alpha_up ? ld_written(a.alpha_up + t.expert) : 1.f);
            // The first accumulator shares its last columns, the second its first: those are read, and given free,
            // before anything is written.
            const int c0 = n & 1 ? 0 : TN - P::OVER;
            {
                uint32_t r[P::OVER / 16][NA * 16];
#pragma unroll
                for (int i = 0; i < P::OVER / 16; ++i)
#pragma unroll
                    for (int h = 0; h < NA; ++h)
                        tmem_ld16(acc + h * TN + c0 + i * 16, *reinterpret_cast<uint32_t(*)[16]>(r[i] + 16 * h));
                tmem_ld_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(lead_free);
#pragma unroll
                for (int i = 0; i < P::OVER / 16; ++i)
                    if (c0 + i * 16 < t.rows)
                        finish16<NA>(a, t.row0 + c0 + i * 16, t.rows - c0 - i * 16, nn, r[i], al, au);
            }
            for (int i = P::OVER; i < TN; i += 16) {
                const int c = c0 + i < TN ? c0 + i : c0 + i - TN;
                if (c >= t.rows) continue;
                uint32_t r[NA * 16];
#pragma unroll
                for (int h = 0; h < NA; ++h) tmem_ld16(acc + h * TN + c, *reinterpret_cast<uint32_t(*)[16]>(r + 16 * h));
                tmem_ld_wait();
                finish16<NA>(a, t.row0 + c, t.rows - c, nn, r, al, au);
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    cluster_sync();                                                // both CTAs are done with each other's memory
    fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
}

// codes [rows][K/2] as bytes, 128-byte columns x `box` rows, 128-byte swizzle; folded (K a multiple of 256): the columns
// are the third dimension and a box takes two of them
bool codes_map(CUtensorMap* m, const uint8_t* codes, long long rows, int K, int box, bool folded) {
    cuuint64_t dims[3] = {folded ? 128ull : (cuuint64_t)K / 2, (cuuint64_t)rows, (cuuint64_t)K / 256};
    cuuint64_t strides[2] = {(cuuint64_t)K / 2, 128};
    cuuint32_t b[3] = {128, (cuuint32_t)box, 2};
    cuuint32_t es[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, folded ? 3 : 2, const_cast<uint8_t*>(codes), dims, strides, b, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// scale tiles [row tiles][ktiles][512 bytes], boxes of box_rows row tiles x one step's tiles
bool scales_map(CUtensorMap* m, const uint8_t* scales, long long row_tiles, int ktiles, int tps, int box_rows) {
    cuuint64_t dims[3] = {64, (cuuint64_t)ktiles, (cuuint64_t)row_tiles};
    cuuint64_t strides[2] = {512, (cuuint64_t)ktiles * 512};
    cuuint32_t b[3] = {64, (cuuint32_t)tps, (cuuint32_t)box_rows};
    cuuint32_t es[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 3, const_cast<uint8_t*>(scales), dims, strides, b, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int NA>
cudaError_t launch(const MxGemmMaps& maps, const MxGemmArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas);
    cfg.blockDim = dim3(a.xraw ? FUSED_THREADS : THREADS);
    cfg.dynamicSmemBytes = a.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (a.S > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = a.S;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (a.wait) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    auto go = [&](auto kernel, Done& done) {
        const cudaError_t e = configure(kernel, done);
        return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kernel, maps, a) : e;
    };
    static Done pair_done = {}, one_done = {}, fused_done = {};
    if (a.pair) return go(mx_gemm_pair_kernel<FMT, NA>, pair_done);
    if constexpr (NA == 1)
        if (a.xraw) return go(mx_gemm_kernel<FMT, 1, true>, fused_done);
    return go(mx_gemm_kernel<FMT, NA, false>, one_done);
}

// Stage count and size of the pair kernel.
template <int NA> void pair_ring(int fmt, MxGemmArgs& a) {
    a.TN = 256 / NA;
    a.smem = 1024 + HEAD + (fmt == UQ_MXFP4 ? Pair<UQ_MXFP4, NA>::STAGES * Pair<UQ_MXFP4, NA>::STAGE
                                            : Pair<UQ_NVFP4, NA>::STAGES * Pair<UQ_NVFP4, NA>::STAGE);
}

// Clusters of s CTAs that run at the same time, one CTA per SM: fewer than SMs / s, since a cluster stays within a GPC
// (16 clusters of 8 took two rounds, 15 us against 9 for clusters of 4).  Asked once per device.
int clusters_at_once(int s) {
    static std::atomic<int> known[64][MAX_SPLIT + 1] = {};
    static Done done = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][s].load(std::memory_order_relaxed);
    if (n) return n - 1;
    if (configure(mx_gemm_kernel<UQ_MXFP4, 1, false>, done) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = 220 * 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, mx_gemm_kernel<UQ_MXFP4, 1, false>, &cfg) != cudaSuccess) return 0;
    known[dev][s].store(n + 1, std::memory_order_relaxed);
    return n;
}

// CTAs per tile, by the time in steps: a CTA's own, longer where all together ask for more than memory delivers (CTAs
// beyond `enough` share it: each takes about 100 GB/s), and for a split the cluster's start and end and the sums' way
// through it, CTA by CTA a share of the token columns.  Ties go to the larger split.  Measured, weights read from DRAM, us
// unsplit / best split, 4 rows, MXFP4: N = 1024, K = 2048 5.0 / 5.5, 4096 6.6 / 6.1, 8192 9.3 / 6.7; N = 4096, K = 4096 6.9 /
// 7.3, 8192 9.6 / 8.5, 14336 13.7 / 10.6; N = 8192, K = 8192 10.8 / 11.2; 64 rows, N = 4096, K = 8192 10.8 / 10.0; gated,
// 8 rows for 8 experts of 1024 x 4096 12.9 / 12.9, x 8192 20.9 / 18.5.
int split_of(long long tiles, int steps, int tokens, bool gated, int sms) {
    if (tiles * 2 > sms) return 1;
    const double enough = gated ? 96 : 70, fixed = gated ? 2.75 : 5;
    int best = 1;
    double least = 0;
    for (int s = 1; s <= std::min(MAX_SPLIT, steps); ++s) {
        if (s > 1 && tiles > clusters_at_once(s)) continue;
        const double t = (steps + s - 1) / s * std::max(1.0, tiles * s / enough) + (s > 1 ? fixed + tokens / (8.0 * s) : 0);
        if (s == 1 || t <= least) best = s, least = t;
    }
    return best;
}

// Whether pairs of CTAs are the faster of the two kernels.
//   One weight for all rows: by waves.  A wave of 128 x 128 tiles takes 715 cycles per 512 k (NVFP4 842), one of 256 x 256
// pair tiles 1026 (less with fewer than 256 token columns; both measured alone), and the pairs' start and end cost about
// 3000 cycles more; where one wave of 128 x 64 tiles does it, pairs were slower at every size.  Measured, us single /
// pairs, MXFP4: N = K = 8192: M = 256 12.1 / 15.8, 512 19.7 / 16.5, 2048 60.7 / 49.7; N = K = 4096: M = 256 7.4 / 11.3, 512
// 8.8 / 11.3, 1024 12.8 / 11.9, 2048 22.6 / 18.6; 14336 x 4096: M = 128 9.3 / 11.3, 256 14.4 / 13.4, 512 18.6 / 19.5, 1024
// 30.8 / 25.0.
//   Rows by expert: from 128 rows an expert on, where there are pair tiles for every pair.  Measured, 8 experts of 4096 x
// 4096, mean rows 64 16.5 / 18.7, 128 20.7 / 20.2, 192 26.7 / 20.7, 512 45.3 / 35.8; gated 128 51.4 / 43.2; 32 experts of
// 2048 x 2048: 64 20.4 / 22.7, 128 24.9 / 24.7, 256 35.1 / 36.9 (the one of these that the rule takes wrongly: it does not
// weigh a short K, where a pair tile's fixed 1900 cycles are half of its steps), 512 51.6 / 47.2.
bool pays_in_pairs(int fmt, bool gated, const MxGemmArgs& a, int mean, int sms) {
    const long long pair_n = (a.N + 255) / 256;
    if (a.offsets) return mean >= 128 && 2 * pair_n * (a.rows / (gated ? 128 : 256) + a.experts / 2) >= sms;
    if (a.rows <= 64 || (long long)((a.N + 127) / 128) * ((a.rows + 63) / 64) <= sms) return false;
    const long long steps = (a.K + 511) / 512, tiles = (long long)((a.N + 127) / 128) * ((a.rows + 127) / 128);
    const long long waves = (tiles + sms - 1) / sms, pair_waves = (2 * pair_n * ((a.rows + 255) / 256) + sms - 1) / sms;
    const long long single = waves * steps * (fmt == UQ_MXFP4 ? 715 : 842);
    return pair_waves * steps * 1026 * std::min(a.rows, 256) / 256 + 3000 < single;
}

// Tiles, ring and grid of one product.
void plan(int fmt, bool gated, MxGemmArgs& a, int sms) {
    const int NA = gated ? 2 : 1;
    a.ktiles = mx_ktiles(a.K, fmt);
    a.row_tiles = (a.N + 127) / 128;
    const int table = a.offsets ? table_bytes(a.experts) : 0;
    // token tile: the rows an expert gets on average (all of them when there is one).  Under 64 only where no second
    // tile can follow: a tile's scale columns then always start at an even column.
    const int mean = a.offsets ? (a.rows + a.experts - 1) / a.experts : a.rows;
    a.pair = pays_in_pairs(fmt, gated, a, mean, sms);
    if (a.pair) {
        if (gated) pair_ring<2>(fmt, a);
        else pair_ring<1>(fmt, a);
        a.smem += table;
        a.steps = (a.K + PAIR_STEP - 1) / PAIR_STEP;
        a.NT = (a.N + 255) / 256;
        a.group = 8;
        a.S = 1;
        const long long most = a.NT * (a.offsets ? std::min((long long)a.rows, a.rows / a.TN + (long long)a.experts)
                                                 : (a.rows + a.TN - 1) / a.TN);
        a.ctas = (int)std::min(2 * most, (long long)(sms & ~1));
        return;
    }
    const int tps = STEP_K / mx_tile_k(fmt);
    a.steps = (a.K + STEP_K - 1) / STEP_K;
    a.group = 16;
    a.NT = (a.N + 127) / 128;
    // token tiles: exact, or the most that any counts give
    const auto token_tiles = [&](int tn) {
        return a.offsets ? std::min((long long)a.rows, a.rows / tn + (long long)a.experts) : (long long)((a.rows + tn - 1) / tn);
    };
    // 64 columns also for more rows where one wave takes all tiles: the epilogue, the longer part of such a call, halves
    // (MXFP4 us, 128 / 64 columns: 512 x 2048 x 2048 6.8 / 6.0, 256 x 4096 x 8192 11.7 / 10.3, 96 x 8192 x 4096 7.8 / 7.4)
    a.TN = a.rows <= 16 ? 16 : (a.rows <= 32 ? 32 : (mean <= 64 || token_tiles(64) * a.NT <= sms ? 64 : 128));
    const long long tiles = token_tiles(a.TN) * a.NT;
    a.S = split_of(tiles, a.steps, std::min(a.TN, mean), gated, sms);
    a.share = a.steps / a.S;
    a.extra = a.steps % a.S;
    a.ctas = a.S > 1 ? (int)tiles * a.S : (int)std::min(tiles, (long long)sms);
    a.folded = a.K % 256 == 0;
    const int stage_bytes = NA * 128 * (STEP_K / 2) + a.TN * (STEP_K / 2) + (NA + 1) * tps * 512;
    // tensor memory: two accumulators where 512 columns hold them beside the scales of the stages that fit (of three)
    const int sf = (NA + 1) * tps * 4, fit = std::min((222 * 1024 - HEAD - table) / stage_bytes, MAX_STAGES);
    a.accs = 2 * NA * a.TN + std::min(fit, 3) * sf <= 512 ? 2 : 1;
    a.stages = std::min(fit, (512 - a.accs * NA * a.TN) / sf);
    const int cols = a.accs * NA * a.TN + a.stages * sf;
    a.tmem_cols = cols <= 64 ? 64 : (cols <= 128 ? 128 : (cols <= 256 ? 256 : 512));
    a.smem = 1024 + HEAD + a.stages * stage_bytes + table;
}

}  // namespace

// One launch instead of two up to FUSED_ROWS tokens: a call then takes 7.4 us of host time instead of 10, and on the GPU
// (graph replay, weights from DRAM, us one launch / two) MXFP4 14336 x 4096 M = 1 9.0 / 9.5, 2 8.8 / 10.2, 3 9.5 / 10.1, 4
// 10.8 / 10.1; 4096 x 14336 10.3 / 11.4, 10.5 / 11.4, 11.1 / 11.5, 12.4 / 11.6; 4096 x 4096 6.9 / 8.0, 7.2 / 8.0, 7.8 / 8.1,
// 9.0 / 8.0; 1024 x 4096 5.6 / 6.7 to 5.8 / 6.9.  From 4 tokens on the quantizing warps hold up long streams of weights.
bool mx_gemm_quantizes(int rows) { return rows <= FUSED_ROWS; }

cudaError_t launch_mx_gemm(int fmt, const uint8_t* xcodes, const uint8_t* wcodes, const uint8_t* wcodes_up,
                           MxGemmArgs a, int sms, cudaStream_t st) {
    if (!encode_fn()) return cudaErrorNotSupported;
    plan(fmt, wcodes_up != nullptr, a, sms);
    MxGemmMaps m;
    const int tps = (a.pair ? PAIR_STEP : STEP_K) / mx_tile_k(fmt);
    const long long wrows = (long long)a.experts * a.N, wtiles = (long long)a.experts * a.row_tiles;
    bool ok = codes_map(&m.w, wcodes, wrows, a.K, 128, a.folded) && scales_map(&m.w_scales, a.wscales, wtiles, a.ktiles, tps, 1);
    if (a.xraw) {
        m.x = m.w;
        m.x_scales = m.w_scales;
    } else {
        ok = ok && codes_map(&m.x, xcodes, a.rows, a.K, a.pair ? a.TN / 2 : a.TN, a.folded) &&
              scales_map(&m.x_scales, a.xscales, mx_row_tiles(a.rows, a.offsets ? a.experts : 0), a.ktiles, tps,
                        a.pair ? a.TN / 128 : 1);
    }
    m.up = m.w;
    m.up_scales = m.w_scales;
    if (wcodes_up)
        ok = ok && codes_map(&m.up, wcodes_up, wrows, a.K, 128, a.folded) &&
             scales_map(&m.up_scales, a.wscales_up, wtiles, a.ktiles, tps, 1);
    if (!ok) return cudaErrorInvalidValue;
    if (fmt == UQ_MXFP4) return wcodes_up ? launch<UQ_MXFP4, 2>(m, a, st) : launch<UQ_MXFP4, 1>(m, a, st);
    return wcodes_up ? launch<UQ_NVFP4, 2>(m, a, st) : launch<UQ_NVFP4, 1>(m, a, st);
}

}  // namespace uq
