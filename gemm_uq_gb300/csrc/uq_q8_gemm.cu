// uq_q8_gemm.cu -- product of 8-bit operands with one scale per row of each:
//     y[m][n] = sx[m] * sw[n] * sum_k x[m][k] * w[n][k].
//
// Few tokens (q8_gemv_kernel): the integer tensor instruction mma.m16n8k32 (s8 x s8 -> s32) on 16 rows of w and 8 tokens.
// Where a lane's k lie in the instruction does not matter as long as both operands agree, so a lane takes 16 consecutive k
// of its rows with one 16-byte load straight from global memory and feeds them to two instructions.
// A CTA takes 32 rows of w: two warps of 16 rows times four shares of k; a cluster of S CTAs shares k further where the
// rows alone would leave SMs idle.  The shares' integer sums are added in shared memory, in any order the same.
// 14336 x 4096, one to eight tokens in codes: 12.9 us (4.6 TB/s, of which 3 us are a kernel's start and end).
//
// More tokens (q8_tc_kernel): this part multiplies integers at a tenth of its 16-bit floating-point rate, and an int8 is
// exact in fp16, so the product runs on tcgen05 kind::f16 with fp32 accumulators.  Products are at most 2^14 and the sums of
// 1024 k at most 2^24: exact.  After each 1024 k the accumulator is added to fp32 sums in registers.
//   A: 128 rows of w per CTA.  Their int8 comes by TMA; eight warps widen it and write it straight to tensor memory, so that
//      of the two operands only the tokens cross shared memory a second time.
//   B: the tokens as fp16, widened once before (launch_q8_widen, or the quantizer writes fp16 at once), by TMA; up to 32 tokens
//      come as codes and are widened in the kernel.
//   D: 128 lanes (rows of w) x TN columns (tokens).
// Stages of 128 k.  Warp 0 loads the weights, warp 2 the tokens, warp 1 issues the MMAs, warps 4..11 widen in two groups that
// take the stages in turn, and read the accumulator when a chunk of 1024 k or a tile is complete: by then they have widened
// all but one of the stages ahead.  A finished tile's outputs are written behind the next tile's stages.
// PAIR: two CTAs work on 256 rows of w x 256 tokens (cta_group::2), each holding its 128 rows and half of the tokens: with
// one CTA per tile a 128 x 256 tile needs 80 KB of shared memory traffic in the 512 cycles that 64 k compute, which is more
// than it delivers; the pair 48.
// Few tiles: a cluster of S CTAs shares a tile's k, and adds its fp32 sums through distributed shared memory in rank order.
// Every wait is bounded; on a timeout the roles stop, copies in flight are waited for (bounded), the tensor memory is freed,
// and the fault word tells.
// 8192^3 621 to 635 us on different boxes (36 of them widening the tokens; 1.75 PFLOP/s, 0.88 of the measured bf16 burst rate);
// 1024 x 4096 x 4096 30 us; 64 x 14336 x 4096 18.8 to 19.8 us; 37 x 4096 x 14336 19.5 us.  What bounds it: the MMAs of pairs (within a tile
// a stage takes 1020 cycles, as long as its MMAs; of 8192^3 the tensor pipe is active in 81 % of the cycles, the rest is between
// tiles), the widening before and 13.5 rounds of tiles that take 14; for up to 128 tokens HBM while it
// streams (5.8 to 6 TB/s: 600 cycles a stage on 112 SMs, of which the MMAs are 480), and besides 8 us for the start, the first
// weights, the outputs and the sums of shared tiles.
#include <algorithm>

#include "uq_q8.cuh"
#include "uq_tcgen05.cuh"

namespace uq {

namespace {

constexpr int THREADS = 256;
constexpr int ROWS = 32, TOKENS = 8;            // of a tile
constexpr int UNROLL = 4;                       // blocks of 64 k requested together
constexpr int HELD = 4;                         // 16-byte parts of a token that a thread holds while it is quantized
constexpr int MAX_SPLIT = 8;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ int ld_cluster(uint32_t addr, uint32_t rank) {
    int v;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.s32 %0, [r];\n\t}"
                 : "=r"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}
// up to four neighbouring outputs (count of them) at element `at`
template <class T> __device__ __forceinline__ void store4(const Q8GemmArgs& a, long long at, int count, const float (&v)[4]) {
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
}
__device__ __forceinline__ void store_one(const Q8GemmArgs& a, long long at, float v) {
    if (a.ytype == UQ_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    else if (a.ytype == UQ_FP16) static_cast<__half*>(a.y)[at] = __float2half_rn(v);
    else static_cast<float*>(a.y)[at] = v;
}

// a load that stays where it is written: ahead of the barriers between it and its use
__device__ __forceinline__ uint4 ldg_now(const int8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// X int8_t: the tokens are codes with scales.  Else there is one token, a row of X, which every CTA quantizes for itself as
// quantize_q8 does: all of it for the scale, its own share of k for the codes, which go to shared memory.  Its first weights
// are on their way meanwhile.
template <class X>
__global__ void __launch_bounds__(THREADS, 3) q8_gemv_kernel(const Q8GemmArgs a, int S) {
    constexpr bool RAW = !std::is_same<X, int8_t>::value;
    __shared__ int parts[8][TOKENS * 16];       // [warp][token][row]
    __shared__ int sums[TOKENS * ROWS];         // [token][row]
    __shared__ uint32_t maxima[THREADS / 32];
    extern __shared__ __align__(16) uint8_t xs[];                  // RAW: the codes of this CTA's k
    float scale = 0.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t rank = S > 1 ? cluster_rank() : 0;
    const int tiles = (a.N + ROWS - 1) / ROWS, blocks = (a.K + 63) / 64, shares = 4 * S, share = (int)rank * 4 + (warp >> 1);
    const int b0 = (int)((long long)blocks * share / shares), b1 = (int)((long long)blocks * (share + 1) / shares);
    const int first = (int)((long long)blocks * rank * 4 / shares), own = (int)((long long)blocks * (rank + 1) * 4 / shares) - first;
    const int8_t* x = a.x + (long long)min(g, a.M - 1) * a.K + 16 * t;
    bool quantized = false;
    for (int tile = blockIdx.x / S; tile < tiles; tile += gridDim.x / S) {
        const int n0 = tile * ROWS, row = n0 + (warp & 1) * 16 + g;
        const int8_t* w0 = a.w + (long long)min(row, a.N - 1) * a.K + 16 * t;
        const int8_t* w1 = a.w + (long long)min(row + 8, a.N - 1) * a.K + 16 * t;
        uint4 p[UNROLL], q[UNROLL];
        auto request = [&](int b) {
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int k = (b + i) * 64;
                const bool in = b + i < b1 && k + 16 * t < a.K;
                p[i] = q[i] = make_uint4(0, 0, 0, 0);
                if (in) {
                    p[i] = ldg_now(w0 + k);
                    q[i] = ldg_now(w1 + k);
                }
            }
        };
        if constexpr (RAW) {
            if (!quantized) {
                // The row's loads go before those of the weights, behind which they would wait.
                quantized = true;
                constexpr int V = 16 / sizeof(X);
                using W = Vec<X, V>;
                const W* xr = static_cast<const W*>(a.raw);
                const int vecs = a.K / V, own0 = first * (64 / V), own1 = min((first + own) * (64 / V), vecs);
                W held[HELD];
#pragma unroll
                for (int i = 0; i < HELD; ++i)
                    if ((int)threadIdx.x + i * THREADS < vecs) held[i] = xr[threadIdx.x + i * THREADS];
                request(b0);
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < HELD; ++i)
                    if ((int)threadIdx.x + i * THREADS < vecs) {
                        float f[V];
                        unpack(held[i], f);
#pragma unroll
                        for (int j = 0; j < V; ++j) most = max(most, magnitude(f[j]));
                    }
                most = __reduce_max_sync(0xffffffffu, most);
                if (lane == 0) maxima[warp] = most;
                __syncthreads();
                most = __reduce_max_sync(0xffffffffu, lane < THREADS / 32 ? maxima[lane] : 0u);
                scale = most >= INF_BITS ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(most), 127.f);
                const Divisor d(scale);
#pragma unroll
                for (int i = 0; i < HELD; ++i) {
                    const int v = threadIdx.x + i * THREADS;
                    if (v < own0 || v >= own1) continue;
                    float f[V];
                    uint32_t c[V];
                    unpack(held[i], f);
                    d.codes(f, c);
                    store_codes<V>(reinterpret_cast<int8_t*>(xs) + (v - own0) * V, c);
                }
                __syncthreads();
            } else {
                request(b0);
            }
        } else {
            request(b0);
        }
        int acc[4] = {};
        for (int b = b0; b < b1; b += UNROLL) {
            uint4 v[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int k = (b + i) * 64;
                const bool in = b + i < b1 && k + 16 * t < a.K && g < a.M;
                v[i] = make_uint4(0, 0, 0, 0);
                if constexpr (RAW) {
                    if (in) v[i] = *reinterpret_cast<const uint4*>(xs + k - first * 64 + 16 * t);
                } else {
                    if (in) v[i] = *reinterpret_cast<const uint4*>(x + k);
                }
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                mma_s8(acc, p[i].x, q[i].x, p[i].y, q[i].y, v[i].x, v[i].y);
                mma_s8(acc, p[i].z, q[i].z, p[i].w, q[i].w, v[i].z, v[i].w);
            }
            if (b + UNROLL < b1) request(b + UNROLL);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) parts[warp][(2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[i];
        __syncthreads();
        const int r = threadIdx.x & 31, c = threadIdx.x >> 5;      // this thread's output: row, token
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += parts[2 * i + (r >> 4)][c * 16 + (r & 15)];
        bool mine = n0 + r < a.N && c < a.M;
        if (S > 1) {
            sums[threadIdx.x] = sum;
            cluster_sync();
            mine = mine && (int)threadIdx.x >= THREADS * (int)rank / S && (int)threadIdx.x < THREADS * ((int)rank + 1) / S;
            if (mine) {
                sum = 0;
                for (int i = 0; i < S; ++i) sum += ld_cluster(smem_u32(&sums[threadIdx.x]), i);
            }
        }
        if (mine) store_one(a, (long long)c * a.N + n0 + r, (float)sum * (RAW ? scale : a.sx[c]) * a.sw[n0 + r]);
        if (S > 1) cluster_sync();
        else __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------------
// tcgen05

constexpr unsigned int FAULT_Q8_WAIT = 32u;
constexpr int TC_THREADS = 384;                 // warpgroups: producers and issuer, and two that widen the weights
constexpr int X_WARPS = 4;                      // of a fourth, which widens few tokens
constexpr int STAGE_K = 128, W_BYTES = 128 * STAGE_K;
constexpr int CHUNK = 1024 / STAGE_K;           // stages whose sums are exact
constexpr int HEAD = 1024;                      // barriers and flags before the stages
constexpr int WIDE_WARPS = 8;
constexpr int MOST_CODES = 32;                  // most tokens that the kernel takes as int8 codes

struct TcArgs8 {
    Q8GemmArgs g;
    int steps;                                  // stages along K
    int NT, MT;                                 // tiles along N and M
    int S, group, ctas;
    int wait;                                   // the kernel before on the stream may still run
};

template <bool PAIR> __device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t on) {
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, " UQ_OPERAND_HI "};\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "elect.sync _|e, 0xffffffff;\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n\t}"
                     :: "r"(d), "r"(a), "r"(b_lo), "r"(idesc), "r"(on) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, " UQ_OPERAND_HI "};\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "elect.sync _|e, 0xffffffff;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
                     :: "r"(d), "r"(a), "r"(b_lo), "r"(idesc), "r"(on) : "memory");
}
template <bool PAIR> __device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (PAIR) pair_commit(bar);
    else uq::commit(bar);
}
__device__ __forceinline__ void arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(addr) : "memory");
}
// An arrival, perhaps on the other CTA's barrier, that orders tensor memory alone (between the tcgen05 fences).  Relaxed: a
// release at cluster scope waits for all of the thread's stores, the outputs of the tile before among them.
__device__ __forceinline__ void arrive_relaxed(uint32_t mapped) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(mapped) : "memory");
}
// A whole warp's wait: false for all lanes once WAIT_LIMIT_NS have passed (the fault word then tells) or the CTA was told to
// stop.  LOCAL: only this CTA arrives; CLUSTER: arrivals of the pair's other CTA count; TENSOR: the wait orders tensor memory
// alone.
enum { LOCAL, CLUSTER, TENSOR };
template <int KIND> __device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned int* fault, volatile int* stop_flag) {
    unsigned long long t0 = 0;
    for (unsigned int i = 0;; ++i) {
        uint32_t ok;
        if constexpr (KIND == TENSOR)
            asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                         "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        else if constexpr (KIND == CLUSTER)
            asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                         "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        else
            asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                         : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
        if (i % 64 == 63) {
            bool stop = *stop_flag != 0;
            if (!t0) t0 = global_ns();
            else if (global_ns() - t0 > WAIT_LIMIT_NS) {
                atomicOr(fault, FAULT_Q8_WAIT);
                stop = true;
            }
            if (__any_sync(0xffffffffu, stop)) return false;
        }
    }
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                    "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}
// four int8 -> two f16x2, exact: a byte with its sign bit turned over is the low byte of 1024 + 128 + v in fp16
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}
__device__ __forceinline__ void after_prior_work(const TcArgs8& a) {
    if (a.wait) asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Writes 16 columns (tokens m0 .. m0 + count) of this lane's output nn; the warp's lanes hold 32 consecutive outputs.  16-bit
// types where N is even: neighbouring lanes exchange every other value and hold pairs of outputs, stored together.  N odd: each
// lane its own outputs (300 x 4095 x 4096 20.1 us; the pairs' halves one after the other 20.6).
template <class T> __device__ __forceinline__ void put16(const Q8GemmArgs& a, int m0, int count, int nn, const float (&v)[16]) {
    if (sizeof(T) == 2 && !(a.N & 1)) {
        const int odd = threadIdx.x & 1, n = nn & ~1;
        T* p = static_cast<T*>(a.y) + (long long)(m0 + odd) * a.N + n;
        const long long step = 2ll * a.N;
#pragma unroll
        for (int j = 0; j < 16; j += 2, p += step) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            if constexpr (sizeof(T) == 2) {
                const uint32_t w = pack2(T(), odd ? got : v[j], odd ? v[j + 1] : got);
                if (j + odd < count && n < a.N) *reinterpret_cast<uint32_t*>(p) = w;
            }
        }
    } else {
        T* p = static_cast<T*>(a.y) + (long long)m0 * a.N + nn;
#pragma unroll
        for (int j = 0; j < 16; ++j, p += a.N)
            if (nn < a.N && j < count) *p = from_f32<T>(v[j]);
    }
}

struct Tile8 { int nt, m0, rows; };
// Tiles are numbered in groups of a.group weight tiles, token tiles within a group, weight tiles fastest, so that CTAs
// running at the same time share both operands in L2.
template <int TN> __device__ __forceinline__ Tile8 find_tile(const TcArgs8& a, int tile) {
    const unsigned per = a.group * a.MT, g = (unsigned)tile / per, in = tile - g * per;
    const unsigned width = min(a.group, a.NT - (int)g * a.group);
    const int tt = in / width;
    return {(int)(g * a.group + in - tt * width), tt * TN, min(TN, a.g.M - tt * TN)};
}

// Rings and tensor memory of a tile shape.
template <int TN, bool PAIR> struct Plan8 {
    // Up to 32 tokens are widened in the kernel, by a warpgroup of their own, in one launch: 10.6 us of host time a call instead
    // of 15.3, and on the GPU 16 x 14336 x 4096 takes 18.7 us and 18.5.  More tokens add to what shared memory delivers: 64 x
    // 14336 x 4096 21.3 us in the kernel and 18.8 with their own, under which the first weights are loaded.
    static constexpr bool CODES = !PAIR && TN <= MOST_CODES;
    static constexpr int THREADS = TC_THREADS + (CODES ? X_WARPS * 32 : 0);
    static constexpr int XR = PAIR ? TN / 2 : TN;                  // token rows of a CTA
    static constexpr int X_BYTES = XR * STAGE_K * 2, C_BYTES = CODES ? XR * STAGE_K : 0;
    static constexpr int XS = TN >= 256 || TN == 64 ? 5 : 4;       // stages of fp16 tokens, of weights, and widened ones
    static constexpr int WS = TN >= 256 ? 3 : (TN == 128 ? 5 : (TN == 64 ? 8 : 10));
    static constexpr int AS = (512 - TN) / 64 < 8 ? (512 - TN) / 64 : 8;
    static constexpr int CS = 4;                                   // of tokens' codes
    static constexpr int RING = WS * W_BYTES + XS * X_BYTES + CS * C_BYTES;
    // Pairs have the accumulator in two halves of columns whose chunks end half a chunk apart: while one is read the MMAs go
    // on with the other, which in the two stages around the end of the chunk come in such an order that twice half a stage
    // lies between (a 256 x 256 tile's 1024 k: 8200 cycles of MMAs, and about 1000 from their end to the next one's start).
    // Not so a CTA alone: an MMA with A in tensor memory takes 60 cycles however few columns it has.
    static constexpr int HALVES = PAIR ? 2 : 1;
    static_assert(1024 + HEAD + RING <= 227 * 1024 && TN + 64 * AS <= 512, "memory");
};
enum { W_FULL = 0, W_EMPTY = 10, X_FULL = 20, X_EMPTY = 28, A_FULL = 36, A_EMPTY = 44, ACC_FULL = 52, ACC_EMPTY = 54,
       C_FULL = 56, C_EMPTY = 60, DRAINED = 64 };

template <class T, int TN, bool PAIR>
__global__ void __launch_bounds__(Plan8<TN, PAIR>::THREADS, 1)
q8_tc_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, const TcArgs8 a) {
    using P = Plan8<TN, PAIR>;
    constexpr int XR = P::XR, XS = P::XS, WS = P::WS, AS = P::AS, HALVES = P::HALVES;
    constexpr int COLS = TN / 2;                                   // accumulator columns of a reading warp
    constexpr int BOX = PAIR ? XR / 2 : XR;                        // token rows of a TMA box
    constexpr int ACROSS = PAIR ? CLUSTER : LOCAL;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* head = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(head);
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int which) { return bar0 + 8 * which; };
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(bars + DRAINED + 1);
    volatile int* stop = reinterpret_cast<volatile int*>(tmem_ptr + 1);
    const uint32_t ring = smem_u32(head + HEAD), xring = ring + WS * W_BYTES, cring = xring + XS * P::X_BYTES;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR || a.S > 1 ? cluster_rank() : 0;
    const uint32_t side = PAIR ? rank : 0;                         // which CTA of the pair
    const int share = PAIR ? 0 : (int)rank;                        // which of the S shares of k
    const bool lead = side == 0;
    unsigned int* fault = a.g.fault;

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];" :: "l"(&wmap) : "memory");
            asm volatile("prefetch.tensormap [%0];" :: "l"(&xmap) : "memory");
            for (int i = 0; i < WS; ++i) {
                mbar_init(bars + W_FULL + i, 1);
                mbar_init(bars + W_EMPTY + i, WIDE_WARPS / 2);
            }
            for (int i = 0; i < XS; ++i) {
                mbar_init(bars + X_FULL + i, P::CODES ? X_WARPS : 1);
                mbar_init(bars + X_EMPTY + i, 1);
            }
            for (int i = 0; i < P::CS; ++i) {
                mbar_init(bars + C_FULL + i, 1);
                mbar_init(bars + C_EMPTY + i, X_WARPS);
            }
            for (int i = 0; i < AS; ++i) {
                mbar_init(bars + A_FULL + i, WIDE_WARPS / 2 * (PAIR ? 2 : 1));
                mbar_init(bars + A_EMPTY + i, 1);
            }
            for (int i = 0; i < HALVES; ++i) {
                mbar_init(bars + ACC_FULL + i, 1);
                mbar_init(bars + ACC_EMPTY + i, WIDE_WARPS / HALVES * (PAIR ? 2 : 1));
            }
            mbar_init(bars + DRAINED, 1);
            *stop = 0;
            fence_barrier_init();
            fence_proxy_async_smem();
        }
        __syncwarp();
    } else if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(tmem_ptr)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_u32(tmem_ptr)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();                            // the other CTA's barriers are ready
    fence_after();
    const uint32_t tmem = (uint32_t)__shfl_sync(0xffffffffu, (int)*tmem_ptr, 0);
    const uint32_t acol = tmem + TN;                               // widened stages, 64 columns each

    // this CTA's tiles, and its k steps of them
    const int tiles = a.NT * a.MT, width = PAIR ? 2 : a.S;         // CTAs of a tile
    const int k0 = (int)((long long)a.steps * share / a.S), k1 = (int)((long long)a.steps * (share + 1) / a.S);
    const int first = blockIdx.x / width, stride = gridDim.x / width;
    // token columns of half h that the MMAs compute
    auto columns = [&](const Tile8& t, int h) { return (min(max(t.rows - h * (TN / HALVES), 0), TN / HALVES) + 15) / 16 * 16; };
    // whether a chunk of half h begins, or ends, with stage j of the tile
    auto begins = [&](int j, int h) { return j == 0 || j % CHUNK == h * (CHUNK / 2); };
    auto ends = [&](int j, int h) { return j == k1 - k0 - 1 || (j + 1) % CHUNK == h * (CHUNK / 2); };

    // 128 sums a thread and the stage being widened take more than a third of the registers: 168 a thread at launch become
    // 56 + 224 + 224 of the three warpgroups.
    if (warp < 4) {
        if constexpr (TN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            // -------------------------------------------------------- weights
            // They do not depend on the kernel before, so they are requested while it may still run.
            int issued = 0, s = 0;
            uint32_t ph = 1;                                       // the first round's stages count as free
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += stride) {
                const int row = find_tile<TN>(a, tile).nt * (PAIR ? 256 : 128) + (int)side * 128;
                for (int kt = k0; kt < k1; ++kt, ++issued) {
                    if (issued >= WS && !warp_wait<LOCAL>(bar(W_EMPTY + s), ph, fault, stop)) { ok = false; break; }
                    expect_bytes(bar(W_FULL + s), W_BYTES);
                    tma_2d(ring + s * W_BYTES, &wmap, kt * STAGE_K, row, bar(W_FULL + s));
                    if (++s == WS) { s = 0; ph ^= 1; }
                }
            }
            if (!ok) *stop = 1;
            // let the last copies land before the CTA can leave
            for (int j = issued - 1; j >= 0 && j >= issued - WS; --j)
                mbar_wait_bounded(bars + W_FULL + j % WS, (uint32_t)((j / WS) & 1), fault, FAULT_Q8_WAIT);
        } else if (warp == 2) {
            // -------------------------------------------------------- tokens, which do
            after_prior_work(a);
            constexpr int SLOTS = P::CODES ? P::CS : XS, FULL = P::CODES ? C_FULL : X_FULL, EMPTY = P::CODES ? C_EMPTY : X_EMPTY;
            int issued = 0, s = 0;
            uint32_t ph = 1;
            bool ok = true;
            const uint32_t lead_full = PAIR ? cluster_addr(bar(FULL), 0) : bar(FULL);
            for (int tile = first; ok && tile < tiles; tile += stride) {
                const Tile8 t = find_tile<TN>(a, tile);
                for (int kt = k0; kt < k1; ++kt, ++issued) {
                    if (issued >= SLOTS && !warp_wait<ACROSS>(bar(EMPTY + s), ph, fault, stop)) { ok = false; break; }
                    if (lead) expect_bytes(bar(FULL + s), P::CODES ? P::C_BYTES : P::X_BYTES * (PAIR ? 2 : 1));
                    if constexpr (P::CODES) {
                        tma_2d(cring + s * P::C_BYTES, &xmap, kt * STAGE_K, t.m0, bar(FULL + s));
                    } else {
                        const uint32_t dst = xring + s * P::X_BYTES;
                        // [64 k][rows], of a pair the CTA's half of the rows of each half of the columns
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if constexpr (PAIR) {
#pragma unroll
                                for (int h = 0; h < HALVES; ++h)
                                    pair_tma_2d(dst + (j * 2 + h) * (BOX * 128), &xmap, kt * STAGE_K + j * 64,
                                                t.m0 + h * (TN / 2) + (int)side * (columns(t, h) >> 1), lead_full + s * 8);
                            } else {
                                tma_2d(dst + j * (XR * 128), &xmap, kt * STAGE_K + j * 64, t.m0, bar(FULL + s));
                            }
                        }
                    }
                    if (++s == SLOTS) { s = 0; ph ^= 1; }
                }
            }
            if (!ok) *stop = 1;
            // (both CTAs' tokens are counted on the even one's barriers, and the CTAs leave together)
            if (lead)
                for (int j = issued - 1; j >= 0 && j >= issued - SLOTS; --j)
                    mbar_wait_bounded(bars + FULL + j % SLOTS, (uint32_t)((j / SLOTS) & 1), fault, FAULT_Q8_WAIT);
        } else if (warp == 1 && lead) {
            // -------------------------------------------------------- MMA issue (PAIR: for both CTAs)
            int xs = 0, as = 0;
            uint32_t used = 0, eph = 3;                            // bit h: half h has had a chunk; parity of its next read
            uint32_t xph = 0, aph = 0;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += stride) {
                const Tile8 t = find_tile<TN>(a, tile);
                // D fp32, A and B fp16, both K-major, M = 128 or 256, N = the half's columns
                const uint32_t base = (1u << 4) | ((PAIR ? 16u : 8u) << 24);
                uint32_t idesc[HALVES];
#pragma unroll
                for (int h = 0; h < HALVES; ++h) idesc[h] = base | ((uint32_t)(columns(t, h) >> 3) << 17);
                for (int j = 0; ok && j < k1 - k0; ++j) {
                    if (!warp_wait<ACROSS>(bar(X_FULL + xs), xph, fault, stop) || !warp_wait<TENSOR>(bar(A_FULL + as), aph, fault, stop)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t b = desc_lo(xring + xs * P::X_BYTES), ac = acol + as * 64;
                    // the half whose chunk has just ended comes last, one whose chunk ends now first
                    const int swap = HALVES == 2 && ((j && begins(j, 0)) || (ends(j, 1) && !ends(j, 0)));
#pragma unroll
                    for (int o = 0; o < HALVES; ++o) {
                        const int h = HALVES == 2 ? o ^ swap : 0;
                        if (begins(j, h)) {
                            // the half's chunk before has been read
                            eph ^= (used >> h & 1u) << h;
                            if ((used >> h & 1u) && !warp_wait<TENSOR>(bar(ACC_EMPTY + h), eph >> h & 1u, fault, stop)) {
                                ok = false;
                                break;
                            }
                            used |= 1u << h;
                            fence_after();
                        }
                        const uint32_t id = h ? idesc[HALVES - 1] : idesc[0], d = tmem + h * (TN / 2);
                        // the half's rows of the first 64 k; the second 64 k follow all rows of the first
                        const uint32_t bh = b + h * (PAIR ? BOX * 8 : XR * 4);
                        const uint32_t more = begins(j, h) ? 0u : 1u;
                        if (id >> 17 & 63u) {
#pragma unroll
                            for (int m = 0; m < 8; ++m) mma<PAIR>(d, ac + m * 8, bh + (m >> 2) * (XR * 8) + (m & 3) * 2, id, more | m);
                        }
                        if (ends(j, h)) commit<PAIR>(bar(ACC_FULL + h));
                    }
                    commit<PAIR>(bar(X_EMPTY + xs));
                    commit<PAIR>(bar(A_EMPTY + as));
                    if (++xs == XS) { xs = 0; xph ^= 1; }
                    if (++as == AS) { as = 0; aph ^= 1; }
                }
            }
            if (!ok) {
                *stop = 1;
                __syncwarp();
                commit<PAIR>(bar(DRAINED));
                mbar_wait_bounded(bars + DRAINED, 0, fault, FAULT_Q8_WAIT);
            }
        }
    } else if (P::CODES && warp >= TC_THREADS / 32) {
        // ------------------------------------------------------------ widening of the tokens: 16 codes of a row at a time
        if constexpr (P::CODES) {
            const int w = warp - TC_THREADS / 32;
            int cs = 0, xs = 0, i = 0;
            uint32_t cph = 0, xph = 1;
            bool ok = true;
            for (int tile = first; ok && tile < tiles; tile += stride)
                for (int kt = k0; kt < k1; ++kt, ++i) {
                    if (!warp_wait<LOCAL>(bar(C_FULL + cs), cph, fault, stop) ||
                        (i >= XS && !warp_wait<LOCAL>(bar(X_EMPTY + xs), xph, fault, stop))) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int j = 0; j < TN / 16; ++j) {
                        const int row = j * 16 + w * 4 + (lane >> 3), c = lane & 7;        // eight lanes to a row's 128 bytes
                        uint4 v, lo, hi;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(cring + cs * P::C_BYTES + row * 128 + ((c ^ (row & 7)) << 4)) : "memory");
                        widen4(v.x, lo.x, lo.y);
                        widen4(v.y, lo.z, lo.w);
                        widen4(v.z, hi.x, hi.y);
                        widen4(v.w, hi.z, hi.w);
                        const uint32_t to = xring + xs * P::X_BYTES + (c >> 2) * (XR * 128) + row * 128, part = (c & 3) * 2;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(to + ((part ^ (row & 7)) << 4)), "r"(lo.x),
                                     "r"(lo.y), "r"(lo.z), "r"(lo.w) : "memory");
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(to + (((part + 1) ^ (row & 7)) << 4)), "r"(hi.x),
                                     "r"(hi.y), "r"(hi.z), "r"(hi.w) : "memory");
                    }
                    fence_proxy_async_smem();                      // the MMAs read through the async proxy
                    __syncwarp();
                    if (lane == 0) {
                        arrive(bar(X_FULL + xs));
                        arrive(bar(C_EMPTY + cs));
                    }
                    if (++cs == P::CS) { cs = 0; cph ^= 1; }
                    if (++xs == XS) { xs = 0; xph ^= 1; }
                }
            if (!ok) *stop = 1;
        }
    } else {
        // ------------------------------------------------------------ widening, and the accumulator: lane = row of w
        if constexpr (TN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int q = warp & 3, half = (warp - 4) >> 2, row = q * 32 + lane;
        const int which = HALVES == 2 ? half : 0;                  // the chunks that this warp's columns belong to
        const uint32_t lanes = (uint32_t)(q * 32) << 16;
        const uint32_t lead_a_full = PAIR ? cluster_addr(bar(A_FULL), 0) : bar(A_FULL);
        const uint32_t lead_acc_empty = PAIR ? cluster_addr(bar(ACC_EMPTY + which), 0) : bar(ACC_EMPTY + which);
        float sums[COLS] = {};
        int ws = 0, as = 0, i = 0, read = 0, boundary = 0;
        uint32_t wph = 0, aph = 1;
        bool pending = false, ok = true, fresh = true, last = false, widened = false;
        Tile8 t = find_tile<TN>(a, first), pt = t, ot = t;         // tile of the stage, of the chunk to be read, of the outputs
        // A finished tile's outputs are written behind the next tile's stages, 32 columns at a time: all at once they would hold
        // up the widening for longer than there are stages ahead.  This code is in the loop once, and for one type: it is
        // executed once a tile, so what it takes is its fetching (a 256 x 256 tile's epilogue, for three types in four places:
        // 18000 cycles).
        constexpr int GROUPS = COLS / 16, READ = COLS < 32 ? COLS : 32;
        int written = GROUPS;
        float sx[(COLS + 31) / 32], sw = 0.f;                      // scales of tokens 32 i + lane, and of this lane's output
        auto write_groups = [&](int to) {
            const int nn = ot.nt * (PAIR ? 256 : 128) + (int)side * 128 + row;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int m = half * COLS + 16 * g;                // token of the tile
                if (g < written || g >= to || m >= ot.rows) continue;
                float v[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = sums[16 * g + c] * __shfl_sync(0xffffffffu, sx[g / 2], (16 * g + c) & 31) * sw;
                put16<T>(a.g, ot.m0 + m, ot.rows - m, nn, v);
            }
            written = min(to, GROUPS);
        };
        for (int tile = first, j = 0; ok;) {
            const bool over = tile >= tiles;
            // What does not happen in every stage is marked so: laid out of the loop's way, a stage's instructions are fetched sooner
            // (8192^3 629 us, then 621).
            // A complete chunk is read when the stages ahead are widened (of pairs, whose group 0 has the first of them, before
            // its second one), or another one ends
            const bool reads = pending && (over || i - boundary >= (PAIR && half == 0 ? AS - 2 : AS - 1) || ends(j, which));
            if (__builtin_expect(written < GROUPS && (reads || over || widened), 0)) write_groups(reads || over ? GROUPS : written + 2);
            widened = false;
            if (__builtin_expect(reads, 0)) {
                pending = false;
                if (!warp_wait<TENSOR>(bar(ACC_FULL + which), (uint32_t)read & 1, fault, stop)) { ok = false; break; }
                ++read;
                fence_after();
                // sums = (a tile's first chunk ? 0 : sums) + chunk, in place: as an expression the sums took twice the registers
#pragma unroll
                for (int c = 0; c < COLS; c += READ) {
                    uint32_t r[READ];
#pragma unroll
                    for (int e = 0; e < READ; e += 16)
                        tmem_ld16(tmem + lanes + half * COLS + c + e, *reinterpret_cast<uint32_t(*)[16]>(r + e));
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int e = 0; e < READ; ++e) asm volatile("{\n\t.reg .pred p;\n\t.reg .f32 t;\n\tsetp.ne.b32 p, %2, 0;\n\tselp.f32 t, 0f00000000, %0, p;\n\tadd.f32 %0, t, %1;\n\t}"
                                     : "+f"(sums[c + e]) : "f"(__uint_as_float(r[e])), "r"((int)fresh));
                }
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(lead_acc_empty);
                fresh = last;
                if (last && (PAIR || a.S == 1)) {
                    after_prior_work(a);                           // the scales may be its output, and y its input
                    ot = pt;
                    written = 0;
#pragma unroll
                    for (int c = 0; c < COLS; c += 32) sx[c / 32] = ld_written(a.g.sx + min(ot.m0 + half * COLS + c + lane, a.g.M - 1));
                    sw = __ldg(a.g.sw + min(ot.nt * (PAIR ? 256 : 128) + (int)side * 128 + row, a.g.N - 1));
                }
            }
            if (__builtin_expect(over, 0)) {
                if (written == GROUPS) break;
                continue;
            }
            // the two groups of four warps take the stages in turn, so that one's loads run under the other's stores
            if ((i & 1) == half) {
                if (!warp_wait<LOCAL>(bar(W_FULL + ws), wph, fault, stop)) { ok = false; break; }
                // this row's 128 k, in the swizzled tile: 32 at a time, the next 32 on their way
                const uint32_t base = ring + ws * W_BYTES + row * 128;
                uint4 v[2][2];
                auto load = [&](uint4 (&to)[2], int from) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(to[c].x), "=r"(to[c].y), "=r"(to[c].z), "=r"(to[c].w)
                                     : "r"(base + (((from + c) ^ (row & 7)) << 4)));
                };
                load(v[0], 0);
                // the MMAs that read these columns before are complete
                if (i >= AS && !warp_wait<TENSOR>(bar(A_EMPTY + as), aph, fault, stop)) { ok = false; break; }
                fence_after();
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t r[16];
                    if (h < 3) load(v[(h + 1) & 1], 2 * h + 2);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 u = v[h & 1][c];
                        widen4(u.x, r[8 * c], r[8 * c + 1]);
                        widen4(u.y, r[8 * c + 2], r[8 * c + 3]);
                        widen4(u.z, r[8 * c + 4], r[8 * c + 5]);
                        widen4(u.w, r[8 * c + 6], r[8 * c + 7]);
                    }
                    tmem_st16(acol + lanes + as * 64 + h * 16, r);
                }
                __syncwarp();
                if (lane == 0) arrive(bar(W_EMPTY + ws));
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(lead_a_full + as * 8);
                widened = true;
            }
            if (__builtin_expect(ends(j, which), 0)) {
                pending = true;
                boundary = i + 1;
                last = j == k1 - k0 - 1;
                pt = t;
            }
            if (++ws == WS) { ws = 0; wph ^= 1; }
            if (++as == AS) { as = 0; aph ^= 1; }
            ++i;
            if (__builtin_expect(++j == k1 - k0, 0)) {
                j = 0;
                tile += stride;
                if (tile < tiles) t = find_tile<TN>(a, tile);
            }
        }
        if (!ok) *stop = 1;
        if (!PAIR && a.S > 1) {
            // when all warps are done with the ring the sums are left there, [token][row]
            asm volatile("bar.sync 1, 256;" ::: "memory");
            float* left = reinterpret_cast<float*>(head + HEAD);
#pragma unroll
            for (int c = 0; c < COLS; ++c)
                if (half * COLS + c < pt.rows) left[(half * COLS + c) * 128 + row] = sums[c];
        }
    }
    __syncwarp();
    fence_before();
    // (split tiles) this thread's four neighbouring outputs, and their scales
    const Tile8 t = find_tile<TN>(a, first);
    const int r = (threadIdx.x & 31) * 4, nn = t.nt * 128 + r;
    float sw4[4] = {};
    if (!PAIR && a.S > 1) {
        after_prior_work(a);
#pragma unroll
        for (int j = 0; j < 4; ++j) sw4[j] = __ldg(a.g.sw + min(nn + j, a.g.N - 1));
    }
    __syncthreads();
    if (PAIR || a.S > 1) cluster_sync();                           // the pair is done with each other's memory; the sums are there
    fence_after();
    if (warp == 1) {
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
    }
    if (!PAIR && a.S > 1) {
        // A thread takes four neighbouring outputs of two tokens at a time; the CTAs' sums of both are requested before they are
        // added.
        for (int it = share * P::THREADS + threadIdx.x; it < t.rows * 32; it += 2 * a.S * P::THREADS) {
            float4 p[2][MAX_SPLIT];
            float sx[2];
            int c[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                c[i] = min((it >> 5) + i * a.S * (P::THREADS / 32), t.rows - 1);
#pragma unroll
                for (int k = 0; k < MAX_SPLIT; ++k)
                    p[i][k] = k < a.S ? ld_cluster4(ring + (c[i] * 128 + r) * 4, k) : make_float4(0.f, 0.f, 0.f, 0.f);
                sx[i] = ld_written(a.g.sx + t.m0 + c[i]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (nn >= a.g.N || (i && (it >> 5) + a.S * (P::THREADS / 32) >= t.rows)) break;
                float v[4] = {};
#pragma unroll
                for (int k = 0; k < MAX_SPLIT; ++k) {
                    v[0] += p[i][k].x; v[1] += p[i][k].y; v[2] += p[i][k].z; v[3] += p[i][k].w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = v[j] * sx[i] * sw4[j];
                store4<T>(a.g, (long long)(t.m0 + c[i]) * a.g.N + nn, a.g.N - nn, v);
            }
        }
        cluster_sync();                                            // nobody leaves while its sums may be read
    }
}

// int8 codes -> fp16, 16 at a time, four of a thread under way together; the product that follows may start meanwhile
__global__ void __launch_bounds__(256) q8_widen_kernel(const uint4* __restrict__ x, uint4* __restrict__ out, long long n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (long long i = blockIdx.x * 1024LL + threadIdx.x; i < n; i += gridDim.x * 1024LL) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j * 256 < n) v[j] = x[i + j * 256];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i + j * 256 >= n) break;
            uint4 lo, hi;
            widen4(v[j].x, lo.x, lo.y);
            widen4(v[j].y, lo.z, lo.w);
            widen4(v[j].z, hi.x, hi.y);
            widen4(v[j].w, hi.z, hi.w);
            out[2 * (i + j * 256)] = lo;
            out[2 * (i + j * 256) + 1] = hi;
        }
    }
}

// rows of `cols` elements of `size` bytes, boxes of 128 bytes x `box` rows, 128-byte swizzle, zeros beyond the ends
bool rows_map(CUtensorMap* m, const void* p, long long rows, int cols, int size, int box) {
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * size};
    cuuint32_t b[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box};
    cuuint32_t es[2] = {1, 1};
    return encode_fn()(m, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(p), dims,
                       strides, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int TN, bool PAIR> cudaError_t launch_tc(TcArgs8 a, const void* x16, int sms, cudaStream_t st) {
    static_assert(Plan8<TN, PAIR>::CODES == (TN <= MOST_CODES), "which form the tokens come in");
    static Done ready = {};
    cudaError_t e = configure(q8_tc_kernel<T, TN, PAIR>, ready);
    if (e != cudaSuccess) return e;
    using P = Plan8<TN, PAIR>;
    const int wide = PAIR ? 256 : 128;
    a.steps = (a.g.K + STAGE_K - 1) / STAGE_K;
    a.NT = (a.g.N + wide - 1) / wide;
    a.MT = (a.g.M + TN - 1) / TN;
    a.group = 8;
    const long long tiles = (long long)a.NT * a.MT;
    a.S = 1;
    while (!PAIR && a.S < MAX_SPLIT && tiles * a.S * 2 <= sms && a.steps >= a.S * 4) a.S *= 2;
    const int width = PAIR ? 2 : a.S;
    a.ctas = a.S > 1 ? (int)tiles * width : (int)std::min(tiles * width, (long long)(sms / width * width));
    CUtensorMap wmap, xmap;
    if (!rows_map(&wmap, a.g.w, a.g.N, a.g.K, 1, 128) || !rows_map(&xmap, P::CODES ? a.g.x : x16, a.g.M, a.g.K, P::CODES ? 1 : 2, PAIR ? P::XR / 2 : P::XR)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ctas);
    cfg.blockDim = dim3(P::THREADS);
    cfg.dynamicSmemBytes = 1024 + HEAD + P::RING;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (width > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = width;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (a.wait) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, q8_tc_kernel<T, TN, PAIR>, wmap, xmap, a);
}

// Whether pairs of CTAs are the faster kernel, by rounds of tiles: a round of 128 x 128 tiles takes about 1.9 us and 0.39 a stage,
// one of 256 x 256 tiles, whose outputs are four times as many, 8.0 us and 0.58 a stage (fitted to K = 2048 to 8192).  Measured, us
// single / pairs: 8192 x 8192 (27 / 14 rounds) K = 512 82 / 126, 1024 122 / 165, 2048 211 / 234, 8192 729 / 633; 2048 x 8192 (7 / 4)
// K = 4096 101 / 107, 8192 189 / 181; 2560 x 8192 (9 / 5) 127 / 133 and 241 / 227; 2500 x 4096 (5 / 3) K = 14336 238 / 224;
// 4096 x 4096 (7 / 4) K = 2048 60 / 71; 1024 x 4096 (2 / 1) K = 1408 17.2 / 18.3, 2048 20.9 / 20.7, 4096 34.0 / 30.5; 512 x 14336
// (3 / 2) K = 4096 47 / 55; 256 x 14336 (2 / 1) 33.2 / 30.3.
bool pays_in_pairs(const Q8GemmArgs& g, int sms) {
    const long long one = (long long)((g.N + 127) / 128) * ((g.M + 127) / 128), two = 2LL * ((g.N + 255) / 256) * ((g.M + 255) / 256);
    const int steps = (g.K + STAGE_K - 1) / STAGE_K;
    return (two + sms - 1) / sms * (206 + 15 * steps) < (one + sms - 1) / sms * (49 + 10 * steps);
}

}  // namespace

Q8Form q8_gemm_form(int M) { return M <= TOKENS ? Q8_GEMV : (M <= MOST_CODES ? Q8_CODES : Q8_WIDE); }

cudaError_t launch_q8_widen(const int8_t* x, void* x16, int M, int K, int sms, cudaStream_t st) {
    const long long n = (long long)M * K / 16, ctas = (n + 1023) / 1024;
    q8_widen_kernel<<<(unsigned)std::min(ctas, 8LL * sms), 256, 0, st>>>(reinterpret_cast<const uint4*>(x), static_cast<uint4*>(x16), n);
    return cudaGetLastError();
}

cudaError_t launch_q8_gemm_tc(const Q8GemmArgs& g, const void* x16, bool wait, int sms, cudaStream_t st) {
    if (!encode_fn()) return cudaErrorNotSupported;
    TcArgs8 a = {};
    a.g = g;
    a.wait = wait;
    return with_dtype(g.ytype, [&](auto t) {
        using T = decltype(t);
        if (g.M <= 32) return launch_tc<T, 32, false>(a, x16, sms, st);
        if (g.M <= 64) return launch_tc<T, 64, false>(a, x16, sms, st);
        if (!pays_in_pairs(g, sms)) return launch_tc<T, 128, false>(a, x16, sms, st);
        return launch_tc<T, 256, true>(a, x16, sms, st);
    });
}

// CTAs sharing a tile's k: up to three CTAs an SM in all.  (Powers of two: clusters of three took 9.3 us for 1 x 4096 x 4096,
// clusters of two 7.6.)
static int gemv_split(int N, int K, int sms) {
    const long long tiles = (N + ROWS - 1) / ROWS;
    int S = 1;
    while (S < MAX_SPLIT && tiles * S * 2 <= 3LL * sms && K >= 64 * 4 * S * 2) S *= 2;
    return S;
}

// One launch instead of two for a single aligned token that the threads can hold: 12.6 us of host time a call instead of 15.7;
// on the GPU 1 x 14336 x 4096 takes 15.0 us instead of 14.3.  (4096 x 14336, the token read twice by each CTA: 21.7 and 19.2.)
bool q8_gemm_quantizes(const void* x, int type, int M, int K) {
    const int bytes = K * (type == UQ_FP32 ? 4 : 2);               // K is below 2^17
    return M == 1 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && bytes <= HELD * THREADS * 16;
}

cudaError_t launch_q8_gemm(const Q8GemmArgs& a, int sms, cudaStream_t st) {
    const long long tiles = (a.N + ROWS - 1) / ROWS;
    const int S = gemv_split(a.N, a.K, sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S > 1 ? (unsigned)tiles * S : (unsigned)std::min(tiles, 3LL * sms));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = a.raw ? ((a.K + 63) / 64 / S + 2) * 64 : 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 1 : 0;
    if (!a.raw) return cudaLaunchKernelEx(&cfg, q8_gemv_kernel<int8_t>, a, S);
    return with_dtype(a.xtype, [&](auto t) { return cudaLaunchKernelEx(&cfg, q8_gemv_kernel<decltype(t)>, a, S); });
}

}  // namespace uq
