// uq_q8_gemm.cu -- product of 8-bit operands with one scale per row of each:
//     y[m][n] = sx[m] * sw[n] * sum_k x[m][k] * w[n][k].
//
// The integer tensor instruction mma.m16n8k32 (s8 x s8 -> s32) on 16 rows of w and 8 tokens.  Where a lane's k lie in the
// instruction does not matter as long as both operands agree, so a lane takes 16 consecutive k of its rows with one
// 16-byte load straight from global memory and feeds them to two instructions.
// A CTA takes 32 rows of w: two warps of 16 rows times four shares of k; a cluster of S CTAs shares k further where the
// rows alone would leave SMs idle.  The shares' integer sums are added in shared memory, in any order the same.
#include "uq_mx.cuh"

namespace uq {

namespace {

constexpr int THREADS = 256;
constexpr int ROWS = 32, TOKENS = 8;            // of a tile
constexpr int UNROLL = 4;                       // blocks of 64 k requested together
constexpr int MAX_SPLIT = 8;

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster(uint32_t addr, uint32_t rank) {
    int v;
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.s32 %0, [r];\n\t}"
                 : "=r"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}
__device__ __forceinline__ void store_one(const Q8GemmArgs& a, long long at, float v) {
    if (a.ytype == UQ_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    else if (a.ytype == UQ_FP16) static_cast<__half*>(a.y)[at] = __float2half_rn(v);
    else static_cast<float*>(a.y)[at] = v;
}

__global__ void __launch_bounds__(THREADS, 3) q8_gemv_kernel(const Q8GemmArgs a, int S) {
    __shared__ int parts[8][TOKENS * 16];       // [warp][token][row]
    __shared__ int sums[TOKENS * ROWS];         // [token][row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t rank = S > 1 ? cluster_rank() : 0;
    const long long NT = (a.N + ROWS - 1) / ROWS, tiles = NT * ((a.M + TOKENS - 1) / TOKENS);
    const int blocks = (a.K + 63) / 64, shares = 4 * S, share = (int)rank * 4 + (warp >> 1);
    const int b0 = (int)((long long)blocks * share / shares), b1 = (int)((long long)blocks * (share + 1) / shares);
    for (long long tile = blockIdx.x / S; tile < tiles; tile += gridDim.x / S) {
        const int n0 = (int)(tile % NT) * ROWS, m0 = (int)(tile / NT) * TOKENS;
        const int row = n0 + (warp & 1) * 16 + g, tok = m0 + g;
        const int8_t* w0 = a.w + (long long)min(row, a.N - 1) * a.K + 16 * t;
        const int8_t* w1 = a.w + (long long)min(row + 8, a.N - 1) * a.K + 16 * t;
        const int8_t* x = a.x + (long long)min(tok, a.M - 1) * a.K + 16 * t;
        int acc[4] = {};
        for (int b = b0; b < b1; b += UNROLL) {
            uint4 p[UNROLL], q[UNROLL], v[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int k = (b + i) * 64;
                const bool in = b + i < b1 && k + 16 * t < a.K;
                p[i] = in ? __ldg(reinterpret_cast<const uint4*>(w0 + k)) : make_uint4(0, 0, 0, 0);
                q[i] = in ? __ldg(reinterpret_cast<const uint4*>(w1 + k)) : make_uint4(0, 0, 0, 0);
                v[i] = in && tok < a.M ? *reinterpret_cast<const uint4*>(x + k) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                mma_s8(acc, p[i].x, q[i].x, p[i].y, q[i].y, v[i].x, v[i].y);
                mma_s8(acc, p[i].z, q[i].z, p[i].w, q[i].w, v[i].z, v[i].w);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) parts[warp][(2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[i];
        __syncthreads();
        const int r = threadIdx.x & 31, c = threadIdx.x >> 5;      // this thread's output: row, token
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += parts[2 * i + (r >> 4)][c * 16 + (r & 15)];
        if (S > 1) {
            sums[threadIdx.x] = sum;
            cluster_sync();
            const int each = THREADS / S;
            if ((int)threadIdx.x / each == (int)rank) {
                sum = 0;
                for (int i = 0; i < S; ++i) sum += ld_cluster(smem_u32(&sums[threadIdx.x]), i);
                if (n0 + r < a.N && m0 + c < a.M)
                    store_one(a, (long long)(m0 + c) * a.N + n0 + r, (float)sum * a.sx[m0 + c] * a.sw[n0 + r]);
            }
            cluster_sync();
        } else {
            if (n0 + r < a.N && m0 + c < a.M)
                store_one(a, (long long)(m0 + c) * a.N + n0 + r, (float)sum * a.sx[m0 + c] * a.sw[n0 + r]);
            __syncthreads();
        }
    }
}

}  // namespace

cudaError_t launch_q8_gemm(const Q8GemmArgs& a, int sms, cudaStream_t st) {
    const long long tiles = (long long)((a.N + ROWS - 1) / ROWS) * ((a.M + TOKENS - 1) / TOKENS);
    int S = 1;
    while (S < MAX_SPLIT && tiles * S * 2 <= 3LL * sms && a.K >= 64 * 4 * S * 2) S *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S > 1 ? (unsigned)tiles * S : (unsigned)(tiles < 3LL * sms ? tiles : 3LL * sms));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, q8_gemv_kernel, a, S);
}

}  // namespace uq
