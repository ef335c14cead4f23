// uq_moe.cu -- expert routing: the stable sort of routes by expert, the rows carried there and back with the router's
// weights applied, and the gradients of both.
//
// All but the sort are memory-bound row copies: a token's row is read once and written to its topk places (or its
// topk rows are read and one row is written), in the widest vectors that rows are whole numbers of.
#include <atomic>
#include <type_traits>

#include "uq_mx.cuh"

namespace uq {

namespace {

// ---- sort --------------------------------------------------------------------------------------
// One cluster of CTAs, each CTA a contiguous range of the routes, each warp a contiguous range of its CTA's, walked
// in strips of 32.  Counting sort: (1) every warp counts its routes per expert (lanes of equal ids find each other by
// one ballot per bit of the id, and the group's first lane adds the group's size), the ids of eight strips requested
// together; (2) per expert the warps' counts become exclusive prefixes, the CTAs'
// totals are read through distributed shared memory, and a scan over the experts gives the offsets; (3) the warps
// walk their strips again, and a route's row is its warp's running count plus its rank within its group.  The order
// of the additions decides nothing: the result is the stable order.  Latency bounds it (a strip and pass cost about
// 0.3 us beside 31 other warps), so warps are added before strips: 8192 x 8 routes over 64 experts 11.0 us on 16 CTAs
// (14.4 on 8; 19.9 with match.any.sync, which took about 60 cycles per distinct id), 4096 routes 6.9 us.
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_BATCH = 8;                   // strips whose ids are requested together

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
    int v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.b32 %0, [a];\n\t}"
                 : "=r"(v) : "r"(smem_u32(p)), "r"(rank) : "memory");
    return v;
}

// the lanes of the warp with the same id as this one (ids below 2^bits)
__device__ __forceinline__ uint32_t same_lanes(int id, int bits) {
    uint32_t same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(0xffffffffu, (id >> b) & 1);
        same &= (id >> b) & 1 ? set : ~set;
    }
    return same;
}

__global__ void __launch_bounds__(SORT_THREADS) moe_sort_kernel(const int32_t* __restrict__ ids, long long n, int E,
                                                                int32_t* __restrict__ order, int32_t* __restrict__ pos,
                                                                int32_t* __restrict__ offsets) {
    extern __shared__ int sm[];
    int* hist = sm;                             // [SORT_WARPS][E]
    int* total = sm + SORT_WARPS * E;           // [E] this CTA's routes per expert
    int* base = total + E;                      // [E + 1] first row of each expert, then of this CTA's routes of it
    __shared__ int scan[SORT_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const long long strips = (n + 31) / 32, workers = (long long)ctas * SORT_WARPS;
    const long long w = (long long)rank * SORT_WARPS + warp;
    const long long s0 = strips * w / workers, s1 = strips * (w + 1) / workers;
    int* mine = hist + warp * E;
    const int bits = 32 - __clz(E);                                // of the ids 0 .. E

    for (int i = tid; i < SORT_WARPS * E; i += SORT_THREADS) hist[i] = 0;
    __syncthreads();
    int id[SORT_BATCH];
    auto load = [&](long long s) {              // ids of strips s .. s + SORT_BATCH; E: dropped, or past the end
#pragma unroll
        for (int j = 0; j < SORT_BATCH; ++j) {
            const long long i = (s + j) * 32 + lane;
            id[j] = s + j < s1 && i < n ? __ldg(ids + i) : E;
            if (id[j] < 0 || id[j] >= E) id[j] = E;
        }
    };
    for (long long s = s0; s < s1; s += SORT_BATCH) {
        load(s);
#pragma unroll
        for (int j = 0; j < SORT_BATCH; ++j) {
            if (s + j >= s1) break;
            const uint32_t same = same_lanes(id[j], bits);
            if (id[j] < E && lane == __ffs(same) - 1) mine[id[j]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += SORT_THREADS) {
        int c[SORT_WARPS], sum = 0;
#pragma unroll
        for (int v = 0; v < SORT_WARPS; ++v) c[v] = hist[v * E + e];
#pragma unroll
        for (int v = 0; v < SORT_WARPS; ++v) {
            hist[v * E + e] = sum;
            sum += c[v];
        }
        total[e] = sum;
    }
    cluster_sync();
    // E <= SORT_THREADS: thread e owns expert e
    int all = 0, before = 0;
    if (tid < E)
        for (uint32_t r = 0; r < ctas; ++r) {
            const int c = ld_cluster(total + tid, r);
            if (r < rank) before += c;
            all += c;
        }
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        scan[lane] = v;
    }
    __syncthreads();
    const int excl = incl - all + (warp ? scan[warp - 1] : 0);
    const int kept = scan[SORT_WARPS - 1];
    if (tid < E) {
        base[tid] = excl + before;
        if (rank == 0) offsets[tid] = excl;
    }
    if (rank == 0 && tid == 0) offsets[E] = kept;
    __syncthreads();
    for (long long s = s0; s < s1; s += SORT_BATCH) {
        if (s1 - s0 > SORT_BATCH) load(s);      // else the ids are still in registers
#pragma unroll
        for (int j = 0; j < SORT_BATCH; ++j) {
            if (s + j >= s1) break;
            const long long i = (s + j) * 32 + lane;
            const int e = id[j];
            const uint32_t same = same_lanes(e, bits);
            int row = -1;
            if (e < E) row = base[e] + mine[e] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (e < E && lane == __ffs(same) - 1) mine[e] += __popc(same);
            __syncwarp();
            if (i < n) pos[i] = row;
            if (row >= 0) order[row] = (int)i;
        }
    }
    for (long long r = kept + (long long)rank * SORT_THREADS + tid; r < n; r += (long long)ctas * SORT_THREADS) order[r] = -1;
    cluster_sync();                             // no CTA leaves while another may read its totals
}

// ---- rows --------------------------------------------------------------------------------------
// A unit is 32 lanes x U vectors of V elements of one row: 32 bytes a lane, or eight vectors.
template <class T, int V> struct Rows {
    static constexpr int U = 32 / (V * (int)sizeof(T)) < 8 ? 32 / (V * (int)sizeof(T)) : 8;
    static constexpr int SPAN = 32 * V * U;     // elements of a row per warp unit
};

template <class T, int V>
__global__ void __launch_bounds__(256) moe_gather_kernel(const T* __restrict__ x, const int32_t* __restrict__ pos,
                                                         const int32_t* __restrict__ offsets, int E, T* __restrict__ xs,
                                                         int T_, int topk, int H) {
    using R = Rows<T, V>;
    using VT = Vec<T, V>;
    const int lane = threadIdx.x & 31;
    const int chunks = (H + R::SPAN - 1) / R::SPAN;
    const int rows = T_ * topk;
    const int kept = min(max(__ldg(offsets + E), 0), rows);
    const long long front = (long long)T_ * chunks, units = front + (long long)(rows - kept) * chunks;
    for (long long u = blockIdx.x * 8LL + (threadIdx.x >> 5); u < units; u += gridDim.x * 8LL) {
        const bool tail = u >= front;
        const long long v = tail ? u - front : u;
        const int row = (int)(v / chunks), h = (int)(v % chunks) * R::SPAN + lane * V;
        VT a[R::U] = {};
        if (!tail) {
#pragma unroll
            for (int i = 0; i < R::U; ++i)
                if (h + i * 32 * V < H) a[i] = *reinterpret_cast<const VT*>(x + (long long)row * H + h + i * 32 * V);
        }
        for (int j = 0; j < (tail ? 1 : topk); ++j) {
            const int dst = tail ? kept + row : __ldg(pos + (long long)row * topk + j);
            if (dst < 0 || dst >= rows) continue;
#pragma unroll
            for (int i = 0; i < R::U; ++i)
                if (h + i * 32 * V < H) *reinterpret_cast<VT*>(xs + (long long)dst * H + h + i * 32 * V) = a[i];
        }
    }
}

// y[t] = sum_j w_j * rows[pos[t][j]] (WEIGHTED) or sum_j rows[pos[t][j]]
template <class T, int V, bool WEIGHTED>
__global__ void __launch_bounds__(256) moe_combine_kernel(const T* __restrict__ ys, const int32_t* __restrict__ pos,
                                                          const float* __restrict__ weights, T* __restrict__ y, int T_,
                                                          int topk, int H) {
    using R = Rows<T, V>;
    using VT = Vec<T, V>;
    const int lane = threadIdx.x & 31;
    const int chunks = (H + R::SPAN - 1) / R::SPAN;
    const int rows = T_ * topk;
    const long long units = (long long)T_ * chunks;
    for (long long u = blockIdx.x * 8LL + (threadIdx.x >> 5); u < units; u += gridDim.x * 8LL) {
        const int t = (int)(u / chunks), h = (int)(u % chunks) * R::SPAN + lane * V;
        float acc[R::U][V] = {};
        for (int j = 0; j < topk; ++j) {
            const int src = __ldg(pos + (long long)t * topk + j);
            if (src < 0 || src >= rows) continue;
            const float w = WEIGHTED ? __ldg(weights + (long long)t * topk + j) : 1.f;
#pragma unroll
            for (int i = 0; i < R::U; ++i)
                if (h + i * 32 * V < H) {
                    const VT a = *reinterpret_cast<const VT*>(ys + (long long)src * H + h + i * 32 * V);
#pragma unroll
                    for (int c = 0; c < V; ++c) acc[i][c] = fmaf(w, to_f32(a.v[c]), acc[i][c]);
                }
        }
#pragma unroll
        for (int i = 0; i < R::U; ++i)
            if (h + i * 32 * V < H) {
                VT a;
#pragma unroll
                for (int c = 0; c < V; ++c) a.v[c] = from_f32<T>(acc[i][c]);
                *reinterpret_cast<VT*>(y + (long long)t * H + h + i * 32 * V) = a;
            }
    }
}

// 8192 tokens of 4 routes, 4096 bf16: 91.5 us (6.4 TB/s, the memory's bound); a CTA per token that took its routes one
// after the other, with a block reduction each, 94.1 us, and 1 token of 8 routes 9.6 us against 4.1.
// One CTA per token (grid-stride), one warp per route: the token's row of dy against the route's row of ys, a dot product
// in a fixed order (lane l takes every 32nd vector, then a tree).  Then the rows nobody owns are zeroed.
template <class T, int V>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(const T* __restrict__ dy, const T* __restrict__ ys,
                                                               const int32_t* __restrict__ pos,
                                                               const float* __restrict__ weights,
                                                               const int32_t* __restrict__ offsets, int E,
                                                               T* __restrict__ dys, float* __restrict__ dw, int T_,
                                                               int topk, int H) {
    using R = Rows<T, V>;
    using VT = Vec<T, V>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rows = T_ * topk;
    for (int t = blockIdx.x; t < T_; t += gridDim.x)
        for (int j = warp; j < topk; j += warps) {
            const long long f = (long long)t * topk + j;
            const int r = __ldg(pos + f);
            const bool on = r >= 0 && r < rows;
            float sum = 0.f;
            if (on) {
                const float w = __ldg(weights + f);
                const T* pg = dy + (long long)t * H;
                const T* pa = ys + (long long)r * H;
                T* po = dys + (long long)r * H;
                for (int h0 = lane * V; h0 < H; h0 += R::SPAN) {
                    VT g[R::U], y[R::U];
#pragma unroll
                    for (int i = 0; i < R::U; ++i) {
                        const int h = h0 + i * 32 * V;
                        g[i] = y[i] = VT{};
                        if (h < H) {
                            g[i] = *reinterpret_cast<const VT*>(pg + h);
                            y[i] = *reinterpret_cast<const VT*>(pa + h);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < R::U; ++i) {
                        const int h = h0 + i * 32 * V;
                        VT o;
#pragma unroll
                        for (int c = 0; c < V; ++c) {
                            const float gf = to_f32(g[i].v[c]);
                            sum = fmaf(gf, to_f32(y[i].v[c]), sum);
                            o.v[c] = from_f32<T>(w * gf);
                        }
                        if (h < H) *reinterpret_cast<VT*>(po + h) = o;
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) dw[f] = sum;         // 0 for a dropped route
        }
    const int kept = min(max(__ldg(offsets + E), 0), rows);
    const VT zero = {};
    for (int r = kept + blockIdx.x; r < rows; r += gridDim.x)
        for (int h = threadIdx.x * V; h < H; h += blockDim.x * V) *reinterpret_cast<VT*>(dys + (long long)r * H + h) = zero;
}

constexpr size_t sort_smem(int E) { return ((size_t)SORT_WARPS * E + 2 * E + 1) * sizeof(int); }

int row_grid(long long rows, int H, int span, int sms) {
    const long long b = (rows * ((H + span - 1) / span) + 7) / 8, most = 64LL * sms;
    return (int)(b < most ? (b < 1 ? 1 : b) : most);
}

}  // namespace

namespace {
// CTAs of the largest cluster that the sort can have on this device: up to 16 (more than 8 are not portable, so they are
// asked for), once per device.  Any size is right.
int sort_cluster(int dev) {
    static std::atomic<int> known[64] = {};
    int n = known[dev].load(std::memory_order_relaxed);
    if (n) return n;
    for (n = 16; n > 1; n /= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n);
        cfg.blockDim = dim3(SORT_THREADS);
        cfg.dynamicSmemBytes = sort_smem(1024);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = n;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int placed = 0;
        if (cudaOccupancyMaxActiveClusters(&placed, moe_sort_kernel, &cfg) == cudaSuccess && placed > 0) break;
        cudaGetLastError();                     // a refusal is an answer
    }
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}
}  // namespace

cudaError_t launch_moe_sort(const int32_t* ids, long long n, int E, int32_t* order, int32_t* pos, int32_t* offsets,
                            cudaStream_t st) {
    static std::atomic<bool> configured[64] = {};  // per device; a second thread that sets the attributes too does no harm
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_relaxed);
    }
    int ctas = 1;                               // CTAs of the cluster: one strip a warp before another is added
    const int most = sort_cluster(dev);
    while (ctas < most && n > (long long)ctas * SORT_THREADS) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(SORT_THREADS);
    cfg.dynamicSmemBytes = sort_smem(E);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_sort_kernel, ids, n, E, order, pos, offsets);
}

namespace {
// calls f(element type, vector width as a constant): the widest vectors, of at most 16 bytes, that rows of H are whole
// numbers of (both gradients of 783 x 8 rows of 1794 bf16: element by element 50.6 us, in pairs 25.9)
template <class F> cudaError_t with_rows(int type, int H, F&& f) {
    return with_dtype(type, [&](auto t) {
        using T = decltype(t);
        constexpr int W = 16 / sizeof(T);
        if (H % W == 0) return f(t, std::integral_constant<int, W>());
        if (H % (W / 2) == 0) return f(t, std::integral_constant<int, W / 2>());
        if constexpr (W == 8)
            if (H % 2 == 0) return f(t, std::integral_constant<int, 2>());
        return f(t, std::integral_constant<int, 1>());
    });
}
}  // namespace

cudaError_t launch_moe_gather(const void* x, int type, const int32_t* pos, const int32_t* offsets, int E, void* xs, int T,
                              int topk, int H, int sms, cudaStream_t st) {
    return with_rows(type, H, [&](auto t, auto v) {
        using D = decltype(t);
        constexpr int V = decltype(v)::value;
        moe_gather_kernel<D, V><<<row_grid(T + (long long)T * topk / 8, H, Rows<D, V>::SPAN, sms), 256, 0, st>>>(
            static_cast<const D*>(x), pos, offsets, E, static_cast<D*>(xs), T, topk, H);
        return cudaGetLastError();
    });
}

cudaError_t launch_moe_combine(const void* ys, int type, const int32_t* pos, const float* weights, void* y, int T,
                               int topk, int H, int sms, cudaStream_t st) {
    return with_rows(type, H, [&](auto t, auto v) {
        using D = decltype(t);
        constexpr int V = decltype(v)::value;
        auto kernel = weights ? moe_combine_kernel<D, V, true> : moe_combine_kernel<D, V, false>;
        kernel<<<row_grid(T, H, Rows<D, V>::SPAN, sms), 256, 0, st>>>(static_cast<const D*>(ys), pos, weights,
                                                                    static_cast<D*>(y), T, topk, H);
        return cudaGetLastError();
    });
}

cudaError_t launch_moe_combine_grad(const void* dy, const void* ys, int type, const int32_t* pos, const float* weights,
                                    const int32_t* offsets, int E, void* dys, float* dw, int T, int topk, int H, int sms,
                                    cudaStream_t st) {
    const int grid = T < 64 * sms ? T : 64 * sms;
    return with_rows(type, H, [&](auto t, auto v) {
        using D = decltype(t);
        constexpr int V = decltype(v)::value;
        moe_combine_grad_kernel<D, V><<<grid, 32 * (topk < 8 ? topk : 8), 0, st>>>(
            static_cast<const D*>(dy), static_cast<const D*>(ys), pos, weights, offsets, E, static_cast<D*>(dys), dw, T, topk, H);
        return cudaGetLastError();
    });
}

}  // namespace uq
