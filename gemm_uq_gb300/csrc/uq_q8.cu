// uq_q8.cu -- rows in 8 bits with one scale each: the quantizer, the norm that ends in it, and the norm's gradient.
//
// RMSNorm with the residual's addition, per row of D values:
//     h = x + residual, rounded to the rows' type (it is the residual stream that the next layer reads, so that the norm
//         is the norm of what was stored),
//     y = h * r * gamma,  r = 1 / sqrt(mean(h^2) + eps),
//     s = max|y| / 127,  code = y / s to the nearest integer, ties to even.
// With m = max|h gamma|: s = r m / 127 and code = rne(h gamma * 127 / m), so the sum of squares and the maximum are one
// pass and one reduction.  The row stays in registers between that pass and the one that writes.
// Its gradient, g = dy gamma and n = h r:  dx = r (g - n mean(g n)) + dh,  dgamma = sum over rows of dy n.
//
// All of it is bound by memory: a row is read once and written once, in the widest accesses that its address, stride and
// length allow.  Small calls are a launch and a chain of latencies: one row of 4096 2.4 us.

#include "uq_q8.cuh"
#include "uq_tcgen05.cuh"

namespace uq {

namespace {

constexpr int MAX_THREADS = 1024;               // of a row; of the gradient's, whose threads hold more
constexpr int GRAD_THREADS = 512;
constexpr int PIPE_THREADS = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// What a row is multiplied with whose squares, or their sum, have left fp32: 2^31 squares of fp32's largest value then stay within
// it, and a sum that had left it is above 2^-32.
// (What rows in range pay for this path, us without / with it: 8192 x 8192 bf16 99.4 / 99.1, 16384 x 512 13.5 / 13.9, 4096 x 4001
// 43.7 / 45.1, 1 x 4096 2.6 / 2.7; gradient of 8192 x 4096 58.3 / 58.9.  fp16 rows cannot leave fp32 and have none of it.)
constexpr float FAR = 0x1p-80f;
// A barrier of one of a CTA's four groups of threads.  (Constant barriers: with a number in a register a CTA claims all 16, and
// fewer CTAs fit an SM, 16384 x 512 18.7 us instead of 13.7.)
__device__ __forceinline__ void group_sync(int group, int threads) {
    switch (group) {
        case 0: asm volatile("bar.sync 1, %0;" :: "r"(threads) : "memory"); break;
        case 1: asm volatile("bar.sync 2, %0;" :: "r"(threads) : "memory"); break;
        case 2: asm volatile("bar.sync 3, %0;" :: "r"(threads) : "memory"); break;
        default: asm volatile("bar.sync 4, %0;" :: "r"(threads) : "memory");
    }
}

// A thread's own prefetches: it copies 16-byte parts of a coming row to shared memory, each row's as one group, and reads back
// what it copied itself, so no other thread is waited for.
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
constexpr int ROWS_AHEAD = 2;                   // groups under way
__device__ __forceinline__ void oldest_copies_landed() { asm volatile("cp.async.wait_group %0;" :: "n"(ROWS_AHEAD - 1) : "memory"); }
template <class W> __device__ __forceinline__ W copied(uint32_t at) {
    static_assert(sizeof(W) == 16, "parts of 16 bytes");
    uint4 u;
    W w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
    memcpy(&w, &u, 16);
    return w;
}

// The 16-byte parts of a row.  A matrix without gaps begins at a 16-byte boundary, its rows need not (ODD): then parts are cut
// at the matrix's boundaries, and those at a row's ends hold elements of its neighbours, which are read as zeros and not written.
// Groups of threads take rows V apart (or a multiple), which all begin at the same place in a part: so a thread's columns stay
// the same.  Rows of an odd length in accesses of one element, and this way: bf16 norm of 4096 x 4097 with all outputs 84 us and
// 60, its gradient 127 and 55, quantizer 48 and 22; 8192 x 1001 fp32 37 and 26, 80 and 29, 20 and 11.  Where it does not pay: plan_of.
template <class T, int V, bool ODD> struct Parts {
    using W = Vec<T, V>;
    int off, D, count;                          // of the row's first element in its first part
    __device__ __forceinline__ Parts(long long row, int d) : D(d) {
        off = ODD ? (int)(row * d & (V - 1)) : 0;
        count = (off + d + (ODD ? V - 1 : 0)) / V;
    }
    __device__ __forceinline__ int column(int part, int j) const { return part * V - off + j; }
    __device__ __forceinline__ bool whole(int part) const { return !ODD || ((part || !off) && (part + 1) * V <= off + D); }
    __device__ __forceinline__ bool in(int part, int j) const { return !ODD || (unsigned)column(part, j) < (unsigned)D; }
    __device__ __forceinline__ void clip(W& w, int part) const {
        if (!whole(part)) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (!in(part, j)) w.v[j] = from_f32<T>(0.f);
        }
    }
    // row: the address of its first part
    __device__ __forceinline__ W load(const T* row, int part) const {
        if (whole(part)) return reinterpret_cast<const W*>(row)[part];
        W w;
#pragma unroll
        for (int j = 0; j < V; ++j) w.v[j] = in(part, j) ? row[part * V + j] : from_f32<T>(0.f);
        return w;
    }
    template <class Y> __device__ __forceinline__ void store(Y* row, int part, const Vec<Y, V>& w) const {
        if (whole(part)) reinterpret_cast<Vec<Y, V>*>(row)[part] = w;
        else
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (in(part, j)) row[part * V + j] = w.v[j];
    }
    __device__ __forceinline__ W of_vector(const T* p, int part) const {           // of gamma
        if constexpr (!ODD) return reinterpret_cast<const W*>(p)[part];
        else {
            W w;
#pragma unroll
            for (int j = 0; j < V; ++j) w.v[j] = in(part, j) ? p[column(part, j)] : from_f32<T>(0.f);
            return w;
        }
    }
    // Copies part `first` + `more` ahead; left: elements of the matrix from the row's first part on (beyond them nothing is read).
    // (Two steps, one of them common to a thread's parts: quantizer 38.8 -> 38.1 us, with the parts' numbers added first.)
    __device__ __forceinline__ void copy(uint32_t dst, const T* row, int first, int more, long long left) const {
        if constexpr (ODD) {
            const int part = first + more;
            const long long here = left - part * V;
            const int bytes = (here < V ? (int)here : V) * (int)sizeof(T);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(reinterpret_cast<const W*>(row) + part), "r"(bytes) : "memory");
        } else {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(reinterpret_cast<const W*>(row) + first + more) : "memory");
        }
    }
};

template <class P, int V> __device__ __forceinline__ void put_codes(const P& parts, int8_t* row, int part, const uint32_t (&c)[V]) {
    if (parts.whole(part)) store_codes<V>(row + (long long)part * V, c);
    else
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (parts.in(part, j)) row[part * V + j] = (int8_t)c[j];
}

struct RowArgs {
    const void *x, *residual, *gamma;
    void *h, *y;
    int8_t* codes;
    float* scales;
    long long ldx;
    int rows, D;
    float eps;
    int group;                                  // threads per row
    __half* wide;                               // the quantizer's codes as fp16 instead
    int early;                                  // the next kernel may start before this one is done
};

// the larger magnitude, NaN if one is
__device__ __forceinline__ float larger(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}

// NORM: the norm; else the plain quantizer (h, y, residual and gamma unused).
// V elements per access, NV accesses of a thread kept in registers; what a longer row has beyond is read again.
// PIPE (16-byte accesses, rows without a rest, many of them): the next rows' loads are under way while a row is reduced and
// written, and gamma stays in registers.  Without, a row is a chain of loads, a reduction, and stores; measured, 8192 rows of 8192
// bf16 with all outputs: PIPE 100 us (6.0 TB/s, 0.89 of the measured copy); else 256 threads a row with four accesses each 134
// us, 512 with two 152; the quantizer 37 (5.4 TB/s) and 44 us.
template <class T, int V, int NV, bool NORM, bool PIPE, bool ODD>
__global__ void __launch_bounds__(PIPE ? PIPE_THREADS : MAX_THREADS, PIPE ? 3 : 1) row_kernel(const RowArgs a) {
    using W = Vec<T, V>;
    __shared__ float sums[2][MAX_THREADS / 32];
    __shared__ float maxima[2][MAX_THREADS / 32];
    constexpr bool WIDE_RANGE = !std::is_same<T, __half>::value;   // squares of fp16 values stay within fp32
    extern __shared__ __align__(16) uint8_t ahead[];               // PIPE: [row][x, residual][part][thread] of 16 bytes
    const int per_cta = blockDim.x / a.group, tid = threadIdx.x % a.group, mine = threadIdx.x / a.group;
    const int warps = a.group >> 5, first_warp = mine * warps, lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * per_cta;
    const Parts<T, V, ODD> parts((long long)blockIdx.x * per_cta + mine, a.D);
    const int nvec = parts.count;
    if constexpr (!NORM)
        if (a.early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const T* gamma = static_cast<const T*>(a.gamma);
    auto x_of = [&](long long row) { return static_cast<const T*>(a.x) + row * a.ldx - parts.off; };
    auto res_of = [&](long long row) { return static_cast<const T*>(a.residual) + row * a.D - parts.off; };
    const bool has_res = NORM && a.residual;
    uint32_t slot = smem_u32(ahead) + threadIdx.x * 16, part = blockDim.x * 16, other = 0;
    auto request = [&](long long row) {
        if (row < a.rows) {
            const long long left = (a.rows - row) * a.D + parts.off;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * a.group < nvec) {
                    parts.copy(slot + other + i * part, x_of(row), tid, i * a.group, left);
                    if (has_res) parts.copy(slot + other + (NV + i) * part, res_of(row), tid, i * a.group, left);
                }
        }
        copies_issued();
        other ^= (has_res ? 2 : 1) * NV * part;
    };
    constexpr bool HELD = NORM && (PIPE || ODD);
    W held[HELD ? NV : 1];
    if constexpr (PIPE)
        for (int i = 0; i < ROWS_AHEAD; ++i) request((long long)blockIdx.x * per_cta + mine + i * step);
    if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * a.group < nvec) held[i] = parts.of_vector(gamma, tid + i * a.group);
    }
    // (this form and no other: written with `if constexpr`, the quantizer, which has no gamma, takes 39 us instead of 37)
    auto gam = [&](int i) { return !NORM ? W() : (HELD ? held[HELD ? i : 0] : parts.of_vector(gamma, tid + i * a.group)); };
    int buf = 0;
    for (long long base = (long long)blockIdx.x * per_cta; base < a.rows; base += step, buf ^= 1) {
        const long long row = base + mine;
        const bool on = row < a.rows;
        const T* x = x_of(on ? row : 0);
        const T* res = has_res ? res_of(on ? row : 0) : nullptr;
        auto add = [&](const W& w, const W& r) {                   // h
            float f[V], g[V];
            unpack(w, f);
            unpack(r, g);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] += g[j];
            return pack<T, V>(f);
        };
        auto load = [&](int v) { return res ? add(parts.load(x, v), parts.load(res, v)) : parts.load(x, v); };
        float sum = 0.f, most = 0.f;
        auto look = [&](const W& w, const W& g) {
            float f[V], c[V];
            unpack(w, f);
            if constexpr (NORM) unpack(g, c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if constexpr (NORM) sum = fmaf(f[j], f[j], sum);
                most = larger(most, NORM ? f[j] * c[j] : f[j]);
            }
        };
        W kept[NV];
        if constexpr (PIPE) {
            oldest_copies_landed();
            if (on) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * a.group < nvec) {
                        kept[i] = copied<W>(slot + other + i * part);
                        if (has_res) kept[i] = add(kept[i], copied<W>(slot + other + (NV + i) * part));
                        parts.clip(kept[i], tid + i * a.group);
                        look(kept[i], gam(i));
                    }
            }
            request(row + ROWS_AHEAD * step);                      // over what has just been read
        } else if (on) {
            if (res) {
                W r[NV];
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * a.group < nvec) {
                        kept[i] = parts.load(x, tid + i * a.group);
                        r[i] = parts.load(res, tid + i * a.group);
                    }
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * a.group < nvec) kept[i] = add(kept[i], r[i]);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * a.group < nvec) kept[i] = parts.load(x, tid + i * a.group);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * a.group < nvec) look(kept[i], gam(i));
            if constexpr (!ODD) {
                for (int v = tid + NV * a.group; v < nvec; v += a.group) look(load(v), NORM ? parts.of_vector(gamma, v) : W());
            }
        }
        if constexpr (NORM) sum = warp_sum(sum);
        most = __uint_as_float(warp_max(__float_as_uint(most)));   // (NaN and infinity are the largest patterns)
        if (warps > 1) {
            // two sets of slots: those of this row are written again only after the barrier of the next one
            if (lane == 0) {
                if constexpr (NORM) sums[buf][threadIdx.x >> 5] = sum;
                maxima[buf][threadIdx.x >> 5] = most;
            }
            __syncthreads();
            const int w = first_warp + lane;
            if constexpr (NORM) sum = warp_sum(lane < warps ? sums[buf][w] : 0.f);
            most = __uint_as_float(warp_max(__float_as_uint(lane < warps ? maxima[buf][w] : 0.f)));
        }
        if (!on) continue;
        const bool bad = !(most < __uint_as_float(INF_BITS));
        const float nan = __uint_as_float(0x7FC00000u);
        if constexpr (NORM) {
            float r = __frsqrt_rn(sum / (float)a.D + a.eps);
            if constexpr (WIDE_RANGE) {
                if (__builtin_expect(!(sum < __uint_as_float(INF_BITS)), 0)) {
                    // The squares, or their sum, have left fp32, which their mean need not: again, from FAR h.
                    sum = 0.f;
                    auto add_far = [&](const W& w) {
                        float f[V];
                        unpack(w, f);
#pragma unroll
                        for (int j = 0; j < V; ++j) sum = fmaf(f[j] * FAR, f[j] * FAR, sum);
                    };
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        if (tid + i * a.group < nvec) add_far(kept[i]);
                    if constexpr (!PIPE && !ODD) {
                        for (int v = tid + NV * a.group; v < nvec; v += a.group) add_far(load(v));
                    }
                    sum = warp_sum(sum);
                    if (warps > 1) {
                        group_sync(mine, a.group);                 // the first sums have been read
                        if (lane == 0) sums[buf][threadIdx.x >> 5] = sum;
                        group_sync(mine, a.group);
                        sum = warp_sum(lane < warps ? sums[buf][first_warp + lane] : 0.f);
                    }
                    r = FAR * __frsqrt_rn(sum / (float)a.D + FAR * (FAR * a.eps));
                }
            }
            if (tid == 0 && a.scales) a.scales[row] = bad ? nan : r * most / 127.f;
            // 127 / most stays finite for the smallest; a bad row's codes are zero
            const float up = most < 0x1p-64f ? 0x1p80f : 1.f;
            const float inv = most > 0.f && !bad ? 127.f / (most * up) : 0.f;
            const long long start = row * a.D - parts.off;
            T* h = a.h ? static_cast<T*>(a.h) + start : nullptr;
            T* y = a.y ? static_cast<T*>(a.y) + start : nullptr;
            int8_t* codes = a.codes ? a.codes + start : nullptr;
            auto write = [&](int v, const W& w, const W& g) {
                float f[V], c[V];
                if (h) parts.store(h, v, w);
                unpack(w, f);
                unpack(g, c);
#pragma unroll
                for (int j = 0; j < V; ++j) c[j] *= f[j];
                if (y) {
                    float o[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = c[j] * r;
                    parts.store(y, v, pack<T, V>(o));
                }
                if (codes) {
                    uint32_t q[V];
                    if (up != 1.f) {
#pragma unroll
                        for (int j = 0; j < V; ++j) c[j] *= up;
                    }
                    if (bad) {
#pragma unroll
                        for (int j = 0; j < V; ++j) c[j] = 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < V; ++j) q[j] = code_bits(c[j], inv);
                    put_codes(parts, codes, v, q);
                }
            };
            // before anything is written, which may be over x or the residual
            if constexpr (!PIPE && !ODD) {
                for (int v = tid + NV * a.group; v < nvec; v += a.group) write(v, load(v), parts.of_vector(gamma, v));
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * a.group < nvec) write(tid + i * a.group, kept[i], gam(i));
        } else {
            const float s = bad ? nan : __fdiv_rn(most, 127.f);
            if (tid == 0) a.scales[row] = s;
            const Divisor d(s);
            const long long start = row * a.D - parts.off;
            auto write = [&](int v, const W& w) {
                float f[V];
                uint32_t c[V];
                unpack(w, f);
                d.codes(f, c);
                if (a.wide) {
#pragma unroll
                    for (int j = 0; j < V; ++j) f[j] = (float)(int8_t)c[j];
                    parts.store(a.wide + start, v, pack<__half, V>(f));
                } else {
                    put_codes(parts, a.codes + start, v, c);
                }
            };
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * a.group < nvec) write(tid + i * a.group, kept[i]);
            if constexpr (!PIPE && !ODD) {
                for (int v = tid + NV * a.group; v < nvec; v += a.group) write(v, load(v));
            }
        }
    }
}

// out = code * scale, rounded once; V codes a thread.  ODD: rows of more than V codes that are not whole V, so that a
// thread's codes may belong to two rows (fp32: 4 codes a thread, whose 16 bytes lie beside its neighbours'; 4096 x 4096 11 us,
// with 16 codes a thread 18).  4096 x 4097 bf16 8.8 us, 27 with a code a thread.
template <class T, int V, bool ODD>
__global__ void __launch_bounds__(256) dequant_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                      T* __restrict__ out, long long n, int K) {
    for (long long i = (blockIdx.x * 256LL + threadIdx.x) * V; i < n; i += gridDim.x * (256LL * V)) {
        const long long row = n <= 0xFFFFFFFFll ? (long long)((uint32_t)i / (uint32_t)K) : i / K;
        const float s = scales[row];
        int own = V;                            // codes of that row
        float next = s;
        if constexpr (ODD) {
            const long long end = (row + 1) * K;
            if (end - i < V && end < n) own = (int)(end - i), next = scales[row + 1];
            if (n - i < V) {
                for (int j = 0; j < (int)(n - i); ++j) out[i + j] = from_f32<T>((float)codes[i + j] * (j < own ? s : next));
                continue;
            }
        }
        const Vec<int8_t, V> c = *reinterpret_cast<const Vec<int8_t, V>*>(codes + i);
        constexpr int O = V * sizeof(T) <= 16 ? V : 16 / sizeof(T);
#pragma unroll
        for (int b = 0; b < V; b += O) {
            Vec<T, O> o;
#pragma unroll
            for (int j = 0; j < O; ++j) o.v[j] = from_f32<T>((float)c.v[b + j] * (b + j < own ? s : next));
            *reinterpret_cast<Vec<T, O>*>(out + i + b) = o;
        }
    }
}

struct GradArgs {
    const void *dy, *h, *gamma, *dh;
    void* dx;
    float* partials;                            // [row groups of the grid][D]
    int rows, D;
    float eps;
    int group;
};

// A group of threads takes every so many-th row; its share of dgamma stays in registers (of a longer row, in its CTA's row of
// `partials`, where a CTA has one group) until its rows are done; then a CTA's groups are added in order.  Named barriers, so
// that a CTA's groups do not wait for one another.  gamma stays in registers: read again for every row, four accesses a thread,
// it kept L1 73 % busy.  PIPE as above.  Measured, 8192 rows of 4096 bf16 with dh: 59 us (4.6 TB/s, the addition of the
// partials in it), without PIPE 68, with gamma read again 96.
template <class T, int V, int NV, bool PIPE, bool ODD>
__global__ void __launch_bounds__(GRAD_THREADS, 1) norm_grad_kernel(const GradArgs a) {
    using W = Vec<T, V>;
    extern __shared__ __align__(16) uint8_t ahead[];               // PIPE: [row][dy, h, dh][part][thread] of 16 bytes; then
    __shared__ float2 sums[2][GRAD_THREADS / 32];
    const int per_cta = blockDim.x / a.group, tid = threadIdx.x % a.group, mine = threadIdx.x / a.group;
    const int warps = a.group >> 5, first_warp = mine * warps, lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * per_cta;
    const Parts<T, V, ODD> parts((long long)blockIdx.x * per_cta + mine, a.D);
    const int nvec = parts.count;
    const uint32_t part16 = blockDim.x * 16, stage = 3 * NV * part16;
    float* together = reinterpret_cast<float*>(ahead + (PIPE ? ROWS_AHEAD * stage : 0));           // several groups: [D]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");                // the kernel that adds the partials
    const T* gamma = static_cast<const T*>(a.gamma);
    float* part = a.partials + (long long)blockIdx.x * a.D;
    const uint32_t slot = smem_u32(ahead) + threadIdx.x * 16;
    uint32_t other = 0;
    auto request = [&](long long row) {
        if (row < a.rows) {
            const long long at = ODD ? row * a.D - parts.off : (row * nvec + tid) * V;     // of the row, or of this thread's first part
            const long long left = (a.rows - row) * a.D + parts.off;
            constexpr int OWN = ODD ? 1 : 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (tid + i * a.group >= nvec) continue;
                parts.copy(slot + other + i * part16, static_cast<const T*>(a.dy) + at, OWN * tid, i * a.group, left);
                parts.copy(slot + other + (NV + i) * part16, static_cast<const T*>(a.h) + at, OWN * tid, i * a.group, left);
                if (a.dh) parts.copy(slot + other + (2 * NV + i) * part16, static_cast<const T*>(a.dh) + at, OWN * tid, i * a.group, left);
            }
        }
        copies_issued();
        other ^= stage;
    };
    if constexpr (PIPE)
        for (int i = 0; i < ROWS_AHEAD; ++i) request((long long)blockIdx.x * per_cta + mine + i * step);
    W gam[NV];
    float dg[NV][V] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (tid + i * a.group < nvec) gam[i] = parts.of_vector(gamma, tid + i * a.group);
    if constexpr (!ODD) {
        for (int v = tid + NV * a.group; v < nvec; v += a.group)
#pragma unroll
            for (int j = 0; j < V; ++j) part[(long long)v * V + j] = 0.f;
    }
    int buf = 0;
    for (long long row = (long long)blockIdx.x * per_cta + mine; row < a.rows; row += step, buf ^= 1) {
        const long long at = row * a.D - parts.off;
        const T *dy = static_cast<const T*>(a.dy) + at, *h = static_cast<const T*>(a.h) + at;
        const T* dh = a.dh ? static_cast<const T*>(a.dh) + at : nullptr;
        T* dx = static_cast<T*>(a.dx) + at;
        float s1 = 0.f, s2 = 0.f;
        auto look = [&](const W& u, const W& w, const W& g) {
            float t[V], f[V], c[V];
            unpack(u, t);
            unpack(w, f);
            unpack(g, c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s1 = fmaf(f[j], f[j], s1);
                s2 = fmaf(t[j] * c[j], f[j], s2);
            }
        };
        W ku[NV], kw[NV], kd[NV];
        if constexpr (PIPE) {
            oldest_copies_landed();
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * a.group < nvec) {
                    ku[i] = copied<W>(slot + other + i * part16);
                    kw[i] = copied<W>(slot + other + (NV + i) * part16);
                    if (dh) kd[i] = copied<W>(slot + other + (2 * NV + i) * part16);
                    parts.clip(ku[i], tid + i * a.group);
                    parts.clip(kw[i], tid + i * a.group);
                }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * a.group < nvec) {
                    ku[i] = parts.load(dy, tid + i * a.group);
                    kw[i] = parts.load(h, tid + i * a.group);
                    if (dh) kd[i] = parts.load(dh, tid + i * a.group);
                }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * a.group < nvec) look(ku[i], kw[i], gam[i]);
        if constexpr (PIPE) request(row + ROWS_AHEAD * step);      // over what has just been read
        if constexpr (!ODD) {
            for (int v = tid + NV * a.group; v < nvec; v += a.group) look(parts.load(dy, v), parts.load(h, v), parts.of_vector(gamma, v));
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (warps > 1) {
            if (lane == 0) sums[buf][threadIdx.x >> 5] = make_float2(s1, s2);
            asm volatile("bar.sync %0, %1;" :: "r"(1 + mine), "r"(a.group) : "memory");
            const float2 p = lane < warps ? sums[buf][first_warp + lane] : make_float2(0.f, 0.f);
            s1 = warp_sum(p.x);
            s2 = warp_sum(p.y);
        }
        float r = __frsqrt_rn(s1 / (float)a.D + a.eps);
        float c = r * r * (s2 / (float)a.D);                       // n mean(g n) = h r (r s2 / D)
        if constexpr (!std::is_same<T, __half>::value) {
            if (__builtin_expect(!(s1 < __uint_as_float(INF_BITS)), 0)) {
                // The squares, or their sum, have left fp32, which their mean need not: both sums again, from FAR h.
                s1 = s2 = 0.f;
                auto look_far = [&](const W& u, const W& w, const W& g) {
                    float t[V], f[V], e[V];
                    unpack(u, t);
                    unpack(w, f);
                    unpack(g, e);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        s1 = fmaf(f[j] * FAR, f[j] * FAR, s1);
                        s2 = fmaf(t[j] * e[j], f[j] * FAR, s2);
                    }
                };
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * a.group < nvec) look_far(ku[i], kw[i], gam[i]);
                if constexpr (!ODD) {
#pragma unroll 1
                    for (int v = tid + NV * a.group; v < nvec; v += a.group) look_far(parts.load(dy, v), parts.load(h, v), parts.of_vector(gamma, v));
                }
                s1 = warp_sum(s1);
                s2 = warp_sum(s2);
                if (warps > 1) {
                    asm volatile("bar.sync %0, %1;" :: "r"(1 + mine), "r"(a.group) : "memory");    // the first sums have been read
                    if (lane == 0) sums[buf][threadIdx.x >> 5] = make_float2(s1, s2);
                    asm volatile("bar.sync %0, %1;" :: "r"(1 + mine), "r"(a.group) : "memory");
                    const float2 p = lane < warps ? sums[buf][first_warp + lane] : make_float2(0.f, 0.f);
                    s1 = warp_sum(p.x);
                    s2 = warp_sum(p.y);
                }
                const float far = __frsqrt_rn(s1 / (float)a.D + FAR * (FAR * a.eps));              // r / FAR
                r = FAR * far;
                c = r * (far * (s2 / (float)a.D));
            }
        }
        auto write = [&](int v, const W& u, const W& w, const W& g, const W& d, float (&out)[V]) {
            float t[V], f[V], e[V];
            unpack(u, t);
            unpack(w, f);
            unpack(g, e);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                out[j] = fmaf(t[j] * r, f[j], out[j]);
                e[j] = r * fmaf(-f[j], c, t[j] * e[j]);
            }
            if (dh) {
                unpack(d, t);
#pragma unroll
                for (int j = 0; j < V; ++j) e[j] += t[j];
            }
            parts.store(dx, v, pack<T, V>(e));
        };
        if constexpr (!ODD) {
            for (int v = tid + NV * a.group; v < nvec; v += a.group) {
                float out[V];
#pragma unroll
                for (int j = 0; j < V; ++j) out[j] = part[(long long)v * V + j];
                write(v, parts.load(dy, v), parts.load(h, v), parts.of_vector(gamma, v), dh ? parts.load(dh, v) : W(), out);
#pragma unroll
                for (int j = 0; j < V; ++j) part[(long long)v * V + j] = out[j];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (tid + i * a.group < nvec) write(tid + i * a.group, ku[i], kw[i], gam[i], kd[i], dg[i]);
    }
    for (int g = 0; g < per_cta; ++g) {
        if (g == mine)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * a.group < nvec)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if (!parts.in(tid + i * a.group, j)) continue;
                        const int col = parts.column(tid + i * a.group, j);
                        const float v = g ? together[col] + dg[i][j] : dg[i][j];
                        if (g == per_cta - 1) part[col] = v;
                        else together[col] = v;
                    }
        if (g < per_cta - 1) __syncthreads();
    }
}

// dgamma = the sum of the P partial rows, in order: a CTA of 32 x 8 threads takes 32 columns, its warps every 8th row, and
// adds the warps' sums in order.
__global__ void __launch_bounds__(256) partials_sum_kernel(const float* __restrict__ partials, float* __restrict__ out, int P, int D) {
    __shared__ float part[8][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float s = 0.f;
    if (col < D) {
#pragma unroll 8
        for (int p = w; p < P; p += 8) s += ld_written(partials + (long long)p * D + col);
    }
    part[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && col < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
        out[col] = s;
    }
}

// Elements per access: 16 bytes, or 4, or one element, whatever divides the row and its addresses' alignment (pointers are
// 16-byte aligned).
template <class T> int access(int D, long long ld) {
    const long long both = (long long)D | ld;
    if (both % (16 / (int)sizeof(T)) == 0) return 16 / sizeof(T);
    return both % (4 / (int)sizeof(T)) == 0 ? 4 / sizeof(T) : 1;
}

// Threads per row and accesses per thread for rows of nvec accesses: `most_nv` of them where there are rows enough, else as many
// threads as the row has accesses.
struct Shape { int group, nv; };
Shape shape_of(int nvec, int most_threads, int most_nv, bool few) {
    Shape s = {32, 1};
    while (s.group < most_threads && s.group * (few ? 1 : most_nv) < nvec) s.group *= 2;
    while (s.nv < 4 && s.group * s.nv < nvec) s.nv *= 2;
    return s;
}

// How rows are taken: elements per access; whether in 16-byte parts that rows do not begin or end with.
// The parts' ends cost each access a test, and gamma, which does not begin where a row's part does, is read by elements.  So the
// norm and its gradient (`plain`: the quantizer) take rows by elements where that is more than the wider accesses save: rows of
// few parts, and 16-bit rows that the forms which copy ahead do not hold, of which gamma and the rows fill the registers.
// Measured, us, by elements / in parts: gradient of 400 x 101 bf16 5.2 / 8.4, 301 8.6 / 7.0; norm of 4000 x 101 3.8 / 4.4; 4000
// x 8191 bf16 139 / 150 and 154 / 211, 16001 226 / 238 and 370 / 357; 4000 x 8003 fp32 153 / 99 and 192 / 84; quantizer 4000 x
// 8191 bf16 85 / 44, 8003 fp32 91 / 36.
// Few elements in all are spread over more threads, as few rows are, and so are norms that do not copy ahead: 400 x 601 bf16 3.4 us
// and 5.5 with four parts a thread, gradient of 400 x 301 7.0 and 12.5, norm of 4000 x 301 7.1 and 10.1.
struct Plan { int v; bool odd; Shape s; };
template <class T> Plan plan_of(bool plain, int D, long long ld, int rows, int most_threads, int most_nv, int sms) {
    constexpr int WIDE = 16 / sizeof(T);
    const bool few = rows <= 2 * sms;
    const int v = access<T>(D, ld);
    if (v < WIDE && (ld == D || rows == 1)) {
        const int most = (int)(((long long)D + 2 * WIDE - 2) / WIDE);              // parts of a row, begun anywhere
        Shape s = shape_of(most, most_threads, most_nv, few || (long long)rows * most <= (long long)sms * (most_threads * 5 / 8));
        if (!plain && s.nv < most_nv) s = shape_of(most, most_threads, most_nv, true);
        const bool pays = plain || (most > 32 && (sizeof(T) == 4 || most <= 1024));
        if (pays && s.group * s.nv >= most) return {WIDE, true, s};
    }
    return {v, false, shape_of(D / v, most_threads, most_nv, few)};
}

// CTAs for rows in groups of `per`, at most `most`; a group's rows V apart or a multiple
int grid_of(long long tiles, long long most, const Plan& p) {
    return (int)(tiles <= most ? tiles : (p.odd && most >= p.v ? most / p.v * p.v : most));
}

// f(integral constants V, NV, ODD)
template <class T, class F> cudaError_t with_plan(const Plan& p, F&& f) {
    auto by_nv = [&](auto V, auto ODD) {
        if (p.s.nv == 1) return f(V, std::integral_constant<int, 1>(), ODD);
        if (p.s.nv == 2) return f(V, std::integral_constant<int, 2>(), ODD);
        return f(V, std::integral_constant<int, 4>(), ODD);
    };
    constexpr int WIDE = 16 / sizeof(T), FOUR = 4 / sizeof(T);
    if (p.odd) return by_nv(std::integral_constant<int, WIDE>(), std::true_type());
    if (p.v == WIDE) return by_nv(std::integral_constant<int, WIDE>(), std::false_type());
    if (FOUR > 1 && p.v == FOUR) return by_nv(std::integral_constant<int, FOUR>(), std::false_type());
    return by_nv(std::integral_constant<int, 1>(), std::false_type());
}

template <bool NORM> cudaError_t launch_rows(const RowArgs& a0, int type, int sms, cudaStream_t st) {
    return with_dtype(type, [&](auto t) {
        using T = decltype(t);
        RowArgs a = a0;
        const Plan p = plan_of<T>(!NORM, a.D, a.ldx, a.rows, MAX_THREADS, 4, sms);
        a.group = p.s.group;
        const int block = a.group < 128 ? 128 : a.group, per = block / a.group;
        const long long tiles = ((long long)a.rows + per - 1) / per;
        return with_plan<T>(p, [&](auto V_, auto NV_, auto ODD_) {
            constexpr int V = decltype(V_)::value, NV = decltype(NV_)::value;
            constexpr bool ODD = decltype(ODD_)::value;
            if constexpr (V * sizeof(T) == 16 && NV == 4) {
                if (block <= PIPE_THREADS && (ODD || a.group * NV >= a.D / V) && a.rows > 2 * sms) {
                    static Done done = {};
                    const cudaError_t e = configure(row_kernel<T, V, NV, NORM, true, ODD>, done, 200 * 1024);
                    if (e != cudaSuccess) return e;
                    row_kernel<T, V, NV, NORM, true, ODD><<<grid_of(tiles, (long long)sms * 3 * (PIPE_THREADS / block), p), block,
                                                           ROWS_AHEAD * (a.residual ? 2 : 1) * NV * 16 * block, st>>>(a);
                    return cudaGetLastError();
                }
            }
            if constexpr (NORM && ODD && sizeof(T) == 2 && NV > 1) {
                return cudaErrorInvalidConfiguration;              // (not among plan_of's)
            } else {
                row_kernel<T, V, NV, NORM, false, ODD><<<grid_of(tiles, (long long)sms * (2048 / block), p), block, 0, st>>>(a);
                return cudaGetLastError();
            }
        });
    });
}

}  // namespace

cudaError_t launch_quantize_q8(const void* x, int type, long long ldx, int8_t* codes, void* wide, float* scales, int rows, int K,
                               bool early, int sms, cudaStream_t st) {
    RowArgs a = {};
    a.x = x;
    a.ldx = ldx;
    a.codes = codes;
    a.scales = scales;
    a.wide = static_cast<__half*>(wide);
    a.early = early;
    a.rows = rows;
    a.D = K;
    return launch_rows<false>(a, type, sms, st);
}

cudaError_t launch_dequant_q8(const int8_t* codes, const float* scales, void* out, int type, int rows, int K, int sms, cudaStream_t st) {
    return with_dtype(type, [&](auto t) {
        using T = decltype(t);
        auto go = [&](auto V, auto ODD) {
            constexpr int N = decltype(V)::value;
            const long long n = (long long)rows * K, ctas = (n + 256 * N - 1) / (256 * N);
            dequant_kernel<T, N, decltype(ODD)::value><<<(unsigned)(ctas < 16LL * sms ? ctas : 16LL * sms), 256, 0, st>>>(codes, scales, static_cast<T*>(out), n, K);
            return cudaGetLastError();
        };
        constexpr int V = sizeof(T) == 4 ? 4 : 16;
        if (K % V == 0) return go(std::integral_constant<int, V>(), std::false_type());
        if (K > V) return go(std::integral_constant<int, V>(), std::true_type());
        return go(std::integral_constant<int, 1>(), std::false_type());
    });
}

cudaError_t launch_rmsnorm_q8(const void* x, const void* residual, const void* gamma, int type, long long ldx, void* h, void* y,
                              int8_t* codes, float* scales, int rows, int D, float eps, int sms, cudaStream_t st) {
    const RowArgs a = {x, residual, gamma, h, y, codes, scales, ldx, rows, D, eps};
    return launch_rows<true>(a, type, sms, st);
}

// CTAs of the gradient, each with a partial row of dgamma.
static Plan grad_plan(int type, int rows, int D, int sms) {
    return type == UQ_FP32 ? plan_of<float>(false, D, D, rows, GRAD_THREADS, 2, sms) : plan_of<__half>(false, D, D, rows, GRAD_THREADS, 2, sms);
}
static int grad_block(const Shape& s) { return s.group < 256 ? 256 : s.group; }
int norm_grad_partials(int type, int rows, int D, int sms) {
    const Plan p = grad_plan(type, rows, D, sms);
    const int block = grad_block(p.s), per = block / p.s.group;
    return grid_of(((long long)rows + per - 1) / per, (long long)sms * (GRAD_THREADS / block), p);
}

cudaError_t launch_rmsnorm_grad(const void* dy, const void* h, const void* gamma, const void* dh, int type, void* dx, float* dgamma,
                                float* partials, int rows, int D, float eps, int sms, cudaStream_t st) {
    const Plan p = grad_plan(type, rows, D, sms);
    const int P = norm_grad_partials(type, rows, D, sms), group = p.s.group;
    const GradArgs a = {dy, h, gamma, dh, dx, partials, rows, D, eps, group};
    cudaError_t e = with_dtype(type, [&](auto t) {
        using T = decltype(t);
        const int block = grad_block(p.s);
        const size_t add = block > group ? (size_t)D * sizeof(float) : 0;
        return with_plan<T>(p, [&](auto V_, auto NV_, auto ODD_) {
            constexpr int V = decltype(V_)::value, NV = decltype(NV_)::value;
            constexpr bool ODD = decltype(ODD_)::value;
            if constexpr (V * sizeof(T) == 16 && NV <= 2) {
                if (rows > 2 * sms) {
                    static Done done = {};
                    const cudaError_t f = configure(norm_grad_kernel<T, V, NV, true, ODD>, done, 200 * 1024);
                    if (f != cudaSuccess) return f;
                    norm_grad_kernel<T, V, NV, true, ODD><<<P, block, ROWS_AHEAD * 3 * NV * 16 * block + add, st>>>(a);
                    return cudaGetLastError();
                }
            }
            if constexpr (ODD && sizeof(T) == 2 && NV > 2) {
                return cudaErrorInvalidConfiguration;              // (not among plan_of's)
            } else {
                norm_grad_kernel<T, V, NV, false, ODD><<<P, block, add, st>>>(a);
                return cudaGetLastError();
            }
        });
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((D + 31) / 32);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, partials_sum_kernel, (const float*)partials, dgamma, P, D);
}

}  // namespace uq
