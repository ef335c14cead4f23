// uq_route.cu -- the router of a mixture of experts: expert ids and weights of each token's logits, and the gradient.
//
// Scores s = softmax(x) or 1 / (1 + e^-x); choice values c = s + bias (the bias balances the experts' load and does not
// enter the weights).  Optionally the experts form groups of equal size: a group counts the sum of its group_top highest c,
// and only the top_groups best groups stay.  The topk highest c are chosen, in that order, equal values by lower index.
// Weights: s of the chosen, divided by their sum where asked, times a factor.
//
// The choice is the one that 64-bit scores give.  Where the order of c is that of x itself (no bias, groups by their best
// member) it needs no scores.  Else c is computed in fp32 with a bound on its error, and where two neighbours in the order,
// or the last group that stays and the first that does not, are nearer than their bounds allow to tell, the token is done
// again in 64 bits (one expert's fp64 exponential costs a warp some thousand cycles: this part has few fp64 units).
//
// One warp per token; its choice values lie in shared memory.
#include "uq_mx.cuh"

namespace uq {

namespace {

constexpr int WARPS = 4;                        // tokens of a CTA
constexpr uint32_t ALL = 0xffffffffu;
__device__ __forceinline__ float low_value() { return __uint_as_float(0xFF800000u); }

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int T, E, topk, sigmoid, groups, top_groups, group_top, renorm;
    float scale;
};

__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
    return v;
}
template <class S> __device__ __forceinline__ S warp_add(S v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
    return v;
}

// 1 / (1 + e^-x) times e^-low for low <= 0 (low = 0: itself): sigmoids far below one keep their ratios
__device__ __forceinline__ float sigmoid_over(float x, float low) {
    return x >= 0.f ? 1.f / (1.f + expf(-x)) : expf(x - low) / (1.f + expf(x));
}

// Choice values are compared as integers in the order of the numbers, fp32 in 32 bits and fp64 in 64 (this part compares
// integers far faster than fp64).  A value of NaN (a NaN logit or bias) ranks below all numbers and above what cannot be chosen,
// which is none_of(): in 32 bits it has minus infinity's place, which no value that can be chosen takes, and in 64 bits that of
// a number far below fp32's, so that even a group's sum of two of them stays above none_of().
__device__ __forceinline__ int key_of(float v) {
    const int k = __float_as_int(v);
    return k < 0 ? k ^ 0x7FFFFFFF : k;
}
__device__ __forceinline__ float value_of(int k) { return __int_as_float(k < 0 ? k ^ 0x7FFFFFFF : k); }
__device__ __forceinline__ long long key_of(double v) {
    const long long k = __double_as_longlong(v);
    return k < 0 ? k ^ 0x7FFFFFFFFFFFFFFFll : k;
}
__device__ __forceinline__ double value_of(long long k) { return __longlong_as_double(k < 0 ? k ^ 0x7FFFFFFFFFFFFFFFll : k); }
template <class S> __device__ __forceinline__ S none_of();
template <> __device__ __forceinline__ int none_of<int>() { return -0x7FFFFFFF - 1; }
template <> __device__ __forceinline__ long long none_of<long long>() { return -0x7FFFFFFFFFFFFFFFll; }
__device__ __forceinline__ int ranked(float c, bool can) { return can ? key_of(fmaxf(c, low_value())) : none_of<int>(); }
__device__ __forceinline__ long long ranked(double c, bool can) {
    return !can ? none_of<long long>() : key_of(c > -1.7e308 ? c : -1.7e308);
}
// the sum of two values, as they are compared
template <class S> __device__ __forceinline__ S together(S a, S b) { return key_of(value_of(a) + value_of(b)); }

// The largest of the lanes' values and, among equal ones, the smallest index; index E where none can be chosen.
__device__ __forceinline__ void best_of(int& c, int& e, int E) {
    const int top = __reduce_max_sync(ALL, c);
    e = __reduce_min_sync(ALL, c == top ? e : E);
    c = top;
    if (c == none_of<int>()) e = E;
}
__device__ __forceinline__ void best_of(long long& c, int& e, int E) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const long long oc = __shfl_xor_sync(ALL, c, o);
        const int oe = __shfl_xor_sync(ALL, e, o);
        if (oc > c || (oc == c && oe < e)) c = oc, e = oe;
    }
    if (c == none_of<long long>()) e = E;
}

// Scores in approximate instructions, with a bound on their error as a part of the largest score, one:
//   sigmoid  e^-x loses 2^-22 and, by its argument's rounding, |x| 2^-23.7, of which s (1 - s) reaches s; the sum 1 + e^-x loses
//            2^-24 s and the reciprocal 2^-23 s: together at most 0.84 of 2^-22, near x = 1.7;
//   softmax  of each score s the same of e^(x - m) (2^-22 and |x - m| 2^-23), and of the sum, which all scores share, its terms'
//            mean loss and E / 32 + 5 roundings.  With u = 2^-24: a part p of the sum at the largest logit and the rest at a distance
//            d lose p (1 - p) d < 2 of 2 u by the distances, the rest at most (4 + 3 + 5 + E / 32) u.
// The addition of the bias loses 2^-24 of its result besides.
__device__ __forceinline__ float exp_about(float x) {
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
    return e;
}
__device__ __forceinline__ float reciprocal_about(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float score_error(const RouteArgs& a) { return a.sigmoid ? 0x1p-22f : (float)(a.E / 32 + 16) * 0x1p-24f; }
// whether fp32 values of this error (`terms` of them in each of the two) are in their order; never where one is infinite or NaN
__device__ __forceinline__ bool apart(const RouteArgs& a, float hi, float lo, float terms, float best = 0.f) {
    return hi - lo > 2.f * terms * ((fmaxf(fabsf(hi), fabsf(lo)) + best) * 0x1p-24f + score_error(a));
}
// The same for the sums of two groups, given the best value of each lane's group.  A sum loses its terms' errors, 2^-24 of each term
// and 2^-24 of itself.  A bias may give the terms opposite signs, so that each is larger than the sum; but the first is at most
// the best of all, and the second at most that and the sum together: group_top times the error of one value, with the sum and the
// best in the place of the value.
__device__ __forceinline__ bool groups_apart(const RouteArgs& a, int hi, int lo, int b1) {
    return apart(a, value_of(hi), value_of(lo), (float)a.group_top, fmaxf(value_of(__reduce_max_sync(ALL, b1)), 0.f));
}

// Chooses from c[0 .. E) (the warp's shared memory; chosen experts are taken out of it), in fp32 or 64 bits.  Lane j returns choice j, -1 for
// none.  `exact`: c is the logits themselves; `sure`: every decision had more distance than the error of the values.
template <class S, class T>
__device__ __forceinline__ int choose(const RouteArgs& a, S* c, const T* x, bool exact, bool& sure) {
    constexpr bool WIDE = sizeof(S) == 8;
    const int lane = threadIdx.x & 31, E = a.E;
    const S none = none_of<S>();
    sure = true;
    if (a.groups > 1) {
        // 2^k lanes per group, each every 2^k-th member; the group's best two by shuffles
        int per = 32;
        while (per * a.groups > 32) per >>= 1;
        const int g = lane / per, size = E / a.groups;
        S b1 = none, b2 = none;
        if (g < a.groups)
            for (int i = lane % per; i < size; i += per) {
                const S v = c[g * size + i];
                b2 = max(b2, min(b1, v));
                b1 = max(b1, v);
            }
        for (int o = 1; o < per; o <<= 1) {
            const S o1 = __shfl_xor_sync(ALL, b1, o), o2 = __shfl_xor_sync(ALL, b2, o);
            b2 = max(min(b1, o1), max(b2, o2));
            b1 = max(b1, o1);
        }
        S total = a.group_top == 2 && b2 > none ? together(b1, b2) : b1;
        if (g >= a.groups) total = none;
        int ahead = 0;                          // groups before this one
        for (int o = 0; o < a.groups; ++o) {
            const S t = __shfl_sync(ALL, total, o * per);
            ahead += t > total || (t == total && o < g);
        }
        const bool stays = total > none && ahead < a.top_groups;
        if constexpr (!WIDE) {
            if (!exact) {
                const int worst = __reduce_min_sync(ALL, stays ? total : 0x7FFFFFFF), next = __reduce_max_sync(ALL, stays ? none : total);
                if (next > none && !groups_apart(a, worst, next, b1)) sure = false;
            }
        }
        const uint32_t open_ = __ballot_sync(ALL, stays && lane % per == 0);
        // without a bias the order within the groups is that of x
        if (!a.bias) exact = true;
        for (int e = lane; e < E; e += 32) {
            const float v = a.bias ? 0.f : to_f32(x[e]) + 0.f;
            if (!(open_ >> (e / size * per) & 1u)) c[e] = none;
            else if constexpr (WIDE) c[e] = a.bias ? c[e] : ranked((double)v, v != low_value());
            else c[e] = a.bias ? c[e] : ranked(v, v != low_value());
        }
        __syncwarp();
    }
    S mine = none;                              // the lane's best remaining expert: of e = lane, lane + 32, ...
    int at = lane;
    auto rescan = [&] {
        mine = none;
        at = lane;
        for (int e = lane; e < E; e += 32) {
            const S v = c[e];
            if (v > mine) mine = v, at = e;
        }
    };
    rescan();
    int id = -1, last = -1;
    float before = 0.f;
    for (int j = 0; j < a.topk; ++j) {
        S v = mine;
        int e = at;
        best_of(v, e, E);
        if (e == E) break;
        if constexpr (!WIDE) {
            const float value = value_of(v);
            if (!exact && j && !apart(a, before, value, 1.f)) {
                // the same logit and bias give the same value: the lower index is right
                if (!(before == value && to_f32(x[e]) == to_f32(x[last]) && (!a.bias || a.bias[e] == a.bias[last]))) sure = false;
            }
            before = value;
            last = e;
        }
        if (lane == j) id = e;
        if (at == e && mine > none) {
            c[e] = none;
            rescan();
        }
    }
    if constexpr (!WIDE) {
        // What is not chosen: near the last choice only where the logit and the bias are its own.  (All of it, since between two
        // of the same there may be a third that fp32 does not tell from them.)
        if (!exact && last >= 0) {
            const float xl = to_f32(x[last]), bl = a.bias ? a.bias[last] : 0.f;
            bool near = false;
            for (int e = lane; e < E; e += 32)
                if (c[e] > none && !apart(a, before, value_of(c[e]), 1.f)) near |= to_f32(x[e]) != xl || (a.bias && a.bias[e] != bl);
            if (__any_sync(ALL, near)) sure = false;
        }
    }
    return id;
}

// Choice values of a token in fp32, into c[] (by_logit: the logits themselves), and in 64 bits.
template <class T> __device__ __forceinline__ void values(const RouteArgs& a, int* c, const T* x, bool by_logit) {
    const int lane = threadIdx.x & 31;
    float m = low_value(), over = 0.f;
    if (!a.sigmoid && !by_logit) {
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, to_f32(x[e]));
        m = warp_max_f(m);
        for (int e = lane; e < a.E; e += 32) {
            const float v = to_f32(x[e]);
            if (v > low_value()) over += exp_about(v - m);
        }
        over = reciprocal_about(warp_add(over));
    }
    for (int e = lane; e < a.E; e += 32) {
        const float v = to_f32(x[e]), b = a.bias ? a.bias[e] : 0.f;
        float s = by_logit || v != v ? v : (a.sigmoid ? reciprocal_about(1.f + exp_about(-v)) : exp_about(v - m) * over);
        c[e] = ranked(s + b, v != low_value() && b != low_value());
    }
    __syncwarp();
}
template <class T> __device__ __forceinline__ void values(const RouteArgs& a, long long* c, const T* x) {
    const int lane = threadIdx.x & 31;
    double m = 0, sum = 1;
    if (!a.sigmoid) {
        float top = low_value();
        for (int e = lane; e < a.E; e += 32) top = fmaxf(top, to_f32(x[e]));
        m = (double)warp_max_f(top);
        sum = 0;
#pragma unroll 4
        for (int e = lane; e < a.E; e += 32) {
            const float v = to_f32(x[e]);
            if (v > low_value()) sum += exp((double)v - m);
        }
        sum = warp_add(sum);
    }
#pragma unroll 4
    for (int e = lane; e < a.E; e += 32) {
        const float v = to_f32(x[e]), b = a.bias ? a.bias[e] : 0.f;
        double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - m) / sum;
        if (v != v) s = (double)v;
        c[e] = ranked(s + (double)b, v != low_value() && b != low_value());
    }
    __syncwarp();
}

// Weight (without the factor) of lane j's choice; `nan`: this lane has seen a NaN among the logits.
template <class T> __device__ __forceinline__ float weight_of(const RouteArgs& a, const T* x, int id, bool nan) {
    const int lane = threadIdx.x & 31;
    const float v = id >= 0 ? to_f32(x[id]) : low_value();
    if (a.renorm) {
        // among the chosen alone, from the largest logit of them: their ratios survive where the scores underflow
        bool bad = id >= 0 && v != v;
        const float m = warp_max_f(v);
        float w = 0.f;
        if (a.sigmoid) {
            if (id >= 0) w = sigmoid_over(v, fminf(m, 0.f));
        } else {
            bad |= nan;                         // makes all of softmax NaN
            if (id >= 0) w = expf(v - m);
        }
        const float all = warp_add(w);
        return __any_sync(ALL, bad) ? __uint_as_float(0x7FC00000u) : (all > 0.f || all != all ? w / all : 0.f);
    }
    if (a.sigmoid) return 1.f / (1.f + expf(-v));
    float m = low_value(), sum = 0.f;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, to_f32(x[e]));
    m = warp_max_f(m);
    for (int e = lane; e < a.E; e += 32) {
        const float u = to_f32(x[e]);
        if (u != low_value()) sum += expf(u - m);
    }
    return expf(v - m) / warp_add(sum);
}

// The same choice with the values in registers: lane l holds experts l NL .. l NL + NL - 1 (of E <= 32 NL), so that the lowest
// of the lanes with the largest value has the lower index.  Groups have to be whole lanes, a power of two of them.
// Scores that need 64 bits: sigmoids of the choices that are too near to tell are done again, a lane each; anything else
// that fp32 leaves open (softmax with a bias, groups, more than 32 near ones) is done by choose() in 64 bits.
template <class T, int NL>
__global__ void __launch_bounds__(WARPS * 32) route_lanes_kernel(const RouteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * NL;
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
    constexpr int V = NL * (int)sizeof(T) < 16 ? NL : 16 / (int)sizeof(T);
    const bool whole = a.E % V == 0;            // rows of whole accesses
    long long* mine = reinterpret_cast<long long*>(smem + (size_t)warp * a.E * 8);
    float bias[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) bias[i] = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.f;
    for (long long t = (long long)blockIdx.x * WARPS + warp; t < a.T; t += (long long)gridDim.x * WARPS) {
        const T* x = static_cast<const T*>(a.logits) + t * a.E;
        float v[NL];
        int c[NL];
#pragma unroll
        for (int i = 0; i < NL; i += V) {
            Vec<T, V> w;
            if (whole) {
                if (e0 + i < a.E) w = *reinterpret_cast<const Vec<T, V>*>(x + e0 + i);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (e0 + i + j < a.E) w.v[j] = x[e0 + i + j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) v[i + j] = e0 + i + j < a.E ? to_f32(w.v[j]) : low_value();
        }
        if (by_logit) {
#pragma unroll
            for (int i = 0; i < NL; ++i) c[i] = ranked(v[i] + 0.f, v[i] != low_value());
        } else {
            float m = 0.f, over = 1.f;
            if (!a.sigmoid) {
                m = v[0];
#pragma unroll
                for (int i = 1; i < NL; ++i) m = fmaxf(m, v[i]);
                m = warp_max_f(m);
                over = 0.f;
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    if (v[i] > low_value()) over += exp_about(v[i] - m);
                over = reciprocal_about(warp_add(over));
            }
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                float s = a.sigmoid ? reciprocal_about(1.f + exp_about(-v[i])) : exp_about(v[i] - m) * over;
                if (v[i] != v[i]) s = v[i];
                c[i] = ranked(s + bias[i], v[i] != low_value() && bias[i] != low_value());
            }
        }
        const int none = none_of<int>();
        bool exact = by_logit, groups_sure = true;
        int doubt = 0;                          // 1: near neighbours; 2: something near behind the 32nd
        if (a.groups > 1) {
            const int per = a.E / a.groups / NL, g = lane / per;   // lanes of a group
            int b1 = none, b2 = none;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                b2 = max(b2, min(b1, c[i]));
                b1 = max(b1, c[i]);
            }
            for (int o = 1; o < per; o <<= 1) {
                const int o1 = __shfl_xor_sync(ALL, b1, o), o2 = __shfl_xor_sync(ALL, b2, o);
                b2 = max(min(b1, o1), max(b2, o2));
                b1 = max(b1, o1);
            }
            int total = a.group_top == 2 && b2 > none ? together(b1, b2) : b1;
            if (g >= a.groups) total = none;
            int ahead = 0;
            for (int o = 0; o < a.groups; ++o) {
                const int other = __shfl_sync(ALL, total, o * per);
                ahead += other > total || (other == total && o < g);
            }
            const bool stays = total > none && ahead < a.top_groups;
            if (!exact) {
                const int worst = __reduce_min_sync(ALL, stays ? total : 0x7FFFFFFF), next = __reduce_max_sync(ALL, stays ? none : total);
                groups_sure = next == none || groups_apart(a, worst, next, b1);
            }
            if (!a.bias) exact = true;          // the order within the groups is that of x
#pragma unroll
            for (int i = 0; i < NL; ++i)
                c[i] = !stays ? none : (a.bias ? c[i] : ranked(v[i] + 0.f, v[i] != low_value()));
        }
        // lane j: choice j; behind the last one, those that are too near to it.  What is near behind the 32nd is looked at below.
        int id = -1, last = -1, found = 0;
        float before = 0.f;
        for (int j = 0; j <= 32; ++j) {
            if (exact && j == a.topk) break;
            int best = c[0], at = 0;
#pragma unroll
            for (int i = 1; i < NL; ++i)
                if (c[i] > best) best = c[i], at = i;
            const int top = __reduce_max_sync(ALL, best), who = __ffs(__ballot_sync(ALL, best == top)) - 1;
            if (top == none) break;
            const float value = value_of(top);
            const int e = __shfl_sync(ALL, e0 + at, who);
            if (!exact && j) {
                if (apart(a, before, value, 1.f)) {
                    if (j >= a.topk) break;
                } else if (j == 32 || !(before == value && to_f32(x[e]) == to_f32(x[last]) && (!a.bias || a.bias[e] == a.bias[last]))) {
                    doubt |= j == 32 ? 2 : 1;   // (the same logit and bias give the same value: the lower index is right)
                }
            }
            before = value;
            last = e;
            if (lane == j) id = e;
            found = j + 1;
            if (lane == who)
#pragma unroll
                for (int i = 0; i < NL; ++i)
                    if (i == at) c[i] = none;
        }
        if (doubt == 2 && groups_sure) {        // all equal, as padding may be?  Then the lower indices are right, too
            const int e31 = __shfl_sync(ALL, id, 31);
            const float xl = to_f32(x[e31]), bl = a.bias ? a.bias[e31] : 0.f;
            bool near = to_f32(x[last]) != xl || (a.bias && a.bias[last] != bl);
#pragma unroll
            for (int i = 0; i < NL; ++i)
                if (c[i] > none && !apart(a, before, value_of(c[i]), 1.f)) near |= v[i] != xl || bias[i] != bl;
            if (!__any_sync(ALL, near)) doubt = 0;
        }
        if (doubt || !groups_sure) {
            const float u = id >= 0 ? to_f32(x[id]) : 0.f;
            const bool odd = u != u || (id >= 0 && a.bias && a.bias[id] != a.bias[id]);
            if (groups_sure && a.sigmoid && found < 32 && !__any_sync(ALL, odd)) {
                double d = id >= 0 ? 1.0 / (1.0 + exp(-(double)u)) + (double)(a.bias ? a.bias[id] : 0.f) : 0.0;
                int rank = 0, got = -1;
                for (int o = 0; o < found; ++o) {
                    const double od = __shfl_sync(ALL, d, o);
                    const int oe = __shfl_sync(ALL, id, o);
                    rank += od > d || (od == d && oe < id);
                }
                for (int o = 0; o < found; ++o) {
                    const int r = __shfl_sync(ALL, rank, o), oe = __shfl_sync(ALL, id, o);
                    if (r == lane) got = oe;
                }
                id = got;
            } else {
                bool yes;
                __syncwarp();
                values(a, mine, x);
                id = choose(a, mine, x, false, yes);
            }
        }
        if (lane >= a.topk) id = -1;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < NL; ++i) nan |= v[i] != v[i];
        const float w = weight_of(a, x, id, nan);
        if (lane < a.topk) {
            a.ids[t * a.topk + lane] = id;
            a.weights[t * a.topk + lane] = id >= 0 ? w * a.scale : 0.f;
        }
    }
}

template <class T>
__global__ void __launch_bounds__(WARPS * 32) route_kernel(const RouteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool by_logit = !a.bias && (a.groups == 1 || a.group_top == 1);
    uint8_t* mine = smem + (size_t)warp * a.E * (by_logit ? 4 : 8);
    for (long long t = (long long)blockIdx.x * WARPS + warp; t < a.T; t += (long long)gridDim.x * WARPS) {
        const T* x = static_cast<const T*>(a.logits) + t * a.E;
        bool sure;
        __syncwarp();
        values(a, reinterpret_cast<int*>(mine), x, by_logit);
        int id = choose(a, reinterpret_cast<int*>(mine), x, by_logit, sure);
        if (!sure) {
            __syncwarp();
            values(a, reinterpret_cast<long long*>(mine), x);
            id = choose(a, reinterpret_cast<long long*>(mine), x, false, sure);
        }
        bool nan = false;
        for (int e = lane; e < a.E; e += 32) nan |= to_f32(x[e]) != to_f32(x[e]);
        const float w = weight_of(a, x, id, nan);
        if (lane < a.topk) {
            a.ids[t * a.topk + lane] = id;
            a.weights[t * a.topk + lane] = id >= 0 ? w * a.scale : 0.f;
        }
    }
}

struct RouteGradArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    void* dlogits;
    int T, E, topk, sigmoid, renorm;
    float scale;
};

// Gradient of a token's logits.  With dw the weights' gradient times the factor, over the routes that have an expert:
//   renormalised, w_j = s_j / sum s: q_j = w_j (dw_j - sum_i w_i dw_i), dx of the chosen q_j (softmax), q_j (1 - s_j) (sigmoid)
//   softmax: ds_e = sum of dw over the routes to e, dx_e = s_e (ds_e - sum s ds);  sigmoid: dx_e = s_e (1 - s_e) ds_e
// Lane j holds route j; an expert's routes are found by all lanes' ids in turn, in order, so one expert may be named twice.
template <class T>
__global__ void __launch_bounds__(WARPS * 32) route_grad_kernel(const RouteGradArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (long long t = (long long)blockIdx.x * WARPS + warp; t < a.T; t += (long long)gridDim.x * WARPS) {
        const T* x = static_cast<const T*>(a.logits) + t * a.E;
        T* dx = static_cast<T*>(a.dlogits) + t * a.E;
        int id = lane < a.topk ? a.ids[t * a.topk + lane] : -1;
        if (id < 0 || id >= a.E) id = -1;
        const float dw = id >= 0 ? a.dweights[t * a.topk + lane] * a.scale : 0.f;
        const float v = id >= 0 ? to_f32(x[id]) : low_value();
        float q = dw;                           // what route j adds to its expert
        float m = low_value(), sum = 0.f, dot = 0.f;
        if (a.renorm) {
            // (from the largest of them; where all are minus infinity the weights are 0 and there is no gradient)
            const float top = warp_max_f(v);
            float w = 0.f;
            if (id >= 0 && top != low_value()) w = a.sigmoid ? sigmoid_over(v, fminf(top, 0.f)) : expf(v - top);
            const float all = warp_add(w);
            w = all > 0.f || all != all ? w / all : 0.f;
            q = w * (dw - warp_add(w * dw));
            if (a.sigmoid) q *= v >= 0.f ? expf(-v) / (1.f + expf(-v)) : 1.f / (1.f + expf(v));        // 1 - s
            if (id < 0) q = 0.f;
        } else if (!a.sigmoid) {
            for (int e = lane; e < a.E; e += 32) m = fmaxf(m, to_f32(x[e]));
            m = warp_max_f(m);
            for (int e = lane; e < a.E; e += 32) {
                const float u = to_f32(x[e]);
                if (u != low_value()) sum += expf(u - m);
            }
            sum = warp_add(sum);
            dot = warp_add(id >= 0 ? expf(v - m) / sum * dw : 0.f);
        }
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            float ds = 0.f;
            for (int j = 0; j < a.topk; ++j) {
                const int at = __shfl_sync(ALL, id, j);
                const float add = __shfl_sync(ALL, q, j);
                if (at == e) ds += add;
            }
            if (e >= a.E) continue;
            const float u = to_f32(x[e]);
            float d = ds;
            if (!a.renorm) {
                if (a.sigmoid) {
                    const float n = expf(-fabsf(u));               // s (1 - s) = n / (1 + n)^2
                    d = ds * (n / ((1.f + n) * (1.f + n)));
                } else {
                    d = u == low_value() ? 0.f : expf(u - m) / sum * (ds - dot);
                }
            }
            dx[e] = from_f32<T>(d);
        }
    }
}

}  // namespace

cudaError_t launch_moe_route(const void* logits, int type, const float* bias, int32_t* ids, float* weights, int T, int E, int topk,
                             bool sigmoid, int groups, int top_groups, int group_top, bool renorm, float scale, int sms,
                             cudaStream_t st) {
    const RouteArgs a = {logits, bias, ids, weights, T, E, topk, sigmoid, groups, top_groups, group_top, renorm, scale};
    const bool by_logit = !bias && (groups == 1 || group_top == 1);
    const size_t smem = (size_t)WARPS * E * (by_logit ? 4 : 8);    // at most 32 KB
    const long long ctas = ((long long)T + WARPS - 1) / WARPS, most = 16LL * sms;
    const unsigned grid = (unsigned)(ctas < most ? ctas : most);
    // values in registers where the groups are whole lanes
    const int nl = E <= 64 ? 2 : (E <= 256 ? 8 : 32);
    const int size = E / groups, per = size / nl;
    const bool lanes = groups == 1 || (size % nl == 0 && (per & (per - 1)) == 0);
    return with_dtype(type, [&](auto t) {
        using T_ = decltype(t);
        if (!lanes) route_kernel<T_><<<grid, WARPS * 32, smem, st>>>(a);
        else if (nl == 2) route_lanes_kernel<T_, 2><<<grid, WARPS * 32, by_logit ? 0 : smem, st>>>(a);
        else if (nl == 8) route_lanes_kernel<T_, 8><<<grid, WARPS * 32, by_logit ? 0 : smem, st>>>(a);
        else route_lanes_kernel<T_, 32><<<grid, WARPS * 32, by_logit ? 0 : smem, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_moe_route_grad(const void* logits, int type, const int32_t* ids, const float* dweights, void* dlogits, int T,
                                  int E, int topk, bool sigmoid, bool renorm, float scale, int sms, cudaStream_t st) {
    const RouteGradArgs a = {logits, ids, dweights, dlogits, T, E, topk, sigmoid, renorm, scale};
    const long long ctas = ((long long)T + WARPS - 1) / WARPS, most = 16LL * sms;
    return with_dtype(type, [&](auto t) {
        route_grad_kernel<decltype(t)><<<(unsigned)(ctas < most ? ctas : most), WARPS * 32, 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace uq
