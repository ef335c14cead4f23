// uq_q8.cuh -- the 8-bit code of a value, and accesses of several elements.
#pragma once

#include <cstring>
#include <type_traits>

#include "uq_mx.cuh"

namespace uq {

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t INF_BITS = 0x7F800000u;

// The low byte of the sum with 1.5 * 2^23 is the nearest integer's two's complement (|v| < 2^22, ties to even).
constexpr float ROUND = 12582912.f;
__device__ __forceinline__ uint32_t code_bits(float v) { return __float_as_uint(v + ROUND); }
// code = t * inv rounded once, to the integer
__device__ __forceinline__ uint32_t code_bits(float t, float inv) { return __float_as_uint(fmaf(t, inv, ROUND)); }

// Quotients x / s as correctly rounded fp32 divisions by Markstein's theorem (1990): r = RN(1 / s), q = x r,
// q + (x - q s) r with the residual by FMA.  Scales far from 1 are divided by the instruction sequence for all values.
struct Divisor {
    float s, r;
    bool fast, zero;
    __device__ __forceinline__ explicit Divisor(float scale) : s(scale) {
        r = 1.f / scale;
        fast = scale >= 0x1p-90f && scale <= 0x1p90f;
        zero = !(scale > 0.f) || scale > 3.0e38f;
    }
    template <int V> __device__ __forceinline__ void codes(const float (&x)[V], uint32_t (&c)[V]) const {
        if (fast) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float q = x[j] * r;
                c[j] = code_bits(fmaf(fmaf(-q, s, x[j]), r, q));
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] = zero ? 0u : code_bits(fminf(fmaxf(__fdiv_rn(x[j], s), -127.f), 127.f));
        }
    }
};

// An access's elements in fp32, and back with one rounding.
template <class T, int V> __device__ __forceinline__ void unpack(const Vec<T, V>& w, float (&f)[V]) {
    if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = to_f32(w.v[j]);
    } else {
        uint32_t u[V / 2];
        memcpy(u, &w, sizeof u);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                f[2 * j] = bf16lo_f32(u[j]);
                f[2 * j + 1] = bf16hi_f32(u[j]);
            } else {
                f[2 * j] = half_bits_f32((uint16_t)u[j]);
                f[2 * j + 1] = half_bits_f32((uint16_t)(u[j] >> 16));
            }
        }
    }
}
template <class T, int V> __device__ __forceinline__ Vec<T, V> pack(const float (&f)[V]) {
    Vec<T, V> w;
    if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) w.v[j] = from_f32<T>(f[j]);
    } else {
        uint32_t u[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(f[2 * j + 1]), "f"(f[2 * j]));
            else
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u[j]) : "f"(f[2 * j + 1]), "f"(f[2 * j]));
        }
        memcpy(&w, u, sizeof u);
    }
    return w;
}

// the low bytes of V words, stored together
template <int V> __device__ __forceinline__ void store_codes(int8_t* p, const uint32_t (&w)[V]) {
    if constexpr (V == 1) {
        *p = (int8_t)w[0];
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)__byte_perm(w[0], w[1], 0x0040);
    } else {
        uint32_t o[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            o[i] = __byte_perm(__byte_perm(w[4 * i], w[4 * i + 1], 0x0040), __byte_perm(w[4 * i + 2], w[4 * i + 3], 0x0040), 0x5410);
        if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = o[0];
        else *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
    }
}

}  // namespace uq
