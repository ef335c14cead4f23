// uq_mx_quant.cuh -- a lane's share of the microscaled quantization: 8 consecutive values of a row, whose block is 4
// lanes (MXFP4) or 2 (NVFP4) of the warp.
#pragma once

#include <cstring>
#include <type_traits>

#include "uq_mx.cuh"

namespace uq {

// 8 values of a row, as loaded
template <class T> struct Raw {
    Vec<T, 16 / sizeof(T)> part[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 w = ld_written(reinterpret_cast<const uint4*>(p) + i);
            memcpy(&part[i], &w, 16);
        }
    }
    __device__ __forceinline__ float at(int i) const {
        constexpr int V = 16 / sizeof(T);
        return to_f32(part[i / V].v[i % V]);
    }
};

// absmax of the 8 values as a bit pattern of fp32: infinities and NaN compare above all numbers
template <class T> __device__ __forceinline__ uint32_t absmax8(const Raw<T>& x) {
    if constexpr (sizeof(T) == 2) {
        // in packed 16-bit patterns: without the sign, their order as integers is the values' order
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
        uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        const uint16_t h = (uint16_t)max(m & 0xFFFFu, m >> 16);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return (uint32_t)h << 16;
        else return __float_as_uint(half_bits_f32(h));
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x.at(i)) & 0x7FFFFFFFu);
        return m;
    }
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 w, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// The divisor of the NVFP4 scales, 6 t, and its reciprocal.  divide() is a correctly rounded quotient by Markstein's
// theorem (1990): with r = RN(1 / t) and q an approximation, q + (a - q t) r, the residual by FMA.  Far from 1 (fast
// false) underflow could spoil the residual.
struct SixT {
    float t, r;
    bool fast;
    __device__ __forceinline__ explicit SixT(float tscale) : t(6.f * tscale), r(1.f / (6.f * tscale)),
                                                               fast(t >= 0x1p-40f && t <= 0x1p40f) {}
    __device__ __forceinline__ float divide(float a) const {
        const float q = a * r;
        return q > 1000.f ? q : fmaf(fmaf(-q, t, a), r, q);        // over 448 it saturates, whatever its last bits
    }
};

// codes of a lane's 8 values and the scale byte of its block (the block's lanes agree on it)
template <int FMT, class T>
__device__ __forceinline__ uint32_t quantize8(const Raw<T>& x, const SixT& six, float tscale, uint32_t& byte) {
    uint32_t am = absmax8(x);
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    float v[8];
    if constexpr (FMT == UQ_MXFP4) {
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const int e = (int)(am >> 23);          // exponent field: floor(log2 a) + 127, 0 for zero and subnormals
        byte = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
        const float inv = __uint_as_float(e == 255 ? 0u : (254u - byte) << 23);    // 2^(127 - byte), a normal number
#pragma unroll
        for (int i = 0; i < 8; i += 2) {                                           // exact: a power of two
            const float2 t = mul2(make_float2(x.at(i), x.at(i + 1)), make_float2(inv, inv));
            v[i] = t.x;
            v[i + 1] = t.y;
        }
    } else {
        const bool bad = am >= 0x7F800000u;
        const float amax = __uint_as_float(am);
        byte = bad ? 0x7Fu : e4m3_of(six.fast ? six.divide(amax) : __fdiv_rn(amax, six.t));
        const float d = e4m3_value(byte) * tscale;
        if (!bad && d >= 0x1p-100f && d <= 0x1p100f && amax <= d * 0x1p100f) {
            // x / d in the same way (with quotients far inside the range: where the block scale has saturated they can
            // exceed it, and the residual of an infinite q is infinite with the other sign).  A tie comes out as a tie:
            // its residual is exact.  For 16-bit types an approximate reciprocal (1 ulp) will do: before its rounding the
            // corrected quotient is within 2^-44 of the true one, and the code changes only if a middle between a tie of
            // the grid and an fp32 neighbour lies in between.  Over all 24-bit divisors and 16-bit values such middles are
            // 2^-43 away, but for one pair (2^-48: 1 / 2 by 2 - 2^-23, times powers of two), which is tested.
            float r;
            if constexpr (sizeof(T) == 2) asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
            else r = __frcp_rn(d);
            const float2 r2 = make_float2(r, r), nd2 = make_float2(-d, -d);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 x2 = make_float2(x.at(i), x.at(i + 1)), q2 = mul2(x2, r2), t = fma2(fma2(q2, nd2, x2), r2, q2);
                v[i] = t.x;
                v[i + 1] = t.y;
            }
        } else {
            const bool zero = bad || !(d > 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = zero ? x.at(i) * 0.f : __fdiv_rn(x.at(i), d);
        }
    }
    return e2m1_pack8(v);
}

// the word of this lane's scale tile (4 blocks) from the blocks' bytes; the same in all of the tile's lanes
template <int FMT> __device__ __forceinline__ uint32_t scale_word(uint32_t byte, int lane) {
    constexpr int LPB = FMT == UQ_MXFP4 ? 4 : 2;                 // lanes per block
    byte <<= 8 * ((lane / LPB) & 3);
    byte |= __shfl_xor_sync(0xffffffffu, byte, LPB);
    return byte | __shfl_xor_sync(0xffffffffu, byte, 2 * LPB);
}

}  // namespace uq
