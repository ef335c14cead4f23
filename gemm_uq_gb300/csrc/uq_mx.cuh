// uq_mx.cuh -- microscaled 4-bit floating point: formats, the scale tile layout, and the PTX wrappers of the
// block-scaled tensor-core product (sm_103a).
//
// A microscaled row of K values is K e2m1 codes (two per byte, low nibble = even k) and one scale byte per
// block: UQ_MXFP4 blocks of 32, scale 2^(byte - 127) (255: NaN); UQ_NVFP4 blocks of 16, scale an e4m3 value.
//
// Scale tiles.  Scales are kept in 512-byte tiles of 128 rows x 4 blocks, byte (r % 32) * 16 + (r / 32) * 4 + b:
// 32 rows of 16 bytes, which is what one tcgen05.cp.32x128b copies into four tensor-memory columns, where the
// block-scaled MMA expects them.  Tiles follow each other along k, then along the rows.  Rows in segments (one
// per expert) start a tile each: segment e, whose first row is o, starts at row tile o / 128 + e.  Since
// floor((o + c) / 128) + 1 >= floor(o / 128) + ceil(c / 128), segments never share a tile, and no prefix sum of
// padded counts is needed to find one.
#pragma once

#include <cuda_fp16.h>

#include "uq_kernels.h"

namespace uq {

constexpr unsigned int FAULT_MX_WAIT = 16u;     // a block-scaled product kernel's bounded wait ran out

__host__ __device__ constexpr int mx_block(int fmt) { return fmt == UQ_NVFP4 ? 16 : 32; }
// k columns of one scale tile (4 blocks), and scale tiles along K
__host__ __device__ constexpr int mx_tile_k(int fmt) { return 4 * mx_block(fmt); }
__host__ __device__ inline int mx_ktiles(int K, int fmt) { return (K + mx_tile_k(fmt) - 1) / mx_tile_k(fmt); }
__host__ __device__ inline long long mx_row_tiles(int rows, int segments) {
    return segments > 0 ? (long long)rows / 128 + segments : ((long long)rows + 127) / 128;
}
// byte offset of the scale of (row in tile coordinates, block)
__host__ __device__ inline long long mx_scale_offset(long long srow, int blk, int ktiles) {
    const int r = (int)(srow & 127);
    return ((srow >> 7) * ktiles + (blk >> 2)) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (blk & 3);
}

// Loads of what the kernel before on the stream may have written (rows, positions, offsets, factors), for kernels that
// may be resident before it is done: plain loads, as the read-only path is for data that nobody writes while the kernel
// runs, and volatile with a memory clobber, which keeps them behind the wait for that kernel.
__device__ __forceinline__ int32_t ld_written(const int32_t* p) {
    int32_t v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float ld_written(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ld_written(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// segment of row r: the last e with offsets[e] <= r (empty segments share their offset with the next one)
__device__ __forceinline__ int mx_segment(const int32_t* offsets, int segments, int r) {
    int lo = 0, hi = segments;                  // offsets[0] <= r assumed; invariant offsets[lo] <= r
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ld_written(offsets + mid) <= r) lo = mid; else hi = mid;
    }
    return lo;
}
// row r of a segmented operand in tile coordinates
__device__ __forceinline__ long long mx_srow(const int32_t* offsets, int segments, int r) {
    const int e = mx_segment(offsets, segments, r);
    const int o = min(max(ld_written(offsets + e), 0), r);
    return ((long long)(o >> 7) + e) * 128 + (r - o);
}

// 8 fp32 values -> 8 e2m1 codes in one word (value i in nibble i; nearest, ties to the even code, |v| > 6 -> 6)
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&v)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}
// 8 e2m1 codes -> fp32 (exact)
__device__ __forceinline__ void e2m1_unpack8(uint32_t w, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = half_bits_f32((uint16_t)h[i]);
        v[2 * i + 1] = half_bits_f32((uint16_t)(h[i] >> 16));
    }
}
// fp32 -> e4m3 byte, nearest even, above 448 -> 448
__device__ __forceinline__ uint32_t e4m3_of(float v) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
    return d & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)byte));
    return half_bits_f32((uint16_t)h);
}
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte ? byte << 23 : 0x00400000u));
}

// ---- element types -----------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements as one (V * sizeof(T) <= 16 bytes) or more 16-byte accesses; V = 1: one element
template <class T, int V> struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Vec { T v[V]; };

// calls f(T()) with the element type of a uq_dtype
template <class F> inline cudaError_t with_dtype(int t, F&& f) {
    switch (t) {
        case UQ_BF16: return f(__nv_bfloat16());
        case UQ_FP16: return f(__half());
        case UQ_FP32: return f(float());
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uq
