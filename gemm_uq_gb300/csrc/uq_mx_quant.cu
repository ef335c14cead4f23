// uq_mx_quant.cu -- microscaled 4-bit quantization of rows (optionally gathered by expert), its inverse, and the
// packing of a checkpoint's scales into tiles.
//
// A lane holds 8 consecutive k (one 16-byte load of a 16-bit type), so a block is 4 lanes (MXFP4) or 2 (NVFP4) and a
// warp step covers 256 k of one row: absmax by one or two shuffles, one 4-byte store of codes per lane, one 4-byte
// store of scales per 4 blocks.  Memory-bound: each value is read once, whatever the number of rows it is written to.
#include "uq_mx.cuh"

namespace uq {

namespace {

constexpr int STEP_K = 256;                     // k of a row per warp step

// 8 values of a row at element offset k (16-byte aligned)
template <class T> __device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        const Vec<T, 8> a = *reinterpret_cast<const Vec<T, 8>*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(a.v[i]);
    } else {
        const Vec<T, 4> a = *reinterpret_cast<const Vec<T, 4>*>(p), b = *reinterpret_cast<const Vec<T, 4>*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a.v[i];
            v[4 + i] = b.v[i];
        }
    }
}

// codes of a lane's 8 values and the scale byte of its block (the block's lanes agree on it)
template <int FMT> __device__ __forceinline__ uint32_t quantize8(float (&v)[8], float six_t, float tscale, uint32_t& byte) {
    uint32_t am = 0;                            // absmax as a bit pattern: infinities and NaN compare above all numbers
#pragma unroll
    for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    if constexpr (FMT == UQ_MXFP4) {
        am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const int e = (int)(am >> 23);          // exponent field: floor(log2 a) + 127, 0 for zero and subnormals
        byte = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
        const float inv = __uint_as_float(e == 255 ? 0u : (254u - byte) << 23);    // 2^(127 - byte), a normal number
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;                                   // exact: a power of two
    } else {
        const bool bad = am >= 0x7F800000u;
        byte = bad ? 0x7Fu : e4m3_of(__fdiv_rn(__uint_as_float(am), six_t));
        const float d = e4m3_value(byte) * tscale;
        const bool zero = bad || !(d > 0.f);
        // A real quotient, not a product with a reciprocal: x / d of a tie is exact, so ties are ties.
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = zero ? v[i] * 0.f : __fdiv_rn(v[i], d);
    }
    return e2m1_pack8(v);
}

template <class T, int FMT>
__global__ void __launch_bounds__(256) quantize_mx_kernel(const T* __restrict__ x, long long ldx, uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales, int rows, int K, float tscale,
                                                          const int32_t* __restrict__ offsets, int segments,
                                                          const int32_t* __restrict__ pos, int topk) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int LPB = FMT == UQ_MXFP4 ? 4 : 2;                 // lanes per block
    const int lane = threadIdx.x & 31;
    const int chunks = (K + STEP_K - 1) / STEP_K, ktiles = mx_ktiles(K, FMT);
    const long long units = (long long)rows * chunks;
    const float six_t = 6.0f * tscale;
    const int total = offsets ? min(__ldg(offsets + segments), pos ? rows * topk : rows) : rows;
    for (long long u = blockIdx.x * 8LL + (threadIdx.x >> 5); u < units; u += gridDim.x * 8LL) {
        const int row = (int)(u / chunks), k = (int)(u % chunks) * STEP_K + lane * 8;
        float v[8] = {};
        if (k < K) load8(x + row * ldx + k, v);
        uint32_t byte;
        const uint32_t q = quantize8<FMT>(v, six_t, tscale, byte);
        if (k >= K) byte = 0;
        // the 4 scale bytes of this lane's scale tile, from the 4 blocks' first lanes
        const int first = lane & ~(4 * LPB - 1);
        uint32_t word = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) word |= __shfl_sync(0xffffffffu, byte, first + b * LPB) << (8 * b);
        const int kt = k / mx_tile_k(FMT);
        const bool puts = lane == first && kt < ktiles;
        const int routes = pos ? topk : 1;
        for (int j = 0; j < routes; ++j) {
            const int dst = pos ? __ldg(pos + (long long)row * topk + j) : row;
            if (dst < 0 || dst >= total) continue;
            const long long srow = offsets ? mx_srow(offsets, segments, dst) : dst;
            if (k < K) *reinterpret_cast<uint32_t*>(codes + (long long)dst * (K >> 1) + (k >> 1)) = q;
            if (puts) *reinterpret_cast<uint32_t*>(scales + mx_scale_offset(srow, kt * 4, ktiles)) = word;
        }
    }
}

template <class T, int FMT>
__global__ void __launch_bounds__(256) dequant_mx_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                         T* __restrict__ out, int rows, int K, float tscale,
                                                         const int32_t* __restrict__ offsets, int segments) {
    const int kw = K >> 3, ktiles = mx_ktiles(K, FMT);
    const long long units = (long long)rows * kw;
    const int total = offsets ? min(__ldg(offsets + segments), rows) : rows;
    for (long long u = blockIdx.x * (long long)blockDim.x + threadIdx.x; u < units; u += gridDim.x * (long long)blockDim.x) {
        const int row = (int)(u / kw), k = (int)(u % kw) * 8;
        float v[8] = {};
        if (row < total) {
            const long long srow = offsets ? mx_srow(offsets, segments, row) : row;
            e2m1_unpack8(__ldg(reinterpret_cast<const uint32_t*>(codes) + u), v);
            const uint32_t b = __ldg(scales + mx_scale_offset(srow, k / mx_block(FMT), ktiles));
            const float s = FMT == UQ_MXFP4 ? e8m0_value(b) : e4m3_value(b) * tscale;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= s;
        }
        constexpr int V = 16 / sizeof(T);
        Vec<T, V>* o = reinterpret_cast<Vec<T, V>*>(out + (long long)row * K + k);
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) {
            Vec<T, V> t;
#pragma unroll
            for (int i = 0; i < V; ++i) t.v[i] = from_f32<T>(v[h * V + i]);
            o[h] = t;
        }
    }
}

// one thread per 4-byte word of the tiles
__global__ void pack_mx_scales_kernel(const uint8_t* __restrict__ nat, uint32_t* __restrict__ tiles, int rows, int nb,
                                      int ktiles, long long words_per_expert, long long words) {
    for (long long w = blockIdx.x * (long long)blockDim.x + threadIdx.x; w < words; w += gridDim.x * (long long)blockDim.x) {
        const long long e = w / words_per_expert, i = w % words_per_expert;
        const int in = (int)(i & 127), kt = (int)((i >> 7) % ktiles);
        const long long row = (i >> 7) / ktiles * 128 + (in & 3) * 32 + (in >> 2);
        uint32_t v = 0;
        if (row < rows)
            for (int b = 0; b < 4; ++b)
                if (kt * 4 + b < nb) v |= (uint32_t)nat[(e * rows + row) * nb + kt * 4 + b] << (8 * b);
        tiles[w] = v;
    }
}

int grid_for(long long units, int per_block, int sms, int waves) {
    const long long b = (units + per_block - 1) / per_block, most = (long long)sms * waves;
    return (int)(b < most ? (b < 1 ? 1 : b) : most);
}

}  // namespace

cudaError_t launch_quantize_mx(int fmt, const void* x, int xtype, long long ldx, uint8_t* codes, uint8_t* scales,
                               int rows, int K, float tscale, const int32_t* offsets, int segments, const int32_t* pos,
                               int topk, int sms, cudaStream_t st) {
    const int grid = grid_for((long long)rows * ((K + STEP_K - 1) / STEP_K), 8, sms, 64);
    return with_dtype(xtype, [&](auto t) {
        using T = decltype(t);
        if (fmt == UQ_MXFP4)
            quantize_mx_kernel<T, UQ_MXFP4><<<grid, 256, 0, st>>>(static_cast<const T*>(x), ldx, codes, scales, rows, K,
                                                                  tscale, offsets, segments, pos, topk);
        else
            quantize_mx_kernel<T, UQ_NVFP4><<<grid, 256, 0, st>>>(static_cast<const T*>(x), ldx, codes, scales, rows, K,
                                                                  tscale, offsets, segments, pos, topk);
        return cudaGetLastError();
    });
}

cudaError_t launch_dequant_mx(int fmt, const uint8_t* codes, const uint8_t* scales, void* out, int type, int rows, int K,
                              float tscale, const int32_t* offsets, int segments, int sms, cudaStream_t st) {
    const int grid = grid_for((long long)rows * (K >> 3), 256, sms, 64);
    return with_dtype(type, [&](auto t) {
        using T = decltype(t);
        if (fmt == UQ_MXFP4)
            dequant_mx_kernel<T, UQ_MXFP4><<<grid, 256, 0, st>>>(codes, scales, static_cast<T*>(out), rows, K, tscale,
                                                                 offsets, segments);
        else
            dequant_mx_kernel<T, UQ_NVFP4><<<grid, 256, 0, st>>>(codes, scales, static_cast<T*>(out), rows, K, tscale,
                                                                 offsets, segments);
        return cudaGetLastError();
    });
}

cudaError_t launch_pack_mx_scales(int fmt, const uint8_t* natural, uint8_t* tiles, int experts, int rows, int K,
                                  cudaStream_t st) {
    const int ktiles = mx_ktiles(K, fmt);
    const long long per = mx_row_tiles(rows, 0) * ktiles * 128, words = per * experts;
    const long long g = (words + 255) / 256;
    pack_mx_scales_kernel<<<(int)(g < 65536 ? g : 65536), 256, 0, st>>>(natural, reinterpret_cast<uint32_t*>(tiles), rows,
                                                                       K / mx_block(fmt), ktiles, per, words);
    return cudaGetLastError();
}

}  // namespace uq
