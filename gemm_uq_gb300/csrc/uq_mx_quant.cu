// uq_mx_quant.cu -- microscaled 4-bit quantization of rows (optionally gathered by expert), its inverse, and the
// packing of a checkpoint's scales into tiles.
//
// A warp takes 2048 k of one row in eight steps of 256 (512 in two steps when there are too few rows to fill the SMs
// otherwise; with two always, bf16 -> MXFP4 at 8192 x 8192 took 42 us), a lane 8 consecutive k of each: one 16-byte load
// of a 16-bit type, all requested before the first is used.  A block is then 4 lanes (MXFP4) or 2 (NVFP4): its absmax
// takes one or two shuffles, the codes one 4-byte store per lane, the scales of 4 blocks one 4-byte store.
// Each value is read once, whatever the number of rows it is written to.  8192 x 8192 bf16 -> MXFP4 29.5 us (5.8 TB/s),
// near the memory's bound; NVFP4 36.7 us (4.7 TB/s), 75 % of the issue slots and 66 % of the ALU pipe taken (a quotient per
// value); fp32 -> MXFP4 45.8 us (6.6 TB/s); read back as bf16 28.6 us (5.9 TB/s).
#include "uq_mx_quant.cuh"

namespace uq {

namespace {

constexpr int STEP_K = 256;                     // k of a row per warp step

template <class T, int FMT, int STEPS>
__global__ void __launch_bounds__(128) quantize_mx_kernel(const T* x, long long ldx, uint8_t* codes, uint8_t* scales,
                                                          int rows, int K, float tscale, const int32_t* offsets,
                                                          int segments, const int32_t* pos, int topk, bool early) {
    // Only a product's own quantizer lets the next kernel, that product, start early: what this one writes may otherwise be
    // the weights that a later kernel requests before it waits for its predecessor.  It may do so at once: the work before
    // this call is what overlap's users promise does not write the weights, and the work before that was complete when
    // this kernel could start.
    if (early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");           // with launch overlap: x follows earlier work
    constexpr int UNIT_K = STEP_K * STEPS;                       // k of a row per warp
    constexpr int LPB = FMT == UQ_MXFP4 ? 4 : 2;                 // lanes per block
    constexpr int TPS = STEP_K / mx_tile_k(FMT);                 // scale tiles per step
    const int lane = threadIdx.x & 31;
    const unsigned units_k = (unsigned)(K + UNIT_K - 1) / UNIT_K;
    const int ktiles = mx_ktiles(K, FMT);
    const SixT six(tscale);
    const int total = offsets ? min(ld_written(offsets + segments), pos ? rows * topk : rows) : rows;
    const unsigned long long units = (unsigned long long)rows * units_k;
    for (unsigned long long u0 = blockIdx.x * 4ull + (threadIdx.x >> 5); u0 < units; u0 += gridDim.x * 4ull) {
        const int row = units <= 0xFFFFFFFFull ? (int)((unsigned)u0 / units_k) : (int)(u0 / units_k);
        const int k0 = (int)(u0 - (unsigned long long)row * units_k) * UNIT_K + lane * 8;
        Raw<T> v[STEPS] = {};
        const T* xr = x + row * ldx;
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            if (k0 + i * STEP_K < K) v[i].load(xr + k0 + i * STEP_K);
        uint32_t q[STEPS], word[STEPS];
        const int first = lane & ~(4 * LPB - 1);                 // first lane of this lane's scale tile
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            uint32_t byte;
            q[i] = quantize8<FMT>(v[i], six, tscale, byte);
            if (k0 + i * STEP_K >= K) byte = 0;
            word[i] = scale_word<FMT>(byte, lane);
        }
        const int kt0 = k0 / mx_tile_k(FMT);
        const int routes = pos ? topk : 1;
        for (int j0 = 0; j0 < routes; j0 += 32) {
            // lane j finds the row of route j0 + j
            int dst = -1;
            long long srow = 0;
            if (j0 + lane < routes) {
                dst = pos ? ld_written(pos + (long long)row * topk + j0 + lane) : row;
                if (dst >= total) dst = -1;
                if (dst >= 0) srow = offsets ? mx_srow(offsets, segments, dst) : dst;
            }
            for (int j = 0; j < min(32, routes - j0); ++j) {
                const int d = __shfl_sync(0xffffffffu, dst, j);
                const long long sr = __shfl_sync(0xffffffffu, srow, j);
                if (d < 0) continue;
                uint8_t* c = codes + (long long)d * (K >> 1) + (k0 >> 1);
                uint8_t* sc = scales + mx_scale_offset(sr, kt0 * 4, ktiles);
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    if (k0 + i * STEP_K < K) *reinterpret_cast<uint32_t*>(c + i * (STEP_K / 2)) = q[i];
                    if (lane == first && kt0 + i * TPS < ktiles) *reinterpret_cast<uint32_t*>(sc + i * TPS * 512) = word[i];
                }
            }
        }
    }
}

template <class T, int FMT, int STEPS>
__global__ void __launch_bounds__(128) dequant_mx_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                         T* __restrict__ out, int rows, int K, float tscale,
                                                         const int32_t* __restrict__ offsets, int segments) {
    constexpr int UNIT_K = STEP_K * STEPS;
    const int lane = threadIdx.x & 31;
    const unsigned units_k = (unsigned)(K + UNIT_K - 1) / UNIT_K;
    const int ktiles = mx_ktiles(K, FMT);
    const int total = offsets ? min(__ldg(offsets + segments), rows) : rows;
    const unsigned long long units = (unsigned long long)rows * units_k;
    for (unsigned long long u0 = blockIdx.x * 4ull + (threadIdx.x >> 5); u0 < units; u0 += gridDim.x * 4ull) {
        const int row = units <= 0xFFFFFFFFull ? (int)((unsigned)u0 / units_k) : (int)(u0 / units_k);
        const int k0 = (int)(u0 - (unsigned long long)row * units_k) * UNIT_K + lane * 8;
        uint32_t q[STEPS] = {}, b[STEPS] = {};
        if (row < total) {
            const long long srow = offsets ? mx_srow(offsets, segments, row) : row;
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
                if (k0 + i * STEP_K < K) {
                    q[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + (long long)row * (K >> 1) + ((k0 + i * STEP_K) >> 1)));
                    b[i] = __ldg(scales + mx_scale_offset(srow, (k0 + i * STEP_K) / mx_block(FMT), ktiles));
                }
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (k0 + i * STEP_K >= K) break;
            float v[8];
            e2m1_unpack8(q[i], v);
            const float s = FMT == UQ_MXFP4 ? e8m0_value(b[i]) : e4m3_value(b[i]) * tscale;
            constexpr int V = 16 / sizeof(T);
            Vec<T, V>* o = reinterpret_cast<Vec<T, V>*>(out + (long long)row * K + k0 + i * STEP_K);
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) {
                Vec<T, V> t;
#pragma unroll
                for (int c = 0; c < V; ++c) t.v[c] = from_f32<T>(v[h * V + c] * s);
                o[h] = t;
            }
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

namespace {
// calls f(steps as a constant, grid): long units where they still give every SM its warps
template <class F> cudaError_t with_steps(int rows, int K, int sms, F&& f) {
    const auto units = [&](int steps) { return (long long)rows * ((K + STEP_K * steps - 1) / (STEP_K * steps)); };
    if (units(8) >= 16LL * sms) return f(std::integral_constant<int, 8>(), grid_for(units(8), 4, sms, 64));
    return f(std::integral_constant<int, 2>(), grid_for(units(2), 4, sms, 64));
}
}  // namespace

cudaError_t launch_quantize_mx(int fmt, const void* x, int xtype, long long ldx, uint8_t* codes, uint8_t* scales,
                               int rows, int K, float tscale, const int32_t* offsets, int segments, const int32_t* pos,
                               int topk, int sms, bool early, bool overlap, cudaStream_t st) {
    return with_steps(rows, K, sms, [&](auto steps, int grid) {
        return with_dtype(xtype, [&](auto t) {
            using T = decltype(t);
            constexpr int S = decltype(steps)::value;
            auto kernel = fmt == UQ_MXFP4 ? quantize_mx_kernel<T, UQ_MXFP4, S> : quantize_mx_kernel<T, UQ_NVFP4, S>;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(grid);
            cfg.blockDim = dim3(128);
            cfg.stream = st;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = overlap ? 1 : 0;
            return cudaLaunchKernelEx(&cfg, kernel, static_cast<const T*>(x), ldx, codes, scales, rows, K, tscale, offsets,
                                      segments, pos, topk, early);
        });
    });
}

cudaError_t launch_dequant_mx(int fmt, const uint8_t* codes, const uint8_t* scales, void* out, int type, int rows, int K,
                              float tscale, const int32_t* offsets, int segments, int sms, cudaStream_t st) {
    return with_steps(rows, K, sms, [&](auto steps, int grid) {
        return with_dtype(type, [&](auto t) {
            using T = decltype(t);
            constexpr int S = decltype(steps)::value;
            auto kernel = fmt == UQ_MXFP4 ? dequant_mx_kernel<T, UQ_MXFP4, S> : dequant_mx_kernel<T, UQ_NVFP4, S>;
            kernel<<<grid, 128, 0, st>>>(codes, scales, static_cast<T*>(out), rows, K, tscale, offsets, segments);
            return cudaGetLastError();
        });
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
