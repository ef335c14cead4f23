// uq_kernels.h -- internal declarations shared by the uq CUDA sources and the C-ABI host code.
#pragma once

#include "uq_common.cuh"

namespace uq {

// records the message uq_last_error() returns on the calling thread (uq_api.cu)
void set_last_error(const char* msg);
// whether GEMV, GEMM and microscaled kernels are launched with programmatic dependent launch (uq_set_launch_overlap)
bool launch_overlap();

// reads and clears the fault word of uq_gemm_noalloc launches on the current device (uq_noalloc.cu)
cudaError_t noalloc_take_fault(unsigned int* v);

// offline kernels (uq_pack.cu)
cudaError_t launch_pack(int fmt, const int8_t* codes, uint8_t* wq, int N, int K, unsigned int* bad,
                        cudaStream_t st);
cudaError_t launch_unpack(int fmt, const uint8_t* wq, int8_t* codes, int N, int K, cudaStream_t st);
cudaError_t launch_pack_gguf(int qtype, const uint8_t* blocks, uint8_t* wq, uint16_t* scales, int N, int K,
                             cudaStream_t st);   // qtype 0 = Q4_0, 1 = Q8_0
cudaError_t launch_dequant(int fmt, const uint8_t* wq, const uint8_t* scales, const uint8_t* zc, float* w,
                           int N, int K, int group, cudaStream_t st);
cudaError_t launch_pack_kmeta(const uint16_t* d, const uint16_t* dmin, const uint8_t* sc, const uint8_t* m,
                              uint8_t* meta, long long count, unsigned int* bad, cudaStream_t st);
cudaError_t launch_pack_zeros(const uint8_t* z, uint8_t* out, int N, int G, cudaStream_t st);
cudaError_t launch_quantize(int fmt, const float* w, int8_t* codes, uint16_t* scales, void* zeros,
                            const float* codebook, int N, int K, int group, cudaStream_t st);
cudaError_t launch_quantize_k4(const float* w, int8_t* codes, uint16_t* d, uint16_t* dmin, uint8_t* sc,
                               uint8_t* m, int N, int K, cudaStream_t st);

// fused RMSNorm + RoPE and its cos/sin table (uq_norm.cu)
cudaError_t launch_rope_table(float* table, int max_pos, int head_dim, double base, cudaStream_t st);
cudaError_t launch_rmsnorm_rope(const uint16_t* x, const uint16_t* gamma, const int32_t* pos, const float* table,
                                uint16_t* y, int M, int D, int head_dim, int max_pos, float eps, unsigned int* fault,
                                int sms, cudaStream_t st);

// small-M GEMV (uq_gemv.cu)
struct GemvArgs {
    const uint16_t* x;        // bf16 [M][ldx]
    const uint8_t* wq;        // packed codes
    const uint8_t* scales;    // fp16 [N][K/group] or K4 records
    const uint8_t* zc;        // zeros / codebook / NULL
    uint16_t* y;              // bf16 [M][ldy]
    int M, N, K, group, ldx, ldy;
    int NB, KB;               // row blocks, k tiles
    long long T;              // tiles = NB * KB
    int P;                    // workers that split the tiles, P <= T: warps (CUDA-core GEMV, W4A8) or
                              // CTAs (mma GEMV)
    float* partials;          // fp32 split-K partial sums: [T][16][M] (mma and W4A8 GEMVs, summed by the
                              // second pass), [2P][16][M] (CUDA-core GEMV: first and last row block of
                              // each worker)
    unsigned int* tickets;    // [NB], zero between calls
    unsigned int* fault;      // device fault word
    int overlap;              // launched with programmatic stream serialization (set by the launcher)
    int cta_rows;             // mma / W4A8 GEMV: > 0 = every CTA owns whole row blocks (combined in shared
                              // memory, no second pass; mma GEMV: the most tiles a CTA gets);
                              // 0 = workers split row blocks anywhere (second pass)
    float* out32;             // gate pass of the gated projection: fp32 results [M][ldy] instead of y
    const float* gate32;      // up pass: y = bf16(silu(gate32) * result), gate32 [M][ldy] fp32
    int gated;                // mma GEMV only: the gated projection in one launch; (wq, scales, zc) are the
                              // gate weight, (wq2, scales2, zc2) the up weight, NB and T count both
    const uint8_t* wq2;
    const uint8_t* scales2;
    const uint8_t* zc2;
    int a8;                   // the W4A8 GEMV (integer x codes):
    const int8_t* xq;         //   x codes [M][Kpq], each 32 k in the integer mma's B fragment order
    const float* sxq;         //   per-row scales of x [M]
    const int* sxl;           //   per (row, group) sums of the codes [M][ceil(Kpq / group)]
    int Kpq;                  //   bytes per row of xq
    int ring_slots;           // mma GEMV: ring slots and x-sum table groups of the launch (set by its launcher)
    int sx_groups;
    int mma_pairs;            // mma GEMV: pairs of compute warps that take tiles (set by its launcher)
};
// formats whose GEMV runs on mma.sync (all six)
inline bool gemv_is_mma(int fmt) {
    return fmt == UQ_INT4_SYM || fmt == UQ_INT4_ASYM || fmt == UQ_INT2_ASYM || fmt == UQ_K4 || fmt == UQ_INT8_SYM ||
           fmt == UQ_NF4;
}
// formats of the mma.sync GEMM (gemm_mma_kernel: 9..64 rows)
inline bool gemm_mma_format(int fmt) {
    return fmt == UQ_INT4_SYM || fmt == UQ_INT4_ASYM || fmt == UQ_INT2_ASYM || fmt == UQ_K4;
}
// Plans one GEMV launch from its shape fields (M, N, K, group, NB, KB, T, gated, a8) and the SM
// count: sets a.P and a.cta_rows.  Returns the grid, or 0 when no plan fits (K too long for the
// kernel's shared memory at this M).
int gemv_plan(GemvArgs& a, int fmt, int sms);
// what a planned launch needs: fp32 partial-sum floats, the per-row-block tickets, kernel launches
size_t gemv_partials_floats(int fmt, const GemvArgs& a);
bool gemv_uses_tickets(int fmt, const GemvArgs& a);
int gemv_launches(int fmt, const GemvArgs& a);
cudaError_t launch_gemv(int fmt, const GemvArgs& a, int grid, cudaStream_t st);
// the second pass of a stream-K split (tile partial sums [T][16][M] summed in k order)
cudaError_t launch_gemv_second_pass(const GemvArgs& a, int sms, cudaStream_t st);

// batched decode on mma.sync for the 4-bit and 2-bit formats, 9 <= M <= 64 (uq_gemm_mma.cu)
struct GemmArgs {
    const uint16_t* x;        // bf16 [M][ldx]
    const uint8_t* wq;        // packed codes
    const uint8_t* scales;    // fp16 [N][K/group] or K4 records
    const uint8_t* zc;        // INT4_ASYM zero nibbles, INT2_ASYM fp16 zeros, else NULL
    uint16_t* y;              // bf16 [M][ldy]
    int M, N, K, group, ldx, ldy;
    int NB;                   // row blocks of 16
    int UB;                   // k units per row (4 chunks of codes each)
    int KS;                   // k splits: CTAs per row group of 8 row blocks
    const float* sx;          // K4: column sums of x per 32-k block [K/32][Mpad], else NULL
    int Mpad;                 // columns of sx (8 x column blocks)
    float* partials;          // KS > 1: [KS][NB * 16][M] fp32
    float* out32;             // gate pass of the gated projection: fp32 results [M][ldy] instead of y
    const float* gate32;      // up pass: y = bf16(silu(gate32) * result)
};
int gemm_mma_units(int fmt, int K);               // k units per row
int gemm_mma_splits(int NB, int UB, int sms);     // k splits per row group
// the kernel, then (KS > 1) the second pass over the splits
cudaError_t launch_gemm_mma(int fmt, const GemmArgs& a, int sms, cudaStream_t st);

// W4A8 / W8A8 (uq_w4a8.cu): x codes and scales, then the integer GEMV
cudaError_t launch_quant_x(const uint16_t* x, int8_t* xq, float* sx, int* sxl, int M, int K, int Kp, int gs, int perm,
                           cudaStream_t st);
cudaError_t launch_gemv_a8(int fmt, const GemvArgs& a, const int8_t* xq, const float* sxs, const int* sxl, int Kp,
                           int grid, cudaStream_t st);


// tensor-core GEMM for M >= 16 (uq_tc.cu)
struct TcArgs {
    const uint8_t* wq;        // packed codes
    long long rowbytes;       // bytes of one padded row of codes
    int NB;                   // row blocks of 16
    const uint8_t* scales;    // fp16 [N][K/group] or K4 records
    const uint8_t* zc;        // INT4_ASYM zero nibbles, else NULL
    uint16_t* y;              // bf16 [M][ldy]
    const float* sx;          // K4: column sums of x per 32-k block [K/32][Mpad], else NULL
    int M, Mpad, N, K, group, ldx, ldy;
    int CH;                   // units (chunks of 128 code bytes) per 128-row block
    long long U;              // units = ceil(N/128) * CH
    int P;                    // CTAs, P <= U
    float* partials;          // [2P][128][Mpad]
    unsigned int* tickets;    // [ceil(N/128)]
    unsigned int* fault;
    float* out32;             // gate pass of the gated projection: fp32 results [M][ldy] instead of y
    const float* gate32;      // up pass: y = bf16(silu(gate32) * result)
};

// silu(g) * u in fp32 (silu(g) = g / (1 + e^-g)), the gated projection's epilogue
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-g))), u);
}

// The one place every kernel writes an output element (row m of x, output column n): bf16 y; or, for
// the gated projection, fp32 g (the gate pass) or bf16 silu(g) * u (the up pass; the product in fp32,
// one rounding to bf16).
template <class Args>
__device__ __forceinline__ void store_out(const Args& a, int m, int n, float v) {
    const long long idx = (long long)m * a.ldy + n;
    if (a.out32) {
        a.out32[idx] = v;
        return;
    }
    if (a.gate32) v = silu_mul(a.gate32[idx], v);
    a.y[idx] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
bool tc_supported(int fmt, int N, int K);
int tc_plan(int fmt, int mpad, int group, size_t* smem);   // dynamic shared memory of the launch
cudaError_t launch_colsum32(const uint16_t* x, float* sx, int M, int mpad, int K, int ldx, cudaStream_t st);
cudaError_t launch_tc(int fmt, const uint16_t* x, const TcArgs& a, size_t smem, int grid, cudaStream_t st);

// microscaled 4-bit quantization (uq_mx_quant.cu)
// early: the next kernel may start before this one is done; overlap: this one before the work before it is
cudaError_t launch_quantize_mx(int fmt, const void* x, int xtype, long long ldx, uint8_t* codes, uint8_t* scales,
                               int rows, int K, float tscale, const int32_t* offsets, int segments, const int32_t* pos,
                               int topk, int sms, bool early, bool overlap, cudaStream_t st);
cudaError_t launch_dequant_mx(int fmt, const uint8_t* codes, const uint8_t* scales, void* out, int type, int rows, int K,
                              float tscale, const int32_t* offsets, int segments, int sms, cudaStream_t st);
cudaError_t launch_pack_mx_scales(int fmt, const uint8_t* natural, uint8_t* tiles, int experts, int rows, int K,
                                  cudaStream_t st);

// product of microscaled 4-bit operands (uq_mx_gemm.cu)
struct MxGemmArgs {
    const uint8_t* xscales;   // scale tiles of x
    const uint8_t* wscales;   // of the weight(s)
    const uint8_t* wscales_up;
    const int32_t* offsets;   // segments of x [experts + 1], NULL: one weight for all rows
    const float* alpha_e;     // per expert, NULL = 1
    const float* alpha_up;
    void* y;                  // [rows][N]
    unsigned int* fault;
    float alpha;
    int ytype, rows, experts, N, K;
    int wait;                 // launched with programmatic serialization: the kernel before may still run
    const void* xraw;         // few tokens that the kernel quantizes itself (xcodes and xscales unused), or NULL
    long long ldx;
    int xtype;
    float tscale;
    // set by launch_mx_gemm:
    int steps;                // k steps
    int ktiles;               // scale tiles along K
    int folded;               // codes come in boxes of two 128-byte columns
    int pair;                 // pairs of CTAs (256 x 256 tiles)
    int TN, NT, S;            // tokens per tile, weight tiles, CTAs sharing a tile's steps
    int share, extra;         // steps of a CTA of them: share, of the first `extra` one more
    int group;                // weight tiles that are numbered together
    int row_tiles;            // scale tiles of 128 rows of one expert's weight
    int accs, stages;         // accumulators, ring stages
    int tmem_cols, smem, ctas;
};
bool mx_gemm_quantizes(int rows);   // whether a product of so many tokens quantizes them itself
cudaError_t launch_mx_gemm(int fmt, const uint8_t* xcodes, const uint8_t* wcodes, const uint8_t* wcodes_up, MxGemmArgs a,
                           int sms, cudaStream_t st);

// expert routing (uq_moe.cu)
cudaError_t launch_moe_sort(const int32_t* ids, long long n, int E, int32_t* order, int32_t* pos, int32_t* offsets,
                            cudaStream_t st);
cudaError_t launch_moe_gather(const void* x, int type, const int32_t* pos, const int32_t* offsets, int E, void* xs, int T,
                              int topk, int H, int sms, cudaStream_t st);
cudaError_t launch_moe_combine(const void* ys, int type, const int32_t* pos, const float* weights, void* y, int T,
                               int topk, int H, int sms, cudaStream_t st);   // weights NULL: plain sum
cudaError_t launch_moe_combine_grad(const void* dy, const void* ys, int type, const int32_t* pos, const float* weights,
                                    const int32_t* offsets, int E, void* dys, float* dw, int T, int topk, int H, int sms,
                                    cudaStream_t st);

// rows in 8 bits, the norm that ends in them and its gradient (uq_q8.cu)
// wide: the codes as fp16 there instead; early: the next kernel may start before this one is done
cudaError_t launch_quantize_q8(const void* x, int type, long long ldx, int8_t* codes, void* wide, float* scales, int rows, int K,
                               bool early, int sms, cudaStream_t st);
cudaError_t launch_dequant_q8(const int8_t* codes, const float* scales, void* out, int type, int rows, int K, int sms, cudaStream_t st);
cudaError_t launch_rmsnorm_q8(const void* x, const void* residual, const void* gamma, int type, long long ldx, void* h, void* y,
                              int8_t* codes, float* scales, int rows, int D, float eps, int sms, cudaStream_t st);
int norm_grad_partials(int type, int rows, int D, int sms);        // rows of D floats of `partials`
cudaError_t launch_rmsnorm_grad(const void* dy, const void* h, const void* gamma, const void* dh, int type, void* dx, float* dgamma,
                                float* partials, int rows, int D, float eps, int sms, cudaStream_t st);

// product of 8-bit operands with a scale per row of each (uq_q8_gemm.cu)
struct Q8GemmArgs {
    const int8_t *x, *w;      // [M][K], [N][K]
    const float *sx, *sw;     // [M], [N]
    void* y;                  // [M][N]
    unsigned int* fault;
    int ytype, M, N, K;
    const void* raw;          // a token that the kernel quantizes itself (x and sx unused), or NULL
    int xtype;
};
// whether launch_q8_gemm quantizes the token itself
bool q8_gemm_quantizes(const void* x, int type, int M, int K);
// how a product of so many tokens takes them: codes, launch_q8_gemm; codes, launch_q8_gemm_tc; as fp16, launch_q8_gemm_tc
enum Q8Form { Q8_GEMV, Q8_CODES, Q8_WIDE };
Q8Form q8_gemm_form(int M);
cudaError_t launch_q8_widen(const int8_t* x, void* x16, int M, int K, int sms, cudaStream_t st);
// wait: the call's own kernel before it may still run
cudaError_t launch_q8_gemm_tc(const Q8GemmArgs& a, const void* x16, bool wait, int sms, cudaStream_t st);
cudaError_t launch_q8_gemm(const Q8GemmArgs& a, int sms, cudaStream_t st);

// the router (uq_route.cu)
cudaError_t launch_moe_route(const void* logits, int type, const float* bias, int32_t* ids, float* weights, int T, int E, int topk,
                             bool sigmoid, int groups, int top_groups, int group_top, bool renorm, float scale, int sms,
                             cudaStream_t st);
cudaError_t launch_moe_route_grad(const void* logits, int type, const int32_t* ids, const float* dweights, void* dlogits, int T,
                                  int E, int topk, bool sigmoid, bool renorm, float scale, int sms, cudaStream_t st);

}  // namespace uq
