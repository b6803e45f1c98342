// Internal launch interface between the C ABI (api.cu) and the kernels.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fp8bs {

// ---- quantize.cu
// Every quantiser streams 128x128 BF16 tiles through shared memory with
// TMA; its waits are bounded by timeout_ns and a wait that expires records
// FP8BS_ERR_TIMEOUT in the status word that quant_take_status reads.
// pow2: power-of-two scales instead of fl32(absmax / 448).
cudaError_t launch_quantize_act_1x128(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* xq,
                                      float* sx, bool pow2, int sm_count, uint64_t timeout_ns, cudaStream_t stream);
cudaError_t launch_quantize_act_dual(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* xq,
                                     float* sx, uint8_t* xq_t, float* sx_t, bool pow2, int sm_count,
                                     uint64_t timeout_ns, cudaStream_t stream);
cudaError_t launch_quantize_weight(const uint16_t* w, int64_t N, int64_t K, int64_t ldw, uint8_t* wq,
                                   float* sw, uint8_t* wq_t, float* sw_t, bool pow2, int sm_count,
                                   uint64_t timeout_ns, cudaStream_t stream);
// One launch quantising X [M][K] in 1x128 groups and W [N][Kw] in 128x128
// blocks (the two operands of an FP8 Linear); either may be empty (M or N 0).
cudaError_t launch_quantize_act_weight(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, uint8_t* xq, float* sx,
                                       const uint16_t* w, int64_t N, int64_t Kw, int64_t ldw, uint8_t* wq, float* sw,
                                       bool pow2, int sm_count, uint64_t timeout_ns, cudaStream_t stream);
// FP8 -> FP8 re-tiling 1x128 -> 128x1 (dequantise, transpose, requantise);
// plain loads, no waits.
cudaError_t launch_requant_1x128_to_128x1(const uint8_t* xq, const float* sx, int64_t M, int64_t K, uint8_t* xq_t,
                                          float* sx_t, bool pow2, int sm_count, cudaStream_t stream);
// Fused SwiGLU (gate columns [0, I), up columns [I, 2I) of h) and 1x128
// quantisation of the BF16-rounded result; plain loads, no waits.
cudaError_t launch_swiglu_quantize(const uint16_t* h, int64_t M, int64_t I, int64_t ldh, uint8_t* q, float* s,
                                   bool pow2, int sm_count, cudaStream_t stream);
// Reads and clears the quantisers' device status word (synchronous copy on
// the current device).
cudaError_t quant_take_status(int* status);

// ---- gemm.cu
struct GemmArgs {
  const uint8_t* a;        // [M][K] E4M3, K-major
  const float* sa;         // [K/128][M] kb-major
  const uint8_t* b;        // [G][N][K] E4M3 (G = 1 for the dense GEMM)
  const float* sb;         // block: [G][N/128][K/128]; row: [K/128][N]
  void* d;                 // [M][N]
  const int32_t* offsets;  // grouped only: device [G+1]
  int64_t M;               // rows of A (M_total for the grouped GEMM)
  int64_t N, K;
  int num_groups;          // 1 for the dense GEMM
  bool grouped;
  bool sb_row;             // FP8BS_SCALE_ROW1x128
  bool out_bf16;
  bool accumulate;
  uint64_t timeout_ns;
};

// Returns cudaSuccess, or an error; *tmap_failed is set when a tensor map
// could not be encoded, *reg_check_failed when the compiled kernel's
// register count does not match the warp-specialised register split.
cudaError_t launch_gemm(const GemmArgs& args, int sm_count, cudaStream_t stream, bool* tmap_failed,
                        bool* reg_check_failed);

// Reads and clears the device status word of the GEMM kernels; synchronous
// copy on the current device.
cudaError_t gemm_take_status(int* status);

// ---- gemm_mx.cu
// The same GEMM for power-of-two scales, with the scales applied by the
// tensor core (tcgen05.mma.kind::mxf8f6f4.block_scale, UE8M0) and all of K
// accumulated in tensor memory.  A scale that is not zero or a power of two
// in [2^-127, 2^127] records FP8BS_ERR_DEVICE_ARG in its status word.
cudaError_t launch_gemm_pow2(const GemmArgs& args, int sm_count, cudaStream_t stream, bool* tmap_failed,
                             bool* reg_check_failed);
// The experts' weight gradients: a [M][K] and b [N][K] hold all experts' rows
// along K (K / 128 blocks, sa [K/128][M], sb [K/128][N]), offsets the segments;
// d [num_groups][M][N].
cudaError_t launch_wgrad_pow2(const GemmArgs& args, int sm_count, cudaStream_t stream, bool* tmap_failed,
                              bool* reg_check_failed);
cudaError_t gemm_mx_take_status(int* status);

// ---- fp4.cu (4-bit quantisers and dequantiser; plain loads, no waits)
// fmt: fp8bs_fp4_format.  rows: see fp8bs_quantize_fp4 (swiglu: the `live`
// list of fp8bs_swiglu_quantize_fp4, x the gate/up matrix).
cudaError_t launch_quantize_fp4(const uint16_t* x, int64_t rows_in, int64_t K, int64_t ldx, const int32_t* rows,
                                int64_t M, int fmt, bool swiglu, uint8_t* q, uint8_t* sf, float* g,
                                cudaStream_t stream);
cudaError_t launch_dequantize_fp4(const uint8_t* q, const uint8_t* sf, const float* g, int64_t M, int64_t K, int fmt,
                                  void* out, bool out_bf16, int64_t ldo, cudaStream_t stream);

// ---- gemm_fp4.cu
struct Fp4GemmArgs {
  const uint8_t* a;        // [M][K / 2] E2M1 pairs
  const uint8_t* sfa;      // blocked scales of A
  const float* ga;         // [M] (E4M3x16)
  const uint8_t* b;        // [G][N][K / 2] (G = 1 for the dense GEMM)
  const uint8_t* sfb;      // [G] blocked scales of B
  const float* gb;         // [G][N] (E4M3x16)
  void* d;                 // [M][N]
  const int32_t* offsets;  // device [G + 1], NULL for the dense GEMM
  int64_t M, N, K;
  int num_groups;
  bool out_bf16;
  uint64_t timeout_ns;
};
// tmap_failed, reg_check_failed: as launch_gemm.
cudaError_t launch_gemm_fp4(const Fp4GemmArgs& args, int fmt, int sm_count, cudaStream_t stream, bool* tmap_failed,
                            bool* reg_check_failed);
cudaError_t gemm_fp4_take_status(int* status);

// ---- route.cu (the MoE router and the layout of its choices; no waits)
struct RouteArgs {
  const void* logits;      // [T][ld] float32 or BF16
  bool bf16;
  int64_t T, ld;
  int E, k, S;
  int score;               // 0 softmax, 1 sigmoid
  const float* bias;       // [E] or NULL
  const uint8_t* valid;    // [T] or NULL
  const int32_t* seq;      // [S + 1] or NULL (one sequence)
  bool normalize;
  float scale, alpha;
  int32_t* idx;            // [T][k] (read by the backward pass)
  float* w;                // [T][k]
  int32_t* counts;         // [S][E]
  int32_t* tokens;         // [S]
  float* loss;             // [1], NULL: no statistics
  const float* dw;         // backward: [T][k]
  const float* dloss;      // backward: [1] or NULL
  void* dlogits;           // backward: [T][ldd], the logits' type
  int64_t ldd;
  // set by the launchers
  int64_t chunk;
  float* part_p;
  int32_t* part_n;
  int32_t* part_t;
  float* share;
  int32_t* done;
};
int64_t route_workspace_bytes(int64_t T, int E, int64_t S);
cudaError_t launch_route(RouteArgs args, void* ws, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteArgs& args, cudaStream_t stream);
// Reads and clears the router's device status word (invalid sequences).
cudaError_t route_take_status(int* status);

struct LayoutArgs {
  const int32_t* idx;      // [pairs]
  int64_t pairs;
  int k, E;
  int32_t* offsets;        // [E + 1]
  int32_t* row_token;      // [rows]
  int64_t rows;
  int32_t* row_of;         // [pairs]
  int32_t* hist;           // workspace
};
int64_t layout_workspace_bytes(int64_t T, int k, int E);
cudaError_t launch_layout(const LayoutArgs& args, cudaStream_t stream);

// ---- moe.cu (row movement of the MoE dispatch and combine; no waits)
cudaError_t launch_gather_q_rows(const uint8_t* q, const float* s, int64_t rows_in, int64_t H, bool s_in_kb_major,
                                 const int32_t* idx, int64_t rows_out, uint8_t* q_out, float* s_out,
                                 bool s_out_kb_major, int sm_count, cudaStream_t stream);
cudaError_t launch_scatter_q_rows(const uint8_t* q, const float* s, int64_t rows_in, int64_t H, bool s_in_kb_major,
                                  const int32_t* pos, int k, const int32_t* zero_rows, int64_t n_zero,
                                  int64_t rows_out, uint8_t* q_out, float* s_out, bool s_out_kb_major, int sm_count,
                                  cudaStream_t stream);
cudaError_t launch_gather_bf16_rows(const uint16_t* y, int64_t rows_in, int64_t N, const int32_t* idx,
                                    int64_t rows_out, uint16_t* out, int sm_count, cudaStream_t stream);
cudaError_t launch_moe_combine(const uint16_t* y, int64_t rows_y, int64_t N, const int32_t* idx, const float* w,
                               int64_t T, int k, uint16_t* out, int sm_count, cudaStream_t stream);

// out[t] = add[t] + the rows of token t (idx < 0: none); add may be NULL.
cudaError_t launch_moe_dispatch_backward(const uint16_t* d, int64_t rows, int64_t N, const int32_t* idx, int64_t T, int k,
                                         const uint16_t* add, uint16_t* out, int sm_count, cudaStream_t stream);

// ---- train.cu (norm, its gradient, gradients of the combine and the SwiGLU; the
// norm and its gradient wait for their own copies, bounded by timeout_ns)
struct NormArgs {
  const uint16_t* x;       // [M][ldx]
  const uint16_t* res;     // [M][ldr] or NULL
  const void* gain;        // [K]
  bool gain_f32;
  int64_t M, K, ldx, ldr;
  float eps;
  bool pow2;
  uint16_t* r;             // [M][K] or NULL
  uint16_t* y;             // [M][K] or NULL
  uint8_t* q;              // [M][K] or NULL
  float* s;                // [K/128][M]
  float* rstd;             // [M] or NULL
  uint64_t timeout_ns;
};
cudaError_t launch_rmsnorm(const NormArgs& args, int sm_count, cudaStream_t stream);
int64_t rmsnorm_max_columns();

struct NormBackwardArgs {
  const uint16_t* dy;      // [M][lddy]
  const uint16_t* r;       // [M][ldr]
  const void* gain;
  bool gain_f32;
  const float* rstd;       // [M]
  const uint16_t* dres;    // [M][lddres] or NULL
  int64_t M, K, lddy, ldr, lddres;
  uint16_t* dx;            // [M][K]
  float* dgain;            // [K] or NULL
  bool accumulate;
  uint64_t timeout_ns;
};
int64_t rmsnorm_backward_workspace_bytes(int64_t M, int64_t K);
cudaError_t launch_rmsnorm_backward(const NormBackwardArgs& args, void* ws, cudaStream_t stream);

struct CombineBackwardArgs {
  const uint16_t* dout;      // [T][ldo]
  int64_t T, N, ldo;
  const uint16_t* y;         // [rows][N] or NULL
  int64_t rows;
  const int32_t* row_of;     // [T][k]
  const int32_t* row_token;  // [rows]
  const float* w;            // [T][k]
  int k;
  bool pow2;
  uint16_t* dy;              // [rows][N] or NULL
  uint8_t* q;                // [rows][N] or NULL
  float* s;                  // [N/128][rows]
  float* dw;                 // [T][k] or NULL
};
cudaError_t launch_combine_backward(const CombineBackwardArgs& args, int sm_count, cudaStream_t stream);

struct SwigluBackwardArgs {
  const uint16_t* h;       // [M][ldh]
  const uint16_t* dv;      // [M][lddv]
  const int32_t* live;     // [M] or NULL
  int64_t M, I, ldh, lddv;
  bool pow2;
  uint16_t* dh;            // [M][2I] or NULL
  uint8_t* q;              // [M][2I] or NULL
  float* s;                // [2I/128][M]
};
cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& args, int sm_count, cudaStream_t stream);
// Reads and clears the status word (a wait that ran out, a row_token that does not
// fit row_of).
cudaError_t train_take_status(int* status);

// Diagnostic: a kernel whose bounded wait runs out (nothing ever arrives on
// its barrier) and records FP8BS_ERR_TIMEOUT in the GEMM status word.
cudaError_t launch_wait_timeout_selftest(uint64_t timeout_ns, cudaStream_t stream);

// Diagnostic GEMM without promotion (diag.cu): D[M][N] = A[M][K] B[N][K]^T
// in FP32, accumulated over all of K in tensor memory; M % 128 == 0,
// N % 256 == 0, K % 128 == 0.
cudaError_t launch_unpromoted_gemm(const uint8_t* a, const uint8_t* b, float* d, int64_t M, int64_t N, int64_t K,
                                   uint64_t timeout_ns, cudaStream_t stream);

// Reads and clears the diagnostic kernel's device status word.
cudaError_t diag_take_status(int* status);

}  // namespace fp8bs
