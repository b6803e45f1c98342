/*
 * fp8bs — fine-grained FP8 quantisation and block-scaled FP8 GEMM for
 * NVIDIA GB300 (sm_103a).  C ABI.
 *
 * The method is DeepSeek-V3's FP8 training scheme ("Infrastructure" §3.3):
 *   - §3.3.2 "fine-grained quantization": activations are scaled per 1x128
 *     tile (one token, 128 channels), weights per 128x128 block, and the
 *     scales vary along the GEMM's inner dimension;
 *   - §3.3.2 "online quantization": the max absolute value of each tile or
 *     block is computed when the tensor is used;
 *   - §3.3.2 "mantissa over exponents": every tensor is E4M3;
 *   - §3.3.2 "increasing accumulation precision" (Figure 7b): every
 *     N_C = 128 elements of K the tensor-core partial sum is promoted to
 *     FP32, multiplied by the two scales and accumulated;
 *   - the explicit formulas are the Figure 7 explainer's ("DeepSeek-V3 FP8
 *     动态量化", "Fine-grained quantization"): s = absmax / F_max,
 *     FP8(x) = round(x / s), out += MMA(FP8(x), FP8(w)) * s_x * s_w.
 * Precise readings used here: F_max = 448 (largest finite E4M3, OCP "FN"
 * encoding); round = nearest-even with saturation to +-448; x / s is an IEEE
 * float32 division; the stored scale is s as float32; a group whose absmax
 * is 0 gets s = 0 and all-zero codes.
 *
 * Conventions shared by every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library allocates no device memory and never synchronises, except
 *     fp8bs_get_device_status().  Every call is asynchronous on `stream`
 *     (a cudaStream_t passed as void*, NULL = legacy default stream).
 *   - Matrices are row-major.  BF16 is IEEE bfloat16 (uint16 bit patterns),
 *     E4M3 codes are bytes, scales are float32.
 *   - "kb-major" scale layout: the scale of row r and 128-column group kb
 *     is stored at s[kb * rows + r] (the rows of one group are contiguous).
 *   - Argument errors are returned before anything is launched.  All device
 *     pointers must be 16-byte aligned, every leading dimension in bytes a
 *     multiple of 16.  The current device must have compute capability
 *     10.3 (FP8BS_ERR_UNSUPPORTED_ARCH otherwise).
 *   - Every wait inside a kernel is bounded in time; a wait that expires, or
 *     a device-side argument check that fails, records a status that
 *     fp8bs_get_device_status() returns.
 *   - Inputs holding NaN or Inf are outside the contract.
 */
#ifndef FP8BS_H_
#define FP8BS_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP8BS_OK = 0,
  FP8BS_ERR_INVALID_ARG = 1,      /* NULL pointer, negative size, unknown enum value */
  FP8BS_ERR_SHAPE = 2,            /* a size breaks a multiple-of rule or a limit of the call */
  FP8BS_ERR_ALIGNMENT = 3,        /* pointer or leading dimension not 16-byte aligned */
  FP8BS_ERR_UNSUPPORTED_ARCH = 4, /* current device is not sm_103 */
  FP8BS_ERR_CUDA = 5,             /* a CUDA runtime or driver call failed */
  FP8BS_ERR_TIMEOUT = 6,          /* a bounded device wait expired */
  FP8BS_ERR_DEVICE_ARG = 7        /* a device-resident argument (group offsets, sequences) was invalid */
} fp8bs_status;

typedef enum { FP8BS_OUT_F32 = 0, FP8BS_OUT_BF16 = 1 } fp8bs_out_dtype;

typedef enum {
  /* B's scale is per 128x128 block: sb[(n / 128) * (K / 128) + kb], i.e. a
   * row-major [ceil(N/128)][K/128] array (weights, §3.3.2 (2)). */
  FP8BS_SCALE_BLOCK128x128 = 0,
  /* B's scale is per row and 1x128 group, kb-major: sb[kb * N + n] (both
   * operands are activations, as in the Wgrad GEMM, §3.3.1 / Figure 6). */
  FP8BS_SCALE_ROW1x128 = 1
} fp8bs_b_scale_kind;

typedef enum {
  /* s = fl32(absmax / 448), the Figure 7 explainer's s = absmax / F_max. */
  FP8BS_SCALE_ABSMAX = 0,
  /* Power-of-two ("rounded") scale, §3.3.3 "low-precision activations" (1)
   * and "low-precision communication": s = 2^k, the smallest power of two
   * with absmax / s <= 448 (k >= -149).  Used for activations that are later
   * re-tiled from 1x128 to 128x1, where it makes the re-tiling lossless. */
  FP8BS_SCALE_POW2 = 1
} fp8bs_scale_mode;

/*
 * Activation quantisation, 1x128 tiles (§3.3.2 "fine-grained quantization"
 * (1) and "online quantization"), optionally also 128x1 tiles of the same
 * input (§3.3.3 "low-precision activations" (1): the backward pass needs the
 * activations grouped along tokens; here they are quantised directly from
 * BF16 in the same pass).
 *
 *   x     [M][ldx] BF16, K columns used.                       (in)
 *   xq    [M][K]   E4M3 codes of the 1x128 tiles.              (out)
 *   sx    [K/128][M] float32, kb-major: sx[kb*M + m].          (out)
 *   xq_t  [K][M]   E4M3 codes of X^T grouped 1x128 along M,    (out, optional)
 *                  i.e. of the 128x1 tiles of X.
 *   sx_t  [M/128][K] float32, kb-major: sx_t[tb*K + k] is the   (out, optional)
 *                  scale of column k, rows 128*tb .. 128*tb+127.
 * Rules: K % 128 == 0; M >= 0 arbitrary, but M % 128 == 0 when xq_t/sx_t
 * are given (both or neither).  ldx >= K, ldx*2 % 16 == 0.
 * Codes and scales are bit-exact with the rule: s = fl32(absmax / 448),
 * code = E4M3_rne_satfinite(fl32(x / s)), s == 0 -> codes 0.
 */
int fp8bs_quantize_act(const void* x, int64_t M, int64_t K, int64_t ldx,
                       uint8_t* xq, float* sx, uint8_t* xq_t, float* sx_t,
                       void* stream);

/* fp8bs_quantize_act with a choice of scale (fp8bs_scale_mode): with
 * FP8BS_SCALE_POW2 every group's scale is a power of two and each code is
 * E4M3_rne_satfinite(x / s) (the quotient is exact).  Same arguments, rules
 * and errors otherwise; an unknown scale_mode is FP8BS_ERR_INVALID_ARG. */
int fp8bs_quantize_act_ex(const void* x, int64_t M, int64_t K, int64_t ldx,
                          uint8_t* xq, float* sx, uint8_t* xq_t, float* sx_t,
                          int scale_mode, void* stream);

/*
 * Weight quantisation, 128x128 blocks (§3.3.2 "fine-grained quantization"
 * (2); weights are quantised online too, "online quantization").
 *
 *   w     [N][ldw] BF16, K columns used.                        (in)
 *   wq    [N][K]   E4M3 codes.                                  (out)
 *   sw    [N/128][K/128] float32, row-major.                    (out)
 *   wq_t  [K][N]   the same codes transposed (optional): B operand of a  (out)
 *                  GEMM that uses the weight transposed (Dgrad, Figure 6).
 *   sw_t  [K/128][N/128] the scales transposed (optional, with wq_t).     (out)
 * Rules: N % 128 == 0, K % 128 == 0, ldw >= K, ldw*2 % 16 == 0.
 */
int fp8bs_quantize_weight(const void* w, int64_t N, int64_t K, int64_t ldw,
                          uint8_t* wq, float* sw, uint8_t* wq_t, float* sw_t,
                          void* stream);

/* fp8bs_quantize_weight with a choice of scale (fp8bs_scale_mode). */
int fp8bs_quantize_weight_ex(const void* w, int64_t N, int64_t K, int64_t ldw,
                             uint8_t* wq, float* sw, uint8_t* wq_t, float* sw_t,
                             int scale_mode, void* stream);

/*
 * Both operands of an FP8 Linear (Figure 6, the online quantisation of
 * §3.3.2) in one launch: X in 1x128 groups exactly as fp8bs_quantize_act_ex
 * without the transposed output, and W in 128x128 blocks exactly as
 * fp8bs_quantize_weight_ex without the transposed copy, with one
 * scale_mode for both.  Codes and scales are bit-identical to the two
 * separate calls; one persistent grid walks X's tiles, then W's.
 *
 *   x  [M][ldx] BF16, K columns;  xq [M][K];  sx [K/128][M] (kb-major).
 *   w  [N][ldw] BF16, Kw columns; wq [N][Kw]; sw [N/128][Kw/128].
 * Rules: the union of the two calls' rules (K, N, Kw multiples of 128,
 * 16-byte aligned pointers and leading dimensions); M == 0 or N == 0 leaves
 * that operand out; errors as those calls.
 */
int fp8bs_quantize_act_weight(const void* x, int64_t M, int64_t K, int64_t ldx,
                              uint8_t* xq, float* sx,
                              const void* w, int64_t N, int64_t Kw, int64_t ldw,
                              uint8_t* wq, float* sw, int scale_mode, void* stream);

/*
 * Backward re-tiling from FP8 (§3.5.2 "support for transposed GEMM
 * operations": read the 1x128-quantised activations, dequantise, transpose,
 * requantise in 128x1 tiles; §3.3.3 "low-precision activations" (1): with
 * power-of-two scales this adds no quantisation error):
 *
 *   v[m][k]       = fl32(dec(xq[m][k]) * sx[kb*M + m])        (kb = k / 128)
 *   group (k, tb) = v[128*tb .. 128*tb+127][k]
 *   sx_t[tb*K + k] = scale of the group (scale_mode), xq_t[k][m] = its codes.
 *
 *   xq    [M][K] E4M3, 1x128 groups.  sx [K/128][M] float32, kb-major.   (in)
 *   xq_t  [K][M] E4M3, 128x1 groups.  sx_t [M/128][K] float32.           (out)
 * The outputs have the layout of fp8bs_quantize_act's xq_t / sx_t, so they
 * feed the Wgrad GEMM (FP8BS_SCALE_ROW1x128) directly.
 * Rules: M % 128 == 0, K % 128 == 0; all pointers 16-byte aligned.
 */
int fp8bs_requant_1x128_to_128x1(const uint8_t* xq, const float* sx, int64_t M, int64_t K,
                                 uint8_t* xq_t, float* sx_t, int scale_mode, void* stream);

/*
 * Fused SwiGLU and 1x128 quantisation: the input of the MoE down projection
 * (§3.3.3 "low-precision activations" (2): the SwiGLU output feeds the
 * down-projection FP8 GEMM; doing the cast in the producer avoids writing and
 * re-reading the BF16 activation, the cost §3.5.2 names):
 *
 *   v[m][i] = BF16_rne( silu(h[m][i]) * h[m][I + i] ),  silu(g) = g / (1 + e^-g)
 *   (xq, sx) = the 1x128 quantisation of v, as fp8bs_quantize_act(_ex).
 *
 *   h   [M][ldh] BF16: the gate/up projection output, gate in columns [0, I),
 *       up in columns [I, 2I).                                        (in)
 *   q   [M][I] E4M3 codes.  s [I/128][M] float32, kb-major.            (out)
 * silu(gate) * up is evaluated in FP32 with a relative error below 2^-16 for
 * every gate (gates below -64 take an overflow-free form g * up * e^g),
 * so a value within that distance of a BF16 rounding boundary may round either
 * way; codes and scales are otherwise those of quantising the rounded v.
 * Rules: I % 128 == 0, ldh >= 2*I, ldh*2 % 16 == 0; pointers 16-byte aligned.
 */
int fp8bs_swiglu_quantize(const void* h, int64_t M, int64_t I, int64_t ldh,
                          uint8_t* q, float* s, int scale_mode, void* stream);

/*
 * Block-scaled FP8 GEMM, D = A * B^T with per-128-K-block dequantisation
 * (§3.3.2 "increasing accumulation precision", Figure 7b; Figure 7 explainer
 * formula out += MMA(FP8(x), FP8(w)) * s_x * s_w):
 *
 *   D[m][n] (+)= sum_kb  P_kb[m][n] * sa[kb*M + m] * s_b(n, kb),
 *   P_kb[m][n]  = sum_{k in 128*kb .. 128*kb+127} A[m][k] * B[n][k]
 * with P_kb computed on the tensor cores and the scaled sum in FP32.
 *
 *   a   [M][K] E4M3, K-major.   sa [K/128][M] float32, kb-major.
 *   b   [N][K] E4M3, K-major.   sb per sb_kind (see fp8bs_b_scale_kind).
 *   d   [M][N] FP32 or BF16 (round-to-nearest-even from FP32).
 *   accumulate: FP32 output only; non-zero -> D += result (Wgrad
 *   accumulation), zero -> D = result.
 * Rules: K % 128 == 0, K > 0; N % 128 == 0; M >= 0 arbitrary.
 */
int fp8bs_gemm(const uint8_t* a, const float* sa,
               const uint8_t* b, const float* sb, int sb_kind,
               void* d, int d_dtype, int64_t M, int64_t N, int64_t K,
               int accumulate, void* stream);

/*
 * Grouped block-scaled FP8 GEMM for MoE experts (the expert GEMMs consume
 * FP8 activations dispatched per expert, §3.3.3 "low-precision
 * communication").  Rows [offsets[g], offsets[g+1]) of A belong to expert
 * g and are multiplied by expert g's weight:
 *
 *   D[r][n] = sum_kb P_kb[r][n] * sa[kb*M_total + r] * sb[g][n/128][kb]
 *
 *   a        [M_total][K] E4M3.  sa [K/128][M_total] float32, kb-major.
 *   offsets  DEVICE int32 [num_groups + 1]: non-decreasing, offsets[0] >= 0,
 *            every offset a multiple of 128, offsets[G] <= M_total.  Checked
 *            on the device: a violation skips the launch's work and records
 *            FP8BS_ERR_DEVICE_ARG.
 *   b        [num_groups][N][K] E4M3.  sb [num_groups][N/128][K/128].
 *   d        [M_total][N] FP32 or BF16; rows outside every group are not written.
 * Rules: K % 128 == 0, N % 128 == 0, 1 <= num_groups <= 512.
 */
int fp8bs_grouped_gemm(const uint8_t* a, const float* sa, int64_t M_total,
                       const int32_t* offsets, int num_groups,
                       const uint8_t* b, const float* sb,
                       void* d, int d_dtype, int64_t N, int64_t K, void* stream);

/*
 * The block-scaled FP8 GEMM for power-of-two scales, with the scales applied
 * by the tensor core: §3.5.2 (compute hardware) asks for tensor cores that
 * take the group scaling factors themselves, so that partial sums need not
 * be promoted to the CUDA cores for dequantisation; §3.3.2 notes the
 * microscaling formats of the Blackwell generation.  Here the MMA is
 * tcgen05.mma.kind::mxf8f6f4.block_scale: each group scale becomes an UE8M0
 * scale (an 8-bit biased exponent) repeated over the group's four
 * 32-element blocks of K, and all of K accumulates in FP32 in tensor memory.
 *
 *   D[m][n] (+)= sum_kb P_kb[m][n] * sa[kb*M + m] * s_b(n, kb)
 *
 * Same arguments, layouts, rules and errors as fp8bs_gemm, and the same
 * result up to FP32 summation order, for operands whose scales are all
 * powers of two: quantised with FP8BS_SCALE_POW2 (fp8bs_quantize_act_ex,
 * fp8bs_quantize_weight_ex, fp8bs_requant_1x128_to_128x1).  Every scale of
 * a row or column inside the output must be 0 (a group of zero codes) or a
 * power of two in [2^-127, 2^127]; any other value is detected on the device
 * and records FP8BS_ERR_DEVICE_ARG for fp8bs_get_device_status(), and D is
 * then undefined.  The quantisers produce scales below 2^-127 only for
 * groups whose absmax is below 448 * 2^-127; such operands need fp8bs_gemm.
 */
int fp8bs_gemm_pow2(const uint8_t* a, const float* sa,
                    const uint8_t* b, const float* sb, int sb_kind,
                    void* d, int d_dtype, int64_t M, int64_t N, int64_t K,
                    int accumulate, void* stream);

/*
 * Grouped (MoE) form of fp8bs_gemm_pow2: arguments, layouts, rules and
 * errors of fp8bs_grouped_gemm, scales as fp8bs_gemm_pow2.  The activations
 * dispatched to the experts carry power-of-two scales (§3.3.3
 * "low-precision communication"); the expert weights must be quantised with
 * FP8BS_SCALE_POW2 as well.
 */
int fp8bs_grouped_gemm_pow2(const uint8_t* a, const float* sa, int64_t M_total,
                            const int32_t* offsets, int num_groups,
                            const uint8_t* b, const float* sb,
                            void* d, int d_dtype, int64_t N, int64_t K, void* stream);

/* Layout of the float32 scales of a matrix of E4M3 codes [rows][H] (1x128
 * groups) in fp8bs_gather_q_rows. */
typedef enum {
  FP8BS_SCALES_KB_MAJOR = 0,  /* s[kb * rows + r]: the layout every GEMM reads */
  FP8BS_SCALES_ROW_MAJOR = 1  /* s[r * (H/128) + kb]: one contiguous record per row */
} fp8bs_scale_layout;

/*
 * Row gather of FP8 codes with their 1x128 scales, the data movement of the
 * MoE dispatch (§3.3.3 "low-precision communication": the activations are
 * quantised to FP8, with power-of-two scales, before they are dispatched to
 * the experts, so the FP8 bytes and scales are what moves; the expert GEMMs
 * consume them directly):
 *
 *   q_out[i][:] = q[idx[i]][:],  scales of out row i = scales of row idx[i];
 *   idx[i] < 0 (or >= rows_in): a row of zero codes with zero scales (the
 *   padding of an expert's segment to a multiple of 128 rows).
 *
 *   q      [rows_in][H] E4M3 codes.  s: float32 scales in s_in_layout.   (in)
 *   idx    DEVICE int32 [rows_out].                                       (in)
 *   q_out  [rows_out][H] E4M3.  s_out: float32 scales in s_out_layout.   (out)
 * Packing the rows a rank sends into one buffer per destination (row-major
 * scales: one record per row travels with it) and unpacking received rows
 * into the experts' padded segments (kb-major scales, as the grouped GEMM
 * reads them) are both this call.
 * Rules: H % 128 == 0; q, q_out 16-byte aligned; the layouts are
 * fp8bs_scale_layout values (FP8BS_ERR_INVALID_ARG otherwise).
 */
int fp8bs_gather_q_rows(const uint8_t* q, const float* s, int64_t rows_in, int64_t H, int s_in_layout,
                        const int32_t* idx, int64_t rows_out, uint8_t* q_out, float* s_out, int s_out_layout,
                        void* stream);

/*
 * Row scatter of FP8 codes with their 1x128 scales: the dispatch written from
 * the sender's side, each token row read once and written to each of its k
 * destinations (§3.3.3 "low-precision communication", as fp8bs_gather_q_rows):
 *
 *   for r < rows_in, j < k:  if 0 <= pos[r*k + j] < rows_out, out row
 *     pos[r*k + j] = q[r][:] with the scales of row r;
 *   for i < n_zero:  if 0 <= zero_rows[i] < rows_out, out row zero_rows[i] =
 *     zero codes with zero scales (the padding of an expert's segment).
 *
 *   q      [rows_in][H] E4M3 codes.  s: float32 scales in s_in_layout.   (in)
 *   pos    DEVICE int32 [rows_in][k]; zero_rows DEVICE int32 [n_zero]
 *          (NULL allowed when n_zero == 0).                               (in)
 *   q_out  [rows_out][H] E4M3.  s_out: float32 scales in s_out_layout.   (out)
 * Out rows named by neither list are left as they are; a row named more than
 * once gets one of its writes, which one is unspecified.
 * Rules: H % 128 == 0; 1 <= k <= 64; n_zero >= 0; q, q_out 16-byte aligned;
 * the layouts are fp8bs_scale_layout values (FP8BS_ERR_INVALID_ARG otherwise).
 */
int fp8bs_scatter_q_rows(const uint8_t* q, const float* s, int64_t rows_in, int64_t H, int s_in_layout,
                         const int32_t* pos, int k, const int32_t* zero_rows, int64_t n_zero, int64_t rows_out,
                         uint8_t* q_out, float* s_out, int s_out_layout, void* stream);

/*
 * Row gather of a BF16 matrix (the expert outputs put back in send order for
 * the combine, which §3.3.3 keeps in BF16):
 *   out[i][:] = y[idx[i]][:], zeros where idx[i] < 0 or >= rows_in.
 *   y [rows_in][N] BF16; idx DEVICE int32 [rows_out]; out [rows_out][N] BF16.
 * Rules: N % 8 == 0; y, out 16-byte aligned.
 */
int fp8bs_gather_bf16_rows(const void* y, int64_t rows_in, int64_t N, const int32_t* idx, int64_t rows_out,
                           void* out, void* stream);

/*
 * The MoE combine in BF16 (§3.3.3: the combine components stay in BF16):
 *   out[t][n] = BF16_rne( sum_{j<k} w[t][j] * y[idx[t][j]][n] ),
 * the products and the sum in FP32 (fused multiply-adds, j ascending) and one
 * rounding to BF16; idx[t][j] < 0 (or >= rows_y) contributes nothing.
 *   y    [rows_y][N] BF16: the expert outputs, one row per (token, expert).
 *   idx  DEVICE int32 [T][k]: the row of y holding token t's j-th expert output.
 *   w    DEVICE float32 [T][k]: the gate weights.
 *   out  [T][N] BF16.
 * Rules: N % 8 == 0; 1 <= k <= 64; y, out 16-byte aligned.
 */
int fp8bs_moe_combine(const void* y, int64_t rows_y, int64_t N, const int32_t* idx, const float* w, int64_t T, int k,
                      void* out, void* stream);

/* ---------------------------------------------------------------- 4 bits
 * Microscaled 4-bit operands: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives) with a scale per block of consecutive elements of K.
 *
 *   codes   [M][K/2] bytes, two codes a byte, the element of even column in
 *           the low four bits.
 *   scales  one byte per row and block, in blocks of 512 bytes that hold 128
 *           rows x 4 groups: with J = K / 16 or K / 32 groups a row, the scale
 *           of row r and group j is byte
 *             ((r / 128) * ceil(J / 4) + j / 4) * 512
 *             + (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4,
 *           fp8bs_fp4_scale_bytes(M, K, fmt) bytes in all.  The quantisers
 *           fill the rows up to a multiple of 128 with zeros.
 *   g       [M] float32, one scale per row (FP8BS_FP4_E4M3X16 only).
 */
typedef enum {
  /* E4M3 scale per 16 elements and a float32 scale per row:
   *   g = max(fl32(rowmax / 2688), 2^-100)            (2688 = 6 * 448)
   *   s = E4M3_rne(fl32(amax / fl32(6 g)))            per 16 elements
   *   code = E2M1_rne_satfinite(fl32(x * fl32(1 / fl32(s g)))), zero if s = 0
   *   value = code * s * g */
  FP8BS_FP4_E4M3X16 = 0,
  /* UE8M0 scale per 32 elements (byte b stands for 2^(b - 127)): s = 2^k, the
   * smallest power of two with amax / s <= 6, k >= -127;
   *   code = E2M1_rne_satfinite(x / s), value = code * s.  g is not used and
   * may be NULL. */
  FP8BS_FP4_UE8M0X32 = 1
} fp8bs_fp4_format;

/* Bytes of the blocked scales of an [M][K] matrix; -1 for arguments that the
 * calls below refuse. */
int64_t fp8bs_fp4_scale_bytes(int64_t M, int64_t K, int fmt);

/*
 * 4-bit quantisation, optionally of gathered rows (the dispatch of tokens into
 * the padded segments of their experts, quantised on the way):
 *
 *   out row i = the codes, scales (and g) of x[rows ? rows[i] : i][:];
 *   rows[i] < 0 (or >= rows_in): a row of zeros (scales 0, g = 2^-100).
 *
 *   x     [rows_in][ldx] BF16, K columns used.                        (in)
 *   rows  DEVICE int32 [M], or NULL: then rows_in must be M.          (in)
 *   q, sf, g: see above.                                              (out)
 * Rules: K % 64 == 0 (FP8BS_ERR_SHAPE); ldx >= K, ldx*2 % 16 == 0; x, q, sf
 * 16-byte aligned.  0 <= M <= 2^30.
 */
int fp8bs_quantize_fp4(const void* x, int64_t rows_in, int64_t K, int64_t ldx, const int32_t* rows, int64_t M,
                       int fmt, uint8_t* q, uint8_t* sf, float* g, void* stream);

/*
 * SwiGLU and 4-bit quantisation in one pass, the input of the experts' down
 * projection: v = BF16_rne(gate / (1 + e^-gate) * up) (float32, IEEE division;
 * below gate = -64 as gate e^(gate/2) e^(gate/2) up, which does not overflow),
 * quantised as by fp8bs_quantize_fp4.
 *
 *   h     [M][ldh] BF16, gate in columns [0, I), up in [I, 2I).       (in)
 *   live  DEVICE int32 [M], or NULL: live[i] < 0 gives a row of zeros and
 *         h's row i is not read (padding; fp8bs_moe_layout's row_token). (in)
 * Rules: I % 64 == 0, ldh >= 2I, ldh*2 % 16 == 0, I*2 % 16 == 0.
 */
int fp8bs_swiglu_quantize_fp4(const void* h, int64_t M, int64_t I, int64_t ldh, const int32_t* live, int fmt,
                              uint8_t* q, uint8_t* sf, float* g, void* stream);

/*
 * The values that 4-bit codes stand for: out[m][k] = code * s (* g), the
 * products in float32, rounded once more for BF16 output (fp8bs_out_dtype).
 * Rules: K % 64 == 0; ldo >= K, ldo * (2 or 4) % 16 == 0; pointers 16-byte
 * aligned (g: 4).
 */
int fp8bs_dequantize_fp4(const uint8_t* q, const uint8_t* sf, const float* g, int64_t M, int64_t K, int fmt,
                         void* out, int out_dtype, int64_t ldo, void* stream);

/*
 * 4-bit GEMM, D = A * B^T of the values that the codes stand for, the block
 * scales applied by the tensor core, all of K accumulated in FP32:
 *
 *   D[m][n] = ga[m] gb[n] sum_k a[m][k] sa(m, k) b[n][k] sb(n, k)
 *
 *   a, sfa, ga: [M][K] as above; b, sfb, gb: [N][K]; ga, gb unused (may be
 *   NULL) with FP8BS_FP4_UE8M0X32.  d [M][N] FP32 or BF16 (fp8bs_out_dtype).
 * Rules: K % 64 == 0, K > 0, N % 8 == 0, M arbitrary; pointers 16-byte aligned
 * (ga: 4).  Scale bytes must not be NaN (E4M3 0x7F, 0xFF; UE8M0 0xFF) in rows
 * below M and N.
 */
int fp8bs_gemm_fp4(const uint8_t* a, const uint8_t* sfa, const float* ga,
                   const uint8_t* b, const uint8_t* sfb, const float* gb, int fmt,
                   void* d, int d_dtype, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * Grouped (MoE) form: rows [offsets[g], offsets[g+1]) of A times expert g's
 * weight, offsets as in fp8bs_grouped_gemm (device int32, multiples of 128,
 * checked on the device).  b [G][N][K/2]; sfb: fp8bs_fp4_scale_bytes(N, K, fmt)
 * bytes per expert, one expert after the other; gb [G][N].
 */
int fp8bs_grouped_gemm_fp4(const uint8_t* a, const uint8_t* sfa, const float* ga, int64_t M_total,
                           const int32_t* offsets, int num_groups,
                           const uint8_t* b, const uint8_t* sfb, const float* gb, int fmt,
                           void* d, int d_dtype, int64_t N, int64_t K, void* stream);

/* ---------------------------------------------------------------- router */
typedef enum { FP8BS_IN_F32 = 0, FP8BS_IN_BF16 = 1 } fp8bs_in_dtype;
typedef enum { FP8BS_SCORE_SOFTMAX = 0, FP8BS_SCORE_SIGMOID = 1 } fp8bs_score_kind;

/*
 * The MoE router: each token's k experts and gate weights, and, for training,
 * the counts and the balance loss of every sequence.
 *
 *   s_i = softmax(z)_i or sigmoid(z_i);  p_i = s_i / sum_j s_j.
 *   The experts chosen are the k of largest z_i, or of largest s_i + bias_i
 *   (bias: sigmoid only), in descending order, ties to the lower index.  A
 *   logit of -inf or NaN is not eligible: p_i = s_i = 0; a slot that finds no
 *   eligible expert holds idx -1 and weight 0.  Tokens with valid[t] == 0 have
 *   no eligible expert, whatever their logits hold.
 *   w[t][j] = scale * s_idx / (normalize ? sum over the token's slots : 1).
 *   Each sum that scores are divided by has 1e-20 added.
 *
 *   loss = alpha / S * sum_q sum_i f_qi P_qi   over the sequences q,
 *     f_qi = E counts[q][i] / (k tokens[q]),  P_qi = sum_t p_i / tokens[q],
 *   tokens[q] the sequence's tokens with an eligible expert (one without any
 *   adds nothing).  counts are those of the experts chosen: with a bias, of the
 *   biased choice, which the bias's own update goes by as well.  (A loss whose
 *   f counts the k largest scores without the bias differs from this one
 *   wherever the bias moves a choice.)  Nothing limits a choice to groups of
 *   experts.
 *
 *   logits [T][ld] float32 or BF16 (fp8bs_in_dtype), E columns.       (in)
 *   bias   [E] float32, finite, or NULL.  valid [T] bytes or NULL.     (in)
 *   seq    DEVICE int32 [S + 1], 0 = seq[0] <= ... <= seq[S] = T, or NULL with
 *          S = 1.  Checked on the device where it is read: a violation
 *          records FP8BS_ERR_DEVICE_ARG and leaves the outputs undefined. (in)
 *   idx    [T][k] int32, w [T][k] float32.                            (out)
 *   counts [S][E] int32, tokens [S] int32, loss [1] float32: all three, or all
 *          NULL to leave the statistics out (seq is then not read).   (out)
 *   ws     scratch of fp8bs_moe_route_workspace_bytes(T, E, S) bytes with
 *          statistics, else NULL.
 * Rules: 1 <= E <= 1024, 1 <= k <= min(E, 32), ld >= E, 1 <= S <= 65535,
 * T < 2^31; pointers aligned to their elements, ws to 16 bytes.  Sums are taken
 * in a fixed order: the same inputs give the same bits.  Logits of +inf are
 * outside the contract.  Weights and biased keys are formed with expf and IEEE
 * divisions; the scores in the sums, here and in the gradient, to 2^-21 relative.
 */
int fp8bs_moe_route(const void* logits, int in_dtype, int64_t T, int E, int64_t ld, int score, const float* bias,
                    const uint8_t* valid, const int32_t* seq, int64_t S, int k, int normalize, float scale,
                    float alpha, int32_t* idx, float* w, int32_t* counts, int32_t* tokens, float* loss,
                    void* ws, int64_t ws_bytes, void* stream);
/* -1 for arguments that fp8bs_moe_route refuses. */
int64_t fp8bs_moe_route_workspace_bytes(int64_t T, int E, int64_t S);

/*
 * Gradient of fp8bs_moe_route with respect to the logits, from those of the
 * weights and of the loss (the counts, and so f, are constants):
 *   dlogits = dw . d w / d z + dloss[0] * d loss / d z,
 * 0 for logits that are not eligible.  The scores are recomputed.
 *
 *   idx, counts, tokens: fp8bs_moe_route's outputs; other arguments as there.
 *   dw      [T][k] float32 (slots with idx < 0 are not read).          (in)
 *   dloss   DEVICE float32 [1], or NULL (counts, tokens may be NULL too). (in)
 *   dlogits [T][ldd], of the logits' type, ldd >= E.                   (out)
 */
int fp8bs_moe_route_backward(const void* logits, int in_dtype, int64_t T, int E, int64_t ld, int score,
                             const uint8_t* valid, const int32_t* seq, int64_t S, int k, int normalize, float scale,
                             float alpha, const int32_t* idx, const int32_t* counts, const int32_t* tokens,
                             const float* dw, const float* dloss, void* dlogits, int64_t ldd, void* stream);

/*
 * Row layout of the chosen experts, on the device: the segments that the
 * grouped GEMMs read, as the host planner lays them out for one rank.
 *
 *   offsets   [E + 1] int32: expert e's segment is rows [offsets[e],
 *             offsets[e+1]), its choices in token order, padded to a multiple
 *             of 128.                                                   (out)
 *   row_token [rows] int32: the token of each row, -1 for padding and for the
 *             rows past offsets[E].                                     (out)
 *   row_of    [T][k] int32: the row of each choice, -1 where idx is negative
 *             or not below E.                                           (out)
 *   idx [T][k] int32 (in); rows >= fp8bs_moe_layout_rows(T, k, E), the most
 *   that any choice of experts can take (FP8BS_ERR_SHAPE otherwise).
 *   ws: scratch of fp8bs_moe_layout_workspace_bytes(T, k, E) bytes.
 * Rules: 1 <= E <= 1024, 1 <= k <= 64, T * k <= 2^24; pointers aligned to 4.
 */
int fp8bs_moe_layout(const int32_t* idx, int64_t T, int k, int E, int32_t* offsets, int32_t* row_token, int64_t rows,
                     int32_t* row_of, void* ws, int64_t ws_bytes, void* stream);
/* Both return -1 for arguments that fp8bs_moe_layout refuses. */
int64_t fp8bs_moe_layout_rows(int64_t T, int k, int E);
int64_t fp8bs_moe_layout_workspace_bytes(int64_t T, int k, int E);

/* -------------------------------------------------------------- training
 * The operators of a training step around the 8-bit products.  Where one
 * quantises, it quantises the BF16 value that it would store: codes and scales
 * are bit for bit those of fp8bs_quantize_act_ex on that value, also where it is
 * an infinity that finite inputs overflowed to: with power-of-two scales its code
 * is E4M3's NaN, with absmax scales its whole group's.  Sums are taken in float32
 * in a fixed order: the same inputs give the same bits.
 *
 * Infinities and NaN in the inputs are outside the contract here too: they leave
 * the rest as it is and show in what they reach, but codes and scales may not be
 * the quantiser's there.  A maximum passes over NaN, so that a NaN among zeros has
 * code 0; an infinity of dout under a weight of zero, which is NaN, has NaN's code,
 * where the quantiser has 0.
 */

#define FP8BS_RMSNORM_MIN_EPS 7.8886090522101181e-31f /* 2^-100: squares that underflow do not count beside it */

/*
 * Root-mean-square norm of the residual stream, quantised for the Linear that
 * reads it:
 *
 *   r    = residual ? BF16_rne(x + residual) : x      (the sum in float32)
 *   rstd = 1 / sqrt(mean_k r^2 + eps)                 (float32)
 *   y    = BF16_rne(r * gain * rstd);   (q, s) = the 1x128 quantisation of y
 *
 *   x        [M][ldx] BF16.  residual [M][ldr] BF16, or NULL.           (in)
 *   gain     [K] float32 or BF16 (fp8bs_in_dtype).                      (in)
 *   r        [M][K] BF16, given exactly with a residual; it may be x or
 *            residual itself where that has K columns a row.           (out)
 *   y        [M][K] BF16 or NULL.                                      (out)
 *   q, s     [M][K] E4M3 and [K/128][M] float32, both or neither.      (out)
 *   rstd     [M] float32 or NULL (the gradient reads it).              (out)
 * At least one of y and q.  Rules: K % 8 == 0, with q K % 128 == 0, K <= 16384;
 * 2^-100 <= eps <= 1e30; the sum of a row's squares and each r * gain have to
 * stay in float32's range.  x, residual, gain, r, y and q 16-byte aligned, s and rstd 4.  K == 0 writes
 * nothing, rstd neither.
 */
int fp8bs_rmsnorm_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, const void* residual, int64_t ldr,
                           const void* gain, int gain_dtype, float eps, void* r, void* y, uint8_t* q, float* s,
                           int scale_mode, float* rstd, void* stream);

/*
 * Its gradient, with t = dy * gain (the gradient through the residual's
 * addition is dx for both summands):
 *
 *   dx      = BF16_rne(rstd t - r rstd^3 mean_k(t r) + dres)
 *   dgain_k = sum_m dy r rstd          (accumulate: added to what dgain holds)
 *
 *   dy    [M][lddy] BF16, the gradient of y.  r [M][ldr] BF16 (x where there
 *         was no residual).  rstd [M].  dres [M][lddres] BF16 or NULL, what
 *         reaches r along the residual stream.                          (in)
 *   dx    [M][K] BF16; it may be dy, r or dres itself where that has K
 *         columns a row.  dgain [K] float32, or NULL.                  (out)
 *   ws    scratch of fp8bs_rmsnorm_backward_workspace_bytes(M, K) bytes, 16-byte
 *         aligned, with dgain; two calls at once need one each.
 * Rules as above, K % 8 == 0; dy * gain, dy * r and the sum of a row's t r have to
 * stay in float32's range.  M == 0 gives a dgain of zeros.
 */
int fp8bs_rmsnorm_backward(const void* dy, int64_t M, int64_t K, int64_t lddy, const void* r, int64_t ldr,
                           const void* gain, int gain_dtype, const float* rstd, const void* dres, int64_t lddres,
                           void* dx, float* dgain, int accumulate, void* ws, int64_t ws_bytes, void* stream);
/* -1 for arguments that fp8bs_rmsnorm_backward refuses. */
int64_t fp8bs_rmsnorm_backward_workspace_bytes(int64_t M, int64_t K);

/*
 * Gradient of the SwiGLU v = silu(gate) * up with respect to its input, the
 * operand of the gate/up projection's gradients:
 *
 *   dgate = BF16_rne(dv up sigma(gate) (1 + gate sigma(-gate)))
 *   dup   = BF16_rne(dv gate sigma(gate));   (q, s) = the 1x128 quantisation
 *
 *   h     [M][ldh] BF16, gate in columns [0, I), up in [I, 2I).
 *   dv    [M][lddv] BF16.  live DEVICE int32 [M] or NULL: live[i] < 0 gives a
 *         row of zeros, and h's and dv's row is not read.               (in)
 *   dh    [M][2I] BF16 or NULL: dgate, then dup.                       (out)
 *   q, s  [M][2I] E4M3 and [2I/128][M] float32, both or neither.       (out)
 * At least one of dh and q; dh is not h or dv, which may be read again.  Rules:
 * I % 128 == 0, ldh >= 2I, lddv >= I; 16-byte rows and pointers (live and s: 4).
 */
int fp8bs_swiglu_backward_quantize(const void* h, int64_t M, int64_t I, int64_t ldh, const void* dv, int64_t lddv,
                                   const int32_t* live, void* dh, uint8_t* q, float* s, int scale_mode, void* stream);

/*
 * Gradient of fp8bs_moe_combine: of the experts' outputs, in their segments and
 * quantised for the products that read them, and of the gate weights.
 *
 *   row i = row_of[t][j]:  dy[i] = BF16_rne(w[t][j] dout[t]);  (q, s) = the 1x128
 *     quantisation of dy;  dw[t][j] = sum_n dout[t][n] y[i][n]
 *   rows with row_token[i] < 0: zeros (codes, scales and dy).
 *   row_of[t][j] < 0 (or >= rows): no row; dw[t][j] = 0.
 *
 *   dout  [T][ldo] BF16.  y [rows][N] BF16, the experts' outputs (NULL with
 *         dw NULL).  row_of [T][k], row_token [rows] int32 as
 *         fp8bs_moe_layout gives them; w [T][k] float32.                (in)
 *   dy    [rows][N] BF16 or NULL.  q, s [rows][N] E4M3 and [N/128][rows]
 *         float32, both or neither.  dw [T][k] float32 or NULL.        (out)
 * At least one of dy and q.  A row that several slots of its token name takes
 * the sum of their weights.  A row that a token names and row_token gives to
 * another records FP8BS_ERR_DEVICE_ARG and is passed over (dw 0).  Rows that
 * row_token gives to a token that does not name them are left as they are.
 * Rules: N % 8 == 0, with q N % 128 == 0; 1 <= k <= 64, T * k <= 2^24, rows <=
 * 2^30; dout, y, dy, q 16-byte aligned, ldo * 2 % 16 == 0, the others 4.  N == 0
 * writes nothing, dw neither.
 */
int fp8bs_moe_combine_backward(const void* dout, int64_t T, int64_t N, int64_t ldo, const void* y, int64_t rows,
                               const int32_t* row_of, const int32_t* row_token, const float* w, int k, void* dy,
                               uint8_t* q, float* s, int scale_mode, float* dw, void* stream);

/*
 * Gradient of the dispatch, which copied each token to the rows of its choices:
 *   dx[t] = BF16_rne(add[t] + sum_j d[row_of[t][j]]),  the sum in float32, j
 * ascending; row_of[t][j] < 0 (or >= rows) adds nothing.
 *   d [rows][N] BF16; add [T][N] BF16 or NULL (it may be dx); dx [T][N] BF16.
 * Rules as fp8bs_moe_combine.
 */
int fp8bs_moe_dispatch_backward(const void* d, int64_t rows, int64_t N, const int32_t* row_of, int64_t T, int k,
                                const void* add, void* dx, void* stream);

/*
 * Gradient of the experts' weights (the grouped form of the Wgrad GEMM): with
 * the rows [offsets[g], offsets[g+1]) of both operands expert g's,
 *
 *   D[g][n][k] (+)= sum_r A[r][n] B[r][k],
 *
 * A the gradients of the experts' outputs and B their inputs, both in 128x1
 * groups with power-of-two scales (fp8bs_requant_1x128_to_128x1, or
 * fp8bs_quantize_act_ex's transposed output), applied by the tensor core as in
 * fp8bs_gemm_pow2, with the same rule for scales.
 *
 *   a_t  [N][R] E4M3, sa_t [R/128][N] float32.
 *   b_t  [K][R] E4M3, sb_t [R/128][K] float32.                          (in)
 *   offsets DEVICE int32 [num_groups + 1], as in fp8bs_grouped_gemm, at most R. (in)
 *   d    [num_groups][N][K] FP32 or BF16.  accumulate: FP32 only; non-zero
 *        adds to D.  An expert without rows gets zeros (or adds nothing). (out)
 * Rows outside every segment are not read.  Rules: R, N, K % 128 == 0, R <= 2^30,
 * 1 <= num_groups <= 512, num_groups * N < 2^31; a_t, b_t, sb_t, d 16-byte aligned.
 */
int fp8bs_grouped_wgrad_pow2(const uint8_t* a_t, const float* sa_t, const uint8_t* b_t, const float* sb_t, int64_t R,
                             const int32_t* offsets, int num_groups, void* d, int d_dtype, int64_t N, int64_t K,
                             int accumulate, void* stream);

/*
 * Synchronises `stream`, then returns and clears the device status of the
 * current device: FP8BS_OK, FP8BS_ERR_TIMEOUT, FP8BS_ERR_DEVICE_ARG, or
 * FP8BS_ERR_CUDA if the synchronisation itself failed.
 */
int fp8bs_get_device_status(void* stream);

/* Diagnostic of the failure path: launches a kernel that waits, through the
 * same bounded mbarrier wait every kernel here uses, on a barrier nothing
 * arrives on.  After `timeout_us` microseconds (1 .. 10^7) the wait gives up,
 * the kernel records FP8BS_ERR_TIMEOUT and returns normally, so the next
 * fp8bs_get_device_status() reports FP8BS_ERR_TIMEOUT and the CUDA context
 * stays usable.  Returns FP8BS_OK once the kernel is launched. */
int fp8bs_selftest_wait_timeout(int64_t timeout_us, void* stream);

/*
 * Diagnostic, not part of the hot path: D = A B^T with the FP8 products of
 * all of K accumulated by the tensor core alone (no promotion to FP32
 * registers every 128 K, no scales), the configuration whose accumulation
 * precision DeepSeek-V3 §3.3.2 "Increasing accumulation precision" measures
 * (a maximum relative error near 2% for K = 4096 on H800).  Comparing its
 * result with the exact sum gives the same measurement on this GPU.
 *
 *   a  [M][K] E4M3, K-major;  b  [N][K] E4M3, K-major;  d  [M][N] float32.
 * Rules: M % 128 == 0, N % 256 == 0, K % 128 == 0, K > 0 (FP8BS_ERR_SHAPE);
 * pointers 16-byte aligned (FP8BS_ERR_ALIGNMENT).  Asynchronous on
 * `stream`; a bounded wait that expires records FP8BS_ERR_TIMEOUT for
 * fp8bs_get_device_status() and leaves d unwritten.  Caller owns all
 * buffers.
 */
int fp8bs_diag_gemm_unpromoted(const uint8_t* a, const uint8_t* b, float* d, int64_t M, int64_t N, int64_t K,
                               void* stream);

/* Sets the limit of every bounded device wait, in milliseconds (default
 * 2000; 0 restores the default).  Applies to launches made after the call. */
int fp8bs_set_wait_timeout_ms(int64_t ms);

/* Static, NUL-terminated description of a status code. */
const char* fp8bs_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_H_ */
