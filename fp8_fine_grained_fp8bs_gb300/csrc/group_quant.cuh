// Quantisation of a group of BF16 values to E4M3 with one float32 scale, shared
// by the quantisers (quantize.cu) and by the operators that quantise what they
// produce (train.cu): the group's maximum, its divisor in either scale mode,
// and the codes of value pairs by correctly rounded quotients.
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace fp8bs {
namespace {

// Two float32 -> two E4M3 codes (RNE, saturating to +-448); a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// Per-group divisor: s and y = RN(1/s).  Quotients use Markstein's
// correctly rounded division by a fused multiply-add correction (P.
// Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Develop. 34(1), 1990):
//   q0 = RN(x * y),  r = x - s * q0 (exact by one FMA),  q1 = RN(q0 + r * y),
// which gives q1 = RN(x / s) when y = RN(1/s) and r does not underflow.  For
// every quotient that can give a non-zero E4M3 code (|x / s| >= 2^-10) r is
// exact once s >= 2^-93, and smaller quotients encode to a signed zero
// either way; groups with s < 2^-93 (and s == 0) take IEEE divisions.  An
// input of -0 yields q1 = +0, so the sign of x is ORed back into its code
// (a no-op for every other input, whose code already has x's sign).
struct Divisor {
  float s;
  float y;    // RN(1/s)
  bool fast;  // s >= 2^-93: Markstein path; otherwise IEEE divisions
};

constexpr float kMinFastScale = 1.0097419586828951e-28f;  // 2^-93

__device__ __forceinline__ Divisor make_divisor(float absmax) {
  Divisor d;
  d.s = __fdiv_rn(absmax, kE4M3Max);  // s = fl32(absmax / 448)
  d.fast = d.s >= kMinFastScale;      // false for s == 0
  d.y = __frcp_rn(d.fast ? d.s : 1.0f);
  return d;
}

// Table-driven divisor.  For a normal BF16 absmax a = (1 + f/128) * 2^e the
// scale is s = fl32(a / 448) = fl32((1 + f/128) / 448) * 2^e exactly, and
// RN(1/s) scales by 2^-e in the same way (scaling by a power of two
// commutes with rounding while everything stays normal).  So the 128
// values fl32((1 + f/128) / 448) and their reciprocals are computed once
// per block with the IEEE intrinsics and the per-group work is an exponent
// add.  Absmax values outside the range where s >= 2^-93 and 1/s is normal
// take make_divisor.
struct DivTable {
  uint32_t s[128];  // bits of fl32((1 + f/128) / 448)
  uint32_t y[128];  // bits of RN(1 / s)
};

__device__ __forceinline__ void div_table_init(DivTable& t) {
  for (int f = threadIdx.x; f < 128; f += blockDim.x) {
    const float sf = __fdiv_rn(1.0f + static_cast<float>(f) * (1.0f / 128.0f), kE4M3Max);
    t.s[f] = __float_as_uint(sf);
    t.y[f] = __float_as_uint(__frcp_rn(sf));
  }
}

// absmax given as BF16 bits (non-negative).
__device__ __forceinline__ Divisor table_divisor(const DivTable& t, uint32_t a16) {
  const uint32_t e = a16 >> 7;  // biased exponent of the absmax
  // biased exponents 43..254 give s >= 2^-93 with a normal reciprocal
  if (e < 43 || e > 254) return make_divisor(__uint_as_float(a16 << 16));
  const uint32_t f = a16 & 0x7Fu;
  const int sh = static_cast<int>(e) - 127;
  Divisor d;
  d.s = __uint_as_float(t.s[f] + (static_cast<uint32_t>(sh) << 23));
  d.y = __uint_as_float(t.y[f] - (static_cast<uint32_t>(sh) << 23));
  d.fast = true;
  return d;
}

// Power-of-two ("rounded") scale, §3.3.3 "low-precision activations" (1):
// s = 2^k, the smallest power of two with absmax / s <= 448, k >= -149 (the
// smallest positive float32).  y = 2^-k is then exact and so is x * y (the
// correction term vanishes); the same s >= 2^-93 bound as for any divisor
// selects the fast path.
__device__ __forceinline__ Divisor pow2_from_exp(int k) {
  k = max(k, -149);
  Divisor d;
  d.s = k >= -126 ? __uint_as_float(static_cast<uint32_t>(k + 127) << 23) : __uint_as_float(1u << (k + 149));
  d.fast = k >= -93 && k <= 126;
  d.y = d.fast ? __uint_as_float(static_cast<uint32_t>(127 - k) << 23) : 1.0f;
  return d;
}

// absmax a = m * 2^e with m in [1, 2): a / 448 = (m / 1.75) * 2^(e - 8) and
// m / 1.75 lies in (0.5, 1.143), so k = e - 8, plus 1 when m > 1.75.
__device__ __forceinline__ Divisor pow2_divisor_f32(float a) {
  if (!(a > 0.0f)) {
    Divisor d;
    d.s = 0.0f;
    d.y = 1.0f;
    d.fast = false;
    return d;
  }
  uint32_t b = __float_as_uint(a);
  int bias = 0;
  if ((b >> 23) == 0) {  // subnormal: scale up by 2^64 (exact) and take it back from the exponent
    b = __float_as_uint(a * 18446744073709551616.0f);
    bias = 64;
  }
  const int e = static_cast<int>(b >> 23) - 127 - bias;
  return pow2_from_exp(e - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}

// The same from BF16 absmax bits (1.75 = 1 + 96/128 in BF16's 7-bit fraction).
__device__ __forceinline__ Divisor pow2_divisor_bits(uint32_t a16) {
  const uint32_t e = a16 >> 7;
  if (e == 0) return pow2_divisor_f32(__uint_as_float(a16 << 16));
  return pow2_from_exp(static_cast<int>(e) - 127 - 8 + ((a16 & 0x7Fu) > 96u ? 1 : 0));
}

// Divisor of a group from its BF16 absmax bits, in the requested scale mode.
__device__ __forceinline__ Divisor group_divisor(const DivTable& t, uint32_t a16, bool pow2) {
  return pow2 ? pow2_divisor_bits(a16) : table_divisor(t, a16);
}

// Largest |x| of BF16 values: for non-negative floats the integer order of
// the bit patterns is the numeric order, so the magnitudes are compared as
// unsigned 16-bit pairs (two per instruction).
__device__ __forceinline__ uint32_t umax16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// |x| maxima of the two halves of a packed BF16 pair, in both halves.
__device__ __forceinline__ uint32_t umax_halves(uint32_t m) { return umax16x2(m, __byte_perm(m, 0u, 0x1032)); }

// Running |x| maximum of BF16 pairs, one instruction per word: the
// magnitude of max.xorsign.abs is max(|a|, |b|); its sign bit is junk that
// abs_bits clears once at the end.
__device__ __forceinline__ uint32_t absmax_step(uint32_t m, uint32_t w) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
  return d;
}

__device__ __forceinline__ uint32_t abs_bits(uint32_t m) { return m & 0x7FFF7FFFu; }

__device__ __forceinline__ uint32_t absmax8_bits(uint4 v) {
  return abs_bits(absmax_step(absmax_step(v.x, v.y), absmax_step(v.z, v.w)));
}

// Codes of the BF16 pair w (low half first) in bits 0..15, by the
// Markstein quotient (see Divisor); ns2 = (-s, -s), y2 = (y, y).  The sign of
// a -0 input is restored by the caller (signs4).
__device__ __forceinline__ uint32_t quant_pair(uint32_t w, float2 y2, float2 ns2) {
  const float2 a = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  const float2 q0 = __fmul2_rn(a, y2);
  const float2 r = __ffma2_rn(q0, ns2, a);
  const float2 q1 = __ffma2_rn(r, y2, q0);
  return e4m3x2(q1.x, q1.y);
}

// Sign bits of the four BF16 values in words w0, w1 at bit 7 of the code
// bytes they map to (byte i = value i).
__device__ __forceinline__ uint32_t signs4(uint32_t w0, uint32_t w1) {
  return __byte_perm(w0, w1, 0x7531) & 0x80808080u;
}

// Codes of one value pair through IEEE divisions (x / s, then E4M3, sign
// from the quotient): groups whose scale is below 2^-93 or zero.
__device__ __forceinline__ uint32_t quant2_exact(uint32_t w, float s) {
  if (s == 0.0f) return 0u;
  return e4m3x2(__fdiv_rn(__uint_as_float(w << 16), s), __fdiv_rn(__uint_as_float(w & 0xFFFF0000u), s));
}

// The BF16 pair w (low half first) widened to float32 and negated: -x is
// what quot_pair_nx takes.
__device__ __forceinline__ float2 neg_widen(uint32_t w) {
  return make_float2(__uint_as_float((w << 16) ^ 0x80000000u), __uint_as_float((w & 0xFFFF0000u) ^ 0x80000000u));
}

// Quotients x / s of a value pair given as nx = -x, with a divisor per half:
// s2 the scales, ny2 = -RN(1/s).  The same Markstein quotient as quant_pair
// with the signs moved: q0 = RN(nx * ny), r = RN(s q0 + nx) = -(x - s q0)
// (exact), q1 = RN(q0 + r * ny).  In this form a zero input keeps its sign
// (x = -0: q0 = -0, r = +0, q1 = -0 + -0 = -0), so no sign restoration
// follows; every other input gives the same q1 as quant_pair.
__device__ __forceinline__ float2 quot_pair_nx(float2 nx, float2 ny2, float2 s2) {
  const float2 q0 = __fmul2_rn(nx, ny2);
  const float2 r = __ffma2_rn(q0, s2, nx);
  return __ffma2_rn(r, ny2, q0);
}

// Quotients of the BF16 pair w through IEEE divisions, a scale per half (a
// zero scale gives +0, hence a zero code).
__device__ __forceinline__ float2 quot2_exact(uint32_t w, float s0, float s1) {
  return make_float2(s0 == 0.0f ? 0.0f : __fdiv_rn(__uint_as_float(w << 16), s0),
                     s1 == 0.0f ? 0.0f : __fdiv_rn(__uint_as_float(w & 0xFFFF0000u), s1));
}

// Four float32 -> four E4M3 codes (RNE, saturating) packed in one word, a
// in the low byte: two conversions written into the two halves of the word.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n}\n"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Eight consecutive values of one group -> eight codes (byte i = value i).
__device__ __forceinline__ uint2 quant8m(uint4 v, const Divisor& d) {
  if (!d.fast)
    return make_uint2(quant2_exact(v.x, d.s) | (quant2_exact(v.y, d.s) << 16),
                      quant2_exact(v.z, d.s) | (quant2_exact(v.w, d.s) << 16));
  const float2 y2 = make_float2(d.y, d.y), ns2 = make_float2(-d.s, -d.s);
  const uint32_t c0 = quant_pair(v.x, y2, ns2), c1 = quant_pair(v.y, y2, ns2);
  const uint32_t c2 = quant_pair(v.z, y2, ns2), c3 = quant_pair(v.w, y2, ns2);
  return make_uint2(__byte_perm(c0, c1, 0x5410) | signs4(v.x, v.y), __byte_perm(c2, c3, 0x5410) | signs4(v.z, v.w));
}

// Word k (0..3) of a 16-byte vector.
__device__ __forceinline__ uint32_t word_of(const uint4& v, int k) {
  return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
}

}  // namespace
}  // namespace fp8bs
