// 4-bit quantisers and the dequantiser (E2M1 codes with block scales along
// K), the operands of the 4-bit GEMMs (gemm_fp4.cu).
//
//   FP8BS_FP4_E4M3X16:   g = max(fl(rowmax / 2688), 2^-100)
//                        s = E4M3(fl(amax_16 / fl(6 g)))
//                        code = E2M1(fl(x * fl(1 / fl(s g)))), 0 where s = 0
//   FP8BS_FP4_UE8M0X32:  s = 2^k, the smallest with amax_32 / s <= 6,
//                        -127 <= k;  code = E2M1(x / s) (exact quotient)
//
// 2688 = 6 * 448: the row's largest element meets the largest code of the
// largest block scale.  The float32 scale of a row keeps E4M3 block scales
// (2^-9 .. 448) in range whatever the row's magnitude, and is found in the
// same pass as the codes, so no earlier pass over the tensor is needed.
//
// All memory-bound streams: a row is read once into registers (16 elements,
// a "unit", per thread and step; rows longer than the registers hold are read
// twice, from L2 the second time), its maximum is reduced across the row's
// warps, and codes and scales leave with 8-byte and 4-byte stores.  [16384][7168]
// in 48.4 us with E4M3 scales (301 MB, 0.92 of the copy bandwidth) and 42.6 with
// UE8M0 ones (1.0); the SwiGLU form is bound by instructions (27 an element, 11 of
// them the plain rows', the rest scalar: expf and the corrected quotient):
// [8191][2048] in 18.3 us, 0.62 of the copy bandwidth.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace fp8bs {
namespace {

constexpr int kUnit = 16;          // elements per thread and step
constexpr int kUnitsPerThread = 2; // steps whose elements stay in registers
constexpr int kQuantThreads = 256; // of the dequantiser
constexpr float kMinRowScale = 7.888609052210118e-31f;  // 2^-100: s * g and its reciprocal stay normal

enum Fp4Source { kRows = 0, kSwiglu = 1 };

struct Fp4QuantParams {
  const uint16_t* x;      // [rows_in][ldx] BF16 (SwiGLU: gate | up)
  const int32_t* rows;    // optional: source row of each output row (SwiGLU: liveness), < 0 a zero row
  int64_t rows_in, ldx, M, K;
  uint8_t* q;             // [M][K / 2]
  uint8_t* sf;            // blocked scales
  float* g;               // [M] (E4M3x16)
};

// Byte offset of the scale word (groups 4w .. 4w+3) of a row in the blocked
// layout: 512-byte blocks of 128 rows x 4 groups, row r at 16 (r % 32) +
// 4 ((r / 32) % 4), the layout tcgen05.cp.32x128b copies into tensor memory.
__device__ __forceinline__ int64_t sf_word_offset(int64_t row, int64_t word, int64_t words) {
  return ((row >> 7) * words + word) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// silu(gate) * up of two BF16 pairs, rounded to BF16: gate / (1 + e^-gate)
// with expf and the IEEE quotient; below -64 (kLow), where 1 adds nothing to
// e^-gate and e^-gate overflows in the end, gate e^(gate/2) e^(gate/2).
// The quotient is Markstein's correction of gate * rcp(1 + e^-gate) on negated
// operands, which keep the sign of a zero; for every finite BF16 gate from -64
// up the result is the IEEE division's (tests/test_fp4_paths_gpu.py goes through
// them).
template <bool kLow>
__device__ __forceinline__ uint32_t swiglu_pair(uint32_t gate, uint32_t up) {
  float v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = __uint_as_float(i == 0 ? gate << 16 : gate & 0xFFFF0000u);
    const float b = __uint_as_float(i == 0 ? up << 16 : up & 0xFFFF0000u);
    if (kLow && a < -64.0f) {
      const float e = expf(0.5f * a);
      v[i] = a * e * e * b;
    } else {
      const float d = 1.0f + expf(-a);
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
      const float q = -a * -r;
      v[i] = fmaf(fmaf(d, q, -a), -r, q) * b;
    }
  }
  const __nv_bfloat162 r = __floats2bfloat162_rn(v[0], v[1]);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int kSrc>
__device__ __forceinline__ void load_unit(const uint16_t* row, int64_t K, int64_t unit, uint32_t (&v)[8]) {
  const uint4* p = reinterpret_cast<const uint4*>(row + unit * kUnit);
  const uint4 a = __ldg(p), b = __ldg(p + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  if (kSrc == kSwiglu) {
    const uint4* u = reinterpret_cast<const uint4*>(row + K + unit * kUnit);
    const uint4 c = __ldg(u), d = __ldg(u + 1);
    const uint32_t w[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
    uint32_t low = v[0];   // BF16 below -64: bits above 0xC280
#pragma unroll
    for (int i = 1; i < 8; ++i) low = __vmaxu2(low, v[i]);
    if ((low >> 16) > 0xC280u || (low & 0xFFFFu) > 0xC280u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = swiglu_pair<true>(v[i], w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = swiglu_pair<false>(v[i], w[i]);
    }
  }
}

// Largest magnitude of a unit, as the upper half of a float32 (BF16 bits).
__device__ __forceinline__ uint32_t unit_absmax(const uint32_t (&v)[8]) {
  uint32_t m = v[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}

// Two products in one instruction, each rounded as a float32 product.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Eight values times r to eight codes, element 0 in the lowest four bits.
__device__ __forceinline__ uint32_t codes8(const uint32_t* v, float r) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 m =
        mul2(make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u)), make_float2(r, r));
    f[2 * i] = m.x;
    f[2 * i + 1] = m.y;
  }
  uint32_t c;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(c)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return c;
}

__device__ __forceinline__ uint32_t e4m3_of(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  float f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n}\n" : "=f"(f) : "r"(h));
  return f;
}

// Scale byte and reciprocal of a group with largest magnitude `amax`; b = 6 g
// and y = 1 / b of its row.  amax / b is Markstein's corrected quotient (IBM J.
// Res. Develop. 34(1), 1990): from a correctly rounded y one correction gives
// the IEEE quotient wherever the remainder is exact, which holds for every
// quotient above 2^-10, half the smallest scale (tests/test_fp4_paths_gpu.py
// goes through all BF16 mantissas of amax and of the row's maximum, up to 26
// binades apart).
template <int kFmt>
__device__ __forceinline__ uint32_t group_scale(float amax, float g, float b, float y, float& r) {
  if (kFmt == 0) {
    const float q = amax * y;
    const uint32_t s = e4m3_of(fmaf(fmaf(-q, b, amax), y, q));
    const float d = e4m3_value(s) * g;
    r = d > 0.0f ? __frcp_rn(d) : 0.0f;
    return s;
  }
  // amax = 1.m x 2^e: 2^(e-2) reaches 6 x 2^(e-2) = 1.5 x 2^e, so one more where
  // the mantissa is above 1.5.  BF16 subnormals (e < -126) come out at k = -127.
  const uint32_t bits = __float_as_uint(amax);
  const int k = static_cast<int>(bits >> 23) - 129 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  const uint32_t byte = static_cast<uint32_t>(max(k, -127) + 127);
  r = __uint_as_float((254u - byte) << 23);   // 2^-k, normal for every k in [-127, 126]
  return byte;
}

// Rows of a CTA: short rows share one (a power of two of them, so that the
// CTAs cover the scale rows up to a multiple of 128 exactly).
constexpr int rows_per_cta(int row_warps) { return row_warps == 1 ? 8 : row_warps == 2 ? 4 : row_warps <= 4 ? 2 : 1; }

// One row per kWarps warps.  kBig: rows longer than the units a thread keeps.
// (kWarps known to the compiler: 40 registers a thread instead of 47, and
// [16384][7168] in 49 us instead of 57.)
template <int kFmt, int kSrc, int kWarps, bool kBig>
__global__ void __launch_bounds__(kWarps * rows_per_cta(kWarps) * 32) fp4_quant_kernel(const Fp4QuantParams p) {
  constexpr int kRows = rows_per_cta(kWarps);
  __shared__ uint32_t s_max[kWarps * kRows];
  griddep_launch_dependents();  // a GEMM launched behind this kernel may start its set-up
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int row_in_cta = warp / kWarps;
  constexpr int kRowThreads = kWarps * 32;
  const int t = threadIdx.x % kRowThreads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + row_in_cta;
  const int64_t units = p.K / kUnit;
  const int64_t words = kFmt == 0 ? units / 4 : (units + 7) / 8;
  int64_t src = row;
  bool live = row < p.M;
  if (live && p.rows != nullptr) {
    const int32_t r = p.rows[row];
    live = r >= 0 && (kSrc == kSwiglu || r < p.rows_in);
    if (kSrc != kSwiglu) src = r;
  }
  const uint16_t* xr = p.x + (live ? src * p.ldx : 0);

  uint32_t v[kUnitsPerThread][8];
  uint32_t am[kUnitsPerThread];
  uint32_t rowmax = 0;
  const int steps = kBig ? static_cast<int>((units + kRowThreads - 1) / kRowThreads) : kUnitsPerThread;
  auto load = [&](int i, uint32_t (&w)[8]) {
    const int64_t u = t + static_cast<int64_t>(i) * kRowThreads;
    if (live && u < units) {
      load_unit<kSrc>(xr, p.K, u, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 0u;
    }
  };
  if (!kBig) {
#pragma unroll
    for (int i = 0; i < kUnitsPerThread; ++i) load(i, v[i]);
#pragma unroll
    for (int i = 0; i < kUnitsPerThread; ++i) {
      am[i] = unit_absmax(v[i]);
      rowmax = max(rowmax, am[i]);
    }
  } else if (kFmt == 0) {
    for (int i = 0; i < steps; ++i) {
      load(i, v[0]);
      rowmax = max(rowmax, unit_absmax(v[0]));
    }
  }
  float g = 0.0f, b = 0.0f, y = 0.0f;
  if (kFmt == 0) {
    rowmax = __reduce_max_sync(0xffffffffu, rowmax);
    if (kWarps > 1) {
      if (lane == 0) s_max[warp] = rowmax;
      __syncthreads();
      rowmax = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) rowmax = max(rowmax, s_max[row_in_cta * kWarps + w]);
    }
    g = fmaxf(__uint_as_float(rowmax << 16) / 2688.0f, kMinRowScale);
    b = g * 6.0f;
    y = __frcp_rn(b);
    if (t == 0 && row < p.M) p.g[row] = g;
  }
  auto emit = [&](int i, const uint32_t (&w)[8], uint32_t amax) {
    const int64_t u = t + static_cast<int64_t>(i) * kRowThreads;
    if (kFmt == 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // two units per group
    float r;
    const uint32_t s = group_scale<kFmt>(__uint_as_float(amax << 16), g, b, y, r);
    uint32_t word;
    if (kFmt == 0) {
      word = s << (8 * (lane & 3));
    } else {
      word = u < units ? s << (8 * ((lane >> 1) & 3)) : 0u;   // a last word of two groups ends in zeros
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
    }
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if (u >= units) return;
    if (row >= p.M) word = 0u;  // scale rows up to a multiple of 128
    if (kFmt == 0) {
      if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(p.sf + sf_word_offset(row, u >> 2, words)) = word;
    } else {
      if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(p.sf + sf_word_offset(row, u >> 3, words)) = word;
    }
    if (row < p.M)
      *reinterpret_cast<uint2*>(p.q + row * (p.K / 2) + u * (kUnit / 2)) = make_uint2(codes8(w, r), codes8(w + 4, r));
  };
  if (!kBig) {
#pragma unroll
    for (int i = 0; i < kUnitsPerThread; ++i) emit(i, v[i], am[i]);
  } else {
    for (int i = 0; i < steps; ++i) {
      load(i, v[0]);
      emit(i, v[0], unit_absmax(v[0]));
    }
  }
}

// value = code * s (* g): the first product is exact (six significant bits),
// the second rounds once, BF16 output once more.  A lane turns 4 bytes of
// codes into 8 consecutive values, so a warp writes 512 (BF16) or 1024
// consecutive bytes; kPieces such pieces of a row are in flight per warp.
// [16384][7168] in 45.7 us, 0.97 of the copy bandwidth (16 elements a lane, 32
// bytes written in two halves: 63 us and 2.7 times the L2 sectors that the bytes
// make).
constexpr int kPieces = 4;
constexpr int kPieceK = 256;   // elements of a row that a warp takes at once

template <int kFmt, bool kBf16>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sf, const float* __restrict__ g,
                       int64_t M, int64_t K, void* __restrict__ out, int64_t ldo, uint32_t segs) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t words = kFmt == 0 ? K / 64 : (K + 127) / 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // warps over the segments of kPieces pieces, row by row; fewer than 2^32 (their bytes fit the memory)
  const uint32_t id = blockIdx.x * (kQuantThreads / 32) + warp;
  const uint32_t row32 = id / segs;
  const int64_t row = row32;
  if (row >= M) return;
  const int64_t k0 = static_cast<int64_t>(id - row32 * segs) * (kPieceK * kPieces);
  const float gr = kFmt == 0 ? __ldg(g + row) : 1.0f;
  const uint8_t* sf_row = sf + sf_word_offset(row, 0, words);
  uint32_t c[kPieces], sb[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int64_t k = k0 + i * kPieceK + 8 * lane;
    if (k < K) {
      c[i] = __ldg(reinterpret_cast<const uint32_t*>(q + row * (K / 2) + k / 2));
      sb[i] = kFmt == 0 ? __ldg(sf_row + (k >> 6) * 512 + ((k >> 4) & 3)) : __ldg(sf_row + (k >> 7) * 512 + ((k >> 5) & 3));
    }
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int64_t k = k0 + i * kPieceK + 8 * lane;
    if (k >= K) break;
    uint32_t h[4];   // pairs of values in FP16, exact
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c[i]));
    float2 f[4];
    if (kFmt == 0) {
      uint32_t s2;   // the scale twice
      asm("{\n\t.reg .b16 t;\n\tmov.b16 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n}\n"
          : "=r"(s2)
          : "h"(static_cast<uint16_t>(sb[i] * 0x101u)));
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // code * s: at most 2688 and a multiple of 2^-10, exact in FP16
        const __half2 m = __hmul2(*reinterpret_cast<const __half2*>(&h[j]), *reinterpret_cast<const __half2*>(&s2));
        f[j] = mul2(__half22float2(m), make_float2(gr, gr));
      }
    } else {
      const float s = __uint_as_float(sb[i] == 0u ? 0x00400000u : sb[i] << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = mul2(__half22float2(*reinterpret_cast<const __half2*>(&h[j])), make_float2(s, s));
    }
    if (kBf16) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 v = __float22bfloat162_rn(f[j]);
        w[j] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * ldo + k) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * ldo + k);
      o[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      o[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
  }
}

template <int kFmt, int kSrc, int kWarps, bool kBig>
cudaError_t run_quant(const Fp4QuantParams& p, cudaStream_t stream) {
  constexpr int kRows = rows_per_cta(kWarps);
  const unsigned ctas = static_cast<unsigned>((p.M + 127) / 128 * (128 / kRows));
  return launch_behind(fp4_quant_kernel<kFmt, kSrc, kWarps, kBig>, ctas, kRows * kWarps * 32, stream, p);
}

template <int kFmt, int kSrc>
cudaError_t pick_quant(const Fp4QuantParams& p, cudaStream_t stream) {
  // the fewest warps that hold a row in registers
  constexpr int64_t kPerWarp = 32 * kUnit * kUnitsPerThread;
  if (p.K > 16 * kPerWarp) return run_quant<kFmt, kSrc, 16, true>(p, stream);
  switch ((p.K + kPerWarp - 1) / kPerWarp) {
    case 1: return run_quant<kFmt, kSrc, 1, false>(p, stream);
    case 2: return run_quant<kFmt, kSrc, 2, false>(p, stream);
    case 3: return run_quant<kFmt, kSrc, 3, false>(p, stream);
    case 4: return run_quant<kFmt, kSrc, 4, false>(p, stream);
    case 5: return run_quant<kFmt, kSrc, 5, false>(p, stream);
    case 6: return run_quant<kFmt, kSrc, 6, false>(p, stream);
    case 7: return run_quant<kFmt, kSrc, 7, false>(p, stream);
    case 8: return run_quant<kFmt, kSrc, 8, false>(p, stream);
    default: return run_quant<kFmt, kSrc, 16, false>(p, stream);
  }
}

}  // namespace

cudaError_t launch_quantize_fp4(const uint16_t* x, int64_t rows_in, int64_t K, int64_t ldx, const int32_t* rows,
                                int64_t M, int fmt, bool swiglu, uint8_t* q, uint8_t* sf, float* g,
                                cudaStream_t stream) {
  Fp4QuantParams p;
  p.x = x; p.rows = rows; p.rows_in = rows_in; p.ldx = ldx; p.M = M; p.K = K;
  p.q = q; p.sf = sf; p.g = g;
  if (fmt == 0)
    return swiglu ? pick_quant<0, kSwiglu>(p, stream) : pick_quant<0, kRows>(p, stream);
  return swiglu ? pick_quant<1, kSwiglu>(p, stream) : pick_quant<1, kRows>(p, stream);
}

cudaError_t launch_dequantize_fp4(const uint8_t* q, const uint8_t* sf, const float* g, int64_t M, int64_t K, int fmt,
                                  void* out, bool out_bf16, int64_t ldo, cudaStream_t stream) {
  const uint32_t segs = static_cast<uint32_t>((K + kPieceK * kPieces - 1) / (kPieceK * kPieces));
  const unsigned grid = static_cast<unsigned>((M * segs + kQuantThreads / 32 - 1) / (kQuantThreads / 32));
  const auto kern = fmt == 0 ? (out_bf16 ? fp4_dequant_kernel<0, true> : fp4_dequant_kernel<0, false>)
                             : (out_bf16 ? fp4_dequant_kernel<1, true> : fp4_dequant_kernel<1, false>);
  return launch_behind(kern, grid, kQuantThreads, stream, q, sf, g, M, K, out, ldo, segs);
}

}  // namespace fp8bs
