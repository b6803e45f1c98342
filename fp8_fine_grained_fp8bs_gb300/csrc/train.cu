// Operators of a training step around the 8-bit products: the root-mean-square
// norm with the residual's addition and 8-bit output, its gradient, the
// gradient of the MoE combine (the experts' output gradients in their
// segments, quantised, and the gate weights' gradient), and the gradient of
// the SwiGLU with 8-bit output.
//
// What is quantised is the BF16 value that the unfused operator would store,
// so codes and scales are those of fp8bs_quantize_act_ex on it (one rounding
// to BF16, then the quantiser's).  Statistics and sums are float32.  All are
// streams bound by memory, or next to it by instructions, that read each input
// once from it: the norms' rows through a ring of bulk copies in shared memory,
// the others straight into registers.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "group_quant.cuh"
#include "kernels.h"
#include "launch.h"
#include "tmap.h"

namespace fp8bs {
namespace {

__device__ int g_train_status;

// Eight BF16 values in packed float32 pairs, and such values rounded to BF16 (nearest,
// ties to even).
__device__ __forceinline__ void widen8x2(const uint4& v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 round8x2(const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Table of absmax divisors, for kernels whose CTAs quantise many groups.
template <bool kPow2>
struct Divisors {
  DivTable table;
  __device__ __forceinline__ void init() { div_table_init(table); }   // a barrier follows before use
  __device__ __forceinline__ Divisor of(uint32_t a16) const { return table_divisor(table, a16); }
};
template <>
struct Divisors<true> {
  __device__ __forceinline__ void init() {}
  __device__ __forceinline__ Divisor of(uint32_t a16) const { return pow2_divisor_bits(a16); }
};

// Eight BF16 values of a group with maximum a16 (BF16 bits) -> eight codes; the
// scale.  A power of two: with e the biased exponent of the smallest power of two
// times 1.75 that is at least the maximum (31 carries where the 7 bits of its
// fraction exceed 96, those of 1.75), s = 2^(e - 135).  The quotient is then one
// exact product, which keeps the sign of a zero.  Groups whose scale or its
// reciprocal is not a normal number, zeros among them, take the general way, and so
// do maxima above 1.75 * 2^127: an infinity among the values has the code of no number
// there, where a product with the conversion's saturation would make 448 of it.  One
// unsigned compare finds both ends.
template <bool kPow2>
__device__ __forceinline__ float quantise8(const uint4& v, uint32_t a16, const Divisors<kPow2>& divisors, uint2& codes) {
  if (kPow2) {
    const uint32_t a = a16 + 31u - (9u << 7);
    if (a < (255u - 9u) << 7) {
      const uint32_t e = (a >> 7) + 9u;
      const float y = __uint_as_float((262u - e) << 23);
      const float2 y2 = make_float2(y, y);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = __fmul2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), y2);
      codes = make_uint2(e4m3x4(f[0].x, f[0].y, f[1].x, f[1].y), e4m3x4(f[2].x, f[2].y, f[3].x, f[3].y));
      return __uint_as_float((e - 8u) << 23);
    }
  }
  const Divisor d = divisors.of(a16);
  codes = quant8m(v, d);
  return d.s;
}

// Eight float32 values times w, rounded to BF16.
__device__ __forceinline__ uint4 times8(const float2 (&a)[4], float w) {
  const float2 w2 = make_float2(w, w);
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(a[i], w2);
  return round8x2(f);
}

// quantise8 of the BF16 values of a * w.  Scaling by a power of two commutes with
// rounding: the quotients are the BF16 values of a * (w / s), as long as those that
// reach a code (|v / s| > 2^-10) are normal numbers, which s >= 2^-103 leaves them,
// w / s stays in range, which |w| < 2^24 does then, and no BF16 value of a * w is
// infinite, since a * (w / s) would not be.
constexpr float kPlainWeight = 16777216.0f;
template <bool kPow2>
__device__ __forceinline__ float quantise8_times(const float2 (&a)[4], float w, uint32_t a16, const Divisors<kPow2>& divisors,
                                                 uint2& codes) {
  if (kPow2) {
    const uint32_t b = a16 + 31u - (32u << 7);
    if (b < (255u - 32u) << 7 && fabsf(w) < kPlainWeight) {
      const uint32_t e = (b >> 7) + 32u;
      float2 f[4];
      widen8x2(times8(a, w * __uint_as_float((262u - e) << 23)), f);
      codes = make_uint2(e4m3x4(f[0].x, f[0].y, f[1].x, f[1].y), e4m3x4(f[2].x, f[2].y, f[3].x, f[3].y));
      return __uint_as_float((e - 8u) << 23);
    }
  }
  return quantise8<kPow2>(times8(a, w), a16, divisors, codes);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum of up to 16 warps' values, by every thread, in a fixed order.
__device__ __forceinline__ float sum_of_warps(const float* part, int warps) {
  const int lane = threadIdx.x & 31;
  float v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o, 16);
  return __shfl_sync(0xffffffffu, v, 0);
}

// A row is held by `warps` warps, kVecs 16-byte pieces a thread; short rows
// share a CTA.  Sums of a row: lanes, then warps, in a fixed order.
constexpr int kNormMaxThreads = 512;
constexpr int kMaxNormK = 16384;   // 512 threads x 4 pieces x 8 values

struct RowPlace {
  int warps;   // warps per row
  int rows;    // rows per CTA
  int vecs;    // pieces per thread
};
inline RowPlace place_rows(int K, int four_from) {   // four pieces a thread from that many pieces a row on
  RowPlace p;
  const int nv = (K + 7) / 8;
  p.vecs = nv > four_from ? 4 : nv > 64 ? 2 : 1;
  p.warps = (nv + 32 * p.vecs - 1) / (32 * p.vecs);
  p.rows = std::max(1, 8 / p.warps);
  return p;
}

constexpr int kNormFour = 1024;   // pieces a row from which a thread of the norm takes four
constexpr int kNormWarps = 32;    // of the norm, per SM
constexpr int kNormStages = 2;    // of the norm's ring, see norm_kernel
constexpr int kRingMaxStages = 4;
constexpr int kRingBytes = 112 * 1024;       // of a CTA, two to an SM
constexpr int kRingMaxBytes = 224 * 1024;    // of a CTA that has an SM for itself

// Eight gains of a thread's columns, kept as they are stored.
template <bool kF32>
struct Gain;
template <>
struct Gain<false> {
  uint4 w;
  __device__ __forceinline__ void load(const void* gain, int c, bool here) {
    w = make_uint4(0u, 0u, 0u, 0u);
    if (here) w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(gain) + c));
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const { widen8x2(w, f); }
};
template <>
struct Gain<true> {
  float2 v[4];
  __device__ __forceinline__ void load(const void* gain, int c, bool here) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(gain) + c);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float4 a = here ? __ldg(p) : zero, b = here ? __ldg(p + 1) : zero;
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  }
};

// The ring of a CTA: step i is the CTA's rows (i * CTAs + CTA) * rows and on, of up to
// three matrices, copied row by row into stage i % stages, one lane of warp 0 per row
// and matrix (kMany: they may be more than 32).  Steps are issued in order and taken in
// order.
template <bool kMany>
struct RowRing {
  uint8_t* base;
  uint64_t* full;
  int64_t M, step_rows;
  int rows, arrays, stages, steps;
  uint32_t row_bytes, array_bytes, stage_bytes;
  // the step to issue next (warp 0) and the one taken last
  int issued, in;
  int64_t in_row;
  int out;
  uint32_t out_phase;
  __device__ __forceinline__ RowRing(uint8_t* ring, uint64_t* bars, int K, int rows_, int arrays_, int stages_, int64_t M_)
      : base(ring), full(bars), M(M_), rows(rows_), arrays(arrays_), stages(stages_) {
    row_bytes = 2u * static_cast<uint32_t>(K);
    array_bytes = rows * row_bytes;
    stage_bytes = arrays * array_bytes;
    step_rows = static_cast<int64_t>(gridDim.x) * rows;
    issued = in = 0;
    in_row = static_cast<int64_t>(blockIdx.x) * rows;
    steps = static_cast<int>((M - in_row + step_rows - 1) / step_rows);
    out = stages - 1;
    out_phase = 1;
  }
  __device__ __forceinline__ void init() const {
    if (threadIdx.x == 0) {
      for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
      fence_barrier_init();
    }
    __syncthreads();
  }
  __device__ __forceinline__ void issue(const uint16_t* const (&src)[3], const int64_t (&ld)[3]) {
    if (threadIdx.x >= 32 || issued == steps) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(rows), M - in_row));
    const int lane = threadIdx.x;
    if (lane == 0) mbar_arrive_expect_tx(&full[in], arrays * n * row_bytes);
    __syncwarp();
    for (int at = lane; at < arrays * n; at += 32) {
      const int which = at >= 2 * n ? 2 : at >= n ? 1 : 0, i = at - which * n;
      const uint16_t* from = which == 0 ? src[0] + (in_row + i) * ld[0] : which == 1 ? src[1] + (in_row + i) * ld[1] : src[2] + (in_row + i) * ld[2];
      bulk_load(base + in * stage_bytes + which * array_bytes + i * row_bytes, from, row_bytes, &full[in]);
      if (!kMany) break;
    }
    __syncwarp();
    ++issued;
    in_row += step_rows;
    if (++in == stages) in = 0;
  }
  // Waits for the next step; its stage is stage().
  __device__ __forceinline__ bool take(uint64_t timeout_ns) {
    if (++out == stages) {
      out = 0;
      out_phase ^= 1u;
    }
    return mbar_wait(&full[out], out_phase, timeout_ns);
  }
  __device__ __forceinline__ const uint8_t* stage() const { return base + out * stage_bytes; }
  // After the wait for step `from` ran out: what is issued lands before the CTA may leave.
  __device__ __forceinline__ void drain(int from, uint64_t timeout_ns) const {
    if (threadIdx.x >= 32) return;
    for (int step = from; step < issued; ++step) (void)mbar_wait(&full[step % stages], (step / stages) & 1, timeout_ns);
  }
};

// ------------------------------------------------------------------- norm
struct NormParams {
  const uint16_t* x;
  const uint16_t* res;   // or NULL
  const void* gain;
  int64_t M, ldx, ldr;
  int K, warps, stages;
  float eps, inv_k;
  uint16_t* r;           // or NULL
  uint16_t* y;           // or NULL
  uint8_t* q;            // or NULL (with s)
  float* s;
  float* rstd;           // or NULL
  uint64_t timeout_ns;
};

// A CTA's rows come by bulk copies into a ring of stages that the next rows fill
// while one is worked on; the sum of x and the residual then stays in registers,
// as the gain does over all rows, and is stored beside the codes.  Two stages, and
// the next copy issued after a row's stores, keep the reads in flight few: with a
// residual it is bound by memory, and [16384][7168] takes 124 us (826 MB, 0.98 of
// the copy bandwidth), with three or four stages 145, with two filled at the
// barrier 139, with the sum stored before the barrier or the maxima of two groups in one
// word 127 to 131.  Without a residual it is bound by instructions, about 170 per
// eight values at 0.7 of the issue slots: 89 us for 355 MB.
template <int kVecs, bool kGainF32, bool kPow2, bool kRes>
__global__ void __launch_bounds__(kNormMaxThreads) norm_kernel(const NormParams p) {
  constexpr int kPair = kVecs == 4 || (kVecs == 2 && !kRes) ? 2 : 1;   // pieces whose maxima share the shuffles
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float s_part[2][kNormMaxThreads / 32];
  __shared__ uint64_t full[kRingMaxStages];
  const int T = 32 * p.warps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x / T, t = threadIdx.x - sub * T;
  const int nv = p.K / 8;
  constexpr int arrays = kRes ? 2 : 1;
  const int rows = blockDim.x / T;
  RowRing<false> rr(ring, full, p.K, rows, arrays, p.stages, p.M);
  const uint16_t* const src[3] = {p.x, p.res, nullptr};
  const int64_t ld[3] = {p.ldx, p.ldr, 0};
  __shared__ Divisors<kPow2> divisors;
  divisors.init();
  rr.init();
  griddep_launch_dependents();
  griddep_wait();
  for (int s = 0; s < p.stages; ++s) rr.issue(src, ld);
  Gain<kGainF32> gain[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = i * T + t;
    gain[i].load(p.gain, 8 * c, c < nv);
  }
  // this thread's place in the row-major outputs, moved on with the rows
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows + sub;
  int64_t at = row * p.K + 8 * t;
  float* ps = p.s + static_cast<int64_t>(t >> 4) * p.M + row;
  const int64_t at_step = rr.step_rows * p.K, s_step = static_cast<int64_t>(T >> 4) * p.M;
  int waited = 0;
  for (int step = 0; step < rr.steps; ++step, row += rr.step_rows, at += at_step, ps += rr.step_rows) {
    const bool live = row < p.M;
    const bool ok = rr.take(p.timeout_ns);
    const uint8_t* stage = rr.stage() + sub * rr.row_bytes;
    uint4 v[kVecs];
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = i * T + t;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (!(ok && live && c < nv)) continue;
      v[i] = *reinterpret_cast<const uint4*>(stage + 16 * c);
      float2 a[4];
      widen8x2(v[i], a);
      if (kRes) {
        float2 b[4];
        widen8x2(*reinterpret_cast<const uint4*>(stage + rr.array_bytes + 16 * c), b);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __fadd2_rn(a[e], b[e]);
        v[i] = round8x2(a);
        widen8x2(v[i], a);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = __ffma2_rn(a[e], a[e], sum);
    }
    const float lanes = warp_sum(sum.x + sum.y);
    const int parity = step & 1;
    if (lane == 0) s_part[parity][warp] = lanes;
    if (!__syncthreads_and(ok)) {
      if (threadIdx.x == 0) atomicCAS(&g_train_status, 0, kStatusTimeout);
      break;
    }
    ++waited;
    // the hardware's reciprocal root (2^-22.9) and one Newton step
    const float m = fmaf(sum_of_warps(&s_part[parity][sub * p.warps], p.warps), p.inv_k, p.eps);
    const float root = rsqrtf(m);
    const float rstd = root * fmaf(-0.5f * m * root, root, 1.5f);
    const float2 rstd2 = make_float2(rstd, rstd);
    if (live && t == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
#pragma unroll
    for (int i0 = 0; i0 < kVecs; i0 += kPair) {
      uint4 y[kPair];
#pragma unroll
      for (int i1 = 0; i1 < kPair; ++i1) {
        const int i = i0 + i1;
        float2 a[4], g[4];
        widen8x2(v[i], a);
        gain[i].get(g);
        // r * gain is exact for a BF16 gain, so y is rounded once before BF16
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __fmul2_rn(__fmul2_rn(a[e], g[e]), rstd2);
        y[i1] = round8x2(a);
        if (live && i * T + t < nv && p.y != nullptr) *reinterpret_cast<uint4*>(p.y + at + 8 * i * T) = y[i1];
      }
      uint32_t top = 0u;
      if (p.q != nullptr) {   // the maxima of two groups in one word
        top = umax_halves(absmax8_bits(y[0]));
        if (kPair == 2) top = __byte_perm(top, umax_halves(absmax8_bits(y[kPair - 1])), 0x5410);
#pragma unroll
        for (int o = 1; o <= 8; o <<= 1) top = umax16x2(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
#pragma unroll
      for (int i1 = 0; i1 < kPair; ++i1) {
        const int i = i0 + i1;
        uint2 codes = make_uint2(0u, 0u);
        float s = 0.0f;
        if (p.q != nullptr) s = quantise8<kPow2>(y[i1], i1 ? top >> 16 : top & 0xFFFFu, divisors, codes);
        if (!(live && i * T + t < nv)) continue;
        if (kRes) *reinterpret_cast<uint4*>(p.r + at + 8 * i * T) = v[i];
        if (p.q != nullptr) {
          *reinterpret_cast<uint2*>(p.q + at + 8 * i * T) = codes;
          if ((lane & 15) == 0) ps[i * s_step] = s;
        }
      }
    }
    rr.issue(src, ld);   // into the stage that was read before the barrier
  }
  if (waited < rr.steps) rr.drain(waited, p.timeout_ns);
}

// ---------------------------------------------------------- norm's gradient
struct NormBackwardParams {
  const uint16_t* dy;
  const uint16_t* r;
  const void* gain;
  const float* rstd;
  const uint16_t* dres;  // or NULL
  int64_t M, lddy, ldr, lddres;
  int K, warps, stages;
  float inv_k;           // 1 / K
  uint16_t* dx;
  float* part;           // [CTAs][K], or NULL: no gain gradient
  uint64_t timeout_ns;
};

// With t = dy gain: dx = rstd t - r rstd^3 mean(t r) + dres.  dy r is exact in
// float32 and serves the mean and the gain's sum, which stays in the thread's
// registers over the CTA's rows.  The rows (dy, r and dres) come by bulk copies
// into a ring of stages that the next rows fill while one is worked on; both
// passes over a row read it from there.  Bound by memory: [16384][7168] with dres
// takes 143 us and the gain's gradient 4 more (940 MB, 0.94 of the copy bandwidth; with
// loads straight into registers 260), [16384][1024] 27.3, [509][1984] 5.9, where the
// two launches' latency counts.
template <int kVecs, bool kGainF32>
__global__ void __launch_bounds__(kNormMaxThreads) norm_backward_kernel(const NormBackwardParams p) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float s_part[2][kNormMaxThreads / 32];
  __shared__ uint64_t full[kRingMaxStages];
  const int T = 32 * p.warps;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x / T, t = threadIdx.x - sub * T;
  const int rows = blockDim.x / T;
  const int nv = p.K / 8;
  const int arrays = p.dres != nullptr ? 3 : 2;
  RowRing<kVecs == 1> rr(ring, full, p.K, rows, arrays, p.stages, p.M);
  const uint16_t* const src[3] = {p.dy, p.r, p.dres};
  const int64_t ld[3] = {p.lddy, p.ldr, p.lddres};
  rr.init();
  griddep_launch_dependents();
  griddep_wait();
  for (int s = 0; s < p.stages; ++s) rr.issue(src, ld);
  float2 acc[kVecs][4];
  Gain<kGainF32> gain[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = i * T + t;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = make_float2(0.0f, 0.0f);
    gain[i].load(p.gain, 8 * c, c < nv);
  }
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows + sub;
  uint16_t* out_row = p.dx + row * p.K + 8 * t;
  const int64_t out_step = rr.step_rows * p.K;
  float rstd_next = row < p.M ? __ldg(p.rstd + row) : 0.0f;
  int waited = 0;
  for (int step = 0; step < rr.steps; ++step, row += rr.step_rows, out_row += out_step) {
    const bool live = row < p.M;
    const float rstd = rstd_next;
    rstd_next = row + rr.step_rows < p.M ? __ldg(p.rstd + row + rr.step_rows) : 0.0f;
    const bool ok = rr.take(p.timeout_ns);
    const uint8_t* stage = rr.stage() + sub * rr.row_bytes;
    float2 sum = make_float2(0.0f, 0.0f);
    const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = i * T + t;
      if (!(ok && live && c < nv)) continue;
      float2 a[4], b[4], g[4];
      gain[i].get(g);
      widen8x2(*reinterpret_cast<const uint4*>(stage + 16 * c), a);
      widen8x2(*reinterpret_cast<const uint4*>(stage + rr.array_bytes + 16 * c), b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 ab = __fmul2_rn(a[e], b[e]);
        sum = __ffma2_rn(ab, g[e], sum);
        acc[i][e] = __ffma2_rn(ab, rstd2, acc[i][e]);
      }
    }
    const float lanes = warp_sum(sum.x + sum.y);
    const int parity = step & 1;
    if (lane == 0) s_part[parity][warp] = lanes;
    if (!__syncthreads_and(ok)) {
      if (threadIdx.x == 0) atomicCAS(&g_train_status, 0, kStatusTimeout);
      break;
    }
    ++waited;
    if (step > 0) rr.issue(src, ld);   // every thread is done with the stage before
    const float total = sum_of_warps(&s_part[parity][sub * p.warps], p.warps);
    const float f = -(rstd * rstd * (rstd * (total * p.inv_k)));
    const float2 f2 = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int c = i * T + t;
      if (!(live && c < nv)) continue;
      float2 a[4], b[4], g[4];
      gain[i].get(g);
      widen8x2(*reinterpret_cast<const uint4*>(stage + 16 * c), a);
      widen8x2(*reinterpret_cast<const uint4*>(stage + rr.array_bytes + 16 * c), b);
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = __ffma2_rn(b[e], f2, __fmul2_rn(__fmul2_rn(a[e], g[e]), rstd2));
      if (arrays == 3) {
        widen8x2(*reinterpret_cast<const uint4*>(stage + 2 * rr.array_bytes + 16 * c), b);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __fadd2_rn(a[e], b[e]);
      }
      *reinterpret_cast<uint4*>(out_row + 8 * i * T) = round8x2(a);
    }
  }
  if (waited < rr.steps) {
    rr.drain(waited, p.timeout_ns);
    return;
  }
  if (p.part == nullptr) return;
  // the CTA's sum over its rows' threads, through the ring where rows share the CTA
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.K;
  float* scratch = reinterpret_cast<float*>(ring);
  if (rows > 1) {
    __syncthreads();
    out = scratch + sub * p.K;
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int c = i * T + t;
    if (c >= nv) continue;
    float4* o = reinterpret_cast<float4*>(out + 8 * c);
    o[0] = make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
    o[1] = make_float4(acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y);
  }
  if (rows == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < p.K; c += blockDim.x) {
    float sum = scratch[c];
    for (int i = 1; i < rows; ++i) sum += scratch[i * p.K + c];
    p.part[static_cast<int64_t>(blockIdx.x) * p.K + c] = sum;
  }
}

// The gain's gradient: the CTAs' partial sums added up, 32 columns a CTA, each group of
// eight lanes every 32nd part, all of its loads in flight, in a fixed order.  Small CTAs
// find room beside those of the gradient and wait there.  304 parts of 7168 columns take
// about 4 us behind it, 255 of 1984 3.1 (in a loop without the loads in flight 5.6 and 4.9).
constexpr int kMaxParts = 304;
constexpr int kGainThreads = 256;
__global__ void __launch_bounds__(kGainThreads) norm_gain_kernel(const float* part, int parts, int K, float* dgain,
                                                                 int accumulate) {
  constexpr int kGroups = kGainThreads / 8;   // of eight lanes, four columns each
  __shared__ float4 s_sum[kGroups][8];
  griddep_launch_dependents();
  griddep_wait();
  const int group = threadIdx.x >> 3, at = threadIdx.x & 7;
  const int c = blockIdx.x * 32 + 4 * at;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v[(kMaxParts + kGroups - 1) / kGroups];
  const float4* p = reinterpret_cast<const float4*>(part + c);
#pragma unroll
  for (int j = 0; j < (kMaxParts + kGroups - 1) / kGroups; ++j) {
    const int i = group + j * kGroups;
    v[j] = c < K && i < parts ? p[static_cast<int64_t>(i) * (K / 4)] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
#pragma unroll
  for (int j = 0; j < (kMaxParts + kGroups - 1) / kGroups; ++j) {
    sum.x += v[j].x;
    sum.y += v[j].y;
    sum.z += v[j].z;
    sum.w += v[j].w;
  }
  s_sum[group][at] = sum;
  __syncthreads();
  const int mine = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || mine >= K) return;
  const float* col = reinterpret_cast<const float*>(s_sum) + threadIdx.x;
  float total = col[0];
#pragma unroll
  for (int i = 1; i < kGroups; ++i) total += col[32 * i];
  dgain[mine] = accumulate ? dgain[mine] + total : total;
}

// ------------------------------------------------------ combine's gradient
struct CombineBackwardParams {
  const uint16_t* dout;
  int64_t T, ldo, N;
  const uint16_t* y;         // NULL: no weight gradient
  int64_t rows;
  const int32_t* row_of;     // [T][k]
  const int32_t* row_token;  // [rows]
  const float* w;            // [T][k]
  int k;
  int zero;                  // rows that a warp looks over at a time
  uint16_t* dy;              // or NULL
  uint8_t* q;                // or NULL (with s)
  float* s;
  float* dw;                 // or NULL
};

constexpr int kCbWarps = 8;       // of a CTA
constexpr int kCbUnroll = 4;      // pieces a lane works on at once
constexpr int kCbZeroRows = 8;    // rows that a warp looks over at a time for those without a token, at most

// A warp takes one slot of a token (with few of them, a CTA's warps share one): it
// multiplies dout's row by the slot's weight into the slot's row, and by the slot's
// row of y into the weight's gradient.  Consecutive slots are a CTA's, so dout's row
// comes from L1 but once.  max |BF16(w x)| over a group is BF16(|w| max |x|), since
// both roundings are monotonic, so the maximum is taken of dout, for two groups in
// one word.  Behind the slots, warps zero the rows without a token.  8192 tokens of
// 8 rows x 7168 take 251 us (1.54 GB, 0.91 of the copy bandwidth), next bound by loads
// waited for and instructions.  A CTA per token took 371, a ring filled by a copying
// warp 352; with the warp's number not known to be uniform (pointers in vector
// registers, spills) 281, with bounds checks on every piece 260; prefetches into L2
// 272, five CTAs an SM 265 to 332.  509 tokens 10.3 us; one token 5.2, its slots
// shared (13 with a warp each).
template <bool kPow2, bool kShared>
__global__ void __launch_bounds__(32 * kCbWarps, 4) combine_backward_kernel(const CombineBackwardParams p) {
  __shared__ float s_dot[kCbWarps];
  __shared__ Divisors<kPow2> divisors;
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // uniform, and known to be: rows and slots are a warp's
  const int nv = static_cast<int>(p.N / 8);
  constexpr int kApart = 32 * (kShared ? kCbWarps : 1);   // between a lane's pieces
  const int64_t slots = p.T * p.k;
  divisors.init();
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  const int64_t first_item = kShared ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kCbWarps + warp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kShared ? 1 : kCbWarps);
  for (int64_t item = first_item; item < slots; item += step) {
    const int64_t t = item / p.k;
    const int j = static_cast<int>(item - t * p.k);
    // the token's slots, to find those that name the same row
    const int32_t* of = p.row_of + t * p.k;
    const int32_t r0 = lane < p.k ? __ldg(of + lane) : -1;
    const int32_t r1 = p.k > 32 && lane + 32 < p.k ? __ldg(of + lane + 32) : -1;
    float w = __ldg(p.w + item);
    int32_t r = __shfl_sync(0xffffffffu, j < 32 ? r0 : r1, j & 31);
    if (r >= p.rows) r = -1;
    const int64_t token = r >= 0 ? __ldg(p.row_token + r) : t;
    const uint64_t same = static_cast<uint64_t>(__ballot_sync(0xffffffffu, r0 == r)) |
                          (static_cast<uint64_t>(__ballot_sync(0xffffffffu, r1 == r)) << 32);
    const bool other = token != t;   // row_token gives the row to another token
    if (other && lane == 0) atomicCAS(&g_train_status, 0, kStatusDeviceArg);
    const bool dots = r >= 0 && !other && p.dw != nullptr;
    // a row named by several slots takes the sum of their weights, from the first of them
    const bool write = r >= 0 && !other && (same & ((uint64_t{1} << j) - 1)) == 0;
    if (write && (same >> j) != 1) {
      w = 0.0f;
      for (uint64_t m = same; m != 0; m &= m - 1) w += __ldg(p.w + t * p.k + __ffsll(static_cast<long long>(m)) - 1);
    }
    float2 dot[kCbUnroll];
#pragma unroll
    for (int i = 0; i < kCbUnroll; ++i) dot[i] = make_float2(0.0f, 0.0f);
    if (dots || write) {
      const int v_first = (kShared ? 32 * warp : 0) + lane;
      const uint4* px = reinterpret_cast<const uint4*>(p.dout + t * p.ldo) + v_first;
      int64_t at = r * p.N + 8 * v_first;      // in y, q and dy
      float* so = p.s + static_cast<int64_t>(v_first >> 4) * p.rows + r;
      const int64_t s_step = kApart / 16 * p.rows;
      // kCbUnroll pieces a lane from piece v on, `all` where the row has them; whole
      // warps come here together (half-warp maxima)
      auto pieces = [&](auto all, int v) {
        constexpr bool kAll = decltype(all)::value;
        uint4 x[kCbUnroll], y[kCbUnroll];
#pragma unroll
        for (int i = 0; i < kCbUnroll; ++i) {
          x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
          if (!kAll && v + i * kApart >= nv) continue;
          x[i] = __ldg(px + i * kApart);
          if (dots) y[i] = __ldg(reinterpret_cast<const uint4*>(p.y + at) + i * kApart);
        }
        uint32_t top[kCbUnroll / 2];
        if (p.q != nullptr) {
#pragma unroll
          for (int i = 0; i < kCbUnroll / 2; ++i) {
            top[i] = __byte_perm(umax_halves(absmax8_bits(x[2 * i])), umax_halves(absmax8_bits(x[2 * i + 1])), 0x5410);
#pragma unroll
            for (int o = 1; o <= 8; o <<= 1) top[i] = umax16x2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
          }
        }
#pragma unroll
        for (int i = 0; i < kCbUnroll; ++i) {
          if (!kAll && v + i * kApart >= nv) continue;
          float2 a[4];
          widen8x2(x[i], a);
          if (dots) {
            float2 b[4];
            widen8x2(y[i], b);
#pragma unroll
            for (int e = 0; e < 4; ++e) dot[i] = __ffma2_rn(a[e], b[e], dot[i]);
          }
          if (!write) continue;
          if (p.dy != nullptr) *reinterpret_cast<uint4*>(p.dy + at + 8 * i * kApart) = times8(a, w);
          if (p.q != nullptr) {
            const uint32_t top16 = i & 1 ? top[i / 2] & 0xFFFF0000u : top[i / 2] << 16;
            const uint32_t a16 = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(top16) * fabsf(w)));
            uint2 codes;
            const float s = quantise8_times<kPow2>(a, w, a16, divisors, codes);
            *reinterpret_cast<uint2*>(p.q + at + 8 * i * kApart) = codes;
            if ((lane & 15) == 0) so[i * s_step] = s;
          }
        }
        px += kCbUnroll * kApart;
        at += 8 * kCbUnroll * kApart;
        so += kCbUnroll * s_step;
      };
      int v0 = v_first - lane;
      for (; v0 + (kCbUnroll - 1) * kApart + 32 <= nv; v0 += kCbUnroll * kApart) pieces(std::true_type{}, v0 + lane);
      for (; v0 < nv; v0 += kCbUnroll * kApart) pieces(std::false_type{}, v0 + lane);
    }
    if (p.dw == nullptr) continue;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kCbUnroll; ++i) sum += dot[i].x + dot[i].y;
    sum = warp_sum(sum);
    if (kShared) {
      if (lane == 0) s_dot[warp] = sum;
      __syncthreads();
      sum = s_dot[0];
#pragma unroll
      for (int i = 1; i < kCbWarps; ++i) sum += s_dot[i];
      __syncthreads();
      if (warp != 0) continue;
    }
    if (lane == 0) p.dw[item] = sum;
  }
  // rows without a token
  const int64_t z_step = static_cast<int64_t>(gridDim.x) * kCbWarps * p.zero;
  for (int64_t z = (static_cast<int64_t>(blockIdx.x) * kCbWarps + warp) * p.zero; z < p.rows; z += z_step) {
    const bool none = lane < p.zero && z + lane < p.rows && __ldg(p.row_token + z + lane) < 0;
    for (uint32_t mask = __ballot_sync(0xffffffffu, none); mask != 0u; mask &= mask - 1u) {
      const int64_t row = z + __ffs(mask) - 1;
      if (p.dy != nullptr)
        for (int v = lane; v < nv; v += 32) *reinterpret_cast<uint4*>(p.dy + row * p.N + 8 * v) = make_uint4(0u, 0u, 0u, 0u);
      if (p.q != nullptr) {
        for (int v = lane; v < nv / 2; v += 32) *reinterpret_cast<uint4*>(p.q + row * p.N + 16 * v) = make_uint4(0u, 0u, 0u, 0u);
        for (int kb = lane; kb < nv / 16; kb += 32) p.s[static_cast<int64_t>(kb) * p.rows + row] = 0.0f;
      }
    }
  }
}

// ------------------------------------------------------- SwiGLU's gradient
struct SwigluBackwardParams {
  const uint16_t* h;
  const uint16_t* dv;
  const int32_t* live;   // or NULL
  int64_t M, I, ldh, lddv;
  int rows;              // rows per CTA and step
  uint32_t step;         // of the grid, in rows, and what that is in elements of h, dv and the outputs
  int64_t step_h, step_v, step_out;
  uint16_t* dh;          // [M][2I] or NULL
  uint8_t* q;            // or NULL (with s)
  float* s;
};

// Hardware base-2 exponential and reciprocal (one instruction each).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Gradients dg, du of silu(g) u times dv for two pairs, in packed float32, for
// gates from -64 up.  With e = e^-g: sigma(g) = 1 / (1 + e), sigma(-g) = e sigma(g);
// neither cancels.  log2 e is taken in two parts: a BF16 gate times the first
// (15 bits) is exact, so the exponential's argument has no rounding, and the
// second enters as a factor 1 - g (log2 e - kHi) ln 2.
__device__ __forceinline__ void swiglu_grad2(uint32_t gw, uint32_t uw, uint32_t vw, uint32_t& dgw, uint32_t& duw) {
  constexpr float kHi = 1.44268798828125f;        // 23637 / 16384
  constexpr float kLo = 4.8884955e-06f;           // (log2 e - kHi) ln 2
  const float2 one = make_float2(1.0f, 1.0f);
  const float2 g = make_float2(__uint_as_float(gw << 16), __uint_as_float(gw & 0xFFFF0000u));
  const float2 u = make_float2(__uint_as_float(uw << 16), __uint_as_float(uw & 0xFFFF0000u));
  const float2 v = make_float2(__uint_as_float(vw << 16), __uint_as_float(vw & 0xFFFF0000u));
  const float2 t = __fmul2_rn(g, make_float2(-kHi, -kHi));
  const float2 e = __fmul2_rn(make_float2(ex2_approx(t.x), ex2_approx(t.y)), __ffma2_rn(g, make_float2(-kLo, -kLo), one));
  const float2 d = __fadd2_rn(e, one);
  const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  const float2 du = __fmul2_rn(v, __fmul2_rn(g, s));
  const float2 f = __fmul2_rn(s, __ffma2_rn(g, __fmul2_rn(e, s), one));
  const float2 dg = __fmul2_rn(__fmul2_rn(v, u), f);
  const __nv_bfloat162 a = __floats2bfloat162_rn(dg.x, dg.y), b = __floats2bfloat162_rn(du.x, du.y);
  dgw = *reinterpret_cast<const uint32_t*>(&a);
  duw = *reinterpret_cast<const uint32_t*>(&b);
}

// The same for what swiglu_grad2 cannot give of a pair: gates below -64, where e^-g
// runs out of float32's range in the end (sigma(g) = e^g to within 2^-92), and
// gradients that came out infinite or NaN, dv * up having left float32's range perhaps
// though the gradient does not, or an infinite gate having made NaN of the exponential's
// correction.  The exponents of dv, up and e^g = 2^n 2^f are kept apart until
// the end, so that nothing overflows or vanishes on the way; below -512 e^g leaves nothing
// of any dv and up.  The other values come back as they are.
constexpr uint32_t kFarGate = 0xC280u;            // BF16 of -64; patterns above it are below -64
constexpr float kLog2Hi = 1.44268798828125f;      // 23637 / 16384
constexpr float kLog2Lo = 7.0526077e-06f;         // log2 e - kLog2Hi
__device__ __noinline__ uint2 swiglu_grad2_wide(uint32_t gw, uint32_t uw, uint32_t vw, uint32_t dgw, uint32_t duw) {
  uint2 out = make_uint2(dgw, duw);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t gb = k ? gw >> 16 : gw & 0xFFFFu;
    const bool far = gb > kFarGate;
    const uint32_t high = k ? 0x7F800000u : 0x7F80u;   // the exponent's bits
    if (!far && (dgw & high) != high && (duw & high) != high) continue;
    const float gate = __uint_as_float(gb << 16);
    const float up = __uint_as_float(k ? uw & 0xFFFF0000u : uw << 16);
    const float dv = __uint_as_float(k ? vw & 0xFFFF0000u : vw << 16);
    int ev, eu;
    const float mv = frexpf(dv, &ev), mu = frexpf(up, &eu);
    float dg, du;
    if (far) {
      const float t = fmaxf(gate, -512.0f) * kLog2Hi, n = rintf(t);    // both exact
      const float s = exp2f(t - n + fmaxf(gate, -512.0f) * kLog2Lo);
      const bool none = gate < -512.0f;
      dg = ldexpf(mv * mu * (1.0f + gate) * (none ? 0.0f : s), ev + eu + static_cast<int>(n));
      du = ldexpf(mv * gate * (none ? 0.0f : s), ev + static_cast<int>(n));
    } else {
      const float e = expf(-gate), s = 1.0f / (1.0f + e);
      dg = ldexpf(mv * mu * (s * fmaf(gate, e * s, 1.0f)), ev + eu);
      du = dv * (gate * s);
    }
    const uint32_t a = __bfloat16_as_ushort(__float2bfloat16_rn(dg));
    const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_rn(du));
    out.x = k ? (out.x & 0xFFFFu) | (a << 16) : (out.x & 0xFFFF0000u) | a;
    out.y = k ? (out.y & 0xFFFFu) | (b << 16) : (out.y & 0xFFFF0000u) | b;
  }
  return out;
}

constexpr int kSbThreads = 512;   // of a CTA, at most

__device__ __forceinline__ void swiglu_grad8(const uint4 (&in)[3], uint4 (&d)[2]) {
  swiglu_grad2(in[0].x, in[1].x, in[2].x, d[0].x, d[1].x);
  swiglu_grad2(in[0].y, in[1].y, in[2].y, d[0].y, d[1].y);
  swiglu_grad2(in[0].z, in[1].z, in[2].z, d[0].z, d[1].z);
  swiglu_grad2(in[0].w, in[1].w, in[2].w, d[0].w, d[1].w);
}

// What a thread writes, of row `row`, and reads, of the row to load next (at most 2^31 rows,
// and a few of the grid's steps).
struct SwigluPlace {
  uint32_t row;
  int64_t out;
  float* ps;
  const uint16_t* ph;
  const uint16_t* pv;
  __device__ __forceinline__ SwigluPlace(const SwigluBackwardParams& p, uint32_t row_, int c)
      : row(row_), out(2 * p.I * row_ + 8 * c), ps(p.s == nullptr ? nullptr : p.s + static_cast<int64_t>(c >> 4) * p.M + row_),
        ph(p.h + row_ * p.ldh + 8 * c), pv(p.dv + row_ * p.lddv + 8 * c) {}
  __device__ __forceinline__ void move_on(const SwigluBackwardParams& p) {
    row += p.step;
    out += p.step_out;
    ps += p.step;
  }
  __device__ __forceinline__ bool live(const SwigluBackwardParams& p, uint32_t ahead) const {
    return row + ahead < p.M && (p.live == nullptr || __ldg(p.live + (row + ahead)) >= 0);
  }
  __device__ __forceinline__ void load(const SwigluBackwardParams& p, bool live, uint4 (&in)[3]) {
    in[0] = in[1] = in[2] = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
      in[0] = __ldg(reinterpret_cast<const uint4*>(ph));
      in[1] = __ldg(reinterpret_cast<const uint4*>(ph + p.I));
      in[2] = __ldg(reinterpret_cast<const uint4*>(pv));
    }
    ph += p.step_h;
    pv += p.step_v;
  }
  // Quantises and stores the row's piece, `top` the halves' largest magnitudes in this
  // thread; whole warps come here together.
  template <bool kPow2>
  __device__ __forceinline__ void finish(const SwigluBackwardParams& p, const Divisors<kPow2>& divisors, const uint4 (&d)[2],
                                         uint32_t top, bool first_of_group, bool here) const {
    if (here && p.dh != nullptr) {
      *reinterpret_cast<uint4*>(p.dh + out) = d[0];
      *reinterpret_cast<uint4*>(p.dh + out + p.I) = d[1];
    }
    if (p.q == nullptr) return;
#pragma unroll
    for (int o = 1; o <= 8; o <<= 1) top = umax16x2(top, __shfl_xor_sync(0xffffffffu, top, o));
    uint2 cg, cu;
    const float sg = quantise8<kPow2>(d[0], top & 0xFFFFu, divisors, cg);
    const float su = quantise8<kPow2>(d[1], top >> 16, divisors, cu);
    if (!here) return;
    *reinterpret_cast<uint2*>(p.q + out) = cg;
    *reinterpret_cast<uint2*>(p.q + out + p.I) = cu;
    if (first_of_group) {
      ps[0] = sg;
      ps[(p.I >> 7) * p.M] = su;
    }
  }
};

// Both halves' largest magnitudes of a thread in one word; kNan: NaN where any value is.
// Without it a number is larger than NaN, as in the quantisers.
__device__ __forceinline__ uint32_t absmax_step_nan(uint32_t m, uint32_t w) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
  return d;
}
template <bool kNan>
__device__ __forceinline__ uint32_t swiglu_top(const uint4 (&d)[2]) {
  uint32_t m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    m[i] = kNan ? abs_bits(absmax_step_nan(absmax_step_nan(d[i].x, d[i].y), absmax_step_nan(d[i].z, d[i].w)))
                : absmax8_bits(d[i]);
  return __byte_perm(umax_halves(m[0]), umax_halves(m[1]), 0x5410);
}
// Whether pieces of rows need the second pass, by the largest of their gates' patterns and
// of their gradients' magnitudes (in the halves of a word each): a gate below -64, or a
// gradient that is infinite or NaN.
__device__ __forceinline__ uint32_t top_gate(const uint4& g) { return umax16x2(umax16x2(g.x, g.y), umax16x2(g.z, g.w)); }
__device__ __forceinline__ bool swiglu_again(uint32_t gate, uint32_t top) {
  return (umax_halves(gate) & 0xFFFFu) > kFarGate || (umax_halves(top) & 0xFFFFu) >= 0x7F80u;
}

// The second pass over a warp's rows: those that need it, one at a time, written anew.
template <bool kPow2>
__device__ __noinline__ void swiglu_rows_again(const SwigluBackwardParams& p, const Divisors<kPow2>& divisors, int sub, int c0,
                                               int step_c) {
  const int upr = static_cast<int>(p.I / 8);
  for (int cc = 0; cc < upr; cc += step_c) {
    const int c = c0 + cc;
    const bool inside = sub < p.rows && c < upr;
    SwigluPlace at(p, blockIdx.x * p.rows + sub, c);
    for (; at.row - sub < p.M; at.move_on(p)) {
      uint4 in[3], d[2];
      at.load(p, inside && at.live(p, 0), in);
      swiglu_grad8(in, d);
      if (!__any_sync(0xffffffffu, swiglu_again(top_gate(in[0]), swiglu_top<true>(d)))) continue;
      uint2 w = swiglu_grad2_wide(in[0].x, in[1].x, in[2].x, d[0].x, d[1].x);
      d[0].x = w.x, d[1].x = w.y;
      w = swiglu_grad2_wide(in[0].y, in[1].y, in[2].y, d[0].y, d[1].y);
      d[0].y = w.x, d[1].y = w.y;
      w = swiglu_grad2_wide(in[0].z, in[1].z, in[2].z, d[0].z, d[1].z);
      d[0].z = w.x, d[1].z = w.y;
      w = swiglu_grad2_wide(in[0].w, in[1].w, in[2].w, d[0].w, d[1].w);
      d[0].w = w.x, d[1].w = w.y;
      at.finish<kPow2>(p, divisors, d, swiglu_top<false>(d), (c & 15) == 0, inside && at.row < p.M);
    }
  }
}

// Thread = eight columns of one half of h: the columns stay, the rows advance by
// the grid, with the next row's loads in flight.  A group of 128 is a half-warp's
// 16 threads; whole warps go through the loop together.  Rows with a gate below -64
// or a gradient that is no finite number are written anew in a second pass, which rarely has any: the
// loop keeps the largest patterns of all rows, two instructions a row, and looks at
// them once.  [67712][2048] takes 167 us (1.12 GB, 0.99 of the copy bandwidth); with a vote a
// row, that kept such rows from being stored, 174 to 187, with a call inside the loop,
// whose results went through local memory, 190 to 228.  With absmax scales 205, bound by
// instructions; by a ring of bulk copies 245, unpacked with expf 325.
template <bool kPow2>
__global__ void __launch_bounds__(kSbThreads, 2) swiglu_backward_kernel(const __grid_constant__ SwigluBackwardParams p) {
  __shared__ Divisors<kPow2> divisors;
  divisors.init();
  __syncthreads();
  griddep_launch_dependents();
  const int upr = static_cast<int>(p.I / 8);          // pieces a row, a multiple of 16
  const bool whole = upr * p.rows <= static_cast<int>(blockDim.x);
  const int sub = whole ? threadIdx.x / upr : 0;
  const int step_c = whole ? upr : blockDim.x;        // rows longer than a CTA: in steps
  const int c0 = threadIdx.x - sub * upr;
  const bool mine = sub < p.rows;
  uint32_t gates = 0u, tops = 0u;                     // the largest of all rows
  griddep_wait();
  for (int cc = 0; cc < upr; cc += step_c) {
    const int c = c0 + cc;
    const bool inside = mine && c < upr;
    SwigluPlace at(p, blockIdx.x * p.rows + sub, c);
    uint4 next[3];
    at.load(p, inside && at.live(p, 0), next);
    bool live_after = inside && at.live(p, p.step);   // a row ahead of the loads that wait for it
    while (at.row - sub < p.M) {                  // as far as any of the CTA's rows goes
      const uint4 in[3] = {next[0], next[1], next[2]};
      at.load(p, live_after, next);
      live_after = inside && at.live(p, 2 * p.step);
      uint4 d[2];
      swiglu_grad8(in, d);
      const uint32_t top = swiglu_top<true>(d);
      gates = umax16x2(gates, top_gate(in[0]));
      tops = umax16x2(tops, top);
      at.finish<kPow2>(p, divisors, d, top, (c & 15) == 0, inside && at.row < p.M);
      at.move_on(p);
    }
  }
  if (__any_sync(0xffffffffu, swiglu_again(gates, tops))) swiglu_rows_again<kPow2>(p, divisors, sub, c0, step_c);
}

// CTAs of `kern` that fit on the device at once.
template <typename Kern>
cudaError_t resident_ctas(Kern kern, int threads, int sm_count, std::atomic<int> (&cache)[kMaxCachedDevices], int64_t* n) {
  int per_sm = 0;
  const cudaError_t e = cached_per_device(
      cache, [&](int* v) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kern, threads, 0); }, &per_sm);
  *n = static_cast<int64_t>(per_sm) * sm_count;
  return e;
}

// Lets `kern` take a ring's shared memory, once per device (the call costs 0.3 us).
template <typename Kern>
cudaError_t allow_ring(Kern kern, std::atomic<int> (&cache)[kMaxCachedDevices]) {
  int done = 0;
  return cached_per_device(
      cache,
      [&](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingMaxBytes);
      },
      &done);
}

template <int kVecs, bool kGainF32, bool kPow2>
cudaError_t run_norm(const NormParams& p, int grid, int threads, int smem, cudaStream_t stream) {
  auto kern = p.res != nullptr ? norm_kernel<kVecs, kGainF32, kPow2, true> : norm_kernel<kVecs, kGainF32, kPow2, false>;
  static std::atomic<int> cache[2][kMaxCachedDevices];
  const cudaError_t e = allow_ring(kern, cache[p.res != nullptr ? 1 : 0]);
  if (e != cudaSuccess) return e;
  return launch_behind_smem(kern, dim3(static_cast<unsigned>(grid)), static_cast<unsigned>(threads), static_cast<size_t>(smem),
                            stream, p);
}

template <int kVecs>
cudaError_t run_norm_kind(const NormParams& p, bool gain_f32, bool pow2, int grid, int threads, int smem, cudaStream_t stream) {
  if (gain_f32)
    return pow2 ? run_norm<kVecs, true, true>(p, grid, threads, smem, stream)
                : run_norm<kVecs, true, false>(p, grid, threads, smem, stream);
  return pow2 ? run_norm<kVecs, false, true>(p, grid, threads, smem, stream)
              : run_norm<kVecs, false, false>(p, grid, threads, smem, stream);
}

// Ring and grid of the gradient: two CTAs an SM where two stages of half an SM's
// shared memory hold the rows, else one.  The grid goes by the sizes alone (152
// SMs), so that the parts, and the bits of their sum, do too.
struct NormBackwardPlan {
  RowPlace at;
  int stages, stage_bytes, grid;
};
NormBackwardPlan plan_norm_backward(int64_t M, int64_t K, bool dres) {
  NormBackwardPlan n;
  n.at = place_rows(static_cast<int>(K), 256);
  // At least eight warps a CTA, sixteen for short rows, where four stages hold their rows
  // and no CTA stays without any:
  // [65536][128] 39 us (51 with eight warps), [16384][512] 17.9 (24.6), [16384][1536] 37.3
  // (43.6 with six).
  const int target = K <= 512 ? 16 : 8, rows = (target + n.at.warps - 1) / n.at.warps;
  if (kRingMaxStages * 6 * rows * K <= kRingBytes && M >= int64_t{kMaxParts} * rows) n.at.rows = rows;
  n.stage_bytes = static_cast<int>((dres ? 3 : 2) * n.at.rows * K * 2);
  const bool two = 12 * n.at.rows * K <= kRingBytes;   // two stages of three arrays, with or without dres
  n.stages = std::min(kRingMaxStages, (two ? kRingBytes : kRingMaxBytes) / n.stage_bytes);
  n.grid = static_cast<int>(std::min<int64_t>((M + n.at.rows - 1) / n.at.rows, two ? kMaxParts : kMaxParts / 2));
  return n;
}

template <int kVecs, bool kGainF32>
cudaError_t run_norm_backward(const NormBackwardParams& p, const NormBackwardPlan& n, cudaStream_t stream) {
  auto kern = norm_backward_kernel<kVecs, kGainF32>;
  const int smem = n.stages * n.stage_bytes;
  static std::atomic<int> cache[kMaxCachedDevices];
  const cudaError_t e = allow_ring(kern, cache);
  if (e != cudaSuccess) return e;
  return launch_behind_smem(kern, dim3(static_cast<unsigned>(n.grid)), static_cast<unsigned>(32 * n.at.warps * n.at.rows),
                            static_cast<size_t>(smem), stream, p);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, int sm_count, cudaStream_t stream) {
  const RowPlace at = place_rows(static_cast<int>(a.K), kNormFour);
  const int threads = 32 * at.warps * at.rows;
  const int stage_bytes = static_cast<int>((a.res != nullptr ? 2 : 1) * at.rows * a.K * 2);
  int ctas = std::max(1, kNormWarps / (at.warps * at.rows));   // per SM
  while (ctas > 1 && 2 * stage_bytes > kRingMaxBytes / ctas - 1024) --ctas;
  NormParams p;
  p.x = a.x; p.res = a.res; p.gain = a.gain; p.M = a.M; p.ldx = a.ldx; p.ldr = a.ldr; p.K = static_cast<int>(a.K);
  p.warps = at.warps; p.eps = a.eps; p.inv_k = 1.0f / static_cast<float>(a.K); p.r = a.r; p.y = a.y; p.q = a.q; p.s = a.s; p.rstd = a.rstd; p.timeout_ns = a.timeout_ns;
  p.stages = std::min(kNormStages, (kRingMaxBytes / ctas - 1024 * (ctas > 1)) / stage_bytes);
  const int smem = p.stages * stage_bytes;
  const int grid = static_cast<int>(std::min<int64_t>((a.M + at.rows - 1) / at.rows, static_cast<int64_t>(ctas) * sm_count));
  return at.vecs == 4   ? run_norm_kind<4>(p, a.gain_f32, a.pow2, grid, threads, smem, stream)
         : at.vecs == 2 ? run_norm_kind<2>(p, a.gain_f32, a.pow2, grid, threads, smem, stream)
                        : run_norm_kind<1>(p, a.gain_f32, a.pow2, grid, threads, smem, stream);
}

int64_t rmsnorm_max_columns() { return kMaxNormK; }

int64_t rmsnorm_backward_workspace_bytes(int64_t M, int64_t K) {
  return M == 0 || K == 0 ? 0 : 4 * K * plan_norm_backward(M, K, true).grid;
}

cudaError_t launch_rmsnorm_backward(const NormBackwardArgs& a, void* ws, cudaStream_t stream) {
  const NormBackwardPlan n = plan_norm_backward(a.M, a.K, a.dres != nullptr);
  NormBackwardParams p;
  p.dy = a.dy; p.r = a.r; p.gain = a.gain; p.rstd = a.rstd; p.dres = a.dres; p.M = a.M; p.lddy = a.lddy; p.ldr = a.ldr;
  p.lddres = a.lddres; p.K = static_cast<int>(a.K); p.warps = n.at.warps; p.stages = n.stages; p.dx = a.dx;
  p.part = a.dgain != nullptr ? static_cast<float*>(ws) : nullptr;
  p.timeout_ns = a.timeout_ns; p.inv_k = 1.0f / static_cast<float>(a.K);
  const cudaError_t e = n.at.vecs == 4   ? (a.gain_f32 ? run_norm_backward<4, true>(p, n, stream) : run_norm_backward<4, false>(p, n, stream))
                        : n.at.vecs == 2 ? (a.gain_f32 ? run_norm_backward<2, true>(p, n, stream) : run_norm_backward<2, false>(p, n, stream))
                                         : (a.gain_f32 ? run_norm_backward<1, true>(p, n, stream) : run_norm_backward<1, false>(p, n, stream));
  if (e != cudaSuccess || a.dgain == nullptr) return e;
  return launch_behind(norm_gain_kernel, dim3(static_cast<unsigned>((a.K + 31) / 32)), kGainThreads, stream,
                       static_cast<const float*>(p.part), n.grid, p.K, a.dgain, a.accumulate ? 1 : 0);
}

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, int sm_count, cudaStream_t stream) {
  CombineBackwardParams p;
  p.dout = a.dout; p.T = a.T; p.ldo = a.ldo; p.N = a.N; p.y = a.y; p.rows = a.rows; p.row_of = a.row_of;
  p.row_token = a.row_token; p.w = a.w; p.k = a.k; p.dy = a.dy; p.q = a.q; p.s = a.s; p.dw = a.dw;
  // with fewer slots than two a warp of every SM, a CTA's warps share one
  const int64_t n = a.T * a.k;
  const bool shared = n < 2 * static_cast<int64_t>(sm_count);
  auto kern = a.pow2 ? (shared ? combine_backward_kernel<true, true> : combine_backward_kernel<true, false>)
                     : (shared ? combine_backward_kernel<false, true> : combine_backward_kernel<false, false>);
  static std::atomic<int> cache[4][kMaxCachedDevices];
  int64_t resident = 0;
  const cudaError_t e = resident_ctas(kern, 32 * kCbWarps, sm_count, cache[(a.pow2 ? 2 : 0) + (shared ? 1 : 0)], &resident);
  if (e != cudaSuccess) return e;
  p.zero = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kCbZeroRows, a.rows / (resident * kCbWarps))));
  const int64_t zero = static_cast<int64_t>(p.zero) * kCbWarps;
  const int64_t grid = std::min(resident, std::max(shared ? n : (n + kCbWarps - 1) / kCbWarps, (a.rows + zero - 1) / zero));
  if (grid <= 0) return cudaSuccess;
  return launch_behind(kern, dim3(static_cast<unsigned>(grid)), 32 * kCbWarps, stream, p);
}

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& a, int sm_count, cudaStream_t stream) {
  SwigluBackwardParams p;
  p.h = a.h; p.dv = a.dv; p.live = a.live; p.M = a.M; p.I = a.I; p.ldh = a.ldh; p.lddv = a.lddv;
  p.dh = a.dh; p.q = a.q; p.s = a.s;
  const int upr = static_cast<int>(a.I / 8);
  // Rows share a CTA of 512 threads, or of 256 where there are few rows or short ones
  // ([67712][2048] 174 us with 512, 178 with 256; [64][2048] 2.4 and 2.1, [312500][128] 57.0
  // and 56.2).  Rows of more than 512 pieces take equal steps of at most as many ([9470][4224]
  // 61 us, in steps of 256 with a short last one 74).
  const int halves = upr >= 64 && a.M >= 2 * static_cast<int64_t>(sm_count) * std::max(1, kSbThreads / upr) ? 1 : 2;
  p.rows = std::max(1, kSbThreads / halves / upr);
  const int steps = (upr + kSbThreads - 1) / kSbThreads;
  const int threads = ((steps > 1 ? (upr + steps - 1) / steps : p.rows * upr) + 31) / 32 * 32;
  auto kern = a.pow2 ? swiglu_backward_kernel<true> : swiglu_backward_kernel<false>;
  static std::atomic<int> cache[2][17][kMaxCachedDevices];
  int64_t slots = 0;
  const cudaError_t e = resident_ctas(kern, threads, sm_count, cache[a.pow2 ? 1 : 0][threads / 32], &slots);
  if (e != cudaSuccess) return e;
  const int64_t grid = std::min((p.M + p.rows - 1) / p.rows, slots);
  p.step = static_cast<uint32_t>(grid * p.rows);
  p.step_h = p.step * p.ldh;
  p.step_v = p.step * p.lddv;
  p.step_out = 2 * p.I * p.step;
  return launch_behind(kern, dim3(static_cast<unsigned>(grid)), threads, stream, p);
}

cudaError_t train_take_status(int* status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_train_status, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_train_status, &zero, sizeof(int));
  }
  *status = v;
  return e;
}

}  // namespace fp8bs
