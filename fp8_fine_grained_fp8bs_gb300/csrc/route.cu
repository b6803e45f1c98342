// The MoE router: expert choice, gate weights, per-expert counts and the
// balance loss with its gradient, and the row layout of the choices.
//
//   scores   softmax: s_i = e^(z_i - max) / (sum + eps);  sigmoid: s_i = 1 / (1 + e^-z_i)
//            p_i = s_i / (sum_j s_j + eps)  (softmax: p = s)
//   choice   the k experts of largest z_i, or s_i + bias_i with a selection
//            bias (sigmoid only); ties go to the lower index; logits that are
//            -inf or NaN are not eligible, a slot without an eligible expert
//            holds -1 with weight 0
//   weights  w_j = scale * s_j / (sum over the chosen s + eps), or scale * s_j
//   loss     alpha / S * sum over sequences of sum_i f_i P_i,
//            f_i = E n_i / (k T_s),  P_i = (1 / T_s) sum_t p_i
//
// with n_i the sequence's choices of expert i and T_s its tokens that have an
// eligible expert.  f is a count and has no gradient:
//   d loss / d p_i = alpha / S * f_i / T_s.
//
// A token takes a group of W lanes: half a warp, or a whole one for more than
// 256 experts or 16 choices.  Expert e is held by lane e % W of the group in
// register e / W, so a lane sees the same experts in every token, and the sums
// of p over a group's tokens stay in registers.  Sums over tokens are taken in
// a fixed order (lane, group, chunk of tokens), counts with integer additions,
// so results do not vary from run to run.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"
#include "launch.h"

namespace fp8bs {
namespace {

__device__ int g_route_status;
__device__ __forceinline__ void record_route_status(int code) { atomicCAS(&g_route_status, 0, code); }

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr float kScoreEps = 1e-20f;    // guards the sums that scores are divided by
constexpr float kLowest = -3.402823466e38f;
constexpr uint32_t kFull = 0xffffffffu;

// Reductions over the W lanes of a group; all lanes of the warp take part.
template <int W>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int W>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (W == 32) {
    return __reduce_max_sync(kFull, v);
  } else {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}
template <int W>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  if constexpr (W == 32) {
    return __reduce_min_sync(kFull, v);
  } else {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}
// The group's votes in the low W bits.
template <int W>
__device__ __forceinline__ uint32_t group_ballot(bool p, int lane) {
  const uint32_t b = __ballot_sync(kFull, p);
  return W == 32 ? b : (b >> (lane & ~(W - 1))) & ((1u << (W & 31)) - 1u);
}
__device__ __forceinline__ float warp_sum(float v) { return group_sum<32>(v); }

__device__ __forceinline__ float load_logit(const void* logits, bool bf16, int64_t at) {
  if (bf16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(logits) + at)) << 16);
  return __ldg(static_cast<const float*>(logits) + at);
}

// IEEE division and expf: the choice with a bias is decided by these bits.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

__device__ __forceinline__ bool eligible(float z) { return z > -INFINITY; }  // false for NaN too

// Order-preserving image of a float, above 0 for every number; -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((b >> 31) != 0u ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float from_key(uint32_t k) { return __uint_as_float((k >> 31) != 0u ? k ^ 0x80000000u : ~k); }

// One token's logits in registers: z[i] is expert W i + g, -inf from expert
// `end` on (E, or 0 for a token that is not there or masked).
// The bits of all loads arrive before any is widened: converted one by one,
// BF16 logits waited for each load in turn (backward 131072 x 256: 103 us
// against 58 for float32).
template <int W, int NL>
__device__ __forceinline__ void load_token(const RouteArgs& a, int64_t t, int g, int end, float (&z)[NL]) {
  uint32_t bits[NL];
  if (a.bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + t * a.ld + g;
#pragma unroll
    for (int i = 0; i < NL; ++i) bits[i] = W * i + g < end ? __ldg(p + W * i) : 0xFF80u;
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(a.logits) + t * a.ld + g;
#pragma unroll
    for (int i = 0; i < NL; ++i) bits[i] = W * i + g < end ? __ldg(p + W * i) : 0xFF800000u;
  }
  const uint32_t shift = a.bf16 ? 16 : 0;
#pragma unroll
  for (int i = 0; i < NL; ++i) z[i] = __uint_as_float(bits[i] << shift);
}

// Two float32 operations in one instruction, each rounded as its scalar form.
#define FP8BS_F32X2_2(name, op)                                                                       \
  __device__ __forceinline__ float2 name(float2 a, float2 b) {                                        \
    float2 d;                                                                                         \
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t" op              \
        " z, x, y;\n\tmov.b64 {%0, %1}, z;\n}\n"                                                      \
        : "=f"(d.x), "=f"(d.y)                                                                        \
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));                                                    \
    return d;                                                                                         \
  }
FP8BS_F32X2_2(add2, "add.rn.f32x2")
FP8BS_F32X2_2(mul2, "mul.rn.f32x2")
#undef FP8BS_F32X2_2
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 w, x, y, z;\n\tmov.b64 w, {%2, %3};\n\tmov.b64 x, {%4, %5};\n\tmov.b64 y, {%6, %7};\n\t"
      "fma.rn.f32x2 z, w, x, y;\n\tmov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
// 1 / x within one ulp, for the scores that only enter sums and gradients and
// for their sums; the weights and the keys of the choice are divided.  (Rounded
// correctly, __frcp_rn: gradient of 131072 x 256 68.7 us against 65.6.)
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// e^x for x <= 0, as 2^t (1 + d) with t = fl(x log2 e) and d = x - t ln 2, at most
// |x| 2^-24: the instruction's 2^-22 of relative error and a rounding, at any x.
// (t alone loses that |x| 2^-24: 2^-19.5 for a logit 22 to 30 below the top.)  d
// is what cancellation leaves of an exact product, with ln 2 in two parts (Cody
// and Waite, Software Manual for the Elementary Functions, 1980).  NaN for
// NaN, -inf and x whose t overflows: the callers' maximum with 0 makes it 0.
// Two at a time as costly as one hardware exponential was (131072 x 256 with
// statistics and biased sigmoids 79.4 us, 79.9 before; the gradient 64.4 and
// 64.0; with expf 83.2 and 73.3).
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2Hi = 0.693147182464599609375f;            // fl(ln 2)
constexpr float kLn2Lo = -1.904654299957767e-9f;              // fl(ln 2 - kLn2Hi)
__device__ __forceinline__ float2 exp_pair(float2 x) {
  const float2 t = mul2(x, both(kLog2e));
  const float2 d = fma2(t, both(-kLn2Lo), fma2(t, both(-kLn2Hi), x));
  const float2 p = make_float2(ex2(t.x), ex2(t.y));
  return fma2(p, d, p);
}
__device__ __forceinline__ float exp_one(float x) {
  const float t = x * kLog2e;
  const float p = ex2(t);
  return fmaf(p, fmaf(t, -kLn2Lo, fmaf(t, -kLn2Hi, x)), p);
}

// f(pair) over NL values two at a time; a single value is paired with itself.
template <int NL, typename F>
__device__ __forceinline__ void in_pairs(float (&v)[NL], F f) {
#pragma unroll
  for (int i = 0; i < NL; i += 2) {
    const float2 r = f(make_float2(v[i], v[i + 1 < NL ? i + 1 : i]));
    v[i] = r.x;
    if (i + 1 < NL) v[i + 1] = r.y;
  }
}

// sigmoid(z) is 1 - q or q, with q = e^-|z| / (1 + e^-|z|) <= 1/2, which cannot
// overflow and loses nothing to cancellation; its derivative is q (1 - q).
// 0 where z is not eligible.  Relative error below 2^-21.4 (exponential,
// reciprocal, sum and product).
__device__ __forceinline__ float part_of(float e) {
  const float t = fmaxf(e, 0.0f);
  return t * fast_rcp(1.0f + t);
}
__device__ __forceinline__ float sigmoid_part(float z) { return part_of(exp_one(-fabsf(z))); }
__device__ __forceinline__ float2 sigmoid_parts(float2 z) {
  const float2 e = exp_pair(make_float2(-fabsf(z.x), -fabsf(z.y)));
  return make_float2(part_of(e.x), part_of(e.y));
}

// sigmoid of two logits for the statistics, negated: 1 / (1 + 2^t), moved by
// the exponent's rest: s' = s - s (1 - s) d.  Half of t is what d is computed
// from, so that nothing is infinite but 2^t, for any finite z.  NaN where z is
// not eligible (z * 0 is NaN for NaN and the infinities).
__device__ __forceinline__ float2 minus_sigmoid_pair(float2 z) {
  const float2 half = mul2(z, both(-0.5f * kLog2e));
  const float2 t = add2(half, half);
  const float2 d = fma2(half, both(2.0f * kLn2Lo), fma2(half, both(2.0f * kLn2Hi), z));   // of opposite sign
  const float2 n = fma2(make_float2(ex2(t.x), ex2(t.y)), both(-1.0f), both(-1.0f));
  const float2 s = make_float2(fast_rcp(n.x), fast_rcp(n.y));
  return fma2(z, both(0.0f), fma2(fma2(s, s, s), d, s));
}

// The sequences of a launch: [seq[s], seq[s + 1]) covers 0 .. T in order.  The
// CTAs share the check; a violation leaves the outputs undefined, so they go on
// meanwhile, and the walk below stays inside the arrays and ends whatever seq
// holds.  (Each CTA of both kernels checking all of them first: 65535 sequences of
// one token, 64 experts, with statistics in 7.3 ms against 1.4.)
__device__ __forceinline__ void check_sequences(const RouteArgs& a) {
  if (a.seq == nullptr) return;
  bool bad = false;
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * kRouteThreads + threadIdx.x; s <= a.S;
       s += static_cast<int64_t>(gridDim.x) * kRouteThreads) {
    const int32_t o = a.seq[s];
    bad |= s == 0 ? o != 0 : o < a.seq[s - 1];
    bad |= s == a.S && o != a.T;
  }
  if (bad) record_route_status(kStatusDeviceArg);
}
// Last sequence that begins at or before token t.
__device__ __forceinline__ int sequence_of(const RouteArgs& a, int64_t t) {
  if (a.seq == nullptr) return 0;
  int lo = 0, hi = a.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (a.seq[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int64_t sequence_end(const RouteArgs& a, int s) { return a.seq == nullptr ? a.T : a.seq[s + 1]; }
// The sequence of token t, at which sequence s ends: the next one, or past
// empty ones the one that a search finds.  a.S or above where there is none
// (invalid sequences).
__device__ __forceinline__ int next_sequence(const RouteArgs& a, int s, int64_t t) {
  ++s;
  return s < a.S && sequence_end(a, s) <= t ? sequence_of(a, t) : s;
}

// The largest key of the group's keys key[i] (expert W i + g; -inf or NaN
// where not eligible) in `most` (0: none is eligible), and candidates for the
// k largest of them: all keys from the k-th largest lane maximum on, less
// `slack`; no key among the k largest lies below it.  Of 256 random keys and
// k = 8 about eleven pass, so that the exact order is worked out on one key per
// lane.  (The bound by sorting the maxima, ten exchanges: 32749 tokens in 18.6
// us; by bisection between the least and the largest of them, 22.0.)  Leaves the
// candidates' experts in `list` (lanes' first ones before their second ones)
// and returns their number, which may be above 32 (ties, k near W): only the
// first 32 are in the list then.
template <int W, int NL>
__device__ __forceinline__ int candidates(const float (&key)[NL], int k, bool slack, int lane, uint16_t* list,
                                          uint32_t& most) {
  float m = key[0];
#pragma unroll
  for (int i = 1; i < NL; ++i) m = fmaxf(m, key[i]);
  const uint32_t mine = eligible(m) ? order_key(m) : 0u;
  // bitonic sort of the lanes' maxima, largest first
  uint32_t sorted = mine;
#pragma unroll
  for (int size = 2; size <= W; size *= 2) {
#pragma unroll
    for (int d = size / 2; d > 0; d /= 2) {
      const uint32_t other = __shfl_xor_sync(kFull, sorted, d);
      const bool upper = ((lane & d) == 0) == (size == W || (lane & size) == 0);
      sorted = upper ? max(sorted, other) : min(sorted, other);
    }
  }
  most = __shfl_sync(kFull, sorted, lane & ~(W - 1));
  const uint32_t low = __shfl_sync(kFull, sorted, (lane & ~(W - 1)) + k - 1);
  float bound = low == 0u ? kLowest : from_key(low);   // 0: fewer than k lanes hold an eligible key
  if (slack) bound = fmaxf(bound - (1e-5f + 1e-6f * fabsf(bound)), kLowest);
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < NL; ++i) mask |= key[i] >= bound ? 1u << i : 0u;
  int n = 0;
  const int g = lane & (W - 1);
  const uint32_t below = (1u << g) - 1u;
  while (__any_sync(kFull, mask != 0u)) {
    const uint32_t who = group_ballot<W>(mask != 0u, lane);
    const int at = n + __popc(who & below);
    if (mask != 0u && at < 32) list[at] = static_cast<uint16_t>(W * (__ffs(mask) - 1) + g);
    mask &= mask - 1u;
    n += __popc(who);
  }
  __syncwarp();
  return n;
}

// CTAs that an SM should hold, which bounds the registers of a thread (32749
// tokens of 256 logits: 15.4 us with four CTAs, 19.3 with three; with the
// statistics' sums four would spill: 31.2 us against 27.0).
template <int NL, bool kStats>
constexpr int kRouteCtas = NL <= 8 ? 4 : NL == 16 ? (kStats ? 3 : 4) : 1;

// CTA c routes tokens [c * chunk, (c + 1) * chunk).  With statistics, each
// stretch of one sequence inside the chunk leaves its sums in row c + s of
// the partial arrays: along the tokens every step from one (chunk, sequence)
// to the next raises c or s, so the rows are distinct.
//
// Bound by instructions (about 290 a token of 256 logits, 450 with statistics
// and biased sigmoids, two thirds of the issue slots busy).  131072 tokens: 154
// us choosing the k experts one by one from all keys, two warp reductions and a
// pass over the keys each; 86 with candidates, a warp per token; 61 with half a
// warp, which shares the per-token steps between two tokens (with statistics
// 166, 108 and 79 us).
template <int W, int NL, int kScore, bool kStats>
__global__ void __launch_bounds__(kRouteThreads, kRouteCtas<NL, kStats>) route_kernel(const RouteArgs a) {
  constexpr int kGroups = kRouteThreads / W;          // tokens at a time
  constexpr int kPerLane = 32 / W;                    // candidates of a lane
  __shared__ float s_p[kStats ? kGroups * W * NL : 1];
  __shared__ int s_n[kStats ? W * NL : 1];
  __shared__ int s_t[kRouteWarps];
  __shared__ uint16_t s_list[kGroups][32];
  __shared__ __align__(16) uint64_t s_order[kGroups][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = threadIdx.x / W, g = threadIdx.x & (W - 1);
  if (kStats) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
    check_sequences(a);
  }
  const bool biased = kScore == 1 && a.bias != nullptr;
  const int64_t hi = min(a.T, static_cast<int64_t>(blockIdx.x + 1) * a.chunk);
  int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  int s = kStats && lo < hi ? sequence_of(a, lo) : 0;
  uint16_t* list = s_list[group];
  uint64_t* order = s_order[group];
  while (lo < hi) {
    const int64_t end = kStats ? min(hi, sequence_end(a, s)) : hi;
    if (kStats && end <= lo) break;   // invalid sequences
    float acc[NL];
    int live_tokens = 0;   // of the group
    if (kStats) {
#pragma unroll
      for (int i = 0; i < NL; ++i) acc[i] = 0.0f;
      for (int e = threadIdx.x; e < a.E; e += kRouteThreads) s_n[e] = 0;
      __syncthreads();
    }
    // warps walk the tokens together; a group without one stays empty.  The
    // mask is read a step ahead, so that the logits' loads do not wait for it.
    auto is_valid = [&](int64_t t) { return t < end && (a.valid == nullptr || a.valid[t] != 0); };
    bool valid_next = is_valid(lo + threadIdx.x / W);
    for (int64_t t0 = lo + warp * (32 / W); t0 < end; t0 += kGroups) {
      const int64_t t = t0 + lane / W;
      const bool here = t < end, valid = valid_next;
      valid_next = is_valid(t + kGroups);
      float v[NL];   // logits, then scores or keys
      load_token<W, NL>(a, here ? t : lo, g, valid ? a.E : 0, v);
      // Scores of all experts for the statistics, for softmax weights that are
      // not normalised over the chosen, and (approximate) for biased keys.
      const bool all = kStats || biased || (kScore == 0 && !a.normalize);
      float total = 1.0f;
      uint32_t most = 0;
      int n = 0;
      if (!biased) n = candidates<W, NL>(v, a.k, false, lane, list, most);
      const float top = from_key(most);   // softmax; not used where most is 0
      if (all) {
        if (kScore == 1 && !kStats) {
          // keys that narrow the candidates, with a margin
#pragma unroll
          for (int i = 0; i < NL; ++i) v[i] = fmaf(v[i], 0.0f, fast_rcp(1.0f + ex2(v[i] * -kLog2e)));
        } else {
          in_pairs(v, [&](float2 z) { return kScore == 0 ? exp_pair(add2(z, both(-top))) : minus_sigmoid_pair(z); });
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          if (kScore == 1 && kStats) v[i] = -v[i];
          sum += fmaxf(v[i], 0.0f);   // 0 for NaN
        }
        total = group_sum<W>(sum) + kScoreEps;
        if (kStats) {
          const float inv = fast_rcp(total);
#pragma unroll
          for (int i = 0; i < NL; ++i) acc[i] = fmaf(fmaxf(v[i], 0.0f), inv, acc[i]);
        }
      }
      if (biased) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if (W * i + g < a.E) v[i] += __ldg(a.bias + W * i + g);
        n = candidates<W, NL>(v, a.k, true, lane, list, most);
      }
      if (kStats) live_tokens += n > 0 ? 1 : 0;
      // Candidates of this lane: expert, logit, score, and place among them all.
      int mine[kPerLane], slot[kPerLane];
      float zm[kPerLane], sm[kPerLane];
      const bool two = kPerLane > 1 && __any_sync(kFull, n > W);
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) {
        mine[r] = -1;
        slot[r] = a.k;
        zm[r] = sm[r] = 0.0f;
        if (r == 0 || two) {
          const int c = W * r + g;
          uint64_t key = 0;
          if (c < n) {
            mine[r] = list[c];
            zm[r] = load_logit(a.logits, a.bf16, t * a.ld + mine[r]);
            if (kScore == 1) sm[r] = sigmoid(zm[r]);
            const uint32_t high = order_key(biased ? sm[r] + __ldg(a.bias + mine[r]) : zm[r]);
            key = static_cast<uint64_t>(high) << 32 | (0xffffffffu - static_cast<uint32_t>(mine[r]));
            slot[r] = 0;
          }
          order[c] = key;
        }
      }
      __syncwarp();
      const int most_n = two ? 32 : min(32, static_cast<int>(__reduce_max_sync(kFull, static_cast<uint32_t>(n))));
      {
        const uint64_t own0 = order[g], own1 = two ? order[W * (kPerLane - 1) + g] : 0;
        int rank0 = 0, rank1 = 0;
        for (int o = 0; o < most_n; o += 2) {   // the orders past n are 0, below every candidate's
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(order + o);
          rank0 += (x.x > own0 ? 1 : 0) + (x.y > own0 ? 1 : 0);
          if (two) rank1 += (x.x > own1 ? 1 : 0) + (x.y > own1 ? 1 : 0);
        }
        if (mine[0] >= 0) slot[0] = rank0;
        if (kPerLane > 1 && mine[kPerLane - 1] >= 0 && two) slot[kPerLane - 1] = rank1;
      }
      if (__any_sync(kFull, n > 32)) {
        // Too many for one group or both: the k largest one by one from the keys
        // themselves; lane j keeps the j-th.
        const bool many = n > 32;
        uint32_t key[NL];
        load_token<W, NL>(a, here ? t : lo, g, many ? a.E : 0, v);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          float x = v[i];
          if (biased && eligible(x)) x = sigmoid(x) + __ldg(a.bias + W * i + g);
          key[i] = eligible(v[i]) ? order_key(x) : 0u;
        }
        for (int j = 0; j < a.k; ++j) {
          uint32_t m = key[0];
#pragma unroll
          for (int i = 1; i < NL; ++i) m = max(m, key[i]);
          m = group_max<W>(m);   // 0 only where not `many`: more than 32 are eligible, and k <= 32
          uint32_t cand = 0xffffffffu;
#pragma unroll
          for (int i = NL - 1; i >= 0; --i)
            if (key[i] == m) cand = static_cast<uint32_t>(W * i + g);
          const uint32_t e = group_min<W>(cand);
#pragma unroll
          for (int i = 0; i < NL; ++i)
            if (e == static_cast<uint32_t>(W * i + g)) key[i] = 0u;
          if (many && g == j) mine[0] = static_cast<int>(e);
        }
        if (many) {
          slot[0] = g;
          if (kPerLane > 1) slot[kPerLane - 1] = a.k;
          if (g < a.k) {
            zm[0] = load_logit(a.logits, a.bf16, t * a.ld + mine[0]);
            if (kScore == 1) sm[0] = sigmoid(zm[0]);
          }
        }
      }
      // normalised softmax weights need no sum over the experts not chosen
      float chosen = 0.0f;
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) {
        if (slot[r] < a.k) {
          if (kScore == 0) sm[r] = expf(zm[r] - top);
          chosen += sm[r];
        }
      }
      // a sigmoid is a weight as it stands
      const float unit = a.normalize ? a.scale / (group_sum<W>(chosen) + kScoreEps) : kScore == 0 ? a.scale / total : a.scale;
      if (here) {
#pragma unroll
        for (int r = 0; r < kPerLane; ++r) {
          if (slot[r] < a.k) {
            a.idx[t * a.k + slot[r]] = mine[r];
            a.w[t * a.k + slot[r]] = sm[r] * unit;
            if (kStats) atomicAdd(&s_n[mine[r]], 1);
          }
        }
        if (g >= n && g < a.k) {   // slots that find no eligible expert
          a.idx[t * a.k + g] = -1;
          a.w[t * a.k + g] = 0.0f;
        }
      }
      __syncwarp();   // the lists are read before the next token's go in
    }
    if (kStats) {
#pragma unroll
      for (int i = 0; i < NL; ++i) s_p[group * W * NL + W * i + g] = acc[i];
      live_tokens = __reduce_add_sync(kFull, g == 0 ? live_tokens : 0);
      if (lane == 0) s_t[warp] = live_tokens;
      __syncthreads();
      const int64_t row = static_cast<int64_t>(blockIdx.x) + s;
      for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kGroups; ++r) sum += s_p[r * W * NL + e];
        a.part_p[row * a.E + e] = sum;
        a.part_n[row * a.E + e] = s_n[e];
      }
      if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < kRouteWarps; ++w) n += s_t[w];
        a.part_t[row] = n;
      }
      __syncthreads();
    }
    lo = end;
    if (kStats && lo < hi) {
      s = next_sequence(a, s, lo);
      if (s >= a.S) break;
    }
  }
}

// Sums the partial rows of a sequence for 32 experts (32 threads share an
// expert, each taking every 32nd chunk), writes its counts and tokens, and
// leaves the slice's share of the loss; the last CTA to finish adds the
// shares in their order.  About 3 us behind the router.
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads) route_finish_kernel(const RouteArgs a) {
  __shared__ float s_p[32][33];
  __shared__ int s_n[32][33];
  __shared__ int s_t[32];
  __shared__ bool s_last;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
  const int64_t lo = a.seq == nullptr ? 0 : a.seq[s], hi = sequence_end(a, s);
  float p = 0.0f;
  int n = 0, tokens = 0;
  if (lo < hi && lo >= 0 && hi <= a.T) {   // the bounds hold for valid sequences
    const int64_t c0 = lo / a.chunk, c1 = (hi - 1) / a.chunk;
    for (int64_t c = c0 + grp; c <= c1; c += 32) {
      const int64_t row = c + s;
      if (e < a.E) {
        p += a.part_p[row * a.E + e];
        n += a.part_n[row * a.E + e];
      }
      tokens += a.part_t[row];
    }
  }
  s_p[grp][lane] = p;
  s_n[grp][lane] = n;
  if (lane == 0) s_t[grp] = tokens;
  __syncthreads();
  if (grp == 0) {
    p = 0.0f;
    n = 0;
    tokens = 0;
    for (int r = 0; r < 32; ++r) {
      p += s_p[r][lane];
      n += s_n[r][lane];
      tokens += s_t[r];
    }
    if (e < a.E) a.counts[static_cast<int64_t>(s) * a.E + e] = n;
    if (blockIdx.x == 0 && lane == 0) a.tokens[s] = tokens;
    const float per = 1.0f / static_cast<float>(max(tokens, 1));
    const float share = warp_sum(e < a.E ? static_cast<float>(n) * per * (p * per) : 0.0f);
    if (lane == 0) {
      a.share[static_cast<int64_t>(s) * gridDim.x + blockIdx.x] = share;
      __threadfence();
      s_last = atomicAdd(a.done, 1) == static_cast<int>(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const int64_t total = static_cast<int64_t>(gridDim.x) * gridDim.y;
  float sum = 0.0f;
  for (int64_t i = threadIdx.x; i < total; i += kFinishThreads) sum += __ldcg(a.share + i);
  sum = warp_sum(sum);
  if (lane == 0) s_p[0][grp] = sum;
  __syncthreads();
  if (grp == 0) {
    sum = warp_sum(s_p[0][lane]);
    if (lane == 0) *a.loss = sum * (static_cast<float>(a.E) / static_cast<float>(a.k)) * (a.alpha / static_cast<float>(a.S));
  }
}

// CTAs on an SM, more of them against more registers a thread: 131072 tokens of
// 256 logits 65.6 us with four, 72.4 with three; of 128 logits (half a warp a
// token) 40.6 and 36.6.
template <int W, int NL>
constexpr int kBackwardCtas = NL <= 4 ? 4 : NL == 8 ? (W == 32 ? 4 : 3) : NL == 16 ? 2 : 1;

// d logits from the gradients of the gate weights and of the balance loss.
// With g_i = d loss / d p_i (the sequence's constants) and d_j the gradients
// of the chosen scores,
//   softmax: dz_i = p_i (g_i + d_i - sum_l p_l (g_l + d_l))
//   sigmoid: dz_i = s_i (1 - s_i) (d_i + (g_i - sum_l p_l g_l) / sum_l s_l).
// Every lane first stores its experts' dz without d_i; the lanes that hold the
// token's choices then store theirs whole over those k.
// Reads and writes T E values: 268 MB for 131072 tokens of 256, 40 us at the
// copy bandwidth; 66 us measured, instructions (about 400 a token) and loads
// waited for in equal parts.
template <int W, int NL, int kScore>
__global__ void __launch_bounds__(kRouteThreads, kBackwardCtas<W, NL>) route_backward_kernel(const RouteArgs a) {
  constexpr int kGroups = kRouteThreads / W;
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = threadIdx.x & (W - 1);
  check_sequences(a);
  const int64_t hi = min(a.T, static_cast<int64_t>(blockIdx.x + 1) * a.chunk);
  int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  int s = lo < hi ? sequence_of(a, lo) : 0;
  const float up = a.dloss == nullptr ? 0.0f
                                      : __ldg(a.dloss) * (a.alpha / static_cast<float>(a.S)) *
                                            (static_cast<float>(a.E) / static_cast<float>(a.k));
  while (lo < hi) {
    const int64_t end = min(hi, sequence_end(a, s));
    if (end <= lo) break;   // invalid sequences
    const int32_t* counts = a.dloss == nullptr ? nullptr : a.counts + static_cast<int64_t>(s) * a.E;
    // g_i = count_i unit, taken from that of the mean count: the p_l sum to one
    // (but for the guard's share), so a part that all g_l share has no effect, and
    // the counts' differences are exact.  (From g_i itself the sum of p_l g_l kept
    // 2^-23 of it, 1.5e-3 of the gradient of loads a thousandth apart.)
    float unit = 0.0f;
    int mean = 0;
    if (counts != nullptr) {
      const float tokens = static_cast<float>(max(a.tokens[s], 1)), per = 1.0f / tokens;
      unit = up * per * per;
      mean = __float2int_rn(tokens * static_cast<float>(a.k) / static_cast<float>(a.E));
    }
    const float guard = kScore == 0 ? 0.0f : kScoreEps * (static_cast<float>(mean) * unit);   // softmax: the sum is 1 or more
    float coef[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i)
      coef[i] = counts != nullptr && W * i + g < a.E ? static_cast<float>(counts[W * i + g] - mean) * unit : 0.0f;
    // the mask, the choice and its gradient are read a step ahead, so that no
    // load of a step waits for another
    bool valid_next = false;
    int mine_next = -1;
    float dw_next = 0.0f;
    auto ahead = [&](int64_t t) {
      valid_next = t < end && (a.valid == nullptr || a.valid[t] != 0);
      mine_next = t < end && g < a.k ? a.idx[t * a.k + g] : -1;
      dw_next = t < end && g < a.k ? a.dw[t * a.k + g] : 0.0f;
    };
    ahead(lo + threadIdx.x / W);
    for (int64_t t0 = lo + warp * (32 / W); t0 < end; t0 += kGroups) {
      const int64_t t = t0 + lane / W;
      const bool here = t < end, valid = valid_next;
      const int mine = valid && mine_next >= 0 && mine_next < a.E ? mine_next : -1;
      const float dw = mine >= 0 ? dw_next : 0.0f;
      float zm = -INFINITY;
      ahead(t + kGroups);
      // softmax: v = e^(z - top), 0 where not eligible.  sigmoid: v = q (see
      // sigmoid_part) with the logit's sign, -0 where not eligible.
      float v[NL];
      load_token<W, NL>(a, here ? t : lo, g, valid ? a.E : 0, v);
      if (mine >= 0) zm = load_logit(a.logits, a.bf16, t * a.ld + mine);
      float top = 0.0f;
      if (kScore == 0) {
        top = v[0];
#pragma unroll
        for (int i = 1; i < NL; ++i) top = fmaxf(top, v[i]);   // ignores NaN
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      }
      float q[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) q[i] = v[i];
      in_pairs(q, [&](float2 z) { return kScore == 0 ? exp_pair(add2(z, both(-top))) : sigmoid_parts(z); });
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        float score;
        if (kScore == 0) {
          v[i] = score = fmaxf(q[i], 0.0f);   // 0 for NaN
        } else {
          score = v[i] >= 0.0f ? 1.0f - q[i] : q[i];
          v[i] = v[i] >= 0.0f ? q[i] : -q[i];
        }
        sum += score;
        dot = fmaf(coef[i], score, dot);
      }
      const float inv = fast_rcp(group_sum<W>(sum) + kScoreEps);
      float ws = 0.0f, slope = 0.0f;
      if (eligible(zm)) {
        if (kScore == 0) {
          ws = fmaxf(exp_one(zm - top), 0.0f) * inv;
        } else {
          const float q = sigmoid_part(zm);
          ws = zm >= 0.0f ? 1.0f - q : q;
          slope = q * (1.0f - q);
        }
      }
      float dws = a.scale * dw;
      if (a.normalize) {
        // d_j = scale / sum (dw_j - sum_l w_l dw_l), the w_l summing to one but for
        // the guard's share of the sum: taken from the first choice's dw, which
        // leaves nothing of a part that all dw share.  (From dw itself: a single
        // choice kept 2^-23 of its dw, more than the loss's gradient has digits.)
        const float first = __shfl_sync(kFull, dw, lane & ~(W - 1));
        const float r = fast_rcp(group_sum<W>(ws) + kScoreEps);
        const float d = dw - first, guard = kScoreEps * r;
        dws = a.scale * r * (d - group_sum<W>(d * ws) * r + (guard > 1e-7f ? first * guard : 0.0f));
      }
      dot *= inv;
      if (kScore == 0 && !a.normalize) dot = fmaf(dws, ws, dot);   // normalised: these add up to zero
      dot = group_sum<W>(dot);
      if (kScore == 1) dot = fmaf(-guard, inv, dot);
#pragma unroll
      for (int i = 0; i < NL; i += 2) {   // (coef - dot) inv q, sigmoid: times 1 - q
        const int j = i + 1 < NL ? i + 1 : i;
        const float2 q = make_float2(fabsf(v[i]), fabsf(v[j]));
        float2 x = mul2(mul2(add2(make_float2(coef[i], coef[j]), both(-dot)), both(inv)), q);
        if (kScore == 1) x = fma2(x, make_float2(-q.x, -q.y), x);
        v[i] = x.x;
        v[j] = x.y;
      }
      if (here) {
        if (a.bf16) {
          __nv_bfloat16* row = static_cast<__nv_bfloat16*>(a.dlogits) + t * a.ldd + g;
#pragma unroll
          for (int i = 0; i < NL; ++i)
            if (W * i + g < a.E) row[W * i] = __float2bfloat16_rn(v[i]);
        } else {
          float* row = static_cast<float*>(a.dlogits) + t * a.ldd + g;
#pragma unroll
          for (int i = 0; i < NL; ++i)
            if (W * i + g < a.E) row[W * i] = v[i];
        }
      }
      __syncwarp();   // orders the stores of one address
      if (mine >= 0) {
        const float gm = counts != nullptr ? static_cast<float>(__ldg(counts + mine) - mean) * unit : 0.0f;
        const float dz = kScore == 0 ? ws * (gm + dws - dot) : (dws + (gm - dot) * inv) * slope;
        if (a.bf16)
          static_cast<__nv_bfloat16*>(a.dlogits)[t * a.ldd + mine] = __float2bfloat16_rn(dz);
        else
          static_cast<float*>(a.dlogits)[t * a.ldd + mine] = dz;
      }
    }
    lo = end;
    if (lo < hi) {
      s = next_sequence(a, s, lo);
      if (s >= a.S) break;
    }
  }
}

// ------------------------------------------------------------------ layout
// A counting sort of the T k choices by expert, stable in token order.  The
// choices are cut into chunks of 2048, one CTA each: layout_count leaves the
// chunks' histograms; layout_scan turns them into the sums of the chunks before;
// layout_place ranks a chunk's choices (each warp its stretch, equal experts
// among 32 choices found with match_any, the warps' counts summed in order) and
// writes them.  A single chunk needs the last kernel alone; its CTAs all rank
// it, the first writes it, and they share the padding (up to 127 rows an
// expert: 256 tokens, 8 of 256 experts, took 9.1 us with one CTA, 5.8 with 16).
// A few chunks get CTAs that only fill, too.  Bound by latency: three launches
// and a few dependent reads, 15 us for 261992 choices (3 MB).
constexpr int kLayoutThreads = 512;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kChunkPairs = 2048;
constexpr int kWarpSteps = kChunkPairs / kLayoutThreads;   // choices of a lane
constexpr int kPadRows = 2048;                             // rows per CTA that helps to fill

__global__ void __launch_bounds__(kLayoutThreads) layout_count_kernel(const LayoutArgs a) {
  __shared__ int s_n[kMaxExperts];
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < a.E; e += kLayoutThreads) s_n[e] = 0;
  __syncthreads();
  griddep_wait();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * kChunkPairs;
#pragma unroll
  for (int j = 0; j < kWarpSteps; ++j) {
    const int64_t i = lo + j * kLayoutThreads + threadIdx.x;
    const int e = i < a.pairs ? a.idx[i] : -1;
    if (e >= 0 && e < a.E) atomicAdd(&s_n[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kLayoutThreads)
    a.hist[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_n[e];
}

// Turns the chunks' histograms hist[c][e] into the sums of the chunks before,
// and leaves the totals in hist[chunks][e].  A CTA per 32 experts; its warps
// share the chunks.
constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanBatch = 8;   // loads in flight
__global__ void __launch_bounds__(kScanThreads) layout_scan_kernel(const LayoutArgs a, int chunks) {
  __shared__ int s_sum[kScanWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = blockIdx.x * 32 + lane;
  const int per = (chunks + kScanWarps - 1) / kScanWarps;
  const int c0 = min(chunks, warp * per), c1 = min(chunks, c0 + per);
  int sum = 0;
  for (int c = c0; c < c1; c += kScanBatch) {
#pragma unroll
    for (int i = 0; i < kScanBatch; ++i) sum += c + i < c1 && e < a.E ? a.hist[static_cast<int64_t>(c + i) * a.E + e] : 0;
  }
  s_sum[warp][lane] = sum;
  __syncthreads();
  int run = 0;
#pragma unroll
  for (int w = 0; w < kScanWarps; ++w) run += w < warp ? s_sum[w][lane] : 0;
  if (e < a.E) {
    for (int c = c0; c < c1; c += kScanBatch) {
      int v[kScanBatch];
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) v[i] = c + i < c1 ? a.hist[static_cast<int64_t>(c + i) * a.E + e] : 0;
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) {
        if (c + i < c1) a.hist[static_cast<int64_t>(c + i) * a.E + e] = run;
        run += v[i];
      }
    }
    if (warp == kScanWarps - 1) a.hist[static_cast<int64_t>(chunks) * a.E + e] = run;
  }
}

__global__ void __launch_bounds__(kLayoutThreads) layout_place_kernel(const LayoutArgs a, int chunks) {
  __shared__ uint16_t s_w[kLayoutWarps][kMaxExperts];   // counts of a warp, then of the warps before it
  __shared__ int s_base[kMaxExperts];                   // first row of an expert
  __shared__ int s_total[kMaxExperts];                  // choices of an expert
  __shared__ int s_before[kMaxExperts];                 // choices of it in earlier chunks
  __shared__ int s_scan[kLayoutWarps];
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = lane; e < a.E; e += 32) s_w[warp][e] = 0;
  __syncwarp();
  griddep_wait();
  const int64_t lo = static_cast<int64_t>(chunks > 1 ? blockIdx.x : 0) * kChunkPairs + warp * (kChunkPairs / kLayoutWarps) + lane;
  int e[kWarpSteps], before[kWarpSteps];   // expert; choices of it earlier in the warp's stretch
#pragma unroll
  for (int j = 0; j < kWarpSteps; ++j) {
    e[j] = lo + 32 * j < a.pairs ? a.idx[lo + 32 * j] : -1;
    if (e[j] < 0 || e[j] >= a.E) e[j] = -1;
  }
  if (chunks > 1) {
    for (int x = threadIdx.x; x < a.E; x += kLayoutThreads) {
      s_before[x] = a.hist[static_cast<int64_t>(min(static_cast<int>(blockIdx.x), chunks)) * a.E + x];
      s_total[x] = a.hist[static_cast<int64_t>(chunks) * a.E + x];
    }
  }
#pragma unroll
  for (int j = 0; j < kWarpSteps; ++j) {
    const uint32_t same = __match_any_sync(kFull, e[j]);
    const int seen = e[j] >= 0 ? s_w[warp][e[j]] : 0;
    before[j] = seen + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e[j] >= 0 && lane == __ffs(same) - 1) s_w[warp][e[j]] = static_cast<uint16_t>(seen + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int x = threadIdx.x; x < a.E; x += kLayoutThreads) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kLayoutWarps; ++w) {
      const int n = s_w[w][x];
      s_w[w][x] = static_cast<uint16_t>(run);
      run += n;
    }
    if (chunks == 1) {
      s_before[x] = 0;
      s_total[x] = run;
    }
  }
  __syncthreads();
  // first rows: exclusive sum of the padded counts, two experts per thread
  const int e0 = 2 * threadIdx.x;
  const int p0 = e0 < a.E ? (s_total[e0] + 127) / 128 * 128 : 0;
  const int p1 = e0 + 1 < a.E ? (s_total[e0 + 1] + 127) / 128 * 128 : 0;
  int x = p0 + p1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_scan[warp] = x;
  __syncthreads();
  int first = x - p0 - p1, end = 0;
#pragma unroll
  for (int w = 0; w < kLayoutWarps; ++w) {
    if (w < warp) first += s_scan[w];
    end += s_scan[w];
  }
  if (e0 < a.E) s_base[e0] = first;
  if (e0 + 1 < a.E) s_base[e0 + 1] = first + p0;
  __syncthreads();
  // padding: a warp per expert, the experts dealt over the CTAs' warps; then the rows past the segments
  for (int y = blockIdx.x * kLayoutWarps + warp; y < a.E; y += gridDim.x * kLayoutWarps) {
    const int from = s_base[y] + s_total[y], to = s_base[y] + (s_total[y] + 127) / 128 * 128;
    for (int r = from + lane; r < to; r += 32) a.row_token[r] = -1;
  }
  for (int64_t r = end + static_cast<int64_t>(blockIdx.x) * kLayoutThreads + threadIdx.x; r < a.rows;
       r += static_cast<int64_t>(gridDim.x) * kLayoutThreads)
    a.row_token[r] = -1;
  if (blockIdx.x == 0) {
    for (int y = threadIdx.x; y < a.E; y += kLayoutThreads) a.offsets[y] = s_base[y];
    if (threadIdx.x == 0) a.offsets[a.E] = end;
  }
  if (chunks == 1 && blockIdx.x != 0) return;
#pragma unroll
  for (int j = 0; j < kWarpSteps; ++j) {
    const int64_t i = lo + 32 * j;
    int row = -1;
    if (e[j] >= 0) {
      row = s_base[e[j]] + s_before[e[j]] + s_w[warp][e[j]] + before[j];
      a.row_token[row] = static_cast<int32_t>(i / a.k);
    }
    if (i < a.pairs) a.row_of[i] = row;
  }
}

unsigned route_grid(const RouteArgs& a) {
  return static_cast<unsigned>(std::max<int64_t>(1, (a.T + a.chunk - 1) / a.chunk));
}

template <int W, int NL>
cudaError_t run_forward(const RouteArgs& a, cudaStream_t stream) {
  const unsigned grid = route_grid(a);
  if (a.loss != nullptr)
    return a.score == 0 ? launch_behind(route_kernel<W, NL, 0, true>, grid, kRouteThreads, stream, a)
                        : launch_behind(route_kernel<W, NL, 1, true>, grid, kRouteThreads, stream, a);
  return a.score == 0 ? launch_behind(route_kernel<W, NL, 0, false>, grid, kRouteThreads, stream, a)
                      : launch_behind(route_kernel<W, NL, 1, false>, grid, kRouteThreads, stream, a);
}

template <int W, int NL>
cudaError_t run_route(RouteArgs a, bool backward, cudaStream_t stream) {
  if (!backward) return run_forward<W, NL>(a, stream);
  // one wave: a CTA looks up its sequence and that one's counts first
  constexpr int64_t kCtas = 152 * kBackwardCtas<W, NL>;
  a.chunk = std::max<int64_t>(8, (a.T + kCtas - 1) / kCtas);
  return a.score == 0 ? launch_behind(route_backward_kernel<W, NL, 0>, route_grid(a), kRouteThreads, stream, a)
                      : launch_behind(route_backward_kernel<W, NL, 1>, route_grid(a), kRouteThreads, stream, a);
}

cudaError_t pick_route(const RouteArgs& a, bool backward, cudaStream_t stream) {
  // Half a warp per token where k lanes can reach the candidates' bound; the
  // backward pass has less to share and needs more registers (131072 tokens of
  // 256 logits: 66.8 us with half a warp, 65.6 with a whole one; BF16 63.2 and
  // 65.0).
  if (a.k <= 16) {
    if (a.E <= 16) return run_route<16, 1>(a, backward, stream);
    if (a.E <= 32) return run_route<16, 2>(a, backward, stream);
    if (a.E <= 64) return run_route<16, 4>(a, backward, stream);
    if (a.E <= 128) return run_route<16, 8>(a, backward, stream);
    if (a.E <= 256 && !backward) return run_forward<16, 16>(a, stream);
  }
  if (a.E <= 64) return run_route<32, 2>(a, backward, stream);
  if (a.E <= 256) return run_route<32, 8>(a, backward, stream);
  if (a.E <= 512) return run_route<32, 16>(a, backward, stream);
  return run_route<32, 32>(a, backward, stream);
}

// Tokens per CTA with statistics: as many CTAs as are resident at once (131072
// tokens of 128 logits: 52.5 us with 608, 60.3 with 456), and at most 30 + T / 64
// (the partial sums stay small beside the logits).
constexpr int kMaxChunks = 456;
int64_t stats_chunk(int64_t T, int E) {
  const int64_t resident = E <= 128 ? 152 * 4 : kMaxChunks;
  const int64_t chunks = std::min<int64_t>(resident, 30 + T / 64);
  return std::max<int64_t>(8, (T + chunks - 1) / chunks);
}
// Without: at most 64, so that the last CTAs to start are short.
int64_t plain_chunk(int64_t T) {
  return std::min<int64_t>(64, std::max<int64_t>(16, (T / kMaxChunks + 15) / 16 * 16));
}

int64_t layout_chunks(int64_t pairs) { return std::max<int64_t>(1, (pairs + kChunkPairs - 1) / kChunkPairs); }

}  // namespace

int64_t route_workspace_bytes(int64_t T, int E, int64_t S) {
  const int64_t chunk = stats_chunk(T, E), rows = (T + chunk - 1) / chunk + S;
  const int64_t slices = (E + 31) / 32;
  return 4 * (rows * (2 * static_cast<int64_t>(E) + 1) + slices * S + 1);
}

cudaError_t launch_route(RouteArgs a, void* ws, cudaStream_t stream) {
  a.chunk = a.loss == nullptr ? plain_chunk(a.T) : stats_chunk(a.T, a.E);
  if (a.loss == nullptr) return pick_route(a, false, stream);
  const int64_t rows = (a.T + a.chunk - 1) / a.chunk + a.S;
  a.part_p = static_cast<float*>(ws);
  a.part_n = reinterpret_cast<int32_t*>(a.part_p + rows * a.E);
  a.part_t = a.part_n + rows * a.E;
  const unsigned slices = static_cast<unsigned>((a.E + 31) / 32);
  a.share = reinterpret_cast<float*>(a.part_t + rows);
  a.done = reinterpret_cast<int32_t*>(a.share + static_cast<int64_t>(slices) * a.S);
  const cudaError_t e = pick_route(a, false, stream);
  if (e != cudaSuccess) return e;
  return launch_behind(route_finish_kernel, dim3(slices, static_cast<unsigned>(a.S)), kFinishThreads, stream, a);
}

cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t stream) { return pick_route(a, true, stream); }

int64_t layout_workspace_bytes(int64_t T, int k, int E) {
  const int64_t chunks = layout_chunks(T * k);
  return chunks > 1 ? 4 * (chunks + 1) * E : 4;
}

cudaError_t launch_layout(const LayoutArgs& a, cudaStream_t stream) {
  const int chunks = static_cast<int>(layout_chunks(a.pairs));
  if (chunks > 1) {
    cudaError_t e = launch_behind(layout_count_kernel, static_cast<unsigned>(chunks), kLayoutThreads, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_behind(layout_scan_kernel, static_cast<unsigned>((a.E + 31) / 32), kScanThreads, stream, a, chunks);
    if (e != cudaSuccess) return e;
  }
  const int64_t fill = std::min<int64_t>(16, a.rows / kPadRows);
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(chunks, fill));
  return launch_behind(layout_place_kernel, grid, kLayoutThreads, stream, a, chunks);
}

cudaError_t route_take_status(int* status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_route_status, sizeof(int));
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_route_status, &zero, sizeof(int));
  }
  *status = v;
  return e;
}

}  // namespace fp8bs
