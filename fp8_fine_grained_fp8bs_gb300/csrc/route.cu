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
// One warp per token: expert e is held by lane e % 32 in register e / 32, so
// a lane sees the same experts in every token, and the sums of p over a
// warp's tokens stay in registers.  Sums over tokens are taken in a fixed
// order (lane, warp, chunk of tokens), counts with integer additions, so
// results do not vary from run to run.
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
constexpr int kMaxChunks = 608;        // chunks of tokens: four CTAs on each of 152 SMs
constexpr float kScoreEps = 1e-20f;    // guards the sums that scores are divided by
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

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

// One token's logits in registers: z[i] is expert 32 i + lane, -inf past E.
template <int NL>
__device__ __forceinline__ void load_token(const RouteArgs& a, int64_t t, int lane, float (&z)[NL]) {
  if (a.bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + t * a.ld + lane;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      z[i] = 32 * i + lane < a.E ? __uint_as_float(static_cast<uint32_t>(__ldg(p + 32 * i)) << 16) : -INFINITY;
  } else {
    const float* p = static_cast<const float*>(a.logits) + t * a.ld + lane;
#pragma unroll
    for (int i = 0; i < NL; ++i) z[i] = 32 * i + lane < a.E ? __ldg(p + 32 * i) : -INFINITY;
  }
}

// e^x and 1 / x by the hardware's base-2 exponential and reciprocal, for the
// scores that only enter sums and gradients (relative error below 2^-21 where
// the result matters); the weights and biased keys use expf and IEEE division.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// sigmoid(z) and its derivative from t = e^-|z|, which cannot overflow.
__device__ __forceinline__ float fast_sigmoid(float z, float& slope) {
  const float t = fast_exp(-fabsf(z)), r = fast_rcp(1.0f + t);
  slope = t * r * r;
  return z >= 0.0f ? r : t * r;
}

// Scores of a token up to a common factor, 0 where not eligible: e^(z - top)
// with top the maximum over all lanes, or sigmoid(z) (and its derivative in
// slope).  Returns 1 / (their sum + eps); p_i is s[i] times that.
template <int NL, int kScore>
__device__ __forceinline__ float scores_of(const float (&z)[NL], float top, float (&s)[NL], float (&slope)[NL]) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const float v = kScore == 0 ? fast_exp(z[i] - top) : fast_sigmoid(z[i], slope[i]);
    s[i] = fmaxf(v, 0.0f);   // NaN logits (and -inf where all are) count as 0
    sum += s[i];
  }
  return fast_rcp(warp_sum(sum) + kScoreEps);
}
template <int NL>
__device__ __forceinline__ float token_max(const float (&z)[NL]) {
  float top = z[0];
#pragma unroll
  for (int i = 1; i < NL; ++i) top = fmaxf(top, z[i]);   // ignores NaN
  return warp_max(top);
}

// The sequences of a launch: [seq[s], seq[s + 1]) covers 0 .. T in order.
__device__ __forceinline__ bool sequences_ok(const RouteArgs& a) {
  if (a.seq == nullptr) return true;
  bool bad = false;
  for (int s = threadIdx.x; s <= a.S; s += blockDim.x) {
    const int32_t o = a.seq[s];
    bad |= s == 0 ? o != 0 : o < a.seq[s - 1];
    bad |= s == a.S && o != a.T;
  }
  const bool ok = __syncthreads_or(bad) == 0;
  if (!ok && threadIdx.x == 0) record_route_status(kStatusDeviceArg);
  return ok;
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

// Candidates for the k largest of a warp's keys key[i] (expert 32 i + lane;
// -inf or NaN where not eligible), at least `slack` below the k-th largest
// lane maximum: no key among the k largest is below that maximum, since k
// lanes hold one that is not.  Of 256 random keys and k = 8 about nine pass,
// so the exact order is worked out on one key per lane.  Leaves the
// candidates' experts in `list` (lanes' first ones before their second ones)
// and returns their number, which may be above 32 (ties, few lanes): only the
// first 32 are in the list then.
template <int NL>
__device__ __forceinline__ int candidates(const float (&key)[NL], int k, bool slack, int lane, uint16_t* list) {
  float m = key[0];
#pragma unroll
  for (int i = 1; i < NL; ++i) m = fmaxf(m, key[i]);
  uint32_t cur = eligible(m) ? order_key(m) : 0u;
  uint32_t t = 0;
  int seen = 0;
  while (seen < k) {
    t = __reduce_max_sync(kFull, cur);
    if (t == 0u) break;       // fewer than k lanes hold an eligible key: all keys are candidates
    const bool at = cur == t;
    seen += __popc(__ballot_sync(kFull, at));
    if (at) cur = 0u;
  }
  constexpr float kLowest = -3.402823466e38f;
  float bound = t == 0u ? kLowest : __uint_as_float((t >> 31) != 0u ? t ^ 0x80000000u : ~t);
  if (slack) bound = fmaxf(bound - (1e-5f + 1e-6f * fabsf(bound)), kLowest);
  uint32_t mask = 0;
#pragma unroll
  for (int i = 0; i < NL; ++i) mask |= key[i] >= bound ? 1u << i : 0u;
  int n = 0;
  const uint32_t below = (1u << lane) - 1u;
  uint32_t who = __ballot_sync(kFull, mask != 0u);
  while (who != 0u) {
    const int at = n + __popc(who & below);
    if (mask != 0u && at < 32) list[at] = static_cast<uint16_t>(32 * (__ffs(mask) - 1) + lane);
    mask &= mask - 1u;
    n += __popc(who);
    who = __ballot_sync(kFull, mask != 0u);
  }
  __syncwarp();
  return n;
}

// CTAs that an SM should hold, which bounds the registers of a thread.
template <int NL>
constexpr int kRouteCtas = NL <= 8 ? 4 : NL == 16 ? 2 : 1;

// CTA c routes tokens [c * chunk, (c + 1) * chunk).  With statistics, each
// stretch of one sequence inside the chunk leaves its sums in row c + s of
// the partial arrays: along the tokens every step from one (chunk, sequence)
// to the next raises c or s, so the rows are distinct.
//
// Bound by instructions: see ROUTE_NOTE
template <int NL, int kScore, bool kStats>
__global__ void __launch_bounds__(kRouteThreads, kRouteCtas<NL>) route_kernel(const RouteArgs a) {
  __shared__ float s_p[kStats ? kRouteWarps * 32 * NL : 1];
  __shared__ int s_n[kStats ? 32 * NL : 1];
  __shared__ int s_t[kRouteWarps];
  __shared__ uint16_t s_list[kRouteWarps][32];
  __shared__ uint64_t s_order[kRouteWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (kStats) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
    if (!sequences_ok(a)) return;
  }
  const bool biased = kScore == 1 && a.bias != nullptr;
  const int64_t hi = min(a.T, static_cast<int64_t>(blockIdx.x + 1) * a.chunk);
  int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  int s = kStats && lo < hi ? sequence_of(a, lo) : 0;
  while (lo < hi) {
    const int64_t end = kStats ? min(hi, sequence_end(a, s)) : hi;
    float acc[NL];
    int live_tokens = 0;
    if (kStats) {
#pragma unroll
      for (int i = 0; i < NL; ++i) acc[i] = 0.0f;
      for (int e = threadIdx.x; e < a.E; e += kRouteThreads) s_n[e] = 0;
      __syncthreads();
    }
    for (int64_t t = lo + warp; t < end; t += kRouteWarps) {
      int32_t* idx = a.idx + t * a.k;
      float* wt = a.w + t * a.k;
      if (a.valid != nullptr && a.valid[t] == 0) {
        if (lane < a.k) {
          idx[lane] = -1;
          wt[lane] = 0.0f;
        }
        continue;
      }
      float z[NL], sc[NL];
      load_token<NL>(a, t, lane, z);
      // scores of all experts: for the statistics, for softmax weights that are
      // not normalised over the chosen, and (approximate) for biased keys
      float top = 0.0f, inv = 1.0f;
      const bool all = kStats || biased || (kScore == 0 && !a.normalize);
      if (all) {
        float slope[NL];
        if (kScore == 0) top = token_max(z);
        inv = scores_of<NL, kScore>(z, top, sc, slope);
      }
      int n;
      if (biased) {
        float key[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i)   // z * 0 is NaN for the infinities and NaN: not eligible
          key[i] = fmaf(z[i], 0.0f, sc[i] + (32 * i + lane < a.E ? __ldg(a.bias + 32 * i + lane) : 0.0f));
        n = candidates<NL>(key, a.k, true, lane, s_list[warp]);
      } else {
        n = candidates<NL>(z, a.k, false, lane, s_list[warp]);
      }
      if (kStats) {
        live_tokens += n > 0 ? 1 : 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) acc[i] += sc[i] * inv;
      }
      // one candidate per lane and its place among them; mine: its expert
      int mine = -1, slot = lane;
      float zm = -INFINITY, sm = 0.0f;   // its logit, its score (softmax: below)
      if (n <= 32) {
        uint64_t order = 0;
        if (lane < n) {
          mine = s_list[warp][lane];
          zm = load_logit(a.logits, a.bf16, t * a.ld + mine);
          if (kScore == 1) sm = sigmoid(zm);
          const uint32_t key = order_key(biased ? sm + __ldg(a.bias + mine) : zm);
          order = static_cast<uint64_t>(key) << 32 | (0xffffffffu - static_cast<uint32_t>(mine));
          slot = 0;
        }
        s_order[warp][lane] = order;
        __syncwarp();
        for (int o = 0; o < n; ++o) slot += s_order[warp][o] > order ? 1 : 0;
        if (lane >= n) slot = lane;
      } else {
        // too many: the k largest one by one; lane j keeps the j-th
        uint32_t key[NL];
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          float v = z[i];
          if (biased && eligible(v)) v = sigmoid(v) + __ldg(a.bias + 32 * i + lane);
          key[i] = eligible(z[i]) ? order_key(v) : 0u;
        }
        for (int j = 0; j < a.k; ++j) {
          uint32_t m = key[0];
#pragma unroll
          for (int i = 1; i < NL; ++i) m = max(m, key[i]);
          m = __reduce_max_sync(kFull, m);   // never 0: more than 32 are eligible, and k <= 32
          uint32_t cand = 0xffffffffu;
#pragma unroll
          for (int i = NL - 1; i >= 0; --i)
            if (key[i] == m) cand = 32u * i + lane;
          const uint32_t e = __reduce_min_sync(kFull, cand);
#pragma unroll
          for (int i = 0; i < NL; ++i)
            if (e == 32u * i + lane) key[i] = 0u;
          if (lane == j) mine = static_cast<int>(e);
        }
        if (lane < a.k) {
          zm = load_logit(a.logits, a.bf16, t * a.ld + mine);
          if (kScore == 1) sm = sigmoid(zm);
        }
      }
      if (slot >= a.k) mine = -1;
      // normalised softmax weights need no sum over the experts not chosen
      if (kScore == 0) {
        if (!all) top = warp_max(mine >= 0 ? zm : -INFINITY);
        sm = expf(zm - top);
        if (!a.normalize) sm *= inv;
      }
      float w = mine >= 0 ? sm : 0.0f;
      if (a.normalize) w *= fast_rcp(warp_sum(w) + kScoreEps);
      if (slot < a.k) {
        idx[slot] = mine;
        wt[slot] = w * a.scale;
        if (kStats && mine >= 0) atomicAdd(&s_n[mine], 1);
      }
      __syncwarp();   // the lists are read before the next token's go in
    }
    if (kStats) {
#pragma unroll
      for (int i = 0; i < NL; ++i) s_p[warp * 32 * NL + 32 * i + lane] = acc[i];
      if (lane == 0) s_t[warp] = live_tokens;
      __syncthreads();
      const int64_t row = static_cast<int64_t>(blockIdx.x) + s;
      for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouteWarps; ++w) sum += s_p[w * 32 * NL + e];
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
    if (kStats)
      while (lo < hi && sequence_end(a, s) <= lo) ++s;   // empty sequences are passed over
  }
}

// Sums the partial rows of a sequence for 32 experts (32 threads share an
// expert, each taking every 32nd chunk), writes its counts and tokens, and
// leaves the slice's share of the loss; the last CTA to finish adds the
// shares in their order.
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads) route_finish_kernel(const RouteArgs a) {
  __shared__ float s_p[32][33];
  __shared__ int s_n[32][33];
  __shared__ int s_t[32];
  __shared__ bool s_last;
  griddep_launch_dependents();
  griddep_wait();
  if (!sequences_ok(a)) return;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
  const int64_t lo = a.seq == nullptr ? 0 : a.seq[s], hi = sequence_end(a, s);
  float p = 0.0f;
  int n = 0, tokens = 0;
  if (lo < hi) {
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

// d logits from the gradients of the gate weights and of the balance loss.
// With g_i = d loss / d p_i (the sequence's constants) and d_j the gradients
// of the chosen scores,
//   softmax: dz_i = p_i (g_i + d_i - sum_l p_l (g_l + d_l))
//   sigmoid: dz_i = s_i (1 - s_i) (d_i + (g_i - sum_l p_l g_l) / sum_l s_l).
// Every lane first stores its experts' dz without d_i; the lanes that hold the
// token's choices then store theirs whole over those k.
template <int NL, int kScore>
__global__ void __launch_bounds__(kRouteThreads, kRouteCtas<NL>) route_backward_kernel(const RouteArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!sequences_ok(a)) return;
  const int64_t hi = min(a.T, static_cast<int64_t>(blockIdx.x + 1) * a.chunk);
  int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  int s = lo < hi ? sequence_of(a, lo) : 0;
  const float up = a.dloss == nullptr ? 0.0f
                                      : __ldg(a.dloss) * (a.alpha / static_cast<float>(a.S)) *
                                            (static_cast<float>(a.E) / static_cast<float>(a.k));
  auto store = [&](int64_t at, float v) {
    if (a.bf16)
      static_cast<__nv_bfloat16*>(a.dlogits)[at] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(a.dlogits)[at] = v;
  };
  while (lo < hi) {
    const int64_t end = min(hi, sequence_end(a, s));
    const int32_t* counts = a.dloss == nullptr ? nullptr : a.counts + static_cast<int64_t>(s) * a.E;
    float unit = 0.0f;   // g_i per count
    if (counts != nullptr) {
      const float per = 1.0f / static_cast<float>(max(a.tokens[s], 1));
      unit = up * per * per;
    }
    float coef[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i)
      coef[i] = counts != nullptr && 32 * i + lane < a.E ? static_cast<float>(counts[32 * i + lane]) * unit : 0.0f;
    for (int64_t t = lo + warp; t < end; t += kRouteWarps) {
      if (a.valid != nullptr && a.valid[t] == 0) {
        for (int e = lane; e < a.E; e += 32) store(t * a.ldd + e, 0.0f);
        continue;
      }
      float z[NL], sc[NL], slope[NL];
      int mine = -1;
      float dw = 0.0f, zm = -INFINITY;
      if (lane < a.k) {
        const int e = a.idx[t * a.k + lane];
        if (e >= 0 && e < a.E) {
          mine = e;
          dw = a.dw[t * a.k + lane];
        }
      }
      load_token<NL>(a, t, lane, z);
      if (mine >= 0) zm = load_logit(a.logits, a.bf16, t * a.ld + mine);
      const float top = kScore == 0 ? token_max(z) : 0.0f;
      const float inv = scores_of<NL, kScore>(z, top, sc, slope);
      float ws = 0.0f, slope_m = 0.0f;
      if (eligible(zm)) ws = kScore == 0 ? fast_exp(zm - top) * inv : fast_sigmoid(zm, slope_m);
      float dws = a.scale * dw;
      if (a.normalize) {
        const float r = fast_rcp(warp_sum(ws) + kScoreEps);
        dws = a.scale * r * (dw - warp_sum(dw * ws) * r);
      }
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NL; ++i) dot += coef[i] * sc[i];
      dot *= inv;
      if (kScore == 0) dot += dws * ws;
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        float dz = kScore == 0 ? sc[i] * inv * (coef[i] - dot) : (coef[i] - dot) * inv * slope[i];
        dz = eligible(z[i]) ? dz : 0.0f;
        if (32 * i + lane < a.E) store(t * a.ldd + 32 * i + lane, dz);
      }
      __syncwarp();   // orders the stores of one address
      if (mine >= 0) {
        const float g = counts != nullptr ? static_cast<float>(__ldg(counts + mine)) * unit : 0.0f;
        const float dz = kScore == 0 ? ws * (g + dws - dot) : (dws + (g - dot) * inv) * slope_m;
        store(t * a.ldd + mine, eligible(zm) ? dz : 0.0f);
      }
    }
    lo = end;
    while (lo < hi && sequence_end(a, s) <= lo) ++s;
  }
}

// ------------------------------------------------------------------ layout
// A counting sort of the T k choices by expert, stable in token order.  The
// choices are cut into chunks of one CTA each: layout_count leaves the chunks'
// histograms, expert by expert; layout_scan, a warp per expert, turns each
// expert's into the sum of the chunks before; layout_place ranks a chunk's
// choices (each warp its stretch, equal experts among 32 choices found with
// match_any, the warps' counts summed in order) and writes them.  One chunk
// needs the last alone.
constexpr int kLayoutThreads = 512;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kChunkPairs = 2048;           // smallest chunk
constexpr int kMaxLayoutChunks = 512;

__global__ void __launch_bounds__(kLayoutThreads) layout_count_kernel(const LayoutArgs a) {
  __shared__ int s_n[kMaxExperts];
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < a.E; e += kLayoutThreads) s_n[e] = 0;
  __syncthreads();
  griddep_wait();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk, hi = min(a.pairs, lo + a.chunk);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kLayoutThreads) {
    const int e = a.idx[i];
    if (e >= 0 && e < a.E) atomicAdd(&s_n[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kLayoutThreads)
    a.hist[static_cast<int64_t>(e) * (gridDim.x + 1) + blockIdx.x] = s_n[e];
}

// hist[e][0 .. chunks): exclusive sums; hist[e][chunks]: the total.
__global__ void __launch_bounds__(32) layout_scan_kernel(const LayoutArgs a, int chunks) {
  griddep_launch_dependents();
  griddep_wait();
  int* h = a.hist + static_cast<int64_t>(blockIdx.x) * (chunks + 1);
  const int lane = threadIdx.x;
  constexpr int kPer = kMaxLayoutChunks / 32;
  int v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = 32 * i + lane < chunks ? h[32 * i + lane] : 0;
  int run = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (32 * i < chunks) {
      int x = v[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
      if (32 * i + lane < chunks) h[32 * i + lane] = run + x - v[i];
      run += __shfl_sync(kFull, x, 31);
    }
  }
  if (lane == 0) h[chunks] = run;
}

__global__ void __launch_bounds__(kLayoutThreads) layout_place_kernel(const LayoutArgs a) {
  __shared__ uint16_t s_w[kLayoutWarps][kMaxExperts];   // counts of a warp, then of the warps before it
  __shared__ int s_base[kMaxExperts];                   // first row of this chunk's choices
  __shared__ int s_total[kMaxExperts];                  // choices of an expert
  __shared__ int s_scan[kLayoutWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = gridDim.x;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t per_warp = (a.chunk + kLayoutWarps * 32 - 1) / (kLayoutWarps * 32) * 32;
  const int64_t wlo = lo + warp * per_warp;
  const int64_t whi = min(min(a.pairs, lo + a.chunk), wlo + per_warp);
  for (int e = lane; e < a.E; e += 32) s_w[warp][e] = 0;
  __syncwarp();
  // choices of this warp by expert
  for (int64_t i0 = wlo; i0 < whi; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = i < whi ? a.idx[i] : -1;
    const uint32_t same = __match_any_sync(kFull, e);
    if (e >= 0 && e < a.E && lane == __ffs(same) - 1) s_w[warp][e] += static_cast<uint16_t>(__popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kLayoutThreads) {
    int run = 0;
    for (int w = 0; w < kLayoutWarps; ++w) {
      const int n = s_w[w][e];
      s_w[w][e] = static_cast<uint16_t>(run);
      run += n;
    }
    const int* h = a.hist + static_cast<int64_t>(e) * (chunks + 1);
    s_base[e] = chunks > 1 ? h[blockIdx.x] : 0;
    s_total[e] = chunks > 1 ? h[chunks] : run;
  }
  __syncthreads();
  // first rows: exclusive sum of the padded counts, two experts per thread
  const int e0 = 2 * threadIdx.x;
  const int n0 = e0 < a.E ? s_total[e0] : 0, n1 = e0 + 1 < a.E ? s_total[e0 + 1] : 0;
  const int p0 = (n0 + 127) / 128 * 128, p1 = (n1 + 127) / 128 * 128;
  int x = p0 + p1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_scan[warp] = x;
  __syncthreads();
  int first = x - p0 - p1;
  for (int w = 0; w < warp; ++w) first += s_scan[w];
  int end = 0;
  for (int w = 0; w < kLayoutWarps; ++w) end += s_scan[w];
  if (e0 < a.E) s_base[e0] += first;
  if (e0 + 1 < a.E) s_base[e0 + 1] += first + p0;
  if (blockIdx.x == 0) {
    if (e0 < a.E) a.offsets[e0] = first;
    if (e0 + 1 < a.E) a.offsets[e0 + 1] = first + p0;
    if (threadIdx.x == 0) a.offsets[a.E] = end;
  }
  // padding rows: those of experts e = blockIdx.x, blockIdx.x + chunks, ... and the rows past the segments
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = e0 + j, f = j == 0 ? first : first + p0, n = j == 0 ? n0 : n1, p = j == 0 ? p0 : p1;
    if (e < a.E && e % chunks == static_cast<int>(blockIdx.x))
      for (int r = f + n; r < f + p; ++r) a.row_token[r] = -1;
  }
  for (int64_t r = end + static_cast<int64_t>(blockIdx.x) * kLayoutThreads + threadIdx.x; r < a.rows;
       r += static_cast<int64_t>(chunks) * kLayoutThreads)
    a.row_token[r] = -1;
  __syncthreads();
  // place: the running count of a warp moves on as its stretch is walked
  for (int64_t i0 = wlo; i0 < whi; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = i < whi ? a.idx[i] : -1;
    const uint32_t same = __match_any_sync(kFull, e);
    const bool ok = e >= 0 && e < a.E;
    int row = -1;
    if (ok) row = s_base[e] + s_w[warp][e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (ok && lane == __ffs(same) - 1) s_w[warp][e] += static_cast<uint16_t>(__popc(same));
    __syncwarp();
    if (i < whi) a.row_of[i] = row;
    if (ok) a.row_token[row] = static_cast<int32_t>(i / a.k);
  }
}

template <int NL>
cudaError_t run_route(const RouteArgs& a, bool backward, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, (a.T + a.chunk - 1) / a.chunk));
  if (backward)
    return a.score == 0 ? launch_behind(route_backward_kernel<NL, 0>, grid, kRouteThreads, stream, a)
                        : launch_behind(route_backward_kernel<NL, 1>, grid, kRouteThreads, stream, a);
  if (a.loss != nullptr)
    return a.score == 0 ? launch_behind(route_kernel<NL, 0, true>, grid, kRouteThreads, stream, a)
                        : launch_behind(route_kernel<NL, 1, true>, grid, kRouteThreads, stream, a);
  return a.score == 0 ? launch_behind(route_kernel<NL, 0, false>, grid, kRouteThreads, stream, a)
                      : launch_behind(route_kernel<NL, 1, false>, grid, kRouteThreads, stream, a);
}

cudaError_t pick_route(const RouteArgs& a, bool backward, cudaStream_t stream) {
  if (a.E <= 32) return run_route<1>(a, backward, stream);
  if (a.E <= 64) return run_route<2>(a, backward, stream);
  if (a.E <= 128) return run_route<4>(a, backward, stream);
  if (a.E <= 256) return run_route<8>(a, backward, stream);
  if (a.E <= 512) return run_route<16>(a, backward, stream);
  return run_route<32>(a, backward, stream);
}

// Tokens per CTA: at most 608 CTAs, and at most 24 + T / 64 (the partial sums
// stay small beside the logits).
int64_t route_chunk(int64_t T) {
  const int64_t chunks = std::min<int64_t>(kMaxChunks, 24 + T / 64);
  const int64_t c = (T + chunks - 1) / chunks;
  return std::max<int64_t>(kRouteWarps, (c + kRouteWarps - 1) / kRouteWarps * kRouteWarps);
}

int64_t layout_chunk(int64_t pairs) {
  const int64_t c = (pairs + kMaxLayoutChunks - 1) / kMaxLayoutChunks;
  return std::max<int64_t>(kChunkPairs, (c + kChunkPairs - 1) / kChunkPairs * kChunkPairs);
}

}  // namespace

int64_t route_workspace_bytes(int64_t T, int E, int64_t S) {
  const int64_t rows = (T + route_chunk(T) - 1) / route_chunk(T) + S;
  const int64_t slices = (E + 31) / 32;
  return 4 * (rows * (2 * static_cast<int64_t>(E) + 1) + slices * S + 1);
}

cudaError_t launch_route(RouteArgs a, void* ws, cudaStream_t stream) {
  a.chunk = route_chunk(a.T);
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

cudaError_t launch_route_backward(RouteArgs a, cudaStream_t stream) {
  a.chunk = route_chunk(a.T);
  return pick_route(a, true, stream);
}

int64_t layout_workspace_bytes(int64_t T, int k, int E) {
  const int64_t pairs = T * k, chunk = layout_chunk(pairs);
  const int64_t chunks = (pairs + chunk - 1) / chunk;
  return chunks > 1 ? 4 * (chunks + 1) * E : 4;
}

cudaError_t launch_layout(LayoutArgs a, cudaStream_t stream) {
  a.chunk = layout_chunk(a.pairs);
  const unsigned chunks = static_cast<unsigned>(std::max<int64_t>(1, (a.pairs + a.chunk - 1) / a.chunk));
  if (chunks > 1) {
    cudaError_t e = launch_behind(layout_count_kernel, chunks, kLayoutThreads, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_behind(layout_scan_kernel, static_cast<unsigned>(a.E), 32, stream, a, static_cast<int>(chunks));
    if (e != cudaSuccess) return e;
  }
  return launch_behind(layout_place_kernel, chunks, kLayoutThreads, stream, a);
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
