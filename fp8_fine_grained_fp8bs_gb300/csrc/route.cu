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
__device__ __forceinline__ void load_token(const RouteArgs& a, int64_t t, int lane, bool live, float (&z)[NL]) {
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = 32 * i + lane;
    z[i] = live && e < a.E ? load_logit(a.logits, a.bf16, t * a.ld + e) : -INFINITY;
  }
}

// Scores of a token (0 where not eligible) and their sum (+ eps).  softmax
// returns them normalised (and the sum 1), with the maximum and the inverse
// of the exponentials' sum, which the score of a single logit needs.
template <int NL, int kScore>
__device__ __forceinline__ float scores_of(const float (&z)[NL], float (&s)[NL], float& top, float& inv) {
  float sum = 0.0f;
  if (kScore == 0) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i) top = fmaxf(top, z[i]);   // fmaxf ignores NaN
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      s[i] = eligible(z[i]) ? expf(z[i] - top) : 0.0f;
      sum += s[i];
    }
    inv = 1.0f / (warp_sum(sum) + kScoreEps);
#pragma unroll
    for (int i = 0; i < NL; ++i) s[i] *= inv;
    return 1.0f;
  }
  top = 0.0f;
  inv = 1.0f;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    s[i] = eligible(z[i]) ? sigmoid(z[i]) : 0.0f;
    sum += s[i];
  }
  return warp_sum(sum) + kScoreEps;
}
template <int kScore>
__device__ __forceinline__ float score_of(float z, float top, float inv) {
  if (!eligible(z)) return 0.0f;
  return kScore == 0 ? expf(z - top) * inv : sigmoid(z);
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

// CTA c routes tokens [c * chunk, (c + 1) * chunk).  With statistics, each
// stretch of one sequence inside the chunk leaves its sums in row c + s of
// the partial arrays: along the tokens every step from one (chunk, sequence)
// to the next raises c or s, so the rows are distinct.
template <int NL, int kScore, bool kStats>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteArgs a) {
  __shared__ float s_p[kStats ? kRouteWarps * 32 * NL : 1];
  __shared__ int s_n[kStats ? 32 * NL : 1];
  __shared__ int s_t[kRouteWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (kStats) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.done = 0;
    if (!sequences_ok(a)) return;
  }
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
      float z[NL], sc[NL];
      load_token<NL>(a, t, lane, a.valid == nullptr || a.valid[t] != 0, z);
      float top = 0.0f, inv = 1.0f, all = 1.0f;
      if (kScore == 0 || kStats || a.bias != nullptr) all = scores_of<NL, kScore>(z, sc, top, inv);
      uint32_t key[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int e = 32 * i + lane;
        float v = z[i];
        if (kScore == 1 && a.bias != nullptr && e < a.E) v = sc[i] + __ldg(a.bias + e);
        key[i] = eligible(z[i]) ? order_key(v) : 0u;
      }
      if (kStats) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < NL; ++i) any |= key[i] != 0u;
        live_tokens += __any_sync(kFull, any) ? 1 : 0;
        const float r = 1.0f / all;
#pragma unroll
        for (int i = 0; i < NL; ++i) acc[i] += sc[i] * r;
      }
      int mine = -1;
      for (int j = 0; j < a.k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < NL; ++i) m = max(m, key[i]);
        m = __reduce_max_sync(kFull, m);
        if (m == 0u) break;   // no eligible expert is left
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
      float ws = 0.0f;
      if (mine >= 0) ws = score_of<kScore>(load_logit(a.logits, a.bf16, t * a.ld + mine), top, inv);
      float w = ws;
      if (a.normalize) w = ws / (warp_sum(ws) + kScoreEps);
      if (lane < a.k) {
        a.idx[t * a.k + lane] = mine;
        a.w[t * a.k + lane] = w * a.scale;
        if (kStats && mine >= 0) atomicAdd(&s_n[mine], 1);
      }
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
template <int NL, int kScore>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(const RouteArgs a) {
  __shared__ float s_d[kRouteWarps][32 * NL];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!sequences_ok(a)) return;
#pragma unroll
  for (int i = 0; i < NL; ++i) s_d[warp][32 * i + lane] = 0.0f;
  __syncwarp();
  const int64_t hi = min(a.T, static_cast<int64_t>(blockIdx.x + 1) * a.chunk);
  int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  int s = lo < hi ? sequence_of(a, lo) : 0;
  const float up = a.dloss == nullptr ? 0.0f
                                      : __ldg(a.dloss) * (a.alpha / static_cast<float>(a.S)) *
                                            (static_cast<float>(a.E) / static_cast<float>(a.k));
  while (lo < hi) {
    const int64_t end = min(hi, sequence_end(a, s));
    float coef[NL];   // d loss / d p of this sequence
    const float per = 1.0f / static_cast<float>(a.tokens != nullptr ? max(a.tokens[s], 1) : 1);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int e = 32 * i + lane;
      coef[i] = a.dloss != nullptr && e < a.E
                    ? static_cast<float>(a.counts[static_cast<int64_t>(s) * a.E + e]) * per * per * up
                    : 0.0f;
    }
    for (int64_t t = lo + warp; t < end; t += kRouteWarps) {
      float z[NL], sc[NL];
      load_token<NL>(a, t, lane, a.valid == nullptr || a.valid[t] != 0, z);
      float top, inv;
      const float all = scores_of<NL, kScore>(z, sc, top, inv);
      int mine = -1;
      float ws = 0.0f, dw = 0.0f;
      if (lane < a.k) {
        const int e = a.idx[t * a.k + lane];
        if (e >= 0 && e < a.E) {
          mine = e;
          dw = a.dw[t * a.k + lane];
          ws = score_of<kScore>(load_logit(a.logits, a.bf16, t * a.ld + e), top, inv);
        }
      }
      float dws = a.scale * dw;
      if (a.normalize) {
        const float r = 1.0f / (warp_sum(ws) + kScoreEps);
        const float mean = warp_sum(dw * ws) * r;
        dws = a.scale * r * (dw - mean);
      }
      if (mine >= 0) s_d[warp][mine] = dws;
      __syncwarp();
      float u[NL];
      float dot = 0.0f;
      const float r = 1.0f / all;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const float d = s_d[warp][32 * i + lane];
        u[i] = kScore == 0 ? d + coef[i] : d;
        dot += (kScore == 0 ? u[i] : coef[i]) * sc[i] * r;
      }
      dot = warp_sum(dot);
      __syncwarp();
      if (mine >= 0) s_d[warp][mine] = 0.0f;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int e = 32 * i + lane;
        float dz = kScore == 0 ? sc[i] * (u[i] - dot) : (u[i] + (coef[i] - dot) * r) * sc[i] * (1.0f - sc[i]);
        if (!eligible(z[i])) dz = 0.0f;
        if (e < a.E) {
          if (a.bf16)
            static_cast<__nv_bfloat16*>(a.dlogits)[t * a.ldd + e] = __float2bfloat16_rn(dz);
          else
            static_cast<float*>(a.dlogits)[t * a.ldd + e] = dz;
        }
      }
      __syncwarp();
    }
    lo = end;
    while (lo < hi && sequence_end(a, s) <= lo) ++s;
  }
}

// ------------------------------------------------------------------ layout
// A counting sort of the T k choices by expert, stable in token order.  The
// choices are cut into chunks of one CTA each; layout_count leaves each
// chunk's histogram, layout_place adds up the histograms before its own and
// places its choices: each warp ranks its stretch (equal experts of 32
// choices found with match_any), the warps' counts are summed in order.
constexpr int kLayoutThreads = 512;
constexpr int kLayoutWarps = kLayoutThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kChunkPairs = 2048;           // smallest chunk
constexpr int kMaxLayoutChunks = 512;

__global__ void __launch_bounds__(kLayoutThreads) layout_count_kernel(const LayoutArgs a) {
  __shared__ int s_n[kMaxExperts];
  for (int e = threadIdx.x; e < a.E; e += kLayoutThreads) s_n[e] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk, hi = min(a.pairs, lo + a.chunk);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kLayoutThreads) {
    const int e = a.idx[i];
    if (e >= 0 && e < a.E) atomicAdd(&s_n[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kLayoutThreads) a.hist[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_n[e];
}

__global__ void __launch_bounds__(kLayoutThreads) layout_place_kernel(const LayoutArgs a) {
  __shared__ uint16_t s_w[kLayoutWarps][kMaxExperts];   // counts of a warp, then of the warps before it
  __shared__ int s_base[kMaxExperts];                   // first row of this chunk's choices
  __shared__ int s_total[kMaxExperts + 1];              // choices of an expert, then first rows
  __shared__ int s_scan[kLayoutWarps];
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
    int before = 0, total = 0;
    if (chunks > 1) {
      for (int c = 0; c < chunks; ++c) {
        const int n = a.hist[static_cast<int64_t>(c) * a.E + e];
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
        total += n;
      }
    }
    int run = 0;
    for (int w = 0; w < kLayoutWarps; ++w) {
      const int n = s_w[w][e];
      s_w[w][e] = static_cast<uint16_t>(run);
      run += n;
    }
    s_base[e] = before;
    s_total[e] = chunks > 1 ? total : run;
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
  if (backward) {
    if (a.score == 0)
      route_backward_kernel<NL, 0><<<grid, kRouteThreads, 0, stream>>>(a);
    else
      route_backward_kernel<NL, 1><<<grid, kRouteThreads, 0, stream>>>(a);
  } else if (a.loss != nullptr) {
    if (a.score == 0)
      route_kernel<NL, 0, true><<<grid, kRouteThreads, 0, stream>>>(a);
    else
      route_kernel<NL, 1, true><<<grid, kRouteThreads, 0, stream>>>(a);
  } else {
    if (a.score == 0)
      route_kernel<NL, 0, false><<<grid, kRouteThreads, 0, stream>>>(a);
    else
      route_kernel<NL, 1, false><<<grid, kRouteThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t pick_route(const RouteArgs& a, bool backward, cudaStream_t stream) {
  if (a.E <= 32) return run_route<1>(a, backward, stream);
  if (a.E <= 64) return run_route<2>(a, backward, stream);
  if (a.E <= 128) return run_route<4>(a, backward, stream);
  if (a.E <= 256) return run_route<8>(a, backward, stream);
  if (a.E <= 512) return run_route<16>(a, backward, stream);
  return run_route<32>(a, backward, stream);
}

int64_t route_chunk(int64_t T) {
  const int64_t c = (T + kMaxChunks - 1) / kMaxChunks;
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
  route_finish_kernel<<<dim3(slices, static_cast<unsigned>(a.S)), kFinishThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_route_backward(RouteArgs a, cudaStream_t stream) {
  a.chunk = route_chunk(a.T);
  return pick_route(a, true, stream);
}

int64_t layout_workspace_bytes(int64_t T, int k, int E) {
  const int64_t pairs = T * k, chunk = layout_chunk(pairs);
  const int64_t chunks = (pairs + chunk - 1) / chunk;
  return chunks > 1 ? 4 * chunks * E : 4;
}

cudaError_t launch_layout(LayoutArgs a, cudaStream_t stream) {
  a.chunk = layout_chunk(a.pairs);
  const unsigned chunks = static_cast<unsigned>(std::max<int64_t>(1, (a.pairs + a.chunk - 1) / a.chunk));
  if (chunks > 1) {
    layout_count_kernel<<<chunks, kLayoutThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  layout_place_kernel<<<chunks, kLayoutThreads, 0, stream>>>(a);
  return cudaGetLastError();
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
