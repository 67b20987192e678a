// route.cu -- router of a mixture of experts: top-k choice, weights, counts and
// the sorted order of the grouped products, balance loss; and its backward pass.
//
//   s = softmax(l) or sigmoid(l) over the open experts,  p = s / sum s,
//   weight_j = scale * s_j (/ sum of the chosen s),
//   loss = E * sum_e (counts_e / sum counts) * (sum_t p_te / N).
//
// A warp takes a token, lane i the V experts from i * V on, in registers.  The
// choice is k rounds of one warp-wide integer maximum over keys that order as the
// logits do (ties: the lowest lane and register is the lowest expert).
//
// The order has to be the same in every run, so rows are counted, not claimed with
// atomics: each warp goes through a contiguous part of the tokens and counts its
// choices per expert, which is a choice's rank among its warp's; prefix sums over a
// CTA's warps and over the CTAs give its row.  Probabilities are summed in the same
// fixed order.  Two launches: choices and counts per CTA, then the prefix over CTAs
// and the rows; one launch where one CTA holds all tokens.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8q.h"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"
#include "fp8q_vec.cuh"

namespace fp8q {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 152;     // one per SM
constexpr int kOneCta = 64;       // tokens that one CTA takes alone
constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;   // one per lane
constexpr float kTiny = 0x1p-126f;
constexpr float kBig = 3.40282347e38f;

struct RouteArgs {
  const void *logits;
  const uint8_t *valid;
  int32_t *idx, *counts, *offs, *order, *slot, *tokens;
  float *weight, *loss;
  int *cta_counts;    // [CTAs][E]
  float *cta_probs;   // [CTAs][E]
  int *cta_tokens;    // [CTAs]
  int64_t ld;
  int T, E, k, ctas, per_cta, per_warp;
  float scale;
  bool sigmoid, normalise, vec;
};

// V consecutive logits of a row from column lane * V on; -inf behind column E.
template <int kKind, int V>
__device__ __forceinline__ void load_logits(const void *row, int E, int lane, bool vec, float (&l)[V]) {
  constexpr int kBytes = V * size_of(kKind);
  const int e0 = lane * V;
  if (vec && e0 + V <= E) {
    uint32_t w[(kBytes + 3) / 4];
    const char *p = static_cast<const char *>(row) + static_cast<int64_t>(e0) * size_of(kKind);
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 u = ld_stream(p + 16 * i);
        w[4 * i] = u.x;
        w[4 * i + 1] = u.y;
        w[4 * i + 2] = u.z;
        w[4 * i + 3] = u.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      w[0] = u.x;
      w[1] = u.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      l[v] = kKind == kFp32 ? __uint_as_float(w[v]) : (v & 1) ? bf16_hi(w[v / 2]) : bf16_lo(w[v / 2]);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = e0 + v;
      if (e >= E) l[v] = -INFINITY;
      else if constexpr (kKind == kFp32) l[v] = static_cast<const float *>(row)[e];
      else l[v] = bf16_lo(static_cast<const uint16_t *>(row)[e]);
    }
  }
}
__device__ __forceinline__ float logit_at(const void *row, int kind, int e) {
  return kind == kFp32 ? static_cast<const float *>(row)[e]
                       : bf16_lo(static_cast<const uint16_t *>(row)[e]);
}

// Unsigned keys in the order of the logits: 0 for a closed expert (-inf or NaN),
// the same for both zeros; +inf becomes the largest finite value.
__device__ __forceinline__ uint32_t key_of(float l) {
  if (!(l > -INFINITY)) return 0;
  l = fminf(l, kBig);
  const uint32_t b = l == 0.0f ? 0u : __float_as_uint(l);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(~0u, v); }

// Exclusive sums over the CTA's threads (at most 1024); `part` holds 32 ints and
// is free again after the caller's next barrier.
__device__ __forceinline__ int cta_exclusive_sum(int v, int *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(~0u, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  const int before = warp_sum(lane < warps && lane < warp ? part[lane] : 0);
  return before + s - v;
}

// counts, offs, tokens and loss, by one CTA of at least E threads: thread e has
// expert e's total, the sum of its probabilities and its first row.
__device__ __forceinline__ void write_totals(const RouteArgs &a, int total, float probs, int first,
                                             int tokens, float *part) {
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5, warps = blockDim.x >> 5;
  if (e < a.E) {
    a.counts[e] = total;
    a.offs[e] = first;
    if (e == a.E - 1) a.offs[a.E] = first + total;
  }
  const float s = warp_sum(e < a.E ? static_cast<float>(total) * probs : 0.0f);
  const float n = warp_sum(e < a.E ? static_cast<float>(total) : 0.0f);
  if (lane == 0) {
    part[warp] = s;
    part[32 + warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    const float all = warp_sum(lane < warps ? part[lane] : 0.0f);
    const float choices = warp_sum(lane < warps ? part[32 + lane] : 0.0f);
    if (lane == 0) {
      a.tokens[0] = tokens;
      a.loss[0] = tokens > 0 ? static_cast<float>(a.E) * (all / choices) / static_cast<float>(tokens) : 0.0f;
    }
  }
}

// Dynamic shared memory: counts [kWarps][E], then probabilities [kWarps][E].
template <int kKind, int V>
__global__ void __launch_bounds__(kThreads)
route_kernel(const RouteArgs a) {
  extern __shared__ int smem[];
  __shared__ int tokens_of[kWarps], scan[32];
  __shared__ float part[64];
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, k = a.k;
  int *counts = smem;
  float *probs = reinterpret_cast<float *>(smem + kWarps * E);
  int *mine = counts + warp * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();

  const int64_t cta_lo = static_cast<int64_t>(blockIdx.x) * a.per_cta;
  const int64_t cta_hi = min(static_cast<int64_t>(a.T), cta_lo + a.per_cta);
  const int64_t lo = min(cta_hi, cta_lo + static_cast<int64_t>(warp) * a.per_warp);
  const int64_t hi = min(cta_hi, lo + a.per_warp);
  float psum[V];
#pragma unroll
  for (int v = 0; v < V; ++v) psum[v] = 0.0f;
  int routed = 0;

  for (int64_t t = lo; t < hi; ++t) {
    const bool valid = !a.valid || a.valid[t] != 0;
    float l[V];
    uint32_t key[V];
    load_logits<kKind, V>(static_cast<const char *>(a.logits) + t * a.ld * size_of(kKind), E, lane, a.vec, l);
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = valid ? key_of(l[v]) : 0u;
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) best = max(best, key[v]);
    uint32_t top = __reduce_max_sync(~0u, best);
    routed += top != 0;
    const float m = logit_of(top);

    // scores and their sum, before the choice clears keys
    float s[V], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float x = logit_of(key[v]);
      s[v] = key[v] == 0 ? 0.0f : a.sigmoid ? sigmoid(x) : expf(x - m);
      sum += s[v];
    }
    sum = warp_sum(sum);
    const float inv = 1.0f / fmaxf(sum, kTiny);
#pragma unroll
    for (int v = 0; v < V; ++v) psum[v] = fmaf(s[v], inv, psum[v]);

    // lane j keeps choice j
    int chosen = -1;
    uint32_t chosen_key = 0;
    for (int j = 0; j < k && top != 0; ++j) {
      const int owner = __ffs(__ballot_sync(~0u, best == top)) - 1;
      int at = 0;
      if (lane == owner) {
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          if (key[v] == top) at = v;
        best = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (v == at) key[v] = 0;
          best = max(best, key[v]);
        }
      }
      at = __shfl_sync(~0u, at, owner);
      if (lane == j) {
        chosen = owner * V + at;
        chosen_key = top;
      }
      top = __reduce_max_sync(~0u, best);
    }
    float w = 0.0f;
    if (chosen >= 0) {
      const float x = logit_of(chosen_key);
      w = a.sigmoid ? sigmoid(x) : expf(x - m) * inv;
    }
    if (a.normalise) w = w / fmaxf(warp_sum(w), kTiny);
    if (lane < k) {
      const int64_t at = t * k + lane;
      a.idx[at] = chosen;
      a.weight[at] = w * a.scale;
      int rank = -1;
      if (chosen >= 0) {
        rank = mine[chosen];  // a token's choices differ
        mine[chosen] = rank + 1;
      }
      a.slot[at] = rank;
    }
    __syncwarp();
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane * V + v < E) probs[warp * E + lane * V + v] = psum[v];
  if (lane == 0) tokens_of[warp] = routed;
  __syncthreads();

  // counts become the warps' first ranks
  const bool alone = gridDim.x == 1;
  int totals[kMaxExperts / kThreads], tokens = 0;
  float p_of[kMaxExperts / kThreads];
#pragma unroll
  for (int i = 0; i < kMaxExperts / kThreads; ++i) {
    const int e = threadIdx.x + i * kThreads;
    int run = 0;
    float p = 0.0f;
    if (e < E) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int c = counts[w * E + e];
        counts[w * E + e] = run;
        run += c;
        p += probs[w * E + e];
      }
      if (!alone) {
        a.cta_counts[static_cast<int64_t>(blockIdx.x) * E + e] = run;
        a.cta_probs[static_cast<int64_t>(blockIdx.x) * E + e] = p;
      }
    }
    totals[i] = run;
    p_of[i] = p;
  }
#pragma unroll
  for (int w = 0; w < kWarps; ++w) tokens += tokens_of[w];
  __syncthreads();

  int rows = 0;
  if (!alone) {
    if (threadIdx.x == 0) a.cta_tokens[blockIdx.x] = tokens;
  } else {
    // one CTA: its totals are all there is; probs holds them by expert from here on
    int *total_of = reinterpret_cast<int *>(probs);
    float *prob_of = probs + E;
#pragma unroll
    for (int i = 0; i < kMaxExperts / kThreads; ++i) {
      const int e = threadIdx.x + i * kThreads;
      if (e < E) {
        total_of[e] = totals[i];
        prob_of[e] = p_of[i];
      }
    }
    __syncthreads();
    // thread i sums the experts 2i and 2i + 1
    const int e0 = 2 * threadIdx.x;
    const int c0 = e0 < E ? total_of[e0] : 0, c1 = e0 + 1 < E ? total_of[e0 + 1] : 0;
    const int first = cta_exclusive_sum(c0 + c1, scan);
    float all = 0.0f;
    if (e0 < E) {
      a.counts[e0] = c0;
      a.offs[e0] = first;
      all = static_cast<float>(c0) * prob_of[e0];
    }
    if (e0 + 1 < E) {
      a.counts[e0 + 1] = c1;
      a.offs[e0 + 1] = first + c0;
      all = fmaf(static_cast<float>(c1), prob_of[e0 + 1], all);
    }
    all = warp_sum(all);
    const int n = warp_sum(c0 + c1);
    if (lane == 0) {
      part[warp] = all;
      part[32 + warp] = __int_as_float(n);
    }
    __syncthreads();
    float loss = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      loss += part[w];
      rows += __float_as_int(part[32 + w]);
    }
    if (threadIdx.x == 0) {
      a.offs[E] = rows;
      a.tokens[0] = tokens;
      a.loss[0] = tokens > 0 ? static_cast<float>(E) * (loss / static_cast<float>(rows)) /
                                   static_cast<float>(tokens)
                             : 0.0f;
    }
    if (e0 < E) total_of[e0] = first;
    if (e0 + 1 < E) total_of[e0 + 1] = first + c0;
    __syncthreads();
    for (int i = rows + threadIdx.x; i < a.T * k; i += kThreads) a.order[i] = -1;
  }

  // the warp's choices again, now with their ranks in the CTA (or their rows)
  const int *first_row = reinterpret_cast<const int *>(probs);
  for (int64_t i = lo * k + lane; i < hi * k; i += 32) {
    const int e = a.idx[i];
    if (e < 0) continue;
    int row = a.slot[i] + mine[e];
    if (alone) {
      row += first_row[e];
      a.order[row] = static_cast<int32_t>(i);
    }
    a.slot[i] = row;
  }
}

constexpr int kRowThreads = 1024;

// CTA b turns ranks into rows: expert e's choices of CTA b start at offs[e] plus
// the counts of the CTAs before it.
__global__ void __launch_bounds__(kRowThreads)
route_rows_kernel(const RouteArgs a) {
  __shared__ int total_of[kRowThreads], before_of[kRowThreads], scan[32];
  __shared__ float prob_of[kRowThreads], part[64];
  wait_for_previous_kernel();
  const int E = a.E, k = a.k, tid = threadIdx.x;
  // the CTAs' counts are added up by as many groups of threads as there is room
  // for, each taking every groups-th CTA
  const int width = (E + 31) / 32 * 32, groups = kRowThreads / width;
  const int e = tid % width, group = tid / width;
  int total = 0, before = 0, tokens = 0;
  float probs = 0.0f;
  if (e < E && group < groups) {
#pragma unroll 8
    for (int b = group; b < a.ctas; b += groups) {
      const int c = a.cta_counts[b * E + e];
      total += c;
      before += b < static_cast<int>(blockIdx.x) ? c : 0;
    }
    if (blockIdx.x == 0) {
#pragma unroll 8
      for (int b = group; b < a.ctas; b += groups) probs += a.cta_probs[b * E + e];
    }
  }
  total_of[tid] = total;
  before_of[tid] = before;
  prob_of[tid] = probs;
  __syncthreads();
  total = before = 0;
  probs = 0.0f;
  if (tid < E)
    for (int g = 0; g < groups; ++g) {
      total += total_of[g * width + tid];
      before += before_of[g * width + tid];
      probs += prob_of[g * width + tid];
    }
  const int first = cta_exclusive_sum(total, scan);
  __syncthreads();
  if (tid < E) total_of[tid] = first + before;
  if (tid == kRowThreads - 1) before_of[0] = first + total;
  if (blockIdx.x == 0) {
    for (int b = 0; b < a.ctas; ++b) tokens += a.cta_tokens[b];
    write_totals(a, total, probs, first, tokens, part);
  }
  __syncthreads();
  const int64_t all = static_cast<int64_t>(a.T) * k;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.per_cta * k;
  const int64_t hi = min(all, lo + static_cast<int64_t>(a.per_cta) * k);
  for (int64_t i = lo + tid; i < hi; i += kRowThreads) {
    const int x = a.idx[i];
    if (x >= 0) {
      const int row = a.slot[i] + total_of[x];
      a.slot[i] = row;
      a.order[row] = static_cast<int32_t>(i);
    }
    if (i >= before_of[0]) a.order[i] = -1;
  }
}

struct BwdArgs {
  const void *logits;
  const uint8_t *valid;
  const int32_t *idx, *counts, *tokens;
  const float *dweight, *dloss;
  void *dlogits;
  int64_t ld, ld_d;
  int T, E, k;
  float scale;
  bool sigmoid, normalise, vec, vec_d;
};

// With u_j and v_e the gradients with respect to the logarithms of the scores, from
// the weights and from the loss,
//   u_j = q_j (dw_j - sum q dw), q = s / (sum of the chosen s)   (normalised)
//         s_j dw_j                                                (else)
//   v_e = p_e (dp_e - sum p dp), dp_e = dloss * E * f_e / N
//   dl  = (u + v) (1 - s) (sigmoid)  or  u - p sum u + v (softmax, sum u = 0 if
//         normalised).
// Nothing is divided by a score, so small ones lose nothing.
template <int kKind, int V>
__global__ void __launch_bounds__(256)
route_bwd_kernel(const BwdArgs a) {
  extern __shared__ float us[];  // [warps][32 * V]
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, k = a.k;
  float *u_of = us + warp * 32 * V;
  float dp[V];
  {
    int c[V], n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane * V + v;
      u_of[e] = 0.0f;
      c[v] = e < E && a.dloss ? a.counts[e] : 0;
      n += c[v];
    }
    n = warp_sum(n);
    const int tokens = a.dloss ? a.tokens[0] : 0;
    const float f = tokens > 0 && n > 0 ? a.dloss[0] * static_cast<float>(E) / static_cast<float>(n) /
                                              static_cast<float>(tokens)
                                        : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) dp[v] = f * static_cast<float>(c[v]);
  }
  __syncwarp();
  const int warps = gridDim.x * (blockDim.x >> 5);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp; t < a.T; t += warps) {
    const bool valid = !a.valid || a.valid[t] != 0;
    const char *row = static_cast<const char *>(a.logits) + t * a.ld * size_of(kKind);
    int at = -1;
    float dw = 0.0f, x = 0.0f;
    if (lane < k && a.dweight && valid) {
      at = a.idx[t * k + lane];
      dw = a.dweight[t * k + lane] * a.scale;
      if (at >= 0 && at < E) {
        x = logit_at(row, kKind, at);
        if (!(x > -INFINITY)) at = -1;
        x = fminf(x, kBig);
      } else {
        at = -1;
      }
    }
    float l[V], s[V];
    load_logits<kKind, V>(row, E, lane, a.vec, l);
    float m = -kBig;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!valid || !(l[v] > -INFINITY)) l[v] = -INFINITY;
      l[v] = fminf(l[v], kBig);
      m = fmaxf(m, l[v]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = !(l[v] > -INFINITY) ? 0.0f : a.sigmoid ? sigmoid(l[v]) : expf(l[v] - m);
      sum += s[v];
    }
    const float inv = 1.0f / fmaxf(warp_sum(sum), kTiny);
    float pdp = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) pdp = fmaf(s[v] * inv, dp[v], pdp);
    pdp = warp_sum(pdp);

    float u = at < 0 ? 0.0f : a.sigmoid ? sigmoid(x) : expf(x - m) * inv;
    if (at < 0) dw = 0.0f;
    if (a.normalise) {
      u = u / fmaxf(warp_sum(u), kTiny);
      u *= dw - warp_sum(u * dw);
    } else {
      u *= dw;
    }
    const float usum = a.sigmoid || a.normalise ? 0.0f : warp_sum(u);
    if (at >= 0) atomicAdd(u_of + at, u);
    __syncwarp();
    float d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float p = s[v] * inv;
      d[v] = fmaf(p, dp[v] - pdp - usum, u_of[lane * V + v]);
      if (a.sigmoid) d[v] *= sigmoid(-l[v]);
      if (!(l[v] > -INFINITY)) d[v] = 0.0f;
    }
    __syncwarp();
    if (at >= 0) u_of[at] = 0.0f;
    __syncwarp();

    char *out = static_cast<char *>(a.dlogits) + t * a.ld_d * size_of(kKind);
    const int e0 = lane * V;
    if (V % 8 == 0 && a.vec_d && e0 + V <= E) {
#pragma unroll
      for (int i = 0; i < V / 8; ++i) {
        float part[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) part[e] = d[8 * i + e];
        store8<kKind>(out, e0 + 8 * i, part);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e0 + v < E) {
          if constexpr (kKind == kFp32) reinterpret_cast<float *>(out)[e0 + v] = d[v];
          else reinterpret_cast<uint16_t *>(out)[e0 + v] = static_cast<uint16_t>(bf16x2(d[v], 0.0f));
        }
    }
  }
}

struct Plan {
  int ctas, per_cta, per_warp;
};
Plan plan(int64_t T) {
  Plan p;
  p.ctas = T <= kOneCta ? 1 : static_cast<int>(T < kMaxCtas * kWarps ? (T + kWarps - 1) / kWarps : kMaxCtas);
  p.per_cta = static_cast<int>((T + p.ctas - 1) / p.ctas);
  p.per_warp = (p.per_cta + kWarps - 1) / kWarps;
  return p;
}

bool shape_ok(int64_t T, int64_t E) {
  return T >= 0 && T <= (int64_t{1} << 26) && E >= 1 && E <= kMaxExperts;
}

template <int kKind, int V>
fp8q_status launch_route(const RouteArgs &a, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kWarps) * a.E * (sizeof(int) + sizeof(float));
  const auto kern = route_kernel<kKind, V>;
  if (smem > 40 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kWarps * kMaxExperts * 8) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  if (fp8q_status st = launch_dependent(kern, dim3(a.ctas), dim3(kThreads), smem, s, a)) return st;
  if (a.ctas == 1) return FP8Q_OK;
  return launch_dependent(route_rows_kernel, dim3(a.ctas), dim3(kRowThreads), 0, s, a);
}

template <int kKind>
fp8q_status launch_route(const RouteArgs &a, cudaStream_t s) {
  if (a.E <= 32) return launch_route<kKind, 1>(a, s);
  if (a.E <= 64) return launch_route<kKind, 2>(a, s);
  if (a.E <= 128) return launch_route<kKind, 4>(a, s);
  if (a.E <= 256) return launch_route<kKind, 8>(a, s);
  if (a.E <= 512) return launch_route<kKind, 16>(a, s);
  return launch_route<kKind, 32>(a, s);
}

template <int kKind, int V>
fp8q_status launch_bwd(const BwdArgs &a, cudaStream_t s) {
  const int warps = 8, need = (a.T + warps - 1) / warps, most = kMaxCtas * 8;
  const size_t smem = static_cast<size_t>(warps) * 32 * V * sizeof(float);
  return launch_dependent(route_bwd_kernel<kKind, V>, dim3(need < most ? need : most), dim3(32 * warps),
                          smem, s, a);
}

template <int kKind>
fp8q_status launch_bwd(const BwdArgs &a, cudaStream_t s) {
  if (a.E <= 32) return launch_bwd<kKind, 1>(a, s);
  if (a.E <= 64) return launch_bwd<kKind, 2>(a, s);
  if (a.E <= 128) return launch_bwd<kKind, 4>(a, s);
  if (a.E <= 256) return launch_bwd<kKind, 8>(a, s);
  if (a.E <= 512) return launch_bwd<kKind, 16>(a, s);
  return launch_bwd<kKind, 32>(a, s);
}

bool kind_ok(int kind) { return kind == kBf16 || kind == kFp32; }
bool row_vectors(const void *p, int64_t ld, int kind) {
  return aligned16(p) && ld * size_of(kind) % 16 == 0;
}
bool at_element(const void *p, int kind) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<unsigned>(size_of(kind)) == 0;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int64_t fp8q_route_workspace_bytes(int64_t T, int64_t E) {
  if (!shape_ok(T, E)) return 0;
  const Plan p = plan(T);
  return p.ctas <= 1 ? 0 : (2 * E + 1) * static_cast<int64_t>(p.ctas) * 4;
}

extern "C" fp8q_status fp8q_route(const void *logits, int64_t ld, int dtype, const uint8_t *valid,
                                  int score, int normalise, float scale, int32_t *idx,
                                  float *weight, int32_t *counts, int32_t *offs, int32_t *order,
                                  int32_t *slot, int32_t *tokens, float *loss, int64_t T, int64_t E,
                                  int64_t k, void *workspace, int64_t workspace_bytes,
                                  void *stream) {
  if (!kind_ok(dtype) || (score != FP8Q_SCORE_SOFTMAX && score != FP8Q_SCORE_SIGMOID))
    return FP8Q_ERR_INVALID;
  if (!shape_ok(T, E) || k < 1 || k > E || k > kMaxChoices || T * k > 0x7FFFFFFFll || ld < E)
    return FP8Q_ERR_SHAPE;
  if (!counts || !offs || !tokens || !loss) return FP8Q_ERR_INVALID;
  if (T > 0 && (!logits || !idx || !weight || !order || !slot)) return FP8Q_ERR_INVALID;
  const int64_t need = fp8q_route_workspace_bytes(T, E);
  if (need > 0) {
    if (!workspace) return FP8Q_ERR_INVALID;
    if (workspace_bytes < need) return FP8Q_ERR_SHAPE;
    if (!aligned16(workspace)) return FP8Q_ERR_ALIGN;
  }
  if (!at_element(logits, dtype) || !aligned4(idx) || !aligned4(weight) || !aligned4(counts) ||
      !aligned4(offs) || !aligned4(order) || !aligned4(slot) || !aligned4(tokens) || !aligned4(loss))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;
  const Plan p = plan(T);
  RouteArgs a{};
  a.logits = logits;
  a.valid = valid;
  a.idx = idx;
  a.counts = counts;
  a.offs = offs;
  a.order = order;
  a.slot = slot;
  a.tokens = tokens;
  a.weight = weight;
  a.loss = loss;
  a.cta_counts = static_cast<int *>(workspace);
  a.cta_probs = static_cast<float *>(workspace) + E * p.ctas;
  a.cta_tokens = static_cast<int *>(workspace) + 2 * E * p.ctas;
  a.ld = ld;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.ctas = p.ctas;
  a.per_cta = p.per_cta;
  a.per_warp = p.per_warp;
  a.scale = scale;
  a.sigmoid = score == FP8Q_SCORE_SIGMOID;
  a.normalise = normalise != 0;
  a.vec = row_vectors(logits, ld, dtype);
  auto st = static_cast<cudaStream_t>(stream);
  return dtype == kBf16 ? launch_route<kBf16>(a, st) : launch_route<kFp32>(a, st);
}

extern "C" fp8q_status fp8q_route_bwd(const void *logits, int64_t ld, int dtype,
                                      const uint8_t *valid, int score, int normalise, float scale,
                                      const int32_t *idx, const int32_t *counts,
                                      const int32_t *tokens, const float *dweight,
                                      const float *dloss, void *dlogits, int64_t ld_d, int64_t T,
                                      int64_t E, int64_t k, void *stream) {
  if (!kind_ok(dtype) || (score != FP8Q_SCORE_SOFTMAX && score != FP8Q_SCORE_SIGMOID))
    return FP8Q_ERR_INVALID;
  if (!shape_ok(T, E) || k < 1 || k > E || k > kMaxChoices || T * k > 0x7FFFFFFFll || ld < E || ld_d < E)
    return FP8Q_ERR_SHAPE;
  if (T == 0) return FP8Q_OK;
  if (!logits || !dlogits || (dweight && !idx) || (dloss && (!counts || !tokens)))
    return FP8Q_ERR_INVALID;
  if (!at_element(logits, dtype) || !at_element(dlogits, dtype) || !aligned4(idx) ||
      !aligned4(counts) || !aligned4(tokens) || !aligned4(dweight) || !aligned4(dloss))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;
  BwdArgs a{};
  a.logits = logits;
  a.valid = valid;
  a.idx = idx;
  a.counts = counts;
  a.tokens = tokens;
  a.dweight = dweight;
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.ld = ld;
  a.ld_d = ld_d;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.scale = scale;
  a.sigmoid = score == FP8Q_SCORE_SIGMOID;
  a.normalise = normalise != 0;
  a.vec = row_vectors(logits, ld, dtype);
  a.vec_d = row_vectors(dlogits, ld_d, dtype);
  auto st = static_cast<cudaStream_t>(stream);
  return dtype == kBf16 ? launch_bwd<kBf16>(a, st) : launch_bwd<kFp32>(a, st);
}
