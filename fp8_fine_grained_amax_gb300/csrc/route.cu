// route.cu -- router of a mixture of experts: top-k choice, weights, counts and
// the sorted order of the grouped products, balance loss; and its backward pass.
//
//   s = softmax(l) or sigmoid(l) over the open experts,  p = s / sum s,
//   weight_j = scale * s_j (/ sum of the chosen s),
//   loss = E * sum_e (counts_e / sum counts) * (sum_t p_te / N).
//
// A warp takes a token, each lane V experts, in registers: of every 128 experts four next
// to each other, so that a warp reads and writes rows without gaps.  Each expert becomes
// one 32-bit word: the logit's upper bits in an order-preserving form, and below them the
// expert's index, falling, so that no two words are alike and the lower index is the
// larger word.  A lane sorts its words (two instructions per comparator), and the choice
// is k rounds of one warp-wide maximum over the lanes' largest words.  BF16 logits fit in
// the upper bits.  Of FP32 logits those that agree with the last choice in the upper bits
// are taken too, and the lanes sort what they keep by the whole logits; where there are
// more of them than lanes, the choice is made again on whole logits.
//
// The order has to be the same in every run, so rows are counted, not claimed with
// atomics: each warp goes through a contiguous part of the tokens and counts its
// choices per expert, which is a choice's rank among its warp's; prefix sums over a
// CTA's warps and over the CTAs give its row.  Probabilities are summed in the same
// fixed order.  Two launches: choices and counts per CTA, then the prefix over CTAs
// and the rows.  Few tokens take one launch, of one CTA or of a cluster of eight that
// read each other's totals from shared memory.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8q.h"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"
#include "fp8q_vec.cuh"

namespace fp8q {
namespace {

constexpr int kSms = 152;         // one CTA each
constexpr int kMaxPerCta = 65535; // tokens of a CTA: its counts are 16 bits
constexpr int kCluster = 8;
constexpr int kOneCtaTokens = 32;  // a token per warp, of the most experts two
constexpr int kFewPerCta = 8;
constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;   // one per lane
constexpr float kTiny = 0x1p-126f;
constexpr float kBig = 3.40282347e38f;

__host__ __device__ constexpr int round_up(int n, int to) { return (n + to - 1) / to * to; }

struct RouteArgs {
  const void *logits;
  const uint8_t *valid;
  int32_t *idx, *counts, *offs, *order, *slot, *tokens;
  float *weight, *loss;
  uint16_t *cta_counts;  // [E][CTAs, rounded up to 8]
  float *cta_probs;      // [E][CTAs, rounded up to 4]
  int *cta_tokens;    // [CTAs]
  int64_t ld;
  int T, E, k, ctas, per_cta;
  float scale;
  bool sigmoid, normalise, vec;
};

// The v-th of a lane's V experts.
__host__ __device__ constexpr int width(int V) { return V < 4 ? V : 4; }
template <int V>
__device__ __forceinline__ constexpr int expert(int lane, int v) {
  constexpr int W = width(V);
  return v / W * 32 * W + lane * W + v % W;
}

// A lane's logits of a row as they lie in memory, -inf behind column E: what is done with
// them would make the load wait, so nothing is until their turn.
template <int kKind, int V>
struct Row {
  static constexpr int W = width(V), kWords = kKind == kFp32 ? V : (V + 1) / 2;
  uint32_t w[kWords];

  // `vec`: the row starts on 16 bytes and E is a multiple of four.
  __device__ __forceinline__ void load(const void *row, int E, int lane, bool vec) {
    constexpr uint32_t kClosed = kKind == kFp32 ? 0xFF800000u : 0xFF80FF80u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = kClosed;
    if (vec) {
      constexpr int kBytes = W * size_of(kKind);
#pragma unroll
      for (int v = 0; v < V; v += W) {
        const int e = expert<V>(lane, v);
        if (e >= E) continue;
        const char *p = static_cast<const char *>(row) + e * size_of(kKind);
        if constexpr (kBytes == 16) {
          const uint4 u = *reinterpret_cast<const uint4 *>(p);
          w[v] = u.x;
          w[v + 1] = u.y;
          w[v + 2] = u.z;
          w[v + 3] = u.w;
        } else if constexpr (kBytes == 8) {
          constexpr int at = kKind == kFp32 ? 1 : 2;
          const uint2 u = *reinterpret_cast<const uint2 *>(p);
          w[v / at] = u.x;
          w[v / at + 1] = u.y;
        } else if constexpr (kBytes == 4) {
          w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
          w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = expert<V>(lane, v);
        if (e >= E) continue;
        if constexpr (kKind == kFp32) {
          w[v] = static_cast<const uint32_t *>(row)[e];
        } else {
          const uint32_t x = static_cast<const uint16_t *>(row)[e];
          w[v / 2] = v & 1 ? (w[v / 2] & 0xFFFFu) | x << 16 : (w[v / 2] & 0xFFFF0000u) | x;
        }
      }
    }
  }
  __device__ __forceinline__ void values(float (&l)[V]) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (kKind == kFp32) l[v] = __uint_as_float(w[v]);
      else l[v] = v & 1 ? bf16_hi(w[v / 2]) : bf16_lo(w[v / 2]);
    }
  }
};
// A row into the L2: its bytes are at most 32 lines.
__device__ __forceinline__ void prefetch_row(const char *row, int bytes, int lane) {
  if (lane * 128 < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + lane * 128));
}
__device__ __forceinline__ float logit_at(const void *row, int kind, int e) {
  return kind == kFp32 ? static_cast<const float *>(row)[e]
                       : bf16_lo(static_cast<const uint16_t *>(row)[e]);
}

// Warps of a CTA: 64 registers per thread for up to 16 experts per lane, 128 for 32.
// Many experts leave no room there for the next row, the sums of the probabilities and
// the words that wait: the row waits in the L2, the others in shared memory.  (16384
// tokens of 1024 experts, all in registers, eight warps: 73.6 us, so 55.1; of 512 31.5 and
// 28.3.  Both figures from before the second launch's CTAs shared their sums.)
__host__ __device__ constexpr bool many(int V) { return V >= 16; }
__host__ __device__ constexpr int warps_for(int V) { return V <= 16 ? 32 : 16; }

// The lanes' sorted words, of one warp, in shared memory: one column per lane and a zero
// behind its words.  Shifted in registers every round, they took 16384 tokens of 1024
// experts 6 us longer with 8 choices and 28 with 32; of 256 they save 0.2, but one token
// takes 4.2 us instead of 3.9.
__host__ __device__ constexpr int queue_words(int V) { return many(V) ? 32 * (V + 1) : 0; }

// Unsigned keys in the order of the logits, the same for both zeros.  -inf is below
// kOpen, +inf and NaN (which the addition makes the positive one) at kSpecial or above.
constexpr uint32_t kOpen = 0x00800000u, kSpecial = 0xFF800000u;
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);  // -0 + 0 = +0
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

// Falling order of V words: Batcher's odd-even merge sort.
template <int V>
__device__ __forceinline__ void sort_falling(uint32_t (&w)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int i = 0; i + k < V; ++i)
        if (i >= k % p && (i - k % p) % (2 * k) < k && i / (2 * p) == (i + k) / (2 * p)) {
          const uint32_t a = max(w[i], w[i + k]);
          w[i + k] = min(w[i], w[i + k]);
          w[i] = a;
        }
}

// The choice on whole keys: lane j gets the j-th expert, or -1.
template <int V>
__device__ __forceinline__ int choose_exactly(uint32_t (&key)[V], int k, int lane) {
  int chosen = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const uint32_t top = __reduce_max_sync(~0u, best);
    if (top < kOpen) break;
    const unsigned e = expert<V>(lane, at), first = __reduce_min_sync(~0u, best == top ? e : ~0u);
    if (e == first) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v == at) key[v] = 0;
    }
    if (lane == j) chosen = static_cast<int>(first);
  }
  return chosen;
}

// The choices of the lanes, nearly in order, into it: falling logits, equal ones by rising
// experts, none (-1) last.  Neighbours are exchanged until two rounds change nothing.
__device__ __forceinline__ bool comes_before(float x, int e, float y, int f) {
  return e >= 0 && (f < 0 || x > y || (x == y && e < f));
}
__device__ __forceinline__ void sort_lanes(float &x, int &e, int lane) {
  for (int odd = 0, still = 0; still < 2; odd ^= 1) {
    const int other = ((lane - odd) ^ 1) + odd;
    const float y = __shfl_sync(~0u, x, other & 31);
    const int f = __shfl_sync(~0u, e, other & 31);
    const bool paired = other >= 0 && other < 32;
    const bool change = paired && (other > lane ? comes_before(y, f, x, e) : comes_before(x, e, y, f));
    if (change) {
      x = y;
      e = f;
    }
    still = __any_sync(~0u, change) ? 0 : still + 1;
  }
}

// Scores of all experts, for the probabilities: exp2 and the reciprocal are right to 2
// units and 1 unit in the last place, and flush what is below 2^-126 to 0; the difference
// and its product with log2(e) are rounded once each, 2 |l - m| 2^-24 relative in the
// result (2 |l| in a sigmoid).
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float exp_above(float l, float m) { return ex2_ftz((l - m) * kLog2e); }
__device__ __forceinline__ float exp_minus(float l) { return ex2_ftz(-kLog2e * l); }
__device__ __forceinline__ float sigmoid(float l) { return rcp_ftz(1.0f + exp_minus(l)); }
// Scores of the choices, one per lane and token, for the weights: their error does not grow
// with the argument (but for the rounding of l - m).  16384 tokens of 256 experts 17.65 us
// with the fast form here too, 17.75 so; backward 8.55 and 8.65; 262144 of 128 in BF16
// 102.0 and 103.8, 68.0 and 69.0.
__device__ __forceinline__ float chosen_above(float l, float m) { return expf(l - m); }
__device__ __forceinline__ float chosen_sigmoid(float l) { return rcp_ftz(1.0f + expf(-l)); }
// x's share of a sum of which it is a part; exactly 1 where it is all of it.
__device__ __forceinline__ float share_of(float x, float sum) {
  sum = fmaxf(sum, kTiny);
  return x == sum ? 1.0f : x * rcp_ftz(sum);
}

// Logits that are no numbers are closed, infinite ones the largest value.  Rare: the
// callers look for one in the row first.
template <int V>
__device__ __forceinline__ void make_finite(float (&l)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = l[v] > -INFINITY ? fminf(l[v], kBig) : -INFINITY;
}

// E * sum_e (counts_e / choices) * (probs_e / tokens) from the sum of their products.
__device__ __forceinline__ float balance(float sum, int E, int choices, int tokens) {
  return tokens > 0 ? static_cast<float>(E) * (sum / static_cast<float>(choices)) / static_cast<float>(tokens)
                    : 0.0f;
}

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

// Who else has tokens of the call: nobody (one CTA), the other CTAs of the cluster, or
// those of a whole grid, whose rows a second launch works out.
enum Mode { kOneCta, kOneCluster, kGrid };

// Dynamic shared memory: counts [warps][E], probabilities [warps][E, rounded up to 4],
// the warps' words that wait.
template <int kKind, int V, int kMode>
__global__ void __launch_bounds__(32 * warps_for(V))
route_kernel(const RouteArgs a) {
  constexpr bool alone = kMode != kGrid, clustered = kMode == kOneCluster;
  constexpr int kWarps = warps_for(V), kThreads = 32 * kWarps;
  constexpr int kEach = 32 * V > kThreads ? 32 * V / kThreads : 1;  // experts per thread, at most
  constexpr uint32_t kIndex = 32 * V - 1;                            // a word's index bits
  extern __shared__ __align__(16) int smem[];
  __shared__ int tokens_of[kWarps], scan[32], all_rows, cta_tokens, all_tokens;
  __shared__ float part[32];
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, k = a.k;
  const int E4 = round_up(E, 4);
  int *counts = smem;
  float *probs = reinterpret_cast<float *>(smem + kWarps * E);
  int *mine = counts + warp * E;
  float *my_probs = probs + warp * E4;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  if constexpr (many(V))
    for (int e = lane; e < E4; e += 32) my_probs[e] = 0.0f;
  __syncwarp();

  const int64_t cta_lo = static_cast<int64_t>(blockIdx.x) * a.per_cta;
  const int64_t cta_hi = min(static_cast<int64_t>(a.T), cta_lo + a.per_cta);
  // the first warps take one more: few tokens are spread over the SM's four schedulers
  const int n = static_cast<int>(cta_hi > cta_lo ? cta_hi - cta_lo : 0), each = n / kWarps, more = n % kWarps;
  const int64_t lo = cta_lo + warp * each + min(warp, more), hi = lo + each + (warp < more);
  const char *row = static_cast<const char *>(a.logits) + lo * a.ld * size_of(kKind);
  constexpr int kAhead = many(V) ? 1 : V;
  float psum[kAhead];
  Row<kKind, V> next;
#pragma unroll
  for (int v = 0; v < kAhead; ++v) psum[v] = 0.0f;
  int routed = 0;
  bool next_valid = true;
  if (lo < hi) {
    if constexpr (!many(V)) next.load(row, E, lane, a.vec);
    if (a.valid) next_valid = a.valid[lo] != 0;
  }

  uint32_t *queue = reinterpret_cast<uint32_t *>(probs + kWarps * E4) + warp * queue_words(V) + lane;
  if constexpr (many(V)) queue[32 * V] = 0;
  const uint32_t below = kIndex - expert<V>(lane, 0);  // index bits of the lane's first word
  for (int64_t t = lo; t < hi; ++t) {
    float l[V];
    const bool valid = next_valid;
    const char *here = row;
    row += a.ld * size_of(kKind);
    if constexpr (many(V)) next.load(here, E, lane, a.vec);
    next.values(l);
    if (t + 1 < hi) {  // in flight while this token is dealt with
      if constexpr (many(V)) prefetch_row(row, E * size_of(kKind), lane);
      else next.load(row, E, lane, a.vec);
      if (a.valid) next_valid = a.valid[t + 1] != 0;
    }
    int chosen = -1;
    float w = 0.0f;
    if (valid) {
      uint32_t word[V];
      const auto make_words = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v) word[v] = (key_of(l[v]) & ~kIndex) | (below - expert<V>(0, v));
        sort_falling(word);
      };
      make_words();
      if (__reduce_max_sync(~0u, word[0]) >= kSpecial) {
        make_finite(l);
        make_words();
      }
      // lane j keeps the j-th largest word; of FP32 logits one round more tells whether
      // the last choice is apart from the rest
      if constexpr (many(V)) {
#pragma unroll
        for (int v = 1; v < V; ++v) queue[32 * v] = word[v];
      }
      uint32_t kept = 0, top = 0;
      int at = 32;
      const auto round = [&](int j) {
        top = __reduce_max_sync(~0u, word[0]);
        if (lane == j) kept = top;
        if (word[0] == top) {
          if constexpr (many(V)) {
            word[0] = queue[at];
            at += 32;
          } else {
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) word[v] = word[v + 1];
            word[V - 1] = 0;
          }
        }
      };
      for (int j = 0; j < k + (kKind == kFp32); ++j) round(j);
      if (lane < k && kept >= kOpen) chosen = static_cast<int>(kIndex - (kept & kIndex));
      if constexpr (kKind == kFp32) {
        uint32_t behind = __shfl_down_sync(~0u, kept, 1);
        if (lane == k - 1) behind = top;
        if (__any_sync(~0u, lane < k && behind >= kOpen && ((kept ^ behind) & ~kIndex) == 0)) {
          const uint32_t last = __shfl_sync(~0u, kept, k - 1);
          int j = k + 1;
          while (top >= kOpen && ((top ^ last) & ~kIndex) == 0 && j < 32) round(j++);
          if (top >= kOpen && ((top ^ last) & ~kIndex) == 0) {
            uint32_t key[V];
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = key_of(l[v]);
            chosen = choose_exactly<V>(key, k, lane);
          } else {
            chosen = kept >= kOpen ? static_cast<int>(kIndex - (kept & kIndex)) : -1;
            float x = chosen >= 0 ? fminf(logit_at(here, kKind, chosen), kBig) : 0.0f;
            sort_lanes(x, chosen, lane);
            if (lane >= k) chosen = -1;
          }
        }
      }
      float x = 0.0f;
      if (chosen >= 0) x = fminf(logit_at(here, kKind, chosen), kBig);
      const float m = __shfl_sync(~0u, x, 0);  // the first choice is the largest
      routed += __shfl_sync(~0u, chosen, 0) >= 0;

      float s[V], sum = 0.0f;
      if (a.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = sigmoid(l[v]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = exp_above(l[v], m);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) sum += s[v];
      const float inv = rcp_ftz(fmaxf(warp_sum(sum), kTiny));
      if constexpr (many(V)) {
#pragma unroll
        for (int v = 0; v < V; v += 4) {
          const int e = expert<V>(lane, v);
          if (e < E) {
            float4 *p = reinterpret_cast<float4 *>(my_probs + e);
            const float4 q = *p;
            *p = make_float4(fmaf(s[v], inv, q.x), fmaf(s[v + 1], inv, q.y), fmaf(s[v + 2], inv, q.z),
                             fmaf(s[v + 3], inv, q.w));
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) psum[v] = fmaf(s[v], inv, psum[v]);
      }

      if (chosen >= 0) w = a.sigmoid ? chosen_sigmoid(x) : chosen_above(x, m) * inv;
      if (a.normalise) w = share_of(w, warp_sum(w));
    }
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
  if constexpr (!many(V)) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (expert<V>(lane, v) < E) my_probs[expert<V>(lane, v)] = psum[v];
  }
  if (lane == 0) tokens_of[warp] = routed;
  __syncthreads();

  // counts become the warps' first ranks; thread i has the experts from i * kEach on
  int total[kEach];
  float prob[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = threadIdx.x * kEach + i;
    int run = 0;
    float p = 0.0f;
    if (e < E) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int c = counts[w * E + e];
        counts[w * E + e] = run;
        run += c;
        p += probs[w * E4 + e];
      }
      if constexpr (!alone) {
        a.cta_counts[e * round_up(a.ctas, 8) + blockIdx.x] = static_cast<uint16_t>(run);
        a.cta_probs[e * round_up(a.ctas, 4) + blockIdx.x] = p;
      }
    }
    total[i] = run;
    prob[i] = p;
  }
  int tokens = warp_sum(lane < kWarps ? tokens_of[lane] : 0);
  __syncthreads();

  // where the probabilities were: each expert's total, probability and first row here
  int *total_of = smem + kWarps * E, *first_row = total_of + 2 * E;
  float *prob_of = reinterpret_cast<float *>(total_of + E);
  if constexpr (!alone) {
    if (threadIdx.x == 0) a.cta_tokens[blockIdx.x] = tokens;
  } else {
    const int rank = clustered ? blockIdx.x : 0;
    int before[kEach] = {};
    if constexpr (clustered) {
      // the totals of the cluster's CTAs, in the order of their tokens
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int e = threadIdx.x * kEach + i;
        if (e < E) {
          total_of[e] = total[i];
          prob_of[e] = prob[i];
        }
      }
      if (threadIdx.x == 0) cta_tokens = tokens;
      __syncwarp();  // whole warps come to a cluster's barriers
      cluster_sync_all();
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int e = threadIdx.x * kEach + i;
        total[i] = 0;
        prob[i] = 0.0f;
        if (e < E) {  // all loads in flight at once
          uint32_t c[kCluster], p[kCluster];
#pragma unroll
          for (int r = 0; r < kCluster; ++r) {
            c[r] = ld_cluster(mapa_shared(smem_u32(total_of + e), r));
            p[r] = ld_cluster(mapa_shared(smem_u32(prob_of + e), r));
          }
#pragma unroll
          for (int r = 0; r < kCluster; ++r) {
            total[i] += static_cast<int>(c[r]);
            before[i] += r < rank ? static_cast<int>(c[r]) : 0;
            prob[i] += __uint_as_float(p[r]);
          }
        }
      }
    }
    int all = 0;
    float loss = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      all += total[i];
      loss = fmaf(static_cast<float>(total[i]), prob[i], loss);
    }
    int first = cta_exclusive_sum(all, scan);
    loss = warp_sum(loss);
    if (lane == 0) part[warp] = loss;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = threadIdx.x * kEach + i;
      if (e < E) {
        if (rank == 0) {
          a.counts[e] = total[i];
          a.offs[e] = first;
        }
        first_row[e] = first + before[i];
      }
      first += total[i];
    }
    if (threadIdx.x == kThreads - 1) all_rows = first;
    if (threadIdx.x == 0) {
      if constexpr (clustered) {
        tokens = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) tokens += static_cast<int>(ld_cluster(mapa_shared(smem_u32(&cta_tokens), r)));
      }
      all_tokens = tokens;
    }
    __syncthreads();
    // what this CTA read of the others has arrived: all of it went into sums that were
    // stored before the barrier
    if constexpr (clustered) cluster_arrive_relaxed();
    const int rows = all_rows;
    if (rank == 0 && threadIdx.x == 0) {
      loss = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) loss += part[w];
      a.offs[E] = rows;
      a.tokens[0] = all_tokens;
      a.loss[0] = balance(loss, E, rows, all_tokens);
    }
    for (int i = rows + rank * kThreads + threadIdx.x; i < a.T * k; i += (clustered ? kCluster : 1) * kThreads)
      a.order[i] = -1;
  }

  // the warp's choices again, now with their ranks in the CTA (or their rows)
  for (int64_t i = lo * k + lane; i < hi * k; i += 32) {
    const int e = a.idx[i];
    if (e < 0) continue;
    int r = a.slot[i] + mine[e];
    if constexpr (alone) {
      r += first_row[e];
      a.order[r] = static_cast<int32_t>(i);
    }
    a.slot[i] = r;
  }
  if constexpr (clustered) {
    __syncwarp();
    cluster_wait();  // a CTA's totals stay until all have read them
  }
}

constexpr int kRowThreads = 1024;

// Sum of the first n (none if negative, eight at most) 16-bit counts.
__device__ __forceinline__ int sum8(uint4 v, int n) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  unsigned s = 0;
#pragma unroll
  for (int h = 0; h < 4; ++h) s = __dp2a_lo(w[h], 2 * h + 1 < n ? 0x0101u : 2 * h < n ? 0x0001u : 0u, s);
  return static_cast<int>(s);
}

// CTA b turns ranks into rows: expert e's choices of CTA b start at offs[e] plus the
// counts of the CTAs before it.  The CTAs of a cluster share the experts: each adds up the
// counts of its part, before the cluster's first CTA and in all, with as many threads per
// expert as there is room for (1 to 32, next to each other, eight CTAs' counts at a time,
// kBatch loads in flight in each), and the others read the sums from its shared memory.
// The last cluster also adds up the probabilities, and its first CTA writes the totals.
// More than 128 experts take clusters of two (16384 tokens of 256 experts 17.7 us, each
// CTA by itself 18.3, clusters of four, which do not all run at once, 21.9; of 1024 44.7,
// 54.8 and 44.7; of 64 13.0, 12.7 and 15.7), and more than 256 need five loads in a thread
// instead of three (of 256: 17.4 with three, 17.7 with five; of 512: 25.4 and 24.9).
template <int kRowCluster, int kBatch>
__global__ void __launch_bounds__(kRowThreads)
route_rows_kernel(const RouteArgs a) {
  constexpr int kPart = kMaxExperts / kRowCluster;
  __shared__ int first_row[kMaxExperts], scan[32], tokens_of[32];
  __shared__ int total_of[kPart], before_of[kRowCluster][kPart];  // of this CTA's part of the experts
  __shared__ float prob_of[kPart], loss_of[32];
  __shared__ int rows;
  wait_for_previous_kernel();
  const int E = a.E, k = a.k, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  const int rank = cta % kRowCluster, base = cta - rank;
  const bool last = base + kRowCluster == gridDim.x;
  const int64_t lo = static_cast<int64_t>(cta) * a.per_cta * k;
  const int64_t hi = min(static_cast<int64_t>(a.T) * k, lo + static_cast<int64_t>(a.per_cta) * k);
  // the thread's first choice, in flight while the counts are added up
  int next_idx = -1, next_slot = 0;
  if (lo + tid < hi) {
    next_idx = a.idx[lo + tid];
    next_slot = a.slot[lo + tid];
  }
  const int part = (E + kRowCluster - 1) / kRowCluster;  // experts of a CTA
  int share = 1;                                         // threads per expert
  while (share < 32 && 2 * share * part <= kRowThreads) share *= 2;
  const int at = tid / share, mine = tid % share, e = rank * part + at;
  const bool adds = at < part && e < E;
  int total = 0, before = 0, tokens = 0;
  float probs = 0.0f;
  if (last && rank == 0)
    for (int b = tid; b < a.ctas; b += kRowThreads) tokens += a.cta_tokens[b];
  int own[kRowCluster] = {};  // counts of the cluster's CTAs
  if (adds) {
    const uint16_t *counts = a.cta_counts + e * round_up(a.ctas, 8);
    const uint4 *c = reinterpret_cast<const uint4 *>(counts);
    if (mine == 0) {
#pragma unroll
      for (int r = 0; r < kRowCluster; ++r)
        if (base + r < a.ctas) own[r] = counts[base + r];
    }
    const int n = round_up(a.ctas, 8) / 8;
    for (int j0 = mine; j0 < n; j0 += kBatch * share) {
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v[i] = c[min(j0 + i * share, n - 1)];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int b0 = 8 * (j0 + i * share);
        total += sum8(v[i], a.ctas - b0);
        before += sum8(v[i], base - b0);
      }
    }
    if (last) {
      const float4 *p = reinterpret_cast<const float4 *>(a.cta_probs + e * round_up(a.ctas, 4));
      const int m = round_up(a.ctas, 4) / 4;
      for (int j0 = mine; j0 < m; j0 += kBatch * share) {
        float4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = p[min(j0 + i * share, m - 1)];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int b0 = j0 + i * share < m ? 4 * (j0 + i * share) : a.ctas;
          const float w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int h = 0; h < 4; ++h) probs += b0 + h < a.ctas ? w[h] : 0.0f;
        }
      }
    }
  }
  for (int o = 1; o < share; o *= 2) {
    total += __shfl_xor_sync(~0u, total, o);
    before += __shfl_xor_sync(~0u, before, o);
    probs += __shfl_xor_sync(~0u, probs, o);
  }
  if (adds && mine == 0) {
    total_of[at] = total;
    prob_of[at] = probs;
#pragma unroll
    for (int r = 0; r < kRowCluster; ++r) {
      before_of[r][at] = before;
      before += own[r];
    }
  }
  __syncwarp();  // whole warps come to a cluster's barriers
  cluster_sync_all();
  // thread i has expert i from here on
  total = before = 0;
  probs = 0.0f;
  if (tid < E) {
    const int owner = tid / part, there = tid % part;
    total = static_cast<int>(ld_cluster(mapa_shared(smem_u32(total_of + there), owner)));
    before = static_cast<int>(ld_cluster(mapa_shared(smem_u32(&before_of[rank][there]), owner)));
    if (last && rank == 0) probs = __uint_as_float(ld_cluster(mapa_shared(smem_u32(prob_of + there), owner)));
  }
  const int first = cta_exclusive_sum(total, scan);
  first_row[tid] = first + before;
  if (tid == kRowThreads - 1) rows = first + total;
  if (last && rank == 0) {
    if (tid < E) {
      a.counts[tid] = total;
      a.offs[tid] = first;
    }
    const float p = warp_sum(static_cast<float>(total) * probs);
    tokens = warp_sum(tokens);
    if (lane == 0) {
      loss_of[warp] = p;
      tokens_of[warp] = tokens;
    }
  }
  __syncthreads();
  // what this CTA read of the others has arrived: it was stored before the barrier
  cluster_arrive_relaxed();
  if (last && rank == 0 && warp == 0) {
    const float loss = warp_sum(loss_of[lane]);
    tokens = warp_sum(tokens_of[lane]);
    if (lane == 0) {
      a.offs[E] = rows;
      a.tokens[0] = tokens;
      a.loss[0] = balance(loss, E, rows, tokens);
    }
  }
  for (int64_t i = lo + tid; i < hi; i += kRowThreads) {
    const int x = next_idx, rank_here = next_slot;
    if (i + kRowThreads < hi) {
      next_idx = a.idx[i + kRowThreads];
      next_slot = a.slot[i + kRowThreads];
    }
    if (x >= 0) {
      const int r = rank_here + first_row[x];
      a.slot[i] = r;
      a.order[r] = static_cast<int32_t>(i);
    }
    if (i >= rows) a.order[i] = -1;
  }
  __syncwarp();
  cluster_wait();  // a CTA's sums stay until all have read them
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
// CTAs of eight warps that an SM's registers hold.  16384 tokens: 512 experts FP32 13.5 us
// with three, 16.2 with four, BF16 12.7 and 11.8; 256 8.7 with three and with four, 10.6
// with five; 1024 24.7 with two, 29.0 with three.
constexpr int bwd_ctas_per_sm(int kind, int V) {
  return V == 1 ? 6 : V <= 8 ? 4 : V == 16 ? (kind == kFp32 ? 3 : 4) : 2;
}

template <int kKind, int V>
__global__ void __launch_bounds__(256, bwd_ctas_per_sm(kKind, V))
route_bwd_kernel(const BwdArgs a) {
  extern __shared__ __align__(16) float of_warps[];  // [warps][32 * V], many experts: and dp [32 * V]
  wait_for_previous_kernel();
  constexpr int W = width(V), kAhead = many(V) ? 1 : V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E, k = a.k;
  float *u_of = of_warps + warp * 32 * V, *dp_of = of_warps + (blockDim.x >> 5) * 32 * V;
  const int warps = gridDim.x * (blockDim.x >> 5);
  // lane j's choice, and the row's logits
  struct {
    Row<kKind, V> l;
    int at;
    float dw;
    bool valid;
  } next;
  const auto fetch = [&](int64_t t) {
    next.valid = !a.valid || a.valid[t] != 0;
    const char *row = static_cast<const char *>(a.logits) + t * a.ld * size_of(kKind);
    if constexpr (many(V)) prefetch_row(row, E * size_of(kKind), lane);
    else next.l.load(row, E, lane, a.vec);
    next.at = -1;
    next.dw = 0.0f;
    if (lane < k && a.dweight) {
      next.at = a.idx[t * k + lane];
      next.dw = a.dweight[t * k + lane];
    }
  };
  int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (t < a.T) fetch(t);
  float dp[kAhead];
  {
    int c[V], n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert<V>(lane, v);
      u_of[e] = 0.0f;
      c[v] = e < E && a.dloss ? a.counts[e] : 0;
      n += c[v];
    }
    n = warp_sum(n);
    const int tokens = a.dloss ? a.tokens[0] : 0;
    const float f = tokens > 0 && n > 0 ? a.dloss[0] * static_cast<float>(E) / static_cast<float>(n) /
                                              static_cast<float>(tokens)
                                        : 0.0f;
    if constexpr (many(V)) {
      if (warp == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) dp_of[expert<V>(lane, v)] = f * static_cast<float>(c[v]);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) dp[v] = f * static_cast<float>(c[v]);
      __syncwarp();
    }
  }
  // W of dp, from the lane's v-th expert on
  const auto dp_at = [&](int v, float (&d)[W]) {
    if constexpr (many(V)) {
      const float4 q = *reinterpret_cast<const float4 *>(dp_of + expert<V>(lane, v));
      d[0] = q.x;
      d[1] = q.y;
      d[2] = q.z;
      d[3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) d[i] = dp[v + i];
    }
  };
  for (; t < a.T; t += warps) {
    float l[V], s[V], c[V];  // c: 1 - s of a sigmoid
    const char *row = static_cast<const char *>(a.logits) + t * a.ld * size_of(kKind);
    const bool valid = next.valid;
    if constexpr (many(V)) next.l.load(row, E, lane, a.vec);
    next.l.values(l);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!valid) l[v] = -INFINITY;
    const int given = valid && next.at < E ? next.at : -1;
    const float given_dw = next.dw * a.scale;
    if (t + warps < a.T) fetch(t + warps);  // in flight while this token is dealt with

    bool special = false;
#pragma unroll
    for (int v = 0; v < V; ++v) special |= !(l[v] < INFINITY);
    if (__any_sync(~0u, special)) make_finite(l);
    float sum = 0.0f, m = 0.0f;
    if (a.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float e = exp_minus(l[v]);
        s[v] = rcp_ftz(1.0f + e);
        c[v] = fminf(e, 0x1p126f) * s[v];  // any value will do where s is 0
        sum += s[v];
      }
    } else {
      m = -kBig;
#pragma unroll
      for (int v = 0; v < V; ++v) m = fmaxf(m, l[v]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = exp_above(l[v], m);
        c[v] = 1.0f;
        sum += s[v];
      }
    }
    float pdp = 0.0f;
#pragma unroll
    for (int v = 0; v < V; v += W) {
      float d[W];
      dp_at(v, d);
#pragma unroll
      for (int i = 0; i < W; ++i) pdp = fmaf(s[v + i], d[i], pdp);
    }
    const float inv = rcp_ftz(fmaxf(warp_sum(sum), kTiny));
    pdp = warp_sum(pdp) * inv;

    // lane j has choice j's score and gradient; the gradients change lanes through
    // shared memory, all zeros but for these
    float x = given >= 0 ? logit_at(row, kKind, given) : -INFINITY;
    // where there is no choice, or of a closed expert, the gradient does not count, whatever it is
    const int at = x > -INFINITY ? given : -1;
    x = fminf(x, kBig);
    const float dw = at >= 0 ? given_dw : 0.0f;
    float u = at < 0 ? 0.0f : a.sigmoid ? chosen_sigmoid(x) : chosen_above(x, m) * inv;
    if (a.normalise) {
      u = share_of(u, warp_sum(u));
      u *= dw - warp_sum(u * dw);
    } else {
      u *= dw;
    }
    const float usum = a.sigmoid || a.normalise ? 0.0f : warp_sum(u);
    // (a choice that comes twice, which the forward pass does not make, adds up)
    if (at >= 0) u_of[at] = __int_as_float(lane);
    __syncwarp();
    const bool twice = at >= 0 && __float_as_int(u_of[at]) != lane;
    __syncwarp();
    if (__any_sync(~0u, twice)) {
      if (at >= 0) u_of[at] = 0.0f;
      __syncwarp();
      if (at >= 0) atomicAdd(u_of + at, u);
    } else if (at >= 0) {
      u_of[at] = u;
    }
    __syncwarp();
    // closed experts have s = 0 and u = 0
    const float z = pdp + usum;
    char *out = static_cast<char *>(a.dlogits) + t * a.ld_d * size_of(kKind);
#pragma unroll
    for (int v = 0; v < V; v += W) {
      const int e = expert<V>(lane, v);
      float d[W], us[W];
      dp_at(v, d);
      if constexpr (W == 4) {
        const float4 q = *reinterpret_cast<const float4 *>(u_of + e);
        us[0] = q.x;
        us[1] = q.y;
        us[2] = q.z;
        us[3] = q.w;
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) us[i] = u_of[e + i];
      }
#pragma unroll
      for (int i = 0; i < W; ++i) d[i] = fmaf(s[v + i] * inv, d[i] - z, us[i]) * c[v + i];
      if (W > 1 && a.vec_d) {
        if (e < E) {
          if constexpr (W == 4 && kKind == kFp32)
            *reinterpret_cast<float4 *>(out + 4 * e) = make_float4(d[0], d[1], d[2], d[3]);
          else if constexpr (W == 4)
            *reinterpret_cast<uint2 *>(out + 2 * e) = make_uint2(bf16x2(d[0], d[1]), bf16x2(d[2], d[3]));
          else if constexpr (W == 2 && kKind == kFp32)
            *reinterpret_cast<float2 *>(out + 4 * e) = make_float2(d[0], d[1]);
          else if constexpr (W == 2)
            *reinterpret_cast<uint32_t *>(out + 2 * e) = bf16x2(d[0], d[1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (e + i < E) {
            if constexpr (kKind == kFp32) reinterpret_cast<float *>(out)[e + i] = d[i];
            else reinterpret_cast<uint16_t *>(out)[e + i] = static_cast<uint16_t>(bf16x2(d[i], 0.0f));
          }
      }
    }
    __syncwarp();
    if (at >= 0) u_of[at] = 0.0f;
    __syncwarp();  // before another lane writes the next token's choice of the same expert
  }
}

// How a call's tokens are spread; the same for every device, so that the probabilities'
// sums are too.  256 experts: 17 tokens take 4.7 us in one CTA and 5.6 in a cluster, 64
// take 7.9, 5.8 and, in two launches, 8.0, 256 take 7.4 in a cluster and 8.4 in two
// launches, 512 9.9 and 8.5.  512 experts: 64 tokens 10.8, 7.9 and 10.0.  The totals of
// more take longer to exchange than a second launch (1024 experts: 32 tokens 11.2 in one
// CTA and 11.9 in two launches, 64 12.4 in a cluster and 12.1, 256 17.7 and 14.2).
struct Plan {
  Mode mode;
  int ctas, per_cta;
};
Plan plan(int64_t T, int64_t E) {
  Plan p;
  if (T <= kOneCtaTokens) {
    p.mode = kOneCta;
    p.ctas = 1;
  } else if (E <= 512 && T <= kCluster * kOneCtaTokens) {
    p.mode = kOneCluster;
    p.ctas = kCluster;
  } else {
    p.mode = kGrid;
    const int64_t full = (T + kFewPerCta - 1) / kFewPerCta, most = (T + kMaxPerCta - 1) / kMaxPerCta;
    p.ctas = static_cast<int>(most > kSms ? most : full < kSms ? full : kSms);
  }
  p.per_cta = static_cast<int>((T + p.ctas - 1) / p.ctas);
  return p;
}

bool shape_ok(int64_t T, int64_t E) {
  return T >= 0 && T <= (int64_t{1} << 26) && E >= 1 && E <= kMaxExperts;
}

template <int kKind, int V, int kMode>
fp8q_status launch_choice(const RouteArgs &a, cudaStream_t s) {
  constexpr int kWarps = warps_for(V), kQueues = kWarps * queue_words(V) * 4, kMost = kWarps * 32 * V * 8 + kQueues;
  constexpr auto kern = route_kernel<kKind, V, kMode>;
  const size_t smem = static_cast<size_t>(kWarps) * (a.E + round_up(a.E, 4)) * 4 + kQueues;
  if (smem > 40 * 1024)
    if (fp8q_status st = allow_smem<kern>(kMost)) return st;
  if constexpr (kMode == kOneCluster)
    return launch_dependent_cluster(kern, dim3(kCluster), dim3(32 * kWarps), smem, s, kCluster, a);
  return launch_dependent(kern, dim3(a.ctas), dim3(32 * kWarps), smem, s, a);
}

template <int kKind, int V>
fp8q_status launch_route(const RouteArgs &a, Mode mode, cudaStream_t s) {
  if (mode == kOneCta) return launch_choice<kKind, V, kOneCta>(a, s);
  if constexpr (V <= 16) {
    if (mode == kOneCluster) return launch_choice<kKind, V, kOneCluster>(a, s);
  }
  if (fp8q_status st = launch_choice<kKind, V, kGrid>(a, s)) return st;
  if constexpr (V <= 4)
    return launch_dependent(route_rows_kernel<1, 3>, dim3(a.ctas), dim3(kRowThreads), 0, s, a);
  else
    return launch_dependent_cluster(route_rows_kernel<2, V <= 8 ? 3 : 5>, dim3(round_up(a.ctas, 2)), dim3(kRowThreads),
                                    0, s, 2, a);
}

template <int kKind>
fp8q_status launch_route(const RouteArgs &a, Mode mode, cudaStream_t s) {
  if (a.E <= 32) return launch_route<kKind, 1>(a, mode, s);
  if (a.E <= 64) return launch_route<kKind, 2>(a, mode, s);
  if (a.E <= 128) return launch_route<kKind, 4>(a, mode, s);
  if (a.E <= 256) return launch_route<kKind, 8>(a, mode, s);
  if (a.E <= 512) return launch_route<kKind, 16>(a, mode, s);
  return launch_route<kKind, 32>(a, mode, s);
}

template <int kKind, int V>
fp8q_status launch_bwd(const BwdArgs &a, cudaStream_t s) {
  const int warps = 8, need = (a.T + warps - 1) / warps, most = kSms * bwd_ctas_per_sm(kKind, V);
  const size_t smem = static_cast<size_t>(warps + many(V)) * 32 * V * sizeof(float);
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
  const Plan p = plan(T, E);
  return p.mode != kGrid ? 0 : E * (2 * round_up(p.ctas, 8) + 4 * round_up(p.ctas, 4)) + 4ll * p.ctas;
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
  const Plan p = plan(T, E);
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
  a.cta_counts = static_cast<uint16_t *>(workspace);
  a.cta_probs = reinterpret_cast<float *>(a.cta_counts + E * round_up(p.ctas, 8));
  a.cta_tokens = reinterpret_cast<int *>(a.cta_probs + E * round_up(p.ctas, 4));
  a.ld = ld;
  a.T = static_cast<int>(T);
  a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.ctas = p.ctas;
  a.per_cta = p.per_cta;
  a.scale = scale;
  a.sigmoid = score == FP8Q_SCORE_SIGMOID;
  a.normalise = normalise != 0;
  a.vec = E % 4 == 0 && row_vectors(logits, ld, dtype);
  auto st = static_cast<cudaStream_t>(stream);
  return dtype == kBf16 ? launch_route<kBf16>(a, p.mode, st) : launch_route<kFp32>(a, p.mode, st);
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
  a.vec = E % 4 == 0 && row_vectors(logits, ld, dtype);
  a.vec_d = E % 4 == 0 && row_vectors(dlogits, ld_d, dtype);
  auto st = static_cast<cudaStream_t>(stream);
  return dtype == kBf16 ? launch_bwd<kBf16>(a, st) : launch_bwd<kFp32>(a, st);
}
