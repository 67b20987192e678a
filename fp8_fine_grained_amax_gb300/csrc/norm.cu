// norm.cu -- root-mean-square norm with the residual's addition and an FP8
// result, and its backward pass.
//
//   forward   h = x + res,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * w
//   backward  xh = x * rstd,  c = mean(dy * w * xh) over the row,
//             dx = rstd * (dy * w - xh * c) + dres,  dw = sum over rows of dy * xh
//
// Both are bound by memory.  A row is read once and stays in registers between
// its sum and its results: a warp holds a short one, a CTA a longer one.  Sums and
// statistics are FP32; the codes quantise the unrounded y.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8q.h"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"
#include "fp8q_vec.cuh"

namespace fp8q {

namespace {

constexpr int kMaxCols = 32768;         // 1024 threads with four 8-column vectors each
constexpr int kWarpCols = 1024;         // backward: one warp with four vectors per lane
constexpr int kForwardWarpCols = 512;   // forward: one warp with two
constexpr int kRowWarps = 8;            // rows per CTA in the warp forms
constexpr int kSms = 152;
constexpr int kRingBytes = 216 * 1024;  // of an SM's shared memory, for rings

// Sum over the row's threads, the same in all of them: a warp, or the CTA's
// warps through shared memory (`part` may be used again after another barrier).
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float *part) {
  v = warp_sum(v);
  if constexpr (!kWarpRow) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum(lane < warps ? part[lane] : 0.0f);
  }
  return v;
}

// ------------------------------------------------------------------ ring
// Rows on their way into shared memory, laid out as in memory, by asynchronous
// 16-byte copies.  A warp copies the vectors that its own lanes read, in whole runs of
// 512 bytes, so a warp barrier between its wait and its reads, and one between its
// reads and the next copies, is all that the ring needs.  (Bulk copies of whole rows
// under barriers of their own were slower: 8192 x 7168 BF16 69 to 76 us forward and
// 80 us backward, for 67 and 75.  So were copies that put the two halves of FP32
// vectors into planes of their own, which reached the L2 one sector at a time.)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
constexpr int kMostStages = 4;
// Until the oldest of the `stages` groups on their way is there.
__device__ __forceinline__ void oldest_wait(int stages) {
  if (stages == 4) copies_wait<3>();
  else if (stages == 3) copies_wait<2>();
  else copies_wait<1>();
}

// A warp's 32 vectors of 8 columns from vec0 on, of one row, to the row's place in the
// ring.
template <int kKind>
__device__ __forceinline__ void fetch32(uint32_t row_at, const void *base, int64_t row_start, int vec0, int nvec,
                                        int lane) {
  constexpr int kBytes = 8 * size_of(kKind);
  const char *p = static_cast<const char *>(base) + row_start * size_of(kKind);
#pragma unroll
  for (int j = 0; j < kBytes / 16; ++j) {
    const int at = vec0 * kBytes + (32 * j + lane) * 16;
    if (at < nvec * kBytes) copy16(row_at + at, p + at);
  }
}

// Eight values of a row in shared memory.  32-byte pieces of FP32 rows would meet on
// the same banks two by two; every other four lanes read theirs the other way round.
template <int kKind>
__device__ __forceinline__ void ring8(uint32_t row, int vec, float (&v)[8]) {
  if constexpr (kKind == kBf16) {
    unpack8(ld_shared_v4(row + vec * 16), v);
  } else {
    const bool turned = vec & 4;
    const uint32_t at = row + vec * 32;
    const uint4 a = ld_shared_v4(at + (turned ? 16 : 0)), b = ld_shared_v4(at + (turned ? 0 : 16));
    unpack8(turned ? b : a, turned ? a : b, v);
  }
}

// ------------------------------------------------------------------ forward
struct NormArgs {
  const void *x, *res, *w;
  void *r, *y;
  uint8_t *q;
  float *s, *rstd;
  int64_t ldx, ld_res, ld_r, ldy, ldq, ld_s, T;
  int nvec;    // C / 8
  int stages;  // of the ring
  float inv_c, eps;
  bool w_fp32, pow2;
};

__device__ __forceinline__ void store_codes(const NormArgs &a, int64_t row, int vec, float inv,
                                            float (&h)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] *= inv;
  *reinterpret_cast<uint2 *>(a.q + row * a.ldq + 8 * vec) =
      make_uint2(codes4(h[0], h[1], h[2], h[3]), codes4(h[4], h[5], h[6], h[7]));
}

// Codes and scales of V vectors per lane, `step` vectors apart, the whole warp
// together.  The 16 lanes of a 1x128 group are all in the row, or none is.  Of two
// vectors' groups each half of the 16 lanes reduces one and takes its scale, so that
// two groups cost four exchanges and two quotients.
template <int V>
__device__ __forceinline__ void quantise(const NormArgs &a, int64_t row, int first, int step, float (&h)[V][8]) {
  const bool upper = threadIdx.x & 8;
  if constexpr (V == 1) {
    float m = absmax8(h[0]), s, inv;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    group_scale(m, a.pow2, s, inv);
    if (first < a.nvec) {
      if ((first & 15) == 0) a.s[static_cast<int64_t>(first >> 4) * a.ld_s + row] = s;
      store_codes(a, row, first, inv, h[0]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float m0 = absmax8(h[i]), m1 = absmax8(h[i + 1]);
      float m = upper ? m1 : m0, s, inv;
      m = fmaxf(m, __shfl_xor_sync(~0u, upper ? m0 : m1, 8));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      group_scale(m, a.pow2, s, inv);
      const float other = __shfl_xor_sync(~0u, inv, 8);
      const int v0 = first + i * step, v1 = v0 + step;
      const int mine = upper ? v1 : v0;
      if ((threadIdx.x & 7) == 0 && mine < a.nvec) a.s[static_cast<int64_t>(mine >> 4) * a.ld_s + row] = s;
      if (v0 < a.nvec) store_codes(a, row, v0, upper ? other : inv, h[i]);
      if (v1 < a.nvec) store_codes(a, row, v1, upper ? inv : other, h[i + 1]);
    }
  }
}

// y = h * rstd * w of one vector, in place.
__device__ __forceinline__ void scale8(float (&h)[8], float rstd, const float (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = h[e] * rstd * w[e];
}

// Rows straight from memory: a warp or a CTA per row, V vectors per thread.
template <int kX, int kRes, int V, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowWarps : 1024)
rmsnorm_kernel(const NormArgs a) {
  __shared__ float part[32];
  wait_for_previous_kernel();
  const int64_t row = kWarpRow ? static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5)
                               : blockIdx.x;
  if (kWarpRow && row >= a.T) return;
  const int first = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
  const int step = kWarpRow ? 32 : blockDim.x;

  float h[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = first + i * step;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
    if (vec < a.nvec) load8<kX>(a.x, row * a.ldx + 8 * vec, h[i]);
  }
  if constexpr (kRes != kNone) {
    float z[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = first + i * step;
      if (vec < a.nvec) {
        load8<kRes>(a.res, row * a.ld_res + 8 * vec, z[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += z[i][e];
      }
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
  if constexpr (kRes != kNone) {
    if (a.r) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int vec = first + i * step;
        if (vec < a.nvec) store8<kRes>(a.r, row * a.ld_r + 8 * vec, h[i]);
      }
    }
  }
  sum = row_sum<kWarpRow>(sum, part);
  const float rstd = rsqrtf(fmaf(sum, a.inv_c, a.eps));
  if (a.rstd && first == 0) a.rstd[row] = rstd;
  if (!a.y && !a.q) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = first + i * step;
    if (vec < a.nvec) {
      float w[8];
      load8_w(a.w, a.w_fp32, 8 * vec, w);
      scale8(h[i], rstd, w);
      if (a.y) store8<kBf16>(a.y, row * a.ldy + 8 * vec, h[i]);
    }
  }
  if (a.q) quantise<V>(a, row, first, step, h);
}

// Rows of more than 512 columns: CTA b takes rows b, b + gridDim, ..., V vectors per
// thread, with the next rows on their way into shared memory while one is dealt with.
// (1024 columns BF16, 16384 rows: 17.7 us; a warp per row straight from memory 23.6.)
template <int kX, int kRes, int V>
__global__ void __launch_bounds__(1024)
rmsnorm_rows_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float part[2][32];
  wait_for_previous_kernel();
  const int threads = blockDim.x, lane = threadIdx.x & 31, vec0 = threadIdx.x - lane, last = a.stages - 1;
  const uint32_t x_bytes = 8 * a.nvec * size_of(kX);
  const uint32_t stage_bytes = x_bytes + (kRes == kNone ? 0 : 8 * a.nvec * size_of(kRes));
  const uint32_t base = smem_u32(ring);
  const auto fetch = [&](int64_t row, int stage) {
    if (row < a.T) {
      const uint32_t at = base + stage * stage_bytes;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        fetch32<kX>(at, a.x, row * a.ldx, vec0 + i * threads, a.nvec, lane);
        if constexpr (kRes != kNone)
          fetch32<kRes>(at + x_bytes, a.res, row * a.ld_res, vec0 + i * threads, a.nvec, lane);
      }
    }
    copies_commit();
  };
  const int64_t step = gridDim.x;
  int64_t row = blockIdx.x;
  for (int i = 0; i < last; ++i) fetch(row + i * step, i);
  constexpr int kHeld = V <= 2 ? V : 1;  // weights stay in registers where there is room
  float w[kHeld][8] = {};
  if constexpr (V <= 2) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = threadIdx.x + i * threads;
      if (vec < a.nvec) load8_w(a.w, a.w_fp32, 8 * vec, w[i]);
    }
  }

  int turn = 0, stage = 0;
  for (; row < a.T; row += step, turn ^= 1) {
    fetch(row + last * step, stage == 0 ? last : stage - 1);
    oldest_wait(a.stages);
    __syncwarp();
    float h[V][8], sum = 0.0f;
    const uint32_t at = base + stage * stage_bytes;
    stage = stage == last ? 0 : stage + 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = threadIdx.x + i * threads;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
      if (vec < a.nvec) {
        ring8<kX>(at, vec, h[i]);
        if constexpr (kRes != kNone) {
          float z[8];
          ring8<kRes>(at + x_bytes, vec, z);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] += z[e];
          if (a.r) store8<kRes>(a.r, row * a.ld_r + 8 * vec, h[i]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
    }
    sum = row_sum<false>(sum, part[turn]);
    const float rstd = rsqrtf(fmaf(sum, a.inv_c, a.eps));
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (!a.y && !a.q) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = threadIdx.x + i * threads;
      if (vec < a.nvec) {
        if constexpr (V <= 2) {
          scale8(h[i], rstd, w[i]);
        } else {
          load8_w(a.w, a.w_fp32, 8 * vec, w[0]);
          scale8(h[i], rstd, w[0]);
        }
        if (a.y) store8<kBf16>(a.y, row * a.ldy + 8 * vec, h[i]);
      }
    }
    if (a.q) quantise<V>(a, row, threadIdx.x, threads, h);
  }
}

// Stages of a ring with `bytes` of each on an SM: what keeps at most `budget` bytes of
// an SM's shared memory in use, from 2 to 4.  More rows on their way were slower: 8192 x
// 7168 BF16 forward 67.2 us with three stages (86 KB), 68.1 with four; backward 73.6
// with three (129 KB), 75.0 with four, 77.0 with two; 16384 x 1024 backward 30.0 with
// two (98 KB), 34.1 with three.  1 or 0 where not even two fit.
int ring_stages(int bytes, int budget) {
  const int n = budget / bytes;
  if (n >= 2) return n < kMostStages ? n : kMostStages;
  return kRingBytes / bytes < 2 ? kRingBytes / bytes : 2;
}
constexpr int kForwardBudget = 96 * 1024, kBackwardBudget = 132 * 1024;

template <auto kKern, typename Args>
fp8q_status launch_ring(int64_t ctas, int threads, int smem, cudaStream_t s, const Args &a) {
  if (smem > 40 * 1024)
    if (fp8q_status st = allow_smem<kKern>(kRingBytes)) return st;
  return launch_dependent(kKern, dim3(static_cast<unsigned>(ctas)), dim3(threads), smem, s, a);
}

// Threads for one row of nvec vectors, V of them each.
int row_threads(int nvec, int V) { return (nvec + 32 * V - 1) / (32 * V) * 32; }

template <int kX, int kRes>
fp8q_status launch_norm(const NormArgs &a, cudaStream_t s) {
  if (a.nvec <= kForwardWarpCols / 8) {
    const dim3 grid(static_cast<unsigned>((a.T + kRowWarps - 1) / kRowWarps)), block(32 * kRowWarps);
    if (a.nvec <= 32) return launch_dependent(rmsnorm_kernel<kX, kRes, 1, true>, grid, block, 0, s, a);
    return launch_dependent(rmsnorm_kernel<kX, kRes, 2, true>, grid, block, 0, s, a);
  }
  // Vectors per thread: two share the row's sum and the codes' exchanges (8192 x 2048
  // BF16 17.8 us against 21.4 with one), one keeps more warps busy in rows of 4096 to
  // 8192 columns (8192 x 7168 67.2 against 69.4) and finishes a lone row sooner.
  const int V = a.nvec <= 1024 && (a.nvec >= 512 || a.T <= kSms) ? 1 : a.nvec <= 2048 ? 2 : 4;
  const int threads = row_threads(a.nvec, V), per_sm = 1024 / threads;
  const int stage = 8 * a.nvec * (size_of(kX) + (kRes == kNone ? 0 : size_of(kRes)));
  NormArgs b = a;
  b.stages = ring_stages(stage * per_sm, kForwardBudget);
  const int smem = b.stages * stage;
  if (b.stages < 2)
    return launch_dependent(rmsnorm_kernel<kX, kRes, 4, false>, dim3(static_cast<unsigned>(a.T)),
                            dim3(row_threads(a.nvec, 4)), 0, s, a);
  const int64_t most = static_cast<int64_t>(kSms) * per_sm, ctas = a.T < most ? a.T : most;
  if (V == 1) return launch_ring<rmsnorm_rows_kernel<kX, kRes, 1>>(ctas, threads, smem, s, b);
  if (V == 2) return launch_ring<rmsnorm_rows_kernel<kX, kRes, 2>>(ctas, threads, smem, s, b);
  return launch_ring<rmsnorm_rows_kernel<kX, kRes, 4>>(ctas, threads, smem, s, b);
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
  const void *dy, *x, *w, *dres;
  const float *rstd;
  void *dx;
  float *part;  // [CTAs][C], null without dw
  int64_t ld_dy, ldx, ld_dres, ld_dx, T;
  int nvec, stages;
  float inv_c;
  bool w_fp32;
};

// The gradient's part of one vector: adds to the row's sum and to dw.
__device__ __forceinline__ void bwd_terms(float (&t)[8], float (&xh)[8], const float (&w)[8],
                                          float rstd, float (&dw)[8], float &sum) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    xh[e] *= rstd;
    dw[e] = fmaf(t[e], xh[e], dw[e]);
    t[e] *= w[e];
    sum = fmaf(t[e], xh[e], sum);
  }
}
__device__ __forceinline__ void bwd_dx(float (&d)[8], const float (&t)[8], const float (&xh)[8],
                                       float rstd, float c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) d[e] = fmaf(rstd, fmaf(-xh[e], c, t[e]), d[e]);
}

// All forms leave the sum of a CTA's rows' dy * xh in part[CTA], over rows that
// depend on T, C and the types alone, so dw is summed in a fixed order.
//
// Rows as in the forward pass's ring, each taken by a CTA, or by one of its eight
// warps with a ring of its own (rows of up to 1024 columns).  Two vectors of a long row
// are read from shared memory again for dx: 1024 threads have 64 registers each.
template <int kDy, int kX, int kDx, int V, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowWarps : 1024)
rmsnorm_bwd_kernel(const BwdArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sums[2][32], rstds[kMostStages][32];  // a warp's own copy of its rows' rstd
  constexpr bool kAgain = !kWarpRow && V > 1;
  constexpr bool kHold = V <= 2;  // the weights, in registers
  constexpr int kKept = kAgain ? 1 : V, kHeld = kHold ? V : 1;
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, last = a.stages - 1;
  const int first_vec = kWarpRow ? lane : threadIdx.x, vec0 = first_vec - lane;
  const int gap = kWarpRow ? 32 : blockDim.x;  // between a thread's vectors
  const uint32_t y_bytes = 8 * a.nvec * size_of(kDy), x_bytes = 8 * a.nvec * size_of(kX);
  const uint32_t stage_bytes = y_bytes + x_bytes + (a.dres ? 8 * a.nvec * size_of(kDx) : 0);
  const uint32_t base = smem_u32(ring) + (kWarpRow ? warp * a.stages * stage_bytes : 0);
  const auto fetch = [&](int64_t row, int stage) {
    if (row < a.T) {
      if (lane == 0) copy4(smem_u32(&rstds[stage][warp]), a.rstd + row);
      const uint32_t at = base + stage * stage_bytes;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int from = vec0 + i * gap;
        fetch32<kDy>(at, a.dy, row * a.ld_dy, from, a.nvec, lane);
        fetch32<kX>(at + y_bytes, a.x, row * a.ldx, from, a.nvec, lane);
        if (a.dres) fetch32<kDx>(at + y_bytes + x_bytes, a.dres, row * a.ld_dres, from, a.nvec, lane);
      }
    }
    copies_commit();
  };
  const int64_t step = kWarpRow ? static_cast<int64_t>(gridDim.x) * kRowWarps : gridDim.x;
  int64_t row = kWarpRow ? static_cast<int64_t>(blockIdx.x) * kRowWarps + warp : blockIdx.x;
  for (int i = 0; i < last; ++i) fetch(row + i * step, i);
  float w[kHeld][8] = {}, dw[V][8] = {};
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = first_vec + i * gap;
      if (vec < a.nvec) load8_w(a.w, a.w_fp32, 8 * vec, w[i]);
    }
  }

  int turn = 0, stage = 0;
  for (; row < a.T; row += step, turn ^= 1) {
    fetch(row + last * step, stage == 0 ? last : stage - 1);
    oldest_wait(a.stages);
    __syncwarp();
    const float rstd = *(volatile float *)&rstds[stage][warp];
    const uint32_t at = base + stage * stage_bytes;
    stage = stage == last ? 0 : stage + 1;
    float t[kKept][8], xh[kKept][8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int k = kAgain ? 0 : i, vec = first_vec + i * gap;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[k][e] = xh[k][e] = 0.0f;
      if (vec < a.nvec) {
        ring8<kDy>(at, vec, t[k]);
        ring8<kX>(at + y_bytes, vec, xh[k]);
        if constexpr (!kHold) load8_w(a.w, a.w_fp32, 8 * vec, w[0]);
      }
      bwd_terms(t[k], xh[k], w[kHold ? i : 0], rstd, dw[i], sum);
    }
    if (a.dx) {
      const float c = row_sum<kWarpRow>(sum, sums[turn]) * a.inv_c;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int k = kAgain ? 0 : i, vec = first_vec + i * gap;
        if (vec >= a.nvec) continue;
        if constexpr (kAgain) {
          ring8<kDy>(at, vec, t[0]);
          ring8<kX>(at + y_bytes, vec, xh[0]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            xh[0][e] *= rstd;
            t[0][e] *= w[i][e];
          }
        }
        float d[8] = {};
        if (a.dres) ring8<kDx>(at + y_bytes + x_bytes, vec, d);
        bwd_dx(d, t[k], xh[k], rstd, c);
        store8<kDx>(a.dx, row * a.ld_dx + 8 * vec, d);
      }
    }
    __syncwarp();
  }
  if (!a.part) return;
  const int C = 8 * a.nvec;
  if constexpr (!kWarpRow) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = first_vec + i * gap;
      if (vec < a.nvec) store8<kFp32>(a.part, static_cast<int64_t>(blockIdx.x) * C + 8 * vec, dw[i]);
    }
  } else {
    // the warps' sums through shared memory, once no warp's ring is in use
    float *cols = reinterpret_cast<float *>(ring);  // [kRowWarps][C]
    copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = lane + 32 * i;
      if (vec < a.nvec) store8<kFp32>(cols + warp * C, 8 * vec, dw[i]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kRowWarps; ++k) v += cols[k * C + c];
      a.part[static_cast<int64_t>(blockIdx.x) * C + c] = v;
    }
  }
}

// Longer rows: dw is summed in shared memory, and dy and x are read again, from
// the L2, for dx.
template <int kDy, int kX, int kDx>
__global__ void __launch_bounds__(1024)
rmsnorm_bwd_long_kernel(const BwdArgs a) {
  __shared__ float sums[2][32];
  extern __shared__ float cols[];  // [C], each element one thread's
  wait_for_previous_kernel();
  for (int vec = threadIdx.x; vec < a.nvec; vec += blockDim.x) {
    const float zero[8] = {};
    store8<kFp32>(cols, 8 * vec, zero);
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, turn ^= 1) {
    const float rstd = a.rstd[row];
    float sum = 0.0f;
    for (int vec = threadIdx.x; vec < a.nvec; vec += blockDim.x) {
      float t[8], xh[8], w[8], dw[8];
      load8<kDy>(a.dy, row * a.ld_dy + 8 * vec, t);
      load8<kX>(a.x, row * a.ldx + 8 * vec, xh);
      load8_w(a.w, a.w_fp32, 8 * vec, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[e] = cols[8 * vec + e];
      bwd_terms(t, xh, w, rstd, dw, sum);
      store8<kFp32>(cols, 8 * vec, dw);
    }
    if (!a.dx) continue;
    const float c = row_sum<false>(sum, sums[turn]) * a.inv_c;
    for (int vec = threadIdx.x; vec < a.nvec; vec += blockDim.x) {
      float t[8], xh[8], w[8], d[8] = {};
      load8<kDy>(a.dy, row * a.ld_dy + 8 * vec, t);
      load8<kX>(a.x, row * a.ldx + 8 * vec, xh);
      load8_w(a.w, a.w_fp32, 8 * vec, w);
      if (a.dres) load8<kDx>(a.dres, row * a.ld_dres + 8 * vec, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[e] *= rstd;
        t[e] *= w[e];
      }
      bwd_dx(d, t, xh, rstd, c);
      store8<kDx>(a.dx, row * a.ld_dx + 8 * vec, d);
    }
  }
  if (!a.part) return;
  for (int vec = threadIdx.x; vec < a.nvec; vec += blockDim.x) {
    float dw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = cols[8 * vec + e];
    store8<kFp32>(a.part, (static_cast<int64_t>(blockIdx.x) * a.nvec + vec) * 8, dw);
  }
}

// dw = (dw +) the sum of n rows of part: 32 columns per CTA, every warps-th row per
// warp, twenty loads in flight in each.  Eight warps for up to 256 rows, 32 for more
// (the backward pass of 1000 x 2048, 608 rows: 10.6 us in all with eight, 7.5 with 32;
// of 8192 x 7168, 152 rows: 74.4 with eight, 76.7 with 32).
__global__ void __launch_bounds__(1024)
rmsnorm_dw_kernel(const float *part, int n, int C, float *dw, bool accumulate) {
  constexpr int kBatch = 20;
  __shared__ float sums[32][32];
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  for (int r0 = warp; r0 < n; r0 += warps * kBatch) {
    float p[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + warps * i;
      p[i] = c < C && r < n ? part[static_cast<int64_t>(r) * C + c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) v += p[i];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < C) {
    float t = 0.0f;
    for (int k = 0; k < warps; ++k) t += sums[k][lane];
    dw[c] = accumulate ? dw[c] + t : t;
  }
}

// How rows of C columns are taken, and by how many CTAs: as many as fit 152 SMs at
// once.  The CTAs depend on T and C alone, the stages on the types' bytes too, nothing on
// the device or on whether there is a dres, so that the sums' order does not either.
struct BwdPlan {
  int V, threads, stages, ctas;  // stages 0: the long form
};
BwdPlan bwd_plan(int64_t T, int64_t C, int value_bytes) {
  BwdPlan p{};
  const int nvec = static_cast<int>(C / 8), row = static_cast<int>(C) * value_bytes;
  int64_t rows = T, most;
  if (C <= kWarpCols) {
    p.V = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
    p.threads = 32 * kRowWarps;
    const int regs = p.V == 1 ? 3 : p.V == 2 ? 2 : 1;  // CTAs that an SM's registers hold
    p.stages = ring_stages(row * kRowWarps * regs, kBackwardBudget);
    most = kSms * regs;
    rows = (T + kRowWarps - 1) / kRowWarps;
  } else {
    p.V = nvec <= 1024 ? 1 : 2;
    p.threads = row_threads(nvec, p.V);
    const int per_sm = p.threads <= 1024 ? 1024 / p.threads : 1;
    p.stages = p.threads > 1024 ? 0 : ring_stages(row * per_sm, kBackwardBudget);
    if (p.stages < 2) p.stages = 0;
    most = kSms * per_sm;
  }
  p.ctas = static_cast<int>(rows < most ? rows : most);
  return p;
}

template <int kDy, int kX, int kDx>
fp8q_status launch_bwd(const BwdArgs &a, const BwdPlan &p, cudaStream_t s) {
  const int C = 8 * a.nvec;
  const int ring = p.stages * C * (size_of(kDy) + size_of(kX) + (a.dres ? size_of(kDx) : 0));
  if (C <= kWarpCols) {
    const int sums = kRowWarps * C * static_cast<int>(sizeof(float)), smem = kRowWarps * ring > sums ? kRowWarps * ring : sums;
    if (p.V == 1) return launch_ring<rmsnorm_bwd_kernel<kDy, kX, kDx, 1, true>>(p.ctas, p.threads, smem, s, a);
    if (p.V == 2) return launch_ring<rmsnorm_bwd_kernel<kDy, kX, kDx, 2, true>>(p.ctas, p.threads, smem, s, a);
    return launch_ring<rmsnorm_bwd_kernel<kDy, kX, kDx, 4, true>>(p.ctas, p.threads, smem, s, a);
  }
  if (p.stages && p.V == 1)
    return launch_ring<rmsnorm_bwd_kernel<kDy, kX, kDx, 1, false>>(p.ctas, p.threads, ring, s, a);
  if (p.stages) return launch_ring<rmsnorm_bwd_kernel<kDy, kX, kDx, 2, false>>(p.ctas, p.threads, ring, s, a);
  return launch_ring<rmsnorm_bwd_long_kernel<kDy, kX, kDx>>(p.ctas, 1024, static_cast<int>(sizeof(float)) * C, s, a);
}

// Whether rows of `kind` at p with pitch ld start on 16-byte boundaries.
bool rows_aligned(const void *p, int64_t ld, int kind) {
  return aligned16(p) && ld % (16 / size_of(kind)) == 0;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_rmsnorm(const void *x, int64_t ldx, int x_dtype, const void *res,
                                    int64_t ld_res, int res_dtype, const void *w, int w_dtype,
                                    float eps, void *r, int64_t ld_r, void *y, int64_t ldy, void *q,
                                    int64_t ldq, float *s, int64_t ld_s, float *rstd,
                                    int scale_mode, int64_t T, int64_t C, void *stream) {
  if (!kind_ok(x_dtype) || !kind_ok(w_dtype) || (res && !kind_ok(res_dtype)) || !(eps >= 0.0f) ||
      (scale_mode != FP8Q_SCALE_FP32 && scale_mode != FP8Q_SCALE_POW2))
    return FP8Q_ERR_INVALID;
  if (T < 0 || T > 0x7FFFFFFFll || C < 0 || C > kMaxCols || C % 8 || (q && C % 128))
    return FP8Q_ERR_SHAPE;
  if (ldx < C || (res && ld_res < C) || (r && ld_r < C) || (y && ldy < C) ||
      (q && (ldq < C || ld_s < T)))
    return FP8Q_ERR_SHAPE;
  if (T > 0 && C == 0 && rstd) return FP8Q_ERR_SHAPE;  // a mean of nothing
  if (T == 0 || C == 0) return FP8Q_OK;
  if (!x || !w || (r && !res) || (!r && !y && !q && !rstd) || !q != !s) return FP8Q_ERR_INVALID;
  if (!rows_aligned(x, ldx, x_dtype) || !aligned16(w) ||
      (res && !rows_aligned(res, ld_res, res_dtype)) || (r && !rows_aligned(r, ld_r, res_dtype)) ||
      (y && !rows_aligned(y, ldy, kBf16)) || (q && (!aligned16(q) || ldq % 16 || !aligned4(s))) ||
      (rstd && !aligned4(rstd)))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;
  NormArgs a{};
  a.x = x;
  a.res = res;
  a.w = w;
  a.r = r;
  a.y = y;
  a.q = static_cast<uint8_t *>(q);
  a.s = s;
  a.rstd = rstd;
  a.ldx = ldx;
  a.ld_res = ld_res;
  a.ld_r = ld_r;
  a.ldy = ldy;
  a.ldq = ldq;
  a.ld_s = ld_s;
  a.T = T;
  a.nvec = static_cast<int>(C / 8);
  a.inv_c = 1.0f / static_cast<float>(C);
  a.eps = eps;
  a.w_fp32 = w_dtype == kFp32;
  a.pow2 = scale_mode == FP8Q_SCALE_POW2;
  auto st = static_cast<cudaStream_t>(stream);
  const int kr = res ? res_dtype : static_cast<int>(kNone);
  if (x_dtype == kBf16)
    return kr == kNone ? launch_norm<kBf16, kNone>(a, st)
                       : kr == kBf16 ? launch_norm<kBf16, kBf16>(a, st)
                                     : launch_norm<kBf16, kFp32>(a, st);
  return kr == kNone ? launch_norm<kFp32, kNone>(a, st)
                     : kr == kBf16 ? launch_norm<kFp32, kBf16>(a, st)
                                   : launch_norm<kFp32, kFp32>(a, st);
}

extern "C" int64_t fp8q_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t C) {
  if (T < 0 || T > 0x7FFFFFFFll || C < 0 || C > kMaxCols || C % 8) return 0;
  // the types change the ring, not the CTAs
  return static_cast<int64_t>(bwd_plan(T, C, 6).ctas) * C * static_cast<int64_t>(sizeof(float));
}

extern "C" fp8q_status fp8q_rmsnorm_bwd(const void *dy, int64_t ld_dy, int dy_dtype, const void *x,
                                        int64_t ldx, int x_dtype, const float *rstd, const void *w,
                                        int w_dtype, const void *dres, int64_t ld_dres, void *dx,
                                        int64_t ld_dx, int out_dtype, float *dw, int accumulate,
                                        int64_t T, int64_t C, void *workspace,
                                        int64_t workspace_bytes, void *stream) {
  if (!kind_ok(dy_dtype) || !kind_ok(x_dtype) || !kind_ok(w_dtype) || !kind_ok(out_dtype))
    return FP8Q_ERR_INVALID;
  if (T < 0 || T > 0x7FFFFFFFll || C < 0 || C > kMaxCols || C % 8) return FP8Q_ERR_SHAPE;
  if (ld_dy < C || ldx < C || (dres && ld_dres < C) || (dx && ld_dx < C)) return FP8Q_ERR_SHAPE;
  if (C == 0) return FP8Q_OK;
  if ((!dx && !dw) || (dres && !dx)) return FP8Q_ERR_INVALID;
  if (T > 0 && (!dy || !x || !rstd || !w)) return FP8Q_ERR_INVALID;
  if (dw && T > 0) {
    if (!workspace) return FP8Q_ERR_INVALID;
    if (workspace_bytes < fp8q_rmsnorm_bwd_workspace_bytes(T, C)) return FP8Q_ERR_SHAPE;
    if (!aligned16(workspace)) return FP8Q_ERR_ALIGN;
  }
  if ((dw && !aligned4(dw)) ||
      (T > 0 && (!rows_aligned(dy, ld_dy, dy_dtype) || !rows_aligned(x, ldx, x_dtype) ||
                 !aligned16(w) || !aligned4(rstd) ||
                 (dres && !rows_aligned(dres, ld_dres, out_dtype)) ||
                 (dx && !rows_aligned(dx, ld_dx, out_dtype)))))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;
  BwdArgs a{};
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.dres = dres;
  a.rstd = rstd;
  a.dx = dx;
  a.part = dw ? static_cast<float *>(workspace) : nullptr;
  a.ld_dy = ld_dy;
  a.ldx = ldx;
  a.ld_dres = ld_dres;
  a.ld_dx = ld_dx;
  a.T = T;
  a.nvec = static_cast<int>(C / 8);
  a.inv_c = 1.0f / static_cast<float>(C);
  a.w_fp32 = w_dtype == kFp32;
  auto st = static_cast<cudaStream_t>(stream);
  const BwdPlan p = bwd_plan(T, C, size_of(dy_dtype) + size_of(x_dtype) + size_of(out_dtype));
  a.stages = p.stages;
  if (T > 0) {
    const int k = (dy_dtype == kFp32) * 4 + (x_dtype == kFp32) * 2 + (out_dtype == kFp32);
    fp8q_status e = FP8Q_OK;
    switch (k) {
      case 0: e = launch_bwd<kBf16, kBf16, kBf16>(a, p, st); break;
      case 1: e = launch_bwd<kBf16, kBf16, kFp32>(a, p, st); break;
      case 2: e = launch_bwd<kBf16, kFp32, kBf16>(a, p, st); break;
      case 3: e = launch_bwd<kBf16, kFp32, kFp32>(a, p, st); break;
      case 4: e = launch_bwd<kFp32, kBf16, kBf16>(a, p, st); break;
      case 5: e = launch_bwd<kFp32, kBf16, kFp32>(a, p, st); break;
      case 6: e = launch_bwd<kFp32, kFp32, kBf16>(a, p, st); break;
      default: e = launch_bwd<kFp32, kFp32, kFp32>(a, p, st); break;
    }
    if (e != FP8Q_OK) return e;
  }
  if (!dw) return FP8Q_OK;
  return launch_dependent(rmsnorm_dw_kernel, dim3(static_cast<unsigned>((C + 31) / 32)), dim3(p.ctas <= 256 ? 256 : 1024), 0, st,
                          static_cast<const float *>(workspace), p.ctas, static_cast<int>(C), dw,
                          accumulate != 0);
}
