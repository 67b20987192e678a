// norm.cu -- root-mean-square norm with the residual's addition and an FP8
// result, and its backward pass.
//
//   forward   h = x + res,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * w
//   backward  xh = x * rstd,  c = mean(dy * w * xh) over the row,
//             dx = rstd * (dy * w - xh * c) + dres,  dw = sum over rows of dy * xh
//
// Both are bound by memory.  A row is read once and stays in registers between
// its sum and its results: a warp holds rows of up to 1024 columns, a CTA longer
// ones.  Sums and statistics are FP32; the codes quantise the unrounded y.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8q.h"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"
#include "fp8q_vec.cuh"

namespace fp8q {
namespace {

constexpr int kMaxCols = 32768;  // 1024 threads with four 8-column vectors each
constexpr int kWarpCols = 1024;  // one warp with four vectors per lane
constexpr int kCtaCols = 8192;   // one CTA with one vector per thread (backward)
constexpr int kRowWarps = 8;     // rows per CTA in the warp form

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

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

struct NormArgs {
  const void *x, *res, *w;
  void *r, *y;
  uint8_t *q;
  float *s, *rstd;
  int64_t ldx, ld_res, ld_r, ldy, ldq, ld_s, T;
  int nvec;  // C / 8
  float inv_c, eps;
  bool w_fp32, pow2;
};

// y of one vector and its code, all lanes of the warp together (the 16 lanes of a
// group are all in the row, or none is).
__device__ __forceinline__ void finish8(const NormArgs &a, int64_t row, int vec, bool in, float rstd,
                                        const float (&w)[8], float (&h)[8]) {
  if (in) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = h[e] * rstd * w[e];
    if (a.y) store8<kBf16>(a.y, row * a.ldy + 8 * vec, h);
  }
  if (!a.q) return;
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) m = max3_abs(m, h[e], h[e + 1]);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  float s, inv;
  group_scale(m, a.pow2, s, inv);
  if (!in) return;
  if ((vec & 15) == 0) a.s[static_cast<int64_t>(vec >> 4) * a.ld_s + row] = s;
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] *= inv;
  *reinterpret_cast<uint2 *>(a.q + row * a.ldq + 8 * vec) =
      make_uint2(codes4(h[0], h[1], h[2], h[3]), codes4(h[4], h[5], h[6], h[7]));
}

// kX, kRes: kinds of x and of the residual; V: 8-column vectors per thread.
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
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = first + i * step;
    if (vec < a.nvec) {
      load8<kX>(a.x, row * a.ldx + 8 * vec, h[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
    }
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
  const float rstd = 1.0f / sqrtf(fmaf(sum, a.inv_c, a.eps));
  if (a.rstd && first == 0) a.rstd[row] = rstd;
  if (!a.y && !a.q) return;

#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = first + i * step;
    const bool in = vec < a.nvec;  // the same for the 16 lanes of a group
    float w[8];
    if (in) load8_w(a.w, a.w_fp32, 8 * vec, w);
    finish8(a, row, vec, in, rstd, w, h[i]);
  }
}

// One 16-byte piece of a row into this thread's own place of the ring.
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

// One array's part of a ring: per stage and thread the 16 or 32 bytes of its
// vector, in planes of 16 bytes (no bank conflicts).  A thread reads back only what
// it has copied itself, so the ring needs no barrier.
template <int kKind>
struct RingPart {
  static constexpr int kPlanes = kKind == kNone ? 0 : kKind == kBf16 ? 1 : 2;
  __device__ __forceinline__ static void fetch(uint32_t at, int threads, const void *base, int64_t from) {
    const char *p = static_cast<const char *>(base) + from * size_of(kKind);
#pragma unroll
    for (int i = 0; i < kPlanes; ++i) copy16(at + i * threads * 16, p + 16 * i);
  }
  __device__ __forceinline__ static void values(uint32_t at, int threads, float (&v)[8]) {
    if constexpr (kKind == kBf16) unpack8(ld_shared_v4(at), v);
    else unpack8(ld_shared_v4(at), ld_shared_v4(at + threads * 16), v);
  }
};

// Rows of up to 8192 columns, one vector per thread: CTA b takes rows b,
// b + gridDim, ..., with kStages - 1 rows on their way into shared memory while one
// is dealt with.
template <int kX, int kRes, int kStages>
__global__ void __launch_bounds__(1024)
rmsnorm_rows_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float part[2][32];
  using X = RingPart<kX>;
  using R = RingPart<kRes>;
  wait_for_previous_kernel();
  const int vec = threadIdx.x, threads = blockDim.x;
  const bool in = vec < a.nvec;  // the same for the 16 lanes of a group
  const uint32_t stage_bytes = (X::kPlanes + R::kPlanes) * 16 * threads;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  const auto fetch = [&](int64_t row, int stage) {
    if (in && row < a.T) {
      const uint32_t at = mine + stage * stage_bytes;
      X::fetch(at, threads, a.x, row * a.ldx + 8 * vec);
      if constexpr (kRes != kNone)
        R::fetch(at + X::kPlanes * 16 * threads, threads, a.res, row * a.ld_res + 8 * vec);
    }
    copies_commit();
  };
  const int64_t step = gridDim.x;
  int64_t row = blockIdx.x;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + i * step, i);
  float w[8] = {};
  if (in) load8_w(a.w, a.w_fp32, 8 * vec, w);

  int turn = 0, stage = 0;
  for (; row < a.T; row += step, turn ^= 1) {
    fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
    copies_wait<kStages - 1>();
    float h[8] = {};
    if (in) {
      const uint32_t at = mine + stage * stage_bytes;
      X::values(at, threads, h);
      if constexpr (kRes != kNone) {
        float z[8];
        R::values(at + X::kPlanes * 16 * threads, threads, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += z[e];
        if (a.r) store8<kRes>(a.r, row * a.ld_r + 8 * vec, h);
      }
    }
    stage = stage == kStages - 1 ? 0 : stage + 1;
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[e], h[e], sum);
    sum = row_sum<false>(sum, part[turn]);
    const float rstd = 1.0f / sqrtf(fmaf(sum, a.inv_c, a.eps));
    if (a.rstd && vec == 0) a.rstd[row] = rstd;
    finish8(a, row, vec, in, rstd, w, h);
  }
}

constexpr int kSms = 152;
constexpr int kRingBytes = 216 * 1024;  // of an SM's shared memory

template <typename... KArgs, typename... Args>
fp8q_status launch_ring(void (*kern)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t s,
                        Args &&...args) {
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  return launch_dependent(kern, grid, dim3(threads), smem, s, args...);
}

// Threads for one row of nvec vectors, V of them each.
int row_threads(int nvec, int V) { return ((nvec + V - 1) / V + 31) / 32 * 32; }

template <int kX, int kRes>
fp8q_status launch_norm(const NormArgs &a, cudaStream_t s) {
  if (a.nvec <= kWarpCols / 8) {
    const dim3 grid(static_cast<unsigned>((a.T + kRowWarps - 1) / kRowWarps));
    if (a.nvec <= 32) return launch_dependent(rmsnorm_kernel<kX, kRes, 1, true>, grid, dim3(32 * kRowWarps), 0, s, a);
    if (a.nvec <= 64) return launch_dependent(rmsnorm_kernel<kX, kRes, 2, true>, grid, dim3(32 * kRowWarps), 0, s, a);
    return launch_dependent(rmsnorm_kernel<kX, kRes, 4, true>, grid, dim3(32 * kRowWarps), 0, s, a);
  }
  const int threads = row_threads(a.nvec, 1);
  if (threads <= 1024) {
    constexpr int kPlanes = RingPart<kX>::kPlanes + RingPart<kRes>::kPlanes;
    const int per_sm = 1024 / threads;
    const int stage = kPlanes * 16 * threads;
    const int64_t most = static_cast<int64_t>(kSms) * per_sm;
    const dim3 grid(static_cast<unsigned>(a.T < most ? a.T : most));
    if (4 * stage * per_sm <= kRingBytes)
      return launch_ring(rmsnorm_rows_kernel<kX, kRes, 4>, grid, threads, 4 * stage, s, a);
    return launch_ring(rmsnorm_rows_kernel<kX, kRes, 2>, grid, threads, 2 * stage, s, a);
  }
  const dim3 grid(static_cast<unsigned>(a.T));
  return launch_dependent(rmsnorm_kernel<kX, kRes, 4, false>, grid, dim3(row_threads(a.nvec, 4)), 0, s, a);
}

struct BwdArgs {
  const void *dy, *x, *w, *dres;
  const float *rstd;
  void *dx;
  float *part;  // [CTAs][C], null without dw
  int64_t ld_dy, ldx, ld_dres, ld_dx, T;
  int nvec;
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

// In all three forms CTA b takes rows b, b + gridDim, ... (a warp each in the
// warp form) and leaves the sum of its rows' dy * xh in part[b], so dw is summed
// in a fixed order.

// Rows of up to 1024 columns: one per warp, V vectors per lane.
template <int kDy, int kX, int kDx, int V>
__global__ void __launch_bounds__(32 * kRowWarps)
rmsnorm_bwd_warp_kernel(const BwdArgs a) {
  extern __shared__ float cols[];  // [kRowWarps][C]
  wait_for_previous_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float w[V][8], dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = lane + 32 * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = dw[i][e] = 0.0f;
    if (vec < a.nvec) load8_w(a.w, a.w_fp32, 8 * vec, w[i]);
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp; row < a.T;
       row += static_cast<int64_t>(gridDim.x) * kRowWarps) {
    float t[V][8], xh[V][8], d[V][8];
    const float rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = lane + 32 * i;
#pragma unroll
      for (int e = 0; e < 8; ++e) t[i][e] = xh[i][e] = d[i][e] = 0.0f;
      if (vec < a.nvec) {
        load8<kDy>(a.dy, row * a.ld_dy + 8 * vec, t[i]);
        load8<kX>(a.x, row * a.ldx + 8 * vec, xh[i]);
        if (a.dres) load8<kDx>(a.dres, row * a.ld_dres + 8 * vec, d[i]);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) bwd_terms(t[i], xh[i], w[i], rstd, dw[i], sum);
    if (!a.dx) continue;
    const float c = warp_sum(sum) * a.inv_c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int vec = lane + 32 * i;
      if (vec >= a.nvec) continue;
      bwd_dx(d[i], t[i], xh[i], rstd, c);
      store8<kDx>(a.dx, row * a.ld_dx + 8 * vec, d[i]);
    }
  }
  if (!a.part) return;
  const int C = 8 * a.nvec;
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

// Rows of up to 8192 columns: one vector per thread, the next rows on their way into
// shared memory as in the forward pass.
template <int kDy, int kX, int kDx, int kStages>
__global__ void __launch_bounds__(1024)
rmsnorm_bwd_kernel(const BwdArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sums[2][32], rstds[kStages][32];  // a warp's own copy of its rows' rstd
  using Y = RingPart<kDy>;
  using X = RingPart<kX>;
  using D = RingPart<kDx>;
  wait_for_previous_kernel();
  const int vec = threadIdx.x, threads = blockDim.x;
  const bool in = vec < a.nvec;
  const uint32_t plane = 16 * threads;
  const uint32_t stage_bytes = (Y::kPlanes + X::kPlanes + (a.dres ? D::kPlanes : 0)) * plane;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t my_rstd = smem_u32(&rstds[0][threadIdx.x >> 5]);
  const auto fetch = [&](int64_t row, int stage) {
    if ((threadIdx.x & 31) == 0 && row < a.T) copy4(my_rstd + stage * 128, a.rstd + row);
    if (in && row < a.T) {
      const uint32_t at = mine + stage * stage_bytes;
      Y::fetch(at, threads, a.dy, row * a.ld_dy + 8 * vec);
      X::fetch(at + Y::kPlanes * plane, threads, a.x, row * a.ldx + 8 * vec);
      if (a.dres)
        D::fetch(at + (Y::kPlanes + X::kPlanes) * plane, threads, a.dres, row * a.ld_dres + 8 * vec);
    }
    copies_commit();
  };
  const int64_t step = gridDim.x;
  int64_t row = blockIdx.x;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + i * step, i);
  float w[8] = {}, dw[8] = {};
  if (in) load8_w(a.w, a.w_fp32, 8 * vec, w);

  int turn = 0, stage = 0;
  for (; row < a.T; row += step, turn ^= 1) {
    fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
    copies_wait<kStages - 1>();
    __syncwarp();  // the copy of rstd is lane 0's; it is overwritten after the row's barrier
    const float rs = *(volatile float *)&rstds[stage][threadIdx.x >> 5];
    float t[8] = {}, xh[8] = {}, d[8] = {};
    if (in) {
      const uint32_t at = mine + stage * stage_bytes;
      Y::values(at, threads, t);
      X::values(at + Y::kPlanes * plane, threads, xh);
      if (a.dres) D::values(at + (Y::kPlanes + X::kPlanes) * plane, threads, d);
    }
    stage = stage == kStages - 1 ? 0 : stage + 1;
    float sum = 0.0f;
    bwd_terms(t, xh, w, rs, dw, sum);
    if (!a.dx) continue;
    const float c = row_sum<false>(sum, sums[turn]) * a.inv_c;
    if (in) {
      bwd_dx(d, t, xh, rs, c);
      store8<kDx>(a.dx, row * a.ld_dx + 8 * vec, d);
    }
  }
  if (a.part && in) store8<kFp32>(a.part, (static_cast<int64_t>(blockIdx.x) * a.nvec + vec) * 8, dw);
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

// dw = (dw +) the sum of n rows of part: 32 columns per CTA, eight warps with a
// share of the rows each.
__global__ void __launch_bounds__(256)
rmsnorm_dw_kernel(const float *part, int n, int C, float *dw, bool accumulate) {
  __shared__ float sums[8][32];
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int r = warp; r < n; r += 8) v += part[static_cast<int64_t>(r) * C + c];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < C) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += sums[k][lane];
    dw[c] = accumulate ? dw[c] + t : t;
  }
}

// CTAs of the backward pass, and rows of its workspace: the CTAs that fit 152 SMs
// at once (64 registers per thread, 1024 threads per SM), for every device alike,
// so that the sums' order is too.
int bwd_ctas(int64_t T, int64_t C) {
  const int64_t rows = C <= kWarpCols ? (T + kRowWarps - 1) / kRowWarps : T;
  const int64_t most =
      kSms * (C <= kWarpCols ? 4 : C <= kCtaCols ? 1024 / row_threads(static_cast<int>(C / 8), 1) : 1);
  return static_cast<int>(rows < most ? rows : most);
}

template <int kDy, int kX, int kDx>
fp8q_status launch_bwd(const BwdArgs &a, cudaStream_t s) {
  const int C = 8 * a.nvec;
  const dim3 grid(bwd_ctas(a.T, C));
  if (C <= kWarpCols) {
    const dim3 block(32 * kRowWarps);
    const size_t smem = a.part ? kRowWarps * sizeof(float) * C : 0;
    if (a.nvec <= 32)
      return launch_dependent(rmsnorm_bwd_warp_kernel<kDy, kX, kDx, 1>, grid, block, smem, s, a);
    if (a.nvec <= 64)
      return launch_dependent(rmsnorm_bwd_warp_kernel<kDy, kX, kDx, 2>, grid, block, smem, s, a);
    return launch_dependent(rmsnorm_bwd_warp_kernel<kDy, kX, kDx, 4>, grid, block, smem, s, a);
  }
  if (C <= kCtaCols) {
    const int threads = row_threads(a.nvec, 1), per_sm = 1024 / threads;
    const int planes = RingPart<kDy>::kPlanes + RingPart<kX>::kPlanes + (a.dres ? RingPart<kDx>::kPlanes : 0);
    const int stage = planes * 16 * threads;
    if (4 * stage * per_sm <= kRingBytes)
      return launch_ring(rmsnorm_bwd_kernel<kDy, kX, kDx, 4>, grid, threads, 4 * stage, s, a);
    return launch_ring(rmsnorm_bwd_kernel<kDy, kX, kDx, 2>, grid, threads, 2 * stage, s, a);
  }
  const auto kern = rmsnorm_bwd_long_kernel<kDy, kX, kDx>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMaxCols * sizeof(float)) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  return launch_dependent(kern, grid, dim3(1024), sizeof(float) * C, s, a);
}

bool kind_ok(int kind) { return kind == kBf16 || kind == kFp32; }

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
  return static_cast<int64_t>(bwd_ctas(T, C)) * C * static_cast<int64_t>(sizeof(float));
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
  if (T > 0) {
    const int k = (dy_dtype == kFp32) * 4 + (x_dtype == kFp32) * 2 + (out_dtype == kFp32);
    fp8q_status e = FP8Q_OK;
    switch (k) {
      case 0: e = launch_bwd<kBf16, kBf16, kBf16>(a, st); break;
      case 1: e = launch_bwd<kBf16, kBf16, kFp32>(a, st); break;
      case 2: e = launch_bwd<kBf16, kFp32, kBf16>(a, st); break;
      case 3: e = launch_bwd<kBf16, kFp32, kFp32>(a, st); break;
      case 4: e = launch_bwd<kFp32, kBf16, kBf16>(a, st); break;
      case 5: e = launch_bwd<kFp32, kBf16, kFp32>(a, st); break;
      case 6: e = launch_bwd<kFp32, kFp32, kBf16>(a, st); break;
      default: e = launch_bwd<kFp32, kFp32, kFp32>(a, st); break;
    }
    if (e != FP8Q_OK) return e;
  }
  if (!dw) return FP8Q_OK;
  return launch_dependent(rmsnorm_dw_kernel, dim3(static_cast<unsigned>((C + 31) / 32)), dim3(256), 0, st,
                          static_cast<const float *>(workspace), bwd_ctas(T, C), static_cast<int>(C), dw,
                          accumulate != 0);
}
