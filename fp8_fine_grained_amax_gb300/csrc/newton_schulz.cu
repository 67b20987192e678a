// newton_schulz.cu -- orthogonalised update of a weight gradient by
// Newton-Schulz steps, for a batch of matrices.
//
//   X = G / (|G|_F + eps), oriented with the shorter side p as its rows;
//   steps times:  A = X X^T,  B = b A + c A^2,  X = a X + B X.
//
// Each step is three products on the tensor cores (tcgen05.mma kind::f16) with
// FP32 sums.  Operands are FP16, not BF16: X, A and B are bounded (the
// iteration keeps the singular values of X near 1), so FP16's three more
// mantissa bits are free, and a fixed factor S = 2^8 keeps the small entries
// of X and A away from FP16's subnormals (1 / sqrt(p q) is 2.6e-4 for a
// 2048 x 7168 matrix; with S the smallest normal entry is 2.4e-7) while values
// up to 255 still fit.  Stored: X^ = S X, A^ = S A, B^ = S B, so
//   A^ = (X^ X^^T) / S,  B^ = b A^ + (c / S) A^ A^^T,  X^ <- a X^ + (B^ X^) / S.
// The diagonals of A and B never pass through FP16.  Near the end A is close to
// the identity and a X nearly cancels against B X, so that rounding B's
// diagonal (2^-12 of 2.7) would cost more than all other roundings together:
// X, the off-diagonal parts O_A and O_B are FP16, the diagonals d_A and d_B FP32
// vectors, and the epilogues add their terms in FP32:
//   A^2 = O_A O_A + d_A O_A + O_A d_A + d_A^2,   X <- (a + d_B) X + O_B X.
// (Error of a 72 x 3303 update against 64 bits before its rounding to BF16:
// 1.8e-3 with FP16 diagonals, 6e-4 so; FP16 X alone gives 5.5e-4.)
//
// A and B are symmetric: only tiles on and above the diagonal are computed,
// and each is stored twice, the second time transposed.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "fp8q.h"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"

namespace fp8q {

// Device status word of these kernels (read by fp8q_sync_status).
__device__ int g_ns_status;

fp8q_status ns_status_take(cudaStream_t s) {
  int v = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_ns_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_ns_status, &zero, sizeof(int)) != cudaSuccess) return FP8Q_ERR_CUDA;
  }
  return static_cast<fp8q_status>(v);
}

namespace {

constexpr float kS = 256.0f;        // scale of the stored FP16 matrices
constexpr int kMaxParts = 256;      // partial sums of squares per matrix

// ------------------------------------------------------------------ set-up
__device__ __forceinline__ float load_in(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_in(const uint16_t *p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum of squares of matrix blockIdx.y, part blockIdx.x of gridDim.x: rows
// blockIdx.x, blockIdx.x + gridDim.x, ...  Fixed order, so repeated calls agree.
template <typename In>
__global__ void __launch_bounds__(256) ns_sumsq_kernel(const In *__restrict__ g, int64_t ldg,
                                                       int64_t batch_stride, int64_t m, int64_t n,
                                                       float *__restrict__ part) {
  __shared__ float sums[8];
  const In *base = g + blockIdx.y * batch_stride;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t r = blockIdx.x; r < m; r += gridDim.x) {
    const In *row = base + r * ldg;
    int64_t c = threadIdx.x;
    for (; c + 768 < n; c += 1024)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = load_in(row + c + 256 * i);
        acc[i] = fmaf(v, v, acc[i]);
      }
    for (; c < n; c += 256) {
      const float v = load_in(row + c);
      acc[0] = fmaf(v, v, acc[0]);
    }
  }
  const float s = warp_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float t = warp_sum(threadIdx.x < 8 ? sums[threadIdx.x] : 0.0f);
    if (threadIdx.x == 0) part[blockIdx.y * kMaxParts + blockIdx.x] = t;
  }
}

// X^ = FP16(S g / (|g|_F + eps)), transposed when kTall.  One 64 x 64 tile of g
// per block (256 threads).
template <typename In, bool kTall>
__global__ void __launch_bounds__(256) ns_load_kernel(const In *__restrict__ g, int64_t ldg,
                                                      int64_t batch_stride, int64_t m, int64_t n,
                                                      const float *__restrict__ part, int parts,
                                                      float eps, __half *__restrict__ x,
                                                      int64_t ldx) {
  __shared__ float s_scale;
  __shared__ float tile[kTall ? 64 : 1][65];
  const int tid = threadIdx.x;
  if (tid < 32) {
    float v = 0.0f;
    for (int i = tid; i < parts; i += 32) v += part[blockIdx.z * kMaxParts + i];
    v = warp_sum(v);
    if (tid == 0) s_scale = kS / (sqrtf(v) + eps);
  }
  __syncthreads();
  const float scale = s_scale;
  const In *base = g + blockIdx.z * batch_stride;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  if (!kTall) {
    __half *dst = x + blockIdx.z * (m * ldx);
    const int64_t c = c0 + 2 * (tid & 31);
    for (int i = tid >> 5; i < 64; i += 8) {
      const int64_t r = r0 + i;
      if (r >= m || c >= n) continue;
      const float v0 = load_in(base + r * ldg + c);
      const float v1 = c + 1 < n ? load_in(base + r * ldg + c + 1) : 0.0f;
      // ldx is a multiple of 8 and c is even: the pair stays inside the row's pitch
      *reinterpret_cast<__half2 *>(dst + r * ldx + c) = __floats2half2_rn(v0 * scale, v1 * scale);
    }
  } else {
    for (int i = tid; i < 64 * 64; i += 256) {
      const int64_t r = r0 + (i >> 6), c = c0 + (i & 63);
      tile[i >> 6][i & 63] = r < m && c < n ? load_in(base + r * ldg + c) * scale : 0.0f;
    }
    __syncthreads();
    __half *dst = x + blockIdx.z * (n * ldx);
    const int j = 2 * (tid & 31);
    const int64_t r = r0 + j;
    for (int i = tid >> 5; i < 64; i += 8) {
      const int64_t c = c0 + i;
      if (c >= n || r >= m) continue;
      *reinterpret_cast<__half2 *>(dst + c * ldx + r) = __floats2half2_rn(tile[j][i], tile[j + 1][i]);
    }
  }
}

// ------------------------------------------------------------------ products
// D = L R^T (A, A^2) or L R (the update) on CTA pairs: a 256 x BN tile per pair
// (tcgen05.mma.cta_group::2, M = 256, K = 16), each CTA staging its 128 rows of
// L and half of R's columns per 64-wide K block (128-byte rows, 128-byte
// swizzle).  R is K-major where it is a row block of X or A, and N-major (64
// columns x 64 K rows per box, as X is stored) in the update, so no transposed
// copy of X exists.  Two TMEM accumulators: the epilogue of one tile runs under
// the MMAs of the next.
//   warp 0 TMA producer, warp 1 MMA issuer (leading CTA), warps 4-11 epilogue
//   (each thread one row, BN / 2 columns).
enum class Op { kGram, kPoly, kUpdate };  // A = X X^T | B = bA + cA^2 | X' = aX + BX

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr uint64_t kDrainNs = 1000000000ull;
constexpr uint32_t kLBytes = 128 * 128;  // L: 128 rows x 64 FP16

template <int BN>
struct Cfg {
  static constexpr int kStages = BN == 256 ? 5 : 7;
  static constexpr uint32_t kRBytes = (BN / 2) * 128;  // R: half of the columns
  static constexpr uint32_t kTx = 2 * (kLBytes + kRBytes);
  static constexpr size_t kRing = static_cast<size_t>(kStages) * (kLBytes + kRBytes);
};

struct alignas(8) Ctl {
  uint64_t full[8], empty[8], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr uint32_t kStageWarp = 32 * 33 * 4;  // staging of one epilogue warp

template <int BN>
constexpr size_t smem_of() {
  return 1024 + Cfg<BN>::kRing + kEpiWarps * kStageWarp + sizeof(Ctl);
}
static_assert(smem_of<256>() <= 227 * 1024 && smem_of<128>() <= 227 * 1024, "shared memory");

struct NsArgs {
  int batch, rows, cols, kblocks;  // D is [rows][cols] per matrix
  int tiles_m, tiles_n, tiles;     // tiles: per matrix
  float c_old, c_acc;              // D = c_old * old + c_acc * (sum + diagonal terms)
  float c_diag;                    // update: weight of d_B
  const __half *old;               // A^ or X^ (not read for the Gram matrix)
  const float *diag;               // S d_A or S d_B of the matrix read, pitch ldd
  float *diag_out;                 // symmetric results: their diagonal
  int64_t ldd;
  __half *dst;                     // FP16 result, or null
  int64_t ld;                      // pitch of old and dst
  void *out;                       // final result (update only), or null
  int64_t ldo, out_stride;
  int out_f32, tall;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// FP16 x FP16 -> FP32, A K-major, B K-major or N-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// N-major operand, 128-byte swizzle: blocks of 64 columns (a 128-byte row per
// K index), `block_bytes` apart (leading byte offset); eight K rows are one
// 1024-byte atom, the next eight follow it (stride byte offset).
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t addr, uint32_t block_bytes) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) |
         (static_cast<uint64_t>(block_bytes >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t smem_dst, const void *tmap,
                                                 uint32_t bar_cluster_addr, int32_t c0, int32_t c1,
                                                 int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster_addr)
      : "memory");
}
__device__ __forceinline__ void mbar_wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kDrainNs) return;
}

struct NsTile {
  int b, row0, col0;  // matrix, first row (of the pair), first column
};
// Symmetric products: row block i (256 rows) has column blocks from its own
// diagonal on (col >= 256 i).
template <int BN, bool kSym>
__device__ __forceinline__ NsTile tile_of(int t, const NsArgs &p) {
  NsTile r;
  r.b = t / p.tiles;
  int w = t - r.b * p.tiles;
  if (kSym) {
    constexpr int kPer = 256 / BN;  // column blocks per row block
    int i = 0;
    while (w >= p.tiles_n - kPer * i) {
      w -= p.tiles_n - kPer * i;
      ++i;
    }
    r.row0 = i * 256;
    r.col0 = (kPer * i + w) * BN;
  } else {
    r.row0 = (w % p.tiles_m) * 256;
    r.col0 = (w / p.tiles_m) * BN;
  }
  return r;
}

template <int BN, Op kOp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmR,
                   const NsArgs p) {
  using C = Cfg<BN>;
  constexpr bool kSym = kOp != Op::kUpdate;
  constexpr uint32_t kTmem = 2 * BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sL = smem_u32(smem), sR = sL + C::kStages * kLBytes;
  float *stage = reinterpret_cast<float *>(smem + C::kRing);
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + C::kRing + kEpiWarps * kStageWarp);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &ctl->abort_flag;
  const uint32_t rank = cluster_ctarank();
  const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);
  const int total = p.tiles * p.batch;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 1);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->tfull[i]), 1);
      mbar_init(smem_u32(&ctl->tempty[i]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmL);
    prefetch_tmap(&tmR);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctl->tmem_base), kTmem);
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp >= 4) {
    // ================================================== epilogue
    const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(&ctl->tempty[0]), 0);
    float *st = stage + ew * (kStageWarp / 4);
    int buf = 0;
    uint32_t phase = 0;
    for (int t = first; t < total; t += step) {
      const NsTile tl = tile_of<BN, kSym>(t, p);
      const bool got = mbar_wait_bounded(smem_u32(&ctl->tfull[buf]), phase, abort_flag,
                                         &g_ns_status, p.timeout_ns, FP8Q_ERR_TIMEOUT);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const int row0 = tl.row0 + static_cast<int>(rank) * 128 + quarter * 32;  // the warp's rows
      const int row = row0 + lane;
      const int cbase = tl.col0 + half * (BN / 2);
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>(buf * BN + half * (BN / 2));
      const int64_t mat = static_cast<int64_t>(tl.b) * p.rows * p.ld;
      // tiles of the diagonal block hold both triangles themselves
      const bool mirror = kSym && tl.col0 >= tl.row0 + 256;
      const float *diag = p.diag + static_cast<int64_t>(tl.b) * p.ldd;
      const float d_row = kOp != Op::kGram && row < p.rows ? diag[row] : 0.0f;
      const float c_old = kOp == Op::kUpdate ? fmaf(p.c_diag, d_row, p.c_old) : p.c_old;
#pragma unroll 1
      for (int c = 0; c < BN / 2; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(taddr + c, r);
        const int col0 = cbase + c;
        const bool live = row0 < p.rows && col0 < p.cols;  // warp-uniform
        float old[32];
        const bool whole = col0 + 32 <= p.cols;
        if (kOp != Op::kGram && live) {
          const __half *src = p.old + mat + static_cast<int64_t>(row) * p.ld + col0;
          // the pitch is a multiple of 8, so an 8-column unit that begins
          // inside the matrix is readable to its end
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < p.rows && col0 + 8 * k < p.cols) v = *reinterpret_cast<const uint4 *>(src + 8 * k);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              old[8 * k + 2 * e] = f16_lo(w[e]);
              old[8 * k + 2 * e + 1] = f16_hi(w[e]);
            }
          }
        }
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
        if (c + 32 == BN / 2) {  // the accumulator has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty0 + static_cast<uint32_t>(buf) * 8u);
        }
        if (!live) continue;
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float s = __uint_as_float(r[i]);
          if (kOp == Op::kGram) v[i] = p.c_acc * s;
          if (kOp == Op::kUpdate) v[i] = fmaf(c_old, old[i], p.c_acc * s);
        }
        // the diagonal crosses this warp's 32 x 32 block (both begin at
        // multiples of 32)
        const bool on_diag = kSym && row0 == col0;
        if (kOp == Op::kPoly) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // the pitch is a multiple of 8; what lies past the matrix is not stored
            const float4 d = col0 + 4 * k < p.cols
                                 ? *reinterpret_cast<const float4 *>(diag + col0 + 4 * k)
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float dc[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 4 * k + e;
              const float s = __uint_as_float(r[i]);
              v[i] = fmaf(p.c_old, old[i], p.c_acc * fmaf(d_row + dc[e], old[i], s));
              if (on_diag && i == lane) v[i] = fmaf(p.c_old, d_row, p.c_acc * fmaf(d_row, d_row, s));
            }
          }
        }
        if (on_diag && row < p.rows) {
          float d = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i == lane) {
              d = v[i];
              v[i] = 0.0f;
            }
          p.diag_out[static_cast<int64_t>(tl.b) * p.ldd + row] = d;
        }
        if (kOp == Op::kUpdate && p.out) {
          // final result, any pitch: column runs (tall) are contiguous over
          // the lanes; row runs go through the staging buffer
          const int64_t obase = static_cast<int64_t>(tl.b) * p.out_stride;
          if (p.tall) {
            if (row < p.rows)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (whole || col0 + i < p.cols) {
                  const int64_t at = obase + static_cast<int64_t>(col0 + i) * p.ldo + row;
                  if (p.out_f32) static_cast<float *>(p.out)[at] = v[i];
                  else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v[i]);
                }
          } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; ++i) st[lane * 33 + i] = v[i];
            __syncwarp();
            if (col0 + lane < p.cols) {
              const int n = min(32, p.rows - row0);
              for (int i = 0; i < n; ++i) {
                const int64_t at = obase + static_cast<int64_t>(row0 + i) * p.ldo + col0 + lane;
                const float f = st[i * 33 + lane];
                if (p.out_f32) static_cast<float *>(p.out)[at] = f;
                else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(f);
              }
            }
          }
          continue;
        }
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(v[8 * k + 2 * e], v[8 * k + 2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&h);
          }
          u[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        warp_store_block64<2, false, false>(smem_u32(st), u, p.dst + mat, p.ld, row0, p.rows, col0,
                                            p.cols, lane);
        if (mirror && row < p.rows) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(u)[i / 2];
            if (whole || col0 + i < p.cols)
              reinterpret_cast<uint16_t *>(p.dst + mat)[static_cast<int64_t>(col0 + i) * p.ld + row] =
                  static_cast<uint16_t>(i & 1 ? w >> 16 : w & 0xFFFFu);
          }
        }
      }
      buf ^= 1;
      if (buf == 0) phase ^= 1;
    }
  } else if (warp == 0) {
    // ================================================== TMA producer
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0, armed = 0, armed_phase = 0;
      bool ok = true;
      for (int t = first; ok && t < total; t += step) {
        const NsTile tl = tile_of<BN, kSym>(t, p);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&ctl->empty[s]), phase ^ 1, abort_flag, &g_ns_status,
                                 p.timeout_ns, FP8Q_ERR_TIMEOUT)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&ctl->full[s]);
          if (rank == 0) mbar_arrive_expect_tx(fb, C::kTx);
          const uint32_t fb0 = mapa_shared(fb, 0);
          tma_load_3d_pair(sL + s * kLBytes, &tmL, fb0, kb * 64,
                           tl.row0 + static_cast<int>(rank) * 128, tl.b);
          const int rc = tl.col0 + static_cast<int>(rank) * (BN / 2);
          if (kSym) {
            tma_load_3d_pair(sR + s * C::kRBytes, &tmR, fb0, kb * 64, rc, tl.b);
          } else {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
              tma_load_3d_pair(sR + s * C::kRBytes + j * 8192, &tmR, fb0, rc + 64 * j, kb * 64, tl.b);
          }
          armed |= 1u << s;
          armed_phase = (armed_phase & ~(1u << s)) | (phase << s);
          if (++s == C::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {
        // this CTA's copies land before it exits (the leading CTA's barriers
        // see both CTAs' copies; the other waits long enough for any copy)
        if (rank == 0)
          for (int i = 0; i < C::kStages; ++i)
            if (armed & (1u << i)) mbar_wait_drain(smem_u32(&ctl->full[i]), (armed_phase >> i) & 1);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ================================================== MMA issuer
    if (lane == 0 && rank == 0) {
      constexpr uint32_t kIdesc = idesc_f16(256, BN, !kSym);
      int s = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true, issued = false;
      for (int t = first; ok && t < total; t += step) {
        if (!mbar_wait_bounded(smem_u32(&ctl->tempty[buf]), tphase ^ 1, abort_flag, &g_ns_status,
                               p.timeout_ns, FP8Q_ERR_TIMEOUT)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!mbar_wait_bounded(smem_u32(&ctl->full[s]), phase, abort_flag, &g_ns_status,
                                 p.timeout_ns, FP8Q_ERR_TIMEOUT)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = smem_desc_sw128(sL + s * kLBytes);
          const uint64_t bd = kSym ? smem_desc_sw128(sR + s * C::kRBytes)
                                   : smem_desc_sw128_mn(sR + s * C::kRBytes, 8192);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 16 K: 32 bytes of a row, or 16 rows of 128 bytes
            mma_f16_pair(d, ad + 2 * k, bd + (kSym ? 2 : 128) * k, kIdesc, (kb | k) != 0 ? 1u : 0u);
          mma_commit_pair_multicast(smem_u32(&ctl->empty[s]), 0x3);
          issued = true;
          if (++s == C::kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        mma_commit_pair_multicast(smem_u32(&ctl->tfull[buf]), 0x3);
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
      }
      if (!ok && issued) {  // MMAs in flight finish before TMEM is freed
        mma_commit_pair_multicast(smem_u32(&ctl->drain), 0x1);
        mbar_wait_drain(smem_u32(&ctl->drain), 0);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmem);
  }
}

// ------------------------------------------------------------------ host
// FP16 [batch][rows][cols], row pitch ld; box 64 x box_rows, 128-byte swizzle.
bool make_tmap_f16(CUtensorMap *m, const void *base, uint64_t batch, uint64_t rows, uint64_t cols,
                   uint64_t ld, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, rows, batch};
  cuuint64_t strides[2] = {ld * 2, rows * ld * 2};
  cuuint32_t box[3] = {64, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, Op kOp>
fp8q_status launch_ns(const CUtensorMap &l, const CUtensorMap &r, const NsArgs &a, cudaStream_t s) {
  auto kern = ns_gemm_kernel<BN, kOp>;
  constexpr size_t smem = smem_of<BN>();
  static int max_pairs[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (max_pairs[dev] == 0) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem)) != cudaSuccess)
        return FP8Q_ERR_CUDA;
      int n = 0;
      cfg.gridDim = dim3(2, 1, 1);
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)
        return FP8Q_ERR_UNSUPPORTED;
      max_pairs[dev] = n;
    }
  }
  const int64_t tiles = static_cast<int64_t>(a.tiles) * a.batch;
  const int64_t pairs = tiles < max_pairs[dev] ? tiles : max_pairs[dev];
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, l, r, a) == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Workspace: X (two copies), O_A, O_B as FP16 with pitches of a multiple of 8,
// d_A, d_B and the partial sums of squares; every part starts at a multiple of
// 256 bytes.
struct Layout {
  int64_t p, q, ldx, lda, x0, x1, a, b, da, db, part, bytes;
};
Layout layout_of(int64_t batch, int64_t m, int64_t n) {
  Layout l{};
  l.p = m < n ? m : n;
  l.q = m < n ? n : m;
  l.ldx = up(l.q, 8);
  l.lda = up(l.p, 8);
  const int64_t xb = up(batch * l.p * l.ldx * 2, 256), ab = up(batch * l.p * l.lda * 2, 256);
  l.x0 = 0;
  l.x1 = xb;
  l.a = 2 * xb;
  l.b = l.a + ab;
  const int64_t db = up(batch * l.lda * 4, 256);
  l.da = l.b + ab;
  l.db = l.da + db;
  l.part = l.db + db;
  l.bytes = l.part + batch * kMaxParts * 4;
  return l;
}

bool shape_ok(int64_t batch, int64_t m, int64_t n) {
  return batch >= 0 && m >= 0 && n >= 0 && batch <= 65535 && m <= (1 << 20) && n <= (1 << 20);
}

template <typename In>
fp8q_status load_x(const In *g, int64_t ldg, int64_t bs, int64_t batch, int64_t m, int64_t n,
                   float eps, const Layout &l, uint8_t *ws, cudaStream_t s) {
  float *part = reinterpret_cast<float *>(ws + l.part);
  __half *x = reinterpret_cast<__half *>(ws + l.x0);
  const int parts = static_cast<int>(m < kMaxParts ? m : kMaxParts);
  fp8q_status st = launch_on(ns_sumsq_kernel<In>, dim3(parts, static_cast<unsigned>(batch)),
                             dim3(256), 0, s, g, ldg, bs, m, n, part);
  if (st) return st;
  const dim3 grid(static_cast<unsigned>((n + 63) / 64), static_cast<unsigned>((m + 63) / 64),
                  static_cast<unsigned>(batch));
  return launch_on(m > n ? ns_load_kernel<In, true> : ns_load_kernel<In, false>, grid, dim3(256), 0,
                   s, g, ldg, bs, m, n, static_cast<const float *>(part), parts, eps, x, l.ldx);
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" int64_t fp8q_newton_schulz_workspace_bytes(int64_t batch, int64_t m, int64_t n) {
  if (!shape_ok(batch, m, n)) return 0;
  return layout_of(batch, m, n).bytes;
}

extern "C" fp8q_status fp8q_newton_schulz(const void *g, int64_t ldg, int64_t g_stride,
                                          int in_dtype, void *out, int64_t ldo, int64_t o_stride,
                                          int out_dtype, int64_t batch, int64_t m, int64_t n,
                                          int steps, float a, float b, float c, float eps,
                                          void *workspace, int64_t workspace_bytes, void *stream) {
  const bool in_f32 = in_dtype == FP8Q_OUT_FP32, out_f32 = out_dtype == FP8Q_OUT_FP32;
  if ((!in_f32 && in_dtype != FP8Q_OUT_BF16) || (!out_f32 && out_dtype != FP8Q_OUT_BF16))
    return FP8Q_ERR_INVALID;
  if (!(eps >= 0.0f) || steps < 1) return FP8Q_ERR_INVALID;
  if (!shape_ok(batch, m, n) || ldg < n || ldo < n) return FP8Q_ERR_SHAPE;
  if (batch == 0 || m == 0 || n == 0) return FP8Q_OK;
  if (batch > 1 && (g_stride < 0 || o_stride < (m - 1) * ldo + n)) return FP8Q_ERR_SHAPE;
  if (!g || !out || !workspace) return FP8Q_ERR_INVALID;
  const Layout l = layout_of(batch, m, n);
  if (workspace_bytes < l.bytes) return FP8Q_ERR_SHAPE;
  const int64_t isz = in_f32 ? 4 : 2, osz = out_f32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(g) % isz || reinterpret_cast<uintptr_t>(out) % osz ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;
  if (dev.max_smem_optin < static_cast<int>(smem_of<256>() > smem_of<128>() ? smem_of<256>()
                                                                            : smem_of<128>()))
    return FP8Q_ERR_UNSUPPORTED;
  auto s = static_cast<cudaStream_t>(stream);
  auto *ws = static_cast<uint8_t *>(workspace);
  const uint64_t B = static_cast<uint64_t>(batch), P = static_cast<uint64_t>(l.p),
                 Q = static_cast<uint64_t>(l.q);
  __half *x[2] = {reinterpret_cast<__half *>(ws + l.x0), reinterpret_cast<__half *>(ws + l.x1)};
  float *da = reinterpret_cast<float *>(ws + l.da), *db = reinterpret_cast<float *>(ws + l.db);
  __half *am = reinterpret_cast<__half *>(ws + l.a), *bm = reinterpret_cast<__half *>(ws + l.b);
  CUtensorMap xl[2], xr[2], xn[2], al, ar, bl;
  for (int i = 0; i < 2; ++i)
    if (!make_tmap_f16(&xl[i], x[i], B, P, Q, l.ldx, 128) ||
        !make_tmap_f16(&xr[i], x[i], B, P, Q, l.ldx, 64))
      return FP8Q_ERR_CUDA;
  xn[0] = xr[0];  // the update's N-major boxes: 64 columns x 64 rows as well
  xn[1] = xr[1];
  if (!make_tmap_f16(&al, am, B, P, P, l.lda, 128) || !make_tmap_f16(&ar, am, B, P, P, l.lda, 64) ||
      !make_tmap_f16(&bl, bm, B, P, P, l.lda, 128))
    return FP8Q_ERR_CUDA;
  const int64_t bs = batch > 1 ? g_stride : 0;
  fp8q_status st = in_f32 ? load_x(static_cast<const float *>(g), ldg, bs, batch, m, n, eps, l, ws, s)
                          : load_x(static_cast<const uint16_t *>(g), ldg, bs, batch, m, n, eps, l,
                                   ws, s);
  if (st) return st;

  NsArgs sym{};
  sym.batch = static_cast<int>(batch);
  sym.rows = sym.cols = static_cast<int>(l.p);
  sym.tiles_m = static_cast<int>((l.p + 255) / 256);
  sym.tiles_n = static_cast<int>((l.p + 127) / 128);
  for (int i = 0; i < sym.tiles_m; ++i) sym.tiles += sym.tiles_n - 2 * i;
  sym.ld = sym.ldd = l.lda;
  sym.timeout_ns = wait_timeout_ns().load();
  NsArgs upd = sym;
  upd.cols = static_cast<int>(l.q);
  upd.tiles_n = static_cast<int>((l.q + 255) / 256);
  upd.tiles = upd.tiles_m * upd.tiles_n;
  upd.ld = l.ldx;
  if (static_cast<int64_t>(upd.tiles) * batch >= (1ll << 31)) return FP8Q_ERR_SHAPE;
  const int kx = static_cast<int>((l.q + 63) / 64), kp = static_cast<int>((l.p + 63) / 64);
  for (int i = 0; i < steps; ++i) {
    const int cur = i & 1;
    NsArgs ga = sym;
    ga.kblocks = kx;
    ga.c_acc = 1.0f / kS;
    ga.dst = am;
    ga.diag = ga.diag_out = da;
    if ((st = launch_ns<128, Op::kGram>(xl[cur], xr[cur], ga, s))) return st;
    NsArgs pa = sym;
    pa.kblocks = kp;
    pa.c_old = b;
    pa.c_acc = c / kS;
    pa.old = am;
    pa.dst = bm;
    pa.diag = da;
    pa.diag_out = db;
    if ((st = launch_ns<128, Op::kPoly>(al, ar, pa, s))) return st;
    NsArgs ua = upd;
    ua.kblocks = kp;
    ua.c_old = a;
    ua.c_acc = 1.0f / kS;
    ua.c_diag = 1.0f / kS;
    ua.diag = db;
    ua.old = x[cur];
    ua.dst = x[cur ^ 1];
    if (i + 1 == steps) {  // the last step leaves as the caller's matrix, unscaled
      ua.c_old = a / kS;
      ua.c_diag = 1.0f / (kS * kS);
      ua.c_acc = 1.0f / (kS * kS);
      ua.out = out;
      ua.ldo = ldo;
      ua.out_stride = batch > 1 ? o_stride : 0;
      ua.out_f32 = out_f32;
      ua.tall = m > n;
    }
    if ((st = launch_ns<256, Op::kUpdate>(bl, xn[cur], ua, s))) return st;
  }
  return FP8Q_OK;
}
