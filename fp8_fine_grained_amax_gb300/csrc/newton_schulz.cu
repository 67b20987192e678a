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

int *ns_status_word() {
  void *p = nullptr;
  return cudaGetSymbolAddress(&p, g_ns_status) == cudaSuccess ? static_cast<int *>(p) : nullptr;
}

namespace {

constexpr float kS = 256.0f;        // scale of the stored FP16 matrices
constexpr int kMaxParts = 608;      // partial sums of squares per matrix

// ------------------------------------------------------------------ set-up
__device__ __forceinline__ float load_in(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_in(const uint16_t *p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}
// 16 bytes of input (4 FP32 or 8 BF16 values), kept in the cache: the matrix is
// read a second time by the next kernel.
__device__ __forceinline__ void load_vec(const float *p, float (&v)[4]) {
  const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
  v[0] = f.x;
  v[1] = f.y;
  v[2] = f.z;
  v[3] = f.w;
}
__device__ __forceinline__ void load_vec(const uint16_t *p, float (&v)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
template <typename In>
constexpr int kVecOf = 16 / static_cast<int>(sizeof(In));

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum of squares of matrix blockIdx.y, part blockIdx.x of gridDim.x; a warp
// takes pieces of a row (8 loads per lane with kVec false, 4 or 8 with kVec),
// all of a piece's loads in flight.  kVec: rows begin on 16-byte boundaries.  The
// order is fixed, so repeated calls agree.  Also zeroes the counters that the steps kernel of this call uses.
template <bool kVec>
constexpr int kPieceOf = kVec ? 1024 : 256;
template <typename In, bool kVec>
__global__ void __launch_bounds__(256) ns_sumsq_kernel(const In *__restrict__ g, int64_t ldg,
                                                       int64_t batch_stride, int64_t m, int64_t n,
                                                       float *__restrict__ part,
                                                       uint32_t *__restrict__ counters,
                                                       int n_counters) {
  constexpr int V = kVec ? kVecOf<In> : 1;
  constexpr int kPiece = kPieceOf<kVec>, kLoads = kPiece / 32 / V;
  __shared__ float sums[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_previous_kernel();
  let_next_kernel_start();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < n_counters; i += 256) counters[i] = 0u;
  const In *base = g + blockIdx.y * batch_stride;
  const int64_t pieces = (n + kPiece - 1) / kPiece, items = m * pieces;
  float acc = 0.0f;
  for (int64_t it = blockIdx.x * 8 + warp; it < items; it += 8 * gridDim.x) {
    const int64_t r = it / pieces, c0 = (it - r * pieces) * kPiece;
    const In *row = base + r * ldg + c0;
    const int left = static_cast<int>(n - c0 < kPiece ? n - c0 : kPiece);
    float v[kLoads][V];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * 32 + lane) * V;
      if constexpr (kVec) {
        if (c + V <= left) {
          load_vec(row + c, v[i]);
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = c + j < left ? load_in(row + c + j) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) acc = fmaf(v[i][j], v[i][j], acc);
  }
  acc = warp_sum(acc);
  if (lane == 0) sums[warp] = acc;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float t = warp_sum(lane < 8 ? sums[lane] : 0.0f);
    if (lane == 0) part[blockIdx.y * kMaxParts + blockIdx.x] = t;
  }
}

// S / (|g|_F + eps) of matrix blockIdx.z from its partial sums, to every thread.
// (The partial sums are the previous kernel's; the matrix itself is not, but the
// kernel before that one may be writing it still: nothing is read ahead.)
__device__ __forceinline__ float ns_scale(const float *part, int parts, float eps, float *shared) {
  if (threadIdx.x < 32) {
    float v = 0.0f;
    for (int i = threadIdx.x; i < parts; i += 32) v += part[blockIdx.z * kMaxParts + i];
    v = warp_sum(v);
    if (threadIdx.x == 0) {
      // below 2^-119 only where v is 0: the quotient would overflow, and 0 * inf is
      // no zero.  (eps = 0 and a zero matrix: 0 / 0, as the formula has it.)
      const float norm = sqrtf(v) + eps;
      *shared = norm > 0.0f && norm < 0x1p-119f ? 0x1p127f : kS / norm;
    }
  }
  __syncthreads();
  return *shared;
}

__device__ __forceinline__ uint4 pack_half8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// X^ = FP16(S g / (|g|_F + eps)), g no taller than wide: blocks of 32 rows x
// 256 columns, eight columns of four rows per thread.  The pitch ldx is a
// multiple of 8, so every 16-byte unit that begins inside the row is whole.
template <typename In, bool kVec>
__global__ void __launch_bounds__(256) ns_load_kernel(const In *__restrict__ g, int64_t ldg,
                                                      int64_t batch_stride, int64_t m, int64_t n,
                                                      const float *__restrict__ part, int parts,
                                                      float eps, __half *__restrict__ x,
                                                      int64_t ldx) {
  constexpr int V = kVecOf<In>;
  __shared__ float s_scale;
  wait_for_previous_kernel();
  let_next_kernel_start();
  const In *base = g + blockIdx.z * batch_stride;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + 8 * (threadIdx.x & 31);
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 32 + (threadIdx.x >> 5);
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 8 * i;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r >= m || c >= n) continue;
    const In *src = base + r * ldg + c;
    if (kVec && c + 8 <= n) {
#pragma unroll
      for (int j = 0; j < 8; j += V) {
        float t[V];
        load_vec(src + j, t);
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][j + k] = t[k];
      }
    } else {
      for (int j = 0; j < 8; ++j)
        if (c + j < n) v[i][j] = load_in(src + j);
    }
  }
  const float scale = ns_scale(part, parts, eps, &s_scale);
  __half *dst = x + blockIdx.z * (m * ldx);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + 8 * i;
    if (r >= m || c >= n) continue;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= scale;
    *reinterpret_cast<uint4 *>(dst + r * ldx + c) = pack_half8(v[i]);
  }
}

// The same, transposed (g taller than wide): 64 x 64 blocks through shared memory.
template <typename In, bool kVec>
__global__ void __launch_bounds__(256) ns_load_tall_kernel(const In *__restrict__ g, int64_t ldg,
                                                           int64_t batch_stride, int64_t m,
                                                           int64_t n,
                                                           const float *__restrict__ part,
                                                           int parts, float eps,
                                                           __half *__restrict__ x, int64_t ldx) {
  constexpr int V = kVecOf<In>;
  constexpr int kLanes = 64 / V;         // threads across a block row
  constexpr int kRows = 256 / kLanes;    // rows per pass
  __shared__ float s_scale;
  __shared__ float tile[64][65];
  wait_for_previous_kernel();
  let_next_kernel_start();
  const In *base = g + blockIdx.z * batch_stride;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int tid = threadIdx.x, j0 = V * (tid % kLanes);
#pragma unroll
  for (int i = 0; i < 64 / kRows; ++i) {
    const int rr = i * kRows + tid / kLanes;
    const int64_t r = r0 + rr, c = c0 + j0;
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = 0.0f;
    if (r < m && c < n) {
      const In *src = base + r * ldg + c;
      if (kVec && c + V <= n) {
        load_vec(src, v);
      } else {
        for (int k = 0; k < V; ++k)
          if (c + k < n) v[k] = load_in(src + k);
      }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) tile[rr][j0 + k] = v[k];
  }
  const float scale = ns_scale(part, parts, eps, &s_scale);  // also: the block is complete
  __half *dst = x + blockIdx.z * (n * ldx);
  const int j = 8 * (tid & 7);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int cc = 32 * i + (tid >> 3);
    if (c0 + cc >= n || r0 + j >= m) continue;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = tile[j + k][cc] * scale;
    *reinterpret_cast<uint4 *>(dst + (c0 + cc) * ldx + r0 + j) = pack_half8(v);
  }
}

// ------------------------------------------------------------------ products
// One persistent kernel runs every step: 3 * steps phases on CTA pairs
// (tcgen05.mma.cta_group::2, tiles of 256 rows x 256, 128 or 64 columns, K = 16
// per instruction), one pair per two SMs.  Against one launch per product this saves the launch, the
// set-up and the pipeline's first fill, which took longer than the products
// themselves for all but the largest matrices (a 301 x 999 update: 9 us per
// launch).
//  - A matrix moves on to its next phase when its own tiles of the last one are
//    done (a counter per matrix), so the matrices of a batch do not wait for
//    one another.
//  - Tiles are dealt out to the pairs in turn, so that a pair's tiles of a phase
//    belong to different matrices of a batch and the first of them are ready
//    when it comes to the next phase.  Where whole tiles would leave pairs idle
//    for long, pair i takes units [i per, (i + 1) per) of (tile, 64-wide K block)
//    instead, an even share that splits tiles.  A pair whose range begins inside a tile
//    writes its FP32 partial sums to its slot of the workspace; the pair that
//    began the tile, which reaches it last in its own range, adds the partials
//    of the pairs after it in order.  The order is fixed, so results repeat bit
//    by bit.
//  - D = L R^T: both operands are row blocks of X or A, K-major.  The update
//    D = L R reads X as an N-major operand (64 columns x 64 K rows per box), so
//    no transposed copy of X exists.
//  - Two TMEM accumulators: the epilogue of one tile runs under the MMAs of the
//    next.  A warp's old values of X or A are fetched and put into shared
//    memory before it waits for the accumulator, the results replace them
//    there, and global accesses are whole 64-byte pieces of rows.
//  - Data written by other SMs in an earlier phase is read past L1 (ld.cg), and
//    by TMA after a proxy fence behind the counter.  One thread per CTA polls the
//    counter and tells the epilogue warps through shared memory.
//  - The operand ring takes what the epilogue's staging leaves: 5 stages of 32 KB
//    for 256-wide tiles, 8 of 24 KB for 128, 10 of 20 KB for 64.  A stage's copy
//    takes about 1.2 us from issue to arrival, so that with 5 stages no tile
//    could run faster than 0.24 us per K block (128-wide tiles: 0.17 us of MMAs).
//    Changing the layout between phases drains the ring, which a single matrix
//    does anyway; a batch, whose phases overlap, keeps its widest tile's layout
//    (16 of 896 x 640: 204 us, 240 with changes).
//  - The tile width is chosen per phase kind (see Plan): 256 columns feed the
//    tensor cores best (62 bytes of operands per clock and SM), narrower tiles
//    cover the matrix with less waste and finish sooner where there are few.
//   warp 0 TMA producer, warp 1 MMA issuer (leading CTA), warp 2 counts done
//   tiles, warps 4-11 epilogue (each thread one row, half of the tile's columns).
constexpr int kGram = 0, kPoly = 1, kUpdate = 2;  // A = X X^T | B = bA + cA^2 | X' = aX + BX

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kTile = 256;               // rows of a pair's tile, and its largest width
constexpr int kMaxStages = 10;
constexpr uint32_t kOpBytes = 128 * 128;  // one operand's share of a CTA: 128 x 64 FP16
constexpr int kMaxPairs = 76;            // slots for partial sums
// Register split as in the GEMMs: built for kLaunchRegs (checked by the build),
// the control warpgroup hands registers to the two epilogue warpgroups.
constexpr int kLaunchRegs = 168;
constexpr int kCtlRegs = 56, kEpiRegs = 224;
static_assert(kCtlRegs + 2 * kEpiRegs <= 3 * kLaunchRegs, "register split must fit the launch");
constexpr uint64_t kDrainNs = 1000000000ull;
// Staging of one epilogue warp: its rows and columns as FP16, in blocks of 32 x
// 32 (2 KB each; also half an FP32 block of the final result).
constexpr uint32_t kStageBlock = 2048;
// Shared memory from a 1024-byte boundary on: the ring, upwards, and at the end
// the staging of the kind's tile width.
constexpr uint32_t kArena = 224 * 1024;
__host__ __device__ constexpr uint32_t staging_bytes(int bn) { return kEpiWarps * (bn / 64) * kStageBlock; }
__host__ __device__ constexpr uint32_t ring_stage(int bn) { return kOpBytes + bn / 2 * 128; }
__host__ __device__ constexpr int ring_stages(int bn) {
  return static_cast<int>((kArena - staging_bytes(bn)) / ring_stage(bn)) < kMaxStages
             ? static_cast<int>((kArena - staging_bytes(bn)) / ring_stage(bn))
             : kMaxStages;
}
static_assert(ring_stages(256) == 5 && ring_stages(128) == 8 && ring_stages(64) == 10, "ring depths");
constexpr int64_t kSlotFloats = 2 * 128 * 256;

struct alignas(8) Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  // counts, not barrier phases: writer and reader may be any number of steps apart
  uint32_t stored[kEpiWarps];  // tiles whose results a warp has written
  uint32_t ready;              // segments whose matrix is ready for its phase
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kSmem = 1024 + kArena + sizeof(Ctl);
static_assert(kSmem <= 227 * 1024, "shared memory");

// Counters in the workspace, zeroed by the set-up kernel of each call; after
// them, per matrix, the number of its tiles done in all phases (two CTAs each).
struct Sync {
  uint32_t part[kMaxPairs][2][kEpiWarps];  // phase + 1 of the partial sums in the slot
  uint32_t used[kMaxPairs][2][kEpiWarps];  // phase + 1 of the partial sums that were added
};

struct NsArgs {
  int batch, p, q, steps;
  int kb_q, kb_p;          // 64-wide K blocks along q and p
  int row_tiles;           // 256-row tiles along p
  int bn[3], tiles[3];     // by phase kind: tile width, tiles per matrix,
  int layout[3];           // the width that the ring and the staging are laid out for,
  int per[3];              // units per pair of an even split, or 0: whole tiles
  float a, b, c;
  __half *x[2], *am, *bm;
  int64_t ldx, lda;
  float *da, *db;        // S d_A, S d_B, pitch lda
  float *partial;        // [pair][CTA][warp][float4 column][lane]
  Sync *sync;
  uint32_t *done;
  void *out;
  int64_t ldo, out_stride;
  int out_f32, tall, out_vec;  // out_vec: 16-byte units of BF16 rows may be stored
  uint64_t timeout_ns;
};

struct Maps {
  CUtensorMap x[2], a, b;  // left operands: 128 rows x 64
  CUtensorMap xr[2], ar;   // right operands of A and A^2: half a tile's columns x 64
  CUtensorMap xn[2];       // right operand of the update: 64 K rows x 64 columns
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
// Order generic-proxy and async-proxy (TMA) accesses of global memory.
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t *p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void red_release(uint32_t *p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}

// Bounded wait until *p has reached `want` (counters only grow within a call).
__device__ __forceinline__ bool wait_count(const uint32_t *p, uint32_t want,
                                           volatile int *abort_flag, uint64_t limit_ns) {
  if (ld_acquire(p) >= want) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (ld_acquire(p) >= want) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      atomicExch(&g_ns_status, FP8Q_ERR_TIMEOUT);
      return false;
    }
  }
}

// The same for a counter in shared memory.
__device__ __forceinline__ uint32_t ld_acquire_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_release_shared(uint32_t addr, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ bool wait_shared(uint32_t addr, uint32_t want, volatile int *abort_flag,
                                            uint64_t limit_ns) {
  if (ld_acquire_shared(addr) >= want) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (ld_acquire_shared(addr) >= want) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      atomicExch(&g_ns_status, FP8Q_ERR_TIMEOUT);
      return false;
    }
  }
}

// True for the whole warp where every lane's wait came true.  What the waiting
// lanes acquired is ordered before the other lanes' accesses by __syncwarp; a
// vote alone orders no memory.
__device__ __forceinline__ bool warp_acquired(bool got) {
  const bool all = __all_sync(0xffffffffu, got) != 0;
  __syncwarp();
  return all;
}

// One pair's walk over its units of a phase, as segments of tiles.
struct Segment {
  int b, row0, col0;  // matrix, first row and column of the tile
  int kb0, kb1;       // its K blocks
};
struct Walk {
  int kind, kblocks, u, end, stride;  // units; stride: to the pair's next whole tile
  uint32_t ready;  // a matrix's count of done tiles that lets it into this phase
  __device__ Walk(const NsArgs &p, int phase, int pair) {
    kind = phase % 3;
    kblocks = kind == kGram ? p.kb_q : p.kb_p;
    const int units = p.tiles[kind] * p.batch * kblocks;
    int before = phase / 3 * (p.tiles[0] + p.tiles[1] + p.tiles[2]);
    if (kind > 0) before += p.tiles[0];
    if (kind > 1) before += p.tiles[1];
    ready = 2u * static_cast<uint32_t>(before);
    if (p.per[kind] > 0) {
      u = min(pair * p.per[kind], units);
      end = min(u + p.per[kind], units);
      stride = 0;
    } else {
      u = pair < p.tiles[kind] * p.batch ? pair * kblocks : units;
      end = units;
      stride = static_cast<int>(gridDim.x >> 1) * kblocks;
    }
  }
  __device__ bool next(const NsArgs &p, Segment &s) {
    if (u >= end) return false;
    const int t = u / kblocks;
    s.kb0 = u - t * kblocks;
    s.kb1 = min(kblocks, s.kb0 + (end - u));
    u = stride == 0 ? u + (s.kb1 - s.kb0) : end - u > stride ? u + stride : end;
    s.b = t / p.tiles[kind];
    int w = t - s.b * p.tiles[kind];
    const int bn = p.bn[kind];
    if (kind == kUpdate) {
      s.row0 = (w % p.row_tiles) * kTile;
      s.col0 = (w / p.row_tiles) * bn;
    } else {  // row tile i has the columns from its own first row on
      const int per_row = kTile / bn, n = (p.p + bn - 1) / bn;
      int i = 0;
      while (w >= n - per_row * i) w -= n - per_row * i++;
      s.row0 = i * kTile;
      s.col0 = (per_row * i + w) * bn;
    }
    return true;
  }
};

// What an epilogue warp knows of its own place.
struct Epi {
  uint32_t stage;   // its staging: four blocks of 32 x 32
  int row0, lane;   // its first row
};
// 16-byte unit k of row r in a staged block (conflict-free by row and by piece).
__device__ __forceinline__ uint32_t unit_at(uint32_t block, uint32_t r, uint32_t k) {
  return block + r * 64 + 16 * (k ^ ((r >> 1) & 3));
}

__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// A warp's old values, 32 rows x 128 columns: lane l fetches 16-byte unit l % 4
// of rows l / 4 + 8 i of each 32-column block.  Pitches are multiples of 8, so a
// unit that begins inside the matrix may be read to its end.
__device__ __forceinline__ void stage_old(const Epi &e, const __half *m, int64_t ld, int rows,
                                          int cols, int cbase, int blocks) {
  uint4 v[4][4];
  const int r0 = e.row0 + (e.lane >> 2);
  const __half *src = m + static_cast<int64_t>(r0) * ld + cbase + 8 * (e.lane & 3);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[c][i] = make_uint4(0, 0, 0, 0);
      if (c < blocks && r0 + 8 * i < rows && cbase + 32 * c + 8 * (e.lane & 3) < cols)
        v[c][i] = __ldcg(reinterpret_cast<const uint4 *>(src + 8 * i * ld + 32 * c));
    }
  __syncwarp();  // the blocks' previous contents have been read
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c < blocks) st_shared_v4(unit_at(e.stage + c * kStageBlock, (e.lane >> 2) + 8 * i, e.lane & 3), v[c][i]);
  __syncwarp();
}
// This lane's row of a staged block, FP16 pairs.
__device__ __forceinline__ void read_row(const Epi &e, int c, uint32_t (&w)[16]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 u = ld_shared_v4(unit_at(e.stage + c * kStageBlock, e.lane, k));
    w[4 * k] = u.x;
    w[4 * k + 1] = u.y;
    w[4 * k + 2] = u.z;
    w[4 * k + 3] = u.w;
  }
}
__device__ __forceinline__ void write_row(const Epi &e, int c, const uint32_t (&w)[16]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    st_shared_v4(unit_at(e.stage + c * kStageBlock, e.lane, k),
                 make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
}
// The staged 16-bit results to rows of m, 64-byte pieces; the last partial unit
// of a row element by element.
__device__ __forceinline__ void store_staged(const Epi &e, uint16_t *m, int64_t ld, int rows,
                                             int cols, int cbase, int blocks) {
  __syncwarp();
  const int r0 = e.row0 + (e.lane >> 2);
  uint16_t *dst = m + static_cast<int64_t>(r0) * ld + cbase + 8 * (e.lane & 3);
#pragma unroll 1
  for (int c = 0; c < blocks; ++c, dst += 32) {
    const int left = cols - (cbase + 32 * c + 8 * (e.lane & 3));
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = ld_shared_v4(unit_at(e.stage + c * kStageBlock, (e.lane >> 2) + 8 * i, e.lane & 3));
    if (left >= 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + 8 * i < rows) *reinterpret_cast<uint4 *>(dst + 8 * i * ld) = u[i];
    } else if (left > 0) {
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        if (r0 + 8 * i >= rows) break;
        const uint32_t at = unit_at(e.stage + c * kStageBlock, (e.lane >> 2) + 8 * i, e.lane & 3);
        for (int k = 0; k < left; ++k) dst[8 * i * ld + k] = ld_shared_u16(at + 2 * k);
      }
    }
  }
}
// r[lane], by halving.
__device__ __forceinline__ float own_column(const uint32_t (&r)[32], int lane) {
  uint32_t v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = lane & 16 ? r[i + 16] : r[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = lane & 8 ? v[i + 8] : v[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = lane & 4 ? v[i + 4] : v[i];
#pragma unroll
  for (int i = 0; i < 2; ++i) v[i] = lane & 2 ? v[i + 2] : v[i];
  return __uint_as_float(lane & 1 ? v[1] : v[0]);
}
// A lane's row of a block, transposed: column runs are contiguous over the lanes.
__device__ __forceinline__ void store_mirror(const Epi &e, const uint32_t (&w)[16], __half *m,
                                             int64_t ld, int n, int col0) {
  const int row = e.row0 + e.lane;
  if (row >= n) return;
  uint16_t *dst = reinterpret_cast<uint16_t *>(m) + static_cast<int64_t>(col0) * ld + row;
  const int left = n - col0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (i < left) *dst = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
    dst += ld;
  }
}

// A 32 x 32 block of the final result into the caller's matrix, any pitch: column
// runs (tall) are contiguous over the lanes; row runs go through shared memory.
__device__ __forceinline__ void store_out(const Epi &e, const float (&v)[32], const NsArgs &p, int b,
                                          int col0, float *st) {
  const int64_t base = static_cast<int64_t>(b) * p.out_stride;
  const int row = e.row0 + e.lane;
  if (p.tall) {
    if (row < p.p) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col0 + i < p.q) {
          const int64_t at = base + static_cast<int64_t>(col0 + i) * p.ldo + row;
          if (p.out_f32) static_cast<float *>(p.out)[at] = v[i];
          else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v[i]);
        }
    }
    return;
  }
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {  // 16 rows at a time: 2 KB
    __syncwarp();
    if ((e.lane >> 4) == half) {
#pragma unroll
      for (int i = 0; i < 32; ++i) st[(e.lane & 15) * 32 + (i ^ e.lane)] = v[i];
    }
    __syncwarp();
    if (col0 + e.lane < p.q) {
      const int r0 = e.row0 + 16 * half, n = min(16, p.p - r0);
      for (int i = 0; i < n; ++i) {
        const int64_t at = base + static_cast<int64_t>(r0 + i) * p.ldo + col0 + e.lane;
        const float f = st[i * 32 + (e.lane ^ (16 * half + i))];
        if (p.out_f32) static_cast<float *>(p.out)[at] = f;
        else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(f);
      }
    }
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_steps_kernel(const __grid_constant__ Maps maps, const NsArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t ring = smem_u32(smem);
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + kArena);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &ctl->abort_flag;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int phases = 3 * p.steps;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_u32(&ctl->full[i]), 1);
      mbar_init(smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctl->tfull[i]), 1);
      mbar_init(smem_u32(&ctl->tempty[i]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort_flag = 0;
    for (int i = 0; i < kEpiWarps; ++i) ctl->stored[i] = 0;
    ctl->ready = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane < static_cast<int>(sizeof(Maps) / sizeof(CUtensorMap)))
    prefetch_tmap(&maps.x[0] + lane);
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctl->tmem_base), 512);
    tc_fence_before();
  }
  __syncwarp();
  wait_for_previous_kernel();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    // ================================================== epilogue
    const int ew = warp - 4, quarter = warp & 3, half = ew >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(&ctl->tempty[0]), 0);
    Epi e;
    e.lane = lane;
    // this warp's part of a pair's slot of partial sums, as float4
    auto slot_of = [&](int pr) {
      return reinterpret_cast<float4 *>(p.partial + pr * kSlotFloats) +
             (static_cast<int>(rank) * kEpiWarps + ew) * 32 * 32 + lane;
    };
    // lane 0 waits for a counter; the answer goes to the whole warp
    auto warp_wait = [&](const uint32_t *count, uint32_t want) {
      const bool got = lane != 0 || wait_count(count, want, abort_flag, p.timeout_ns);
      return warp_acquired(got);
    };
    int buf = 0, tile_no = 0, seg_no = 0;
    uint32_t tphase = 0, given = 0;  // given: phase + 1 of this warp's last partial sums
    bool ok = true;
    for (int phase = 0; ok && phase < phases; ++phase) {
      const int kind = phase % 3, cur = (phase / 3) & 1;
      const bool last = phase + 1 == phases;
      Walk walk(p, phase, pair);
      Segment s;
      const uint32_t staging = staging_bytes(p.layout[kind]);
      uint8_t *stage = smem + kArena - staging + staging / kEpiWarps * ew;
      e.stage = smem_u32(stage);
      for (; walk.next(p, s); ++seg_no) {
        e.row0 = s.row0 + static_cast<int>(rank) * 128 + quarter * 32;
        const int bn = p.bn[kind], blocks = bn / 64;  // 32-column blocks of this warp
        const int row = e.row0 + lane, cbase = s.col0 + half * (bn / 2);
        const int cols = kind == kUpdate ? p.q : p.p;
        const bool live = e.row0 < p.p && cbase < cols;  // warp-uniform
        const bool owner = s.kb0 == 0;
        const int64_t xmat = static_cast<int64_t>(s.b) * p.p * p.ldx,
                      amat = static_cast<int64_t>(s.b) * p.p * p.lda;
        const float *diag = (kind == kUpdate ? p.db : p.da) + static_cast<int64_t>(s.b) * p.lda;
        float d_row = 0.0f;
        float4 d_col = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // c/S d_A of columns 4 lane .. + 3
        if (owner && live && kind != kGram) {
          // old values are on their way, or in place, before the accumulator is
          // waited for: under the MMAs' own traffic a load takes over a microsecond
          const bool there = lane != 0 || wait_shared(smem_u32(&ctl->ready),
                                                      static_cast<uint32_t>(seg_no) + 1, abort_flag,
                                                      p.timeout_ns);
          if (!(ok = warp_acquired(there))) break;
          if (row < p.p) d_row = __ldcg(diag + row);
          if (kind == kPoly) {  // the pitch is whole
            const int dc = cbase + 4 * lane;
            if (dc < cols && lane < 8 * blocks)
              d_col = __ldcg(reinterpret_cast<const float4 *>(diag + dc));
            const float cs = p.c / kS;
            d_col = make_float4(cs * d_col.x, cs * d_col.y, cs * d_col.z, cs * d_col.w);
          }
          if (kind == kUpdate) stage_old(e, p.x[cur] + xmat, p.ldx, p.p, cols, cbase, blocks);
          else stage_old(e, p.am + amat, p.lda, p.p, cols, cbase, blocks);
        }

        const bool got = mbar_wait_bounded(smem_u32(&ctl->tfull[buf]), tphase, abort_flag,
                                           &g_ns_status, p.timeout_ns, FP8Q_ERR_TIMEOUT);
        if (!(ok = __all_sync(0xffffffffu, got))) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                               static_cast<uint32_t>(buf * kTile + half * (bn / 2));
        // block c of the accumulator; the last one releases it
        auto load_block = [&](int c, uint32_t (&r)[32]) {
          tmem_ld_32x32b_x32(taddr + 32 * c, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
          if (c == blocks - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty0 + static_cast<uint32_t>(buf) * 8u);
          }
        };
        if (!owner) {  // partial sums for the pair that began the tile
          // ... once it has added this warp's last ones
          if (given && !(ok = warp_wait(&p.sync->used[pair][rank][ew], given))) break;
          float4 *slot = slot_of(pair);
#pragma unroll 1
          for (int c = 0; c < blocks; ++c, slot += 8 * 32) {
            uint32_t r[32];
            load_block(c, r);
            if (!live) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              __stcg(slot + k * 32,
                     make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                                 __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3])));
          }
          given = static_cast<uint32_t>(phase) + 1;
          __syncwarp();
          if (lane == 0) st_release(&p.sync->part[pair][rank][ew], given);
          buf ^= 1;
          if (buf == 0) tphase ^= 1;
          continue;
        }
        // pairs after this one that hold the rest of the tile
        const int helpers =
            s.kb1 == walk.kblocks ? 0 : (walk.kblocks - s.kb1 + p.per[kind] - 1) / p.per[kind];
        for (int h = 1; ok && h <= helpers; ++h)
          ok = warp_wait(&p.sync->part[pair + h][rank][ew], static_cast<uint32_t>(phase) + 1);
        if (!ok) break;
        const bool bf16_rows = last && p.out_vec;
        // tiles on the diagonal hold both triangles themselves
        const bool mirror = kind != kUpdate && s.col0 >= s.row0 + kTile;
        if (kind == kGram) __syncwarp();  // the blocks' previous contents have been read
        {
          // one block at a time, the loop not unrolled: this code runs once per
          // tile, and fetching it costs more than running it
#pragma unroll 1
          for (int c = 0; c < blocks; ++c) {
            uint32_t r[32];
            load_block(c, r);
            if (!live) continue;
            for (int h = 1; h <= helpers; ++h) {
              const float4 *src = slot_of(pair + h) + 8 * 32 * c;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 f = __ldcg(src + k * 32);
                r[4 * k] = __float_as_uint(__uint_as_float(r[4 * k]) + f.x);
                r[4 * k + 1] = __float_as_uint(__uint_as_float(r[4 * k + 1]) + f.y);
                r[4 * k + 2] = __float_as_uint(__uint_as_float(r[4 * k + 2]) + f.z);
                r[4 * k + 3] = __float_as_uint(__uint_as_float(r[4 * k + 3]) + f.w);
              }
            }
            const int col0 = cbase + 32 * c;
            uint32_t w[16];
            if (kind == kUpdate) {
              const float scale = last ? 1.0f / (kS * kS) : 1.0f / kS;
              float co = fmaf(1.0f / kS, d_row, p.a);
              if (last) co *= 1.0f / kS;
              read_row(e, c, w);
              if (!last || bf16_rows) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const float x = fmaf(co, f16_lo(w[k]), scale * __uint_as_float(r[2 * k]));
                  const float y = fmaf(co, f16_hi(w[k]), scale * __uint_as_float(r[2 * k + 1]));
                  if (last) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                  } else {
                    const __half2 h = __floats2half2_rn(x, y);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                  }
                }
                write_row(e, c, w);
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  r[i] = __float_as_uint(fmaf(co, i & 1 ? f16_hi(w[i / 2]) : f16_lo(w[i / 2]),
                                              scale * __uint_as_float(r[i])));
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                if (col0 < cols) store_out(e, v, p, s.b, col0, reinterpret_cast<float *>(stage + c * kStageBlock));
              }
              continue;
            }
            float d_new = 0.0f;
            if (kind == kGram) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                r[i] = __float_as_uint((1.0f / kS) * __uint_as_float(r[i]));
            } else {
              const float cs = p.c / kS, co = fmaf(cs, d_row, p.b);
              read_row(e, c, w);
              if (e.row0 == col0)  // b d_A + c/S (sum + d_A^2) on the diagonal
                d_new = fmaf(p.b, d_row, cs * fmaf(d_row, d_row, own_column(r, lane)));
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float dc[4] = {__shfl_sync(0xffffffffu, d_col.x, 8 * c + k),
                                     __shfl_sync(0xffffffffu, d_col.y, 8 * c + k),
                                     __shfl_sync(0xffffffffu, d_col.z, 8 * c + k),
                                     __shfl_sync(0xffffffffu, d_col.w, 8 * c + k)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int i = 4 * k + j;
                  const float o = i & 1 ? f16_hi(w[i / 2]) : f16_lo(w[i / 2]);
                  r[i] = __float_as_uint(fmaf(co + dc[j], o, cs * __uint_as_float(r[i])));
                }
              }
            }
            // the diagonal crosses this block (both begin at multiples of 32): its
            // values leave as FP32, the FP16 matrix holds zeros there
            const bool on_diag = e.row0 == col0;
            if (on_diag) {
              if (kind == kGram) d_new = own_column(r, lane);
              if (row < p.p)
                __stcg((kind == kGram ? p.da : p.db) + static_cast<int64_t>(s.b) * p.lda + row, d_new);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const __half2 h = __floats2half2_rn(__uint_as_float(r[2 * k]),
                                                  __uint_as_float(r[2 * k + 1]));
              w[k] = *reinterpret_cast<const uint32_t *>(&h);
            }
            write_row(e, c, w);
            if (on_diag)
              st_shared_u16(unit_at(e.stage + c * kStageBlock, lane, lane >> 3) + 2 * (lane & 7), 0u);
            if (mirror) store_mirror(e, w, (kind == kGram ? p.am : p.bm) + amat, p.lda, p.p, col0);
          }
          if (live && (!last || bf16_rows)) {
            uint16_t *dst = static_cast<uint16_t *>(p.out) + static_cast<int64_t>(s.b) * p.out_stride;
            int64_t ld = p.ldo;
            if (!last) {
              dst = reinterpret_cast<uint16_t *>(
                  kind == kUpdate ? p.x[cur ^ 1] + xmat : (kind == kGram ? p.am : p.bm) + amat);
              ld = kind == kUpdate ? p.ldx : p.lda;
            }
            store_staged(e, dst, ld, p.p, cols, cbase, blocks);
          }
        }
        for (int h = 1; h <= helpers; ++h) {  // the slots may be written again
          __syncwarp();
          if (lane == 0)
            st_release(&p.sync->used[pair + h][rank][ew], static_cast<uint32_t>(phase) + 1);
        }
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
        // warp 2 counts the tile as done
        __syncwarp();
        if (lane == 0)
          st_release_shared(smem_u32(&ctl->stored[ew]), static_cast<uint32_t>(tile_no) + 1);
        ++tile_no;
      }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    return;
  }
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
  if (warp == 0) {
    // ================================================== TMA producer
    if (lane == 0) {
      int st = 0, seg_no = 0, tile_no = 0, before = p.layout[0];
      uint32_t phases_of = 0, armed = 0;  // bit i: parity of stage i's next use; used so far
      bool ok = true;
      auto wait_empty = [&](int i) {
        return mbar_wait_bounded(smem_u32(&ctl->empty[i]), ((phases_of >> i) & 1u) ^ 1u, abort_flag,
                                 &g_ns_status, p.timeout_ns, FP8Q_ERR_TIMEOUT);
      };
      for (int phase = 0; ok && phase < phases; ++phase) {
        const int kind = phase % 3, cur = (phase / 3) & 1;
        const CUtensorMap *ml = kind == kGram ? &maps.x[cur] : kind == kPoly ? &maps.a : &maps.b;
        const CUtensorMap *mr = kind == kGram   ? &maps.xr[cur]
                                : kind == kPoly ? &maps.ar
                                                : &maps.xn[cur];
        const int half_cols = p.bn[kind] / 2, layout = p.layout[kind], stages = ring_stages(layout);
        const uint32_t stage_bytes = ring_stage(layout), tx = 2 * ring_stage(p.bn[kind]);
        if (layout != before) {
          // another layout: every stage has been used up, and the last tile's
          // results have left the staging that the ring may now reach into
          for (int i = 0; ok && i < kMaxStages; ++i)
            if (armed >> i & 1u) ok = wait_empty(i);
          for (int i = 0; ok && i < kEpiWarps; ++i)
            ok = wait_shared(smem_u32(&ctl->stored[i]), static_cast<uint32_t>(tile_no), abort_flag,
                             p.timeout_ns);
          if (!ok) break;
          before = layout;
          st = 0;
        }
        Walk walk(p, phase, pair);
        Segment s;
        while (ok && walk.next(p, s)) {
          if (!(ok = wait_count(&p.done[s.b], walk.ready, abort_flag, p.timeout_ns))) break;
          st_release_shared(smem_u32(&ctl->ready), static_cast<uint32_t>(++seg_no));
          if (s.kb0 == 0) ++tile_no;
          fence_proxy_async_all();
          for (int kb = s.kb0; kb < s.kb1; ++kb) {
            if (!(ok = wait_empty(st))) break;
            const uint32_t fb = smem_u32(&ctl->full[st]);
            if (rank == 0) mbar_arrive_expect_tx(fb, tx);
            const uint32_t fb0 = mapa_shared(fb, 0), sl = ring + st * stage_bytes, sr = sl + kOpBytes;
            tma_load_3d_pair(sl, ml, fb0, kb * 64, s.row0 + static_cast<int>(rank) * 128, s.b);
            const int rc = s.col0 + static_cast<int>(rank) * half_cols;
            if (kind != kUpdate) {
              tma_load_3d_pair(sr, mr, fb0, kb * 64, rc, s.b);
            } else {
              tma_load_3d_pair(sr, mr, fb0, rc, kb * 64, s.b);
              if (half_cols > 64) tma_load_3d_pair(sr + 8192, mr, fb0, rc + 64, kb * 64, s.b);
            }
            armed |= 1u << st;
            phases_of ^= 1u << st;
            if (++st == stages) st = 0;
          }
        }
      }
      if (!ok) {
        // this CTA's copies land before it exits (the leading CTA's barriers
        // see both CTAs' copies; the other waits long enough for any copy)
        if (rank == 0)
          for (int i = 0; i < kMaxStages; ++i)
            if (armed >> i & 1u)
              mbar_wait_drain(smem_u32(&ctl->full[i]), ((phases_of >> i) & 1u) ^ 1u);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
      }
    }
  } else if (warp == 2) {
    // ================================================== counts of done tiles
    // One device-wide fence per tile covers all epilogue warps' writes, seen
    // through their counts; the epilogue does not wait for it (about 1 us).
    int tile_no = 0;
    bool ok = true;
    for (int phase = 0; ok && phase + 1 < phases; ++phase) {
      Walk walk(p, phase, pair);
      Segment s;
      while (ok && walk.next(p, s)) {
        if (s.kb0 != 0) continue;  // the pair that began the tile counts it
        ++tile_no;
        const bool there =
            lane >= kEpiWarps || wait_shared(smem_u32(&ctl->stored[lane]),
                                             static_cast<uint32_t>(tile_no), abort_flag, p.timeout_ns);
        if (!(ok = warp_acquired(there))) break;
        if (lane == 0) {
          __threadfence();
          red_release(&p.done[s.b]);
        }
      }
    }
  } else if (warp == 1) {
    // ================================================== MMA issuer
    if (lane == 0 && rank == 0) {
      int st = 0, buf = 0, before = p.layout[0];
      uint32_t phases_of = 0, tphase = 0;  // bit i: parity of stage i's next use
      bool ok = true, issued = false;
      for (int phase = 0; ok && phase < phases; ++phase) {
        Walk walk(p, phase, pair);
        const bool n_major = walk.kind == kUpdate;
        const int layout = p.layout[walk.kind], stages = ring_stages(layout);
        const uint32_t idesc = idesc_f16(256, p.bn[walk.kind], n_major),
                       stage_bytes = ring_stage(layout);
        if (layout != before) {
          before = layout;
          st = 0;
        }
        Segment s;
        while (ok && walk.next(p, s)) {
          if (!mbar_wait_bounded(smem_u32(&ctl->tempty[buf]), tphase ^ 1, abort_flag, &g_ns_status,
                                 p.timeout_ns, FP8Q_ERR_TIMEOUT)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(buf * kTile);
          for (int kb = s.kb0; kb < s.kb1; ++kb) {
            if (!mbar_wait_bounded(smem_u32(&ctl->full[st]), (phases_of >> st) & 1u, abort_flag,
                                   &g_ns_status, p.timeout_ns, FP8Q_ERR_TIMEOUT)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sl = ring + st * stage_bytes;
            const uint64_t ad = smem_desc_sw128(sl);
            const uint64_t bd = n_major ? smem_desc_sw128_mn(sl + kOpBytes, 8192)
                                        : smem_desc_sw128(sl + kOpBytes);
            const uint64_t bstep = n_major ? 128 : 2;  // 16 K: 16 rows of 128 bytes, or 32 bytes
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_pair(d, ad + 2 * k, bd + bstep * k, idesc,
                           kb != s.kb0 || k != 0 ? 1u : 0u);
            mma_commit_pair_multicast(smem_u32(&ctl->empty[st]), 0x3);
            issued = true;
            phases_of ^= 1u << st;
            if (++st == stages) st = 0;
          }
          if (!ok) break;
          mma_commit_pair_multicast(smem_u32(&ctl->tfull[buf]), 0x3);
          buf ^= 1;
          if (buf == 0) tphase ^= 1;
        }
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
    tmem_dealloc_pair(tmem_base, 512);
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

// Pairs that can run at once on the current device (at most kMaxPairs).
fp8q_status max_pairs(int &pairs) {
  static int known[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    if (cudaFuncSetAttribute(ns_steps_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem)) != cudaSuccess)
      return FP8Q_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.gridDim = dim3(2, 1, 1);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, ns_steps_kernel, &cfg) != cudaSuccess || n < 1)
      return FP8Q_ERR_UNSUPPORTED;
    known[dev] = n < kMaxPairs ? n : kMaxPairs;
  }
  pairs = known[dev];
  return FP8Q_OK;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Tile width and share of each phase kind, by an estimate of its time: rounds of
// tiles, each the longer of its MMAs and its epilogue, and the last epilogue.  A
// K block of a 256-row tile measured 0.34 us at 256 columns (tensor cores), 0.2
// at 128 and 0.14 at 64 (operand traffic); an epilogue about 1.5 us and 0.45 per 64
// columns; handing split tiles over 9 us (every pair's 256 KB of partial sums go
// through L2 at once).  With every SM reading operands at once (the Gram product of
// a 2048 x 7168 update, about 14 TB/s from L2) a 128-wide block takes 0.27, not 0.2:
// by that figure the estimate would be 33 us for its 128-wide tiles and 31 for an
// even split of 256-wide ones; which of the two is faster has not been measured.
struct Plan {
  int bn[3];
  int64_t tiles[3], per[3], pairs;
};
// A split saves at most one tile's MMAs, so it never pays for short sums (which
// then need no room for partial sums either).
bool may_split(int64_t kblocks) { return kblocks > 26; }
Plan plan_of(int64_t batch, int64_t p, int64_t q, int64_t pairs) {
  Plan r{};
  const int64_t row_tiles = (p + kTile - 1) / kTile;
  for (int k = 0; k < 3; ++k) {
    const int64_t kblocks = ((k == kGram ? q : p) + 63) / 64, cols = k == kUpdate ? q : p;
    double best = 0;
    for (int bn = kTile; bn >= (k == kUpdate ? 128 : 64); bn /= 2) {
      const int64_t n = (cols + bn - 1) / bn;
      int64_t tiles = row_tiles * n;
      if (k != kUpdate) tiles -= kTile / bn * (row_tiles * (row_tiles - 1) / 2);
      const int64_t all = tiles * batch, rounds = (all + pairs - 1) / pairs;
      const double block = bn == 256 ? 0.34 : bn == 128 ? 0.2 : 0.14;
      const double epi = 1.5 + 0.45 * (bn / 64);
      const double mma = block * static_cast<double>(kblocks);
      double t = static_cast<double>(rounds) * (mma > epi ? mma : epi) + epi;
      int64_t per = 0;
      const int64_t even = (all * kblocks + pairs - 1) / pairs;
      const double split = block * static_cast<double>(even) + epi + 9.0;
      if (bn == kTile && may_split(kblocks) && split < t) {
        t = split;
        per = even;
      }
      if (bn == kTile || t < best) {
        best = t;
        r.bn[k] = bn;
        r.tiles[k] = tiles;
        r.per[k] = per;
      }
    }
    int64_t busy = r.tiles[k] * batch;
    if (r.per[k] > 0) busy = (busy * kblocks + r.per[k] - 1) / r.per[k];
    if (busy > pairs) busy = pairs;
    if (busy > r.pairs) r.pairs = busy;
  }
  return r;
}

// Workspace: X (two copies), O_A, O_B as FP16 with pitches of a multiple of 8,
// d_A, d_B, the partial sums of squares and of split tiles, and the counters;
// every part starts at a multiple of 256 bytes.
struct Layout {
  int64_t p, q, ldx, lda, x0, x1, a, b, da, db, part, sync, split, bytes;
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
  l.sync = up(l.part + batch * kMaxParts * 4, 256);
  l.split = up(l.sync + static_cast<int64_t>(sizeof(Sync)) + 4 * batch, 256);
  l.bytes = l.split + (may_split((l.q + 63) / 64) ? kMaxPairs * kSlotFloats * 4 : 0);
  return l;
}

// Sizes are bounded so that every count of units (of the narrowest tiles) is an int.
bool shape_ok(int64_t batch, int64_t m, int64_t n) {
  if (batch < 0 || m < 0 || n < 0 || batch > 65535 || m > (1 << 20) || n > (1 << 20)) return false;
  const int64_t p = m < n ? m : n, q = m < n ? n : m;
  const int64_t units = batch * ((p + 255) / 256) * ((q + 63) / 64) * ((p + 63) / 64);
  return units < (1ll << 30);
}

template <typename In, bool kVec>
fp8q_status load_x(const In *g, int64_t ldg, int64_t bs, int64_t batch, int64_t m, int64_t n,
                   float eps, const Layout &l, uint8_t *ws, cudaStream_t s) {
  float *part = reinterpret_cast<float *>(ws + l.part);
  __half *x = reinterpret_cast<__half *>(ws + l.x0);
  const int64_t blocks = (m * ((n + kPieceOf<kVec> - 1) / kPieceOf<kVec>) + 7) / 8;
  const int parts = static_cast<int>(blocks < kMaxParts ? blocks : kMaxParts);
  const unsigned b = static_cast<unsigned>(batch);
  if (fp8q_status st = launch_dependent(ns_sumsq_kernel<In, kVec>, dim3(parts, b), dim3(256), 0, s, g, ldg,
                                 bs, m, n, part, reinterpret_cast<uint32_t *>(ws + l.sync),
                                 static_cast<int>(sizeof(Sync) / 4 + batch)))
    return st;
  if (m > n)
    return launch_dependent(ns_load_tall_kernel<In, kVec>,
                     dim3(static_cast<unsigned>((n + 63) / 64), static_cast<unsigned>((m + 63) / 64), b),
                     dim3(256), 0, s, g, ldg, bs, m, n, static_cast<const float *>(part), parts, eps,
                     x, l.ldx);
  return launch_dependent(ns_load_kernel<In, kVec>,
                   dim3(static_cast<unsigned>((n + 255) / 256), static_cast<unsigned>((m + 31) / 32), b),
                   dim3(256), 0, s, g, ldg, bs, m, n, static_cast<const float *>(part), parts, eps, x,
                   l.ldx);
}

template <typename In>
fp8q_status load_any(const void *g, int64_t ldg, int64_t bs, int64_t batch, int64_t m, int64_t n,
                     float eps, const Layout &l, uint8_t *ws, cudaStream_t s) {
  const In *in = static_cast<const In *>(g);
  constexpr int64_t V = kVecOf<In>;
  return aligned16(g) && ldg % V == 0 && bs % V == 0
             ? load_x<In, true>(in, ldg, bs, batch, m, n, eps, l, ws, s)
             : load_x<In, false>(in, ldg, bs, batch, m, n, eps, l, ws, s);
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
  if (!(eps >= 0.0f) || steps < 1 || steps > 1000) return FP8Q_ERR_INVALID;
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
  if (dev.max_smem_optin < static_cast<int>(kSmem)) return FP8Q_ERR_UNSUPPORTED;
  int pairs = 0;
  if (fp8q_status st = max_pairs(pairs)) return st;
  auto s = static_cast<cudaStream_t>(stream);
  auto *ws = static_cast<uint8_t *>(workspace);
  NsArgs v{};
  v.batch = static_cast<int>(batch);
  v.p = static_cast<int>(l.p);
  v.q = static_cast<int>(l.q);
  v.steps = steps;
  v.row_tiles = (v.p + kTile - 1) / kTile;
  v.kb_p = (v.p + 63) / 64;
  v.kb_q = (v.q + 63) / 64;
  const Plan plan = plan_of(batch, l.p, l.q, pairs);
  for (int k = 0; k < 3; ++k) {
    v.bn[k] = plan.bn[k];
    v.layout[k] = plan.bn[k];
    for (int j = 0; batch > 1 && j < 3; ++j)
      if (plan.bn[j] > v.layout[k]) v.layout[k] = plan.bn[j];
    v.tiles[k] = static_cast<int>(plan.tiles[k]);
    v.per[k] = static_cast<int>(plan.per[k]);
  }
  v.a = a;
  v.b = b;
  v.c = c;
  v.x[0] = reinterpret_cast<__half *>(ws + l.x0);
  v.x[1] = reinterpret_cast<__half *>(ws + l.x1);
  v.am = reinterpret_cast<__half *>(ws + l.a);
  v.bm = reinterpret_cast<__half *>(ws + l.b);
  v.ldx = l.ldx;
  v.lda = l.lda;
  v.da = reinterpret_cast<float *>(ws + l.da);
  v.db = reinterpret_cast<float *>(ws + l.db);
  v.partial = reinterpret_cast<float *>(ws + l.split);
  v.sync = reinterpret_cast<Sync *>(ws + l.sync);
  v.done = reinterpret_cast<uint32_t *>(v.sync + 1);
  v.out = out;
  v.ldo = ldo;
  v.out_stride = batch > 1 ? o_stride : 0;
  v.out_f32 = out_f32;
  v.tall = m > n;
  v.out_vec = !v.tall && !out_f32 && aligned16(out) && ldo % 8 == 0 && v.out_stride % 8 == 0;
  v.timeout_ns = wait_timeout_ns().load();
  Maps maps;
  for (int i = 0; i < 2; ++i)
    if (!make_tmap_f16(&maps.x[i], v.x[i], batch, l.p, l.q, l.ldx, 128) ||
        !make_tmap_f16(&maps.xr[i], v.x[i], batch, l.p, l.q, l.ldx, plan.bn[kGram] / 2) ||
        !make_tmap_f16(&maps.xn[i], v.x[i], batch, l.p, l.q, l.ldx, 64))
      return FP8Q_ERR_CUDA;
  if (!make_tmap_f16(&maps.a, v.am, batch, l.p, l.p, l.lda, 128) ||
      !make_tmap_f16(&maps.ar, v.am, batch, l.p, l.p, l.lda, plan.bn[kPoly] / 2) ||
      !make_tmap_f16(&maps.b, v.bm, batch, l.p, l.p, l.lda, 128))
    return FP8Q_ERR_CUDA;
  const int64_t bs = batch > 1 ? g_stride : 0;
  if (fp8q_status st = in_f32 ? load_any<float>(g, ldg, bs, batch, m, n, eps, l, ws, s)
                              : load_any<uint16_t>(g, ldg, bs, batch, m, n, eps, l, ws, s))
    return st;
  // the pairs wait for one another: a cooperative launch runs all of them at once
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_dependent
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * plan.pairs), 1, 1);
  return cudaLaunchKernelEx(&cfg, ns_steps_kernel, maps, v) == cudaSuccess ? FP8Q_OK
                                                                           : FP8Q_ERR_CUDA;
}
