// swiglu.cu -- the gated feed-forward block (SwiGLU) around the FP8 GEMMs:
// argument checks of the forward calls, the forward kernel for few tokens, and
// the backward pass down to the gradients of the two projections' outputs.
//
//   forward   g = X Wg^T, u = X Wu^T (per-128-K-group scales, FP32 sums),
//             h = silu(g) * u,  silu(g) = g s,  s = 1 / (1 + exp(-g))
//   backward  du = dh g s,  dg = dh u s (1 + g (1 - s))
//
// The forward pass for more than kFewTokens tokens runs on the tensor-core
// GEMMs of gemm.cu / gemm_mx.cu with the gated epilogue of fp8q_glu.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "fp8q.h"
#include "fp8q_glu.cuh"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"

namespace fp8q {

// Device status word of the few-token kernel (read by fp8q_sync_status).
__device__ int g_glu_status;

fp8q_status glu_status_take(cudaStream_t s) {
  int v = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_glu_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  if (v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_glu_status, &zero, sizeof(int)) != cudaSuccess) return FP8Q_ERR_CUDA;
  }
  return static_cast<fp8q_status>(v);
}

namespace {

__device__ __forceinline__ uint4 ld_stream_v4(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&p);
}

// One FP32 value into the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_f32(uint32_t local_addr, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(local_addr, rank)), "f"(v)
               : "memory");
}

// ------------------------------------------------------------------ few tokens
// With few tokens the block only streams its weights (2 F K bytes), and a
// 256-row tensor-core tile would leave most SMs idle: a CTA here takes 16
// columns of h (16 gate rows and 16 up rows of the weights) and every token,
// its warps split K by 128-wide groups, and a cluster of eight CTAs covers a
// 1x128 group of h, exchanging one max-abs per token through distributed
// shared memory.
//  - mma.sync m16n8k32 (E4M3, FP32 sums): rows 0-7 are eight gate rows, rows
//    8-15 the up rows of the same eight columns, so g and u of one (token,
//    column) land in the same thread; columns are eight tokens.  The tensor
//    cores are far from busy; the form only saves the decode and FMAs.
//  - Within a group the K order is free (the same for both operands): lane
//    4r + t loads bytes 16t and 64 + 16t of row r's 128, whole 64-byte pieces
//    of eight rows per instruction, and feeds the words to the MMAs in pairs.
//  - Each group's FP32 sums are scaled by sa * sb and added to FP32
//    accumulators; the warps' accumulators are summed in warp order.
constexpr int kFewWarps = 8;
constexpr int kFewTokens = 32;

struct FewArgs {
  const uint8_t *a;
  int64_t lda;
  const float *sa;
  int64_t ld_sa;
  const uint8_t *b;
  int64_t ldb;
  const float *sb;
  int64_t ld_sb;
  int M, num_kb;
  GluOut out;
};

__device__ __forceinline__ void mma_e4m3_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1,
                                                 uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A power-of-two scale, or, for any other value, the power of two of its
// exponent field with `bad` set (as the block-scaled MMA path treats it).
__device__ __forceinline__ float pow2_of(float s, bool &bad) {
  const uint32_t b = __float_as_uint(s);
  if (b == 0x00400000u) return s;  // 2^-127
  const uint32_t e = (b >> 23) & 0xFFu;
  if ((b & 0x807FFFFFu) == 0u && e != 0u && e != 0xFFu) return s;
  bad = true;
  if (e == 0u) return __uint_as_float(0x00400000u);
  return __uint_as_float((e < 0xFFu ? e : 0xFEu) << 23);
}

// NT: token blocks of eight (M <= 8 NT).
template <int NT, bool kPow2>
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kFewWarps * 32)
    glu_few_tokens_kernel(const FewArgs p) {
  constexpr int R = 2;  // blocks of eight columns of h per CTA
  __shared__ float red[kFewWarps][R * NT * 4][32];
  __shared__ float cl_amax[8][8 * NT];  // [CTA of the cluster][token]
  __shared__ int tok_amax[8 * NT];      // bits of this CTA's max-abs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane >> 2, t4 = lane & 3;
  const int F = p.out.F;
  const int c0 = static_cast<int>(blockIdx.x) * (8 * R);
  const int nb = c0 / 128, NB = F / 128;
  const float *sbg = p.sb + static_cast<int64_t>(nb) * p.ld_sb;
  const float *sbu = p.sb + static_cast<int64_t>(NB + nb) * p.ld_sb;
  if (threadIdx.x < 8 * NT) tok_amax[threadIdx.x] = 0;
  if (p.out.q) cluster_arrive_relaxed();

  const uint8_t *wg[R], *wu[R], *xp[NT];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    wg[r] = p.b + static_cast<int64_t>(c0 + 8 * r + r8) * p.ldb + 16 * t4;
    wu[r] = wg[r] + static_cast<int64_t>(F) * p.ldb;
  }
  bool tok_in[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    tok_in[n] = 8 * n + r8 < p.M;
    xp[n] = p.a + static_cast<int64_t>(tok_in[n] ? 8 * n + r8 : 0) * p.lda + 16 * t4;
  }
  float acc[R][NT][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.0f;
  bool bad = false;

#pragma unroll 2
  for (int kb = warp; kb < p.num_kb; kb += kFewWarps) {
    const int64_t off = static_cast<int64_t>(kb) * 128;
    uint4 g[R][2], u[R][2], x[NT][2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        g[r][i] = ld_stream_v4(wg[r] + off + 64 * i);
        u[r][i] = ld_stream_v4(wu[r] + off + 64 * i);
      }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[n][i] = tok_in[n] ? __ldg(reinterpret_cast<const uint4 *>(xp[n] + off + 64 * i))
                            : make_uint4(0, 0, 0, 0);
    float s_g = __ldg(sbg + kb), s_u = __ldg(sbu + kb);
    if (kPow2) {
      s_g = pow2_of(s_g, bad);
      s_u = pow2_of(s_u, bad);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      // scales of this thread's two tokens, 8n + 2t and + 1
      float s_x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = 8 * n + 2 * t4 + i;
        s_x[i] = m < p.M ? __ldg(p.sa + static_cast<int64_t>(kb) * p.ld_sa + m) : 0.0f;
        if (kPow2 && m < p.M) s_x[i] = pow2_of(s_x[i], bad);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma_e4m3_16x8x32(d, g[r][i].x, u[r][i].x, g[r][i].y, u[r][i].y, x[n][i].x, x[n][i].y);
          mma_e4m3_16x8x32(d, g[r][i].z, u[r][i].z, g[r][i].w, u[r][i].w, x[n][i].z, x[n][i].w);
        }
        acc[r][n][0] = fmaf(d[0], s_x[0] * s_g, acc[r][n][0]);
        acc[r][n][1] = fmaf(d[1], s_x[1] * s_g, acc[r][n][1]);
        acc[r][n][2] = fmaf(d[2], s_x[0] * s_u, acc[r][n][2]);
        acc[r][n][3] = fmaf(d[3], s_x[1] * s_u, acc[r][n][3]);
      }
    }
  }
  if (kPow2 && bad) atomicCAS(&g_glu_status, 0, FP8Q_ERR_INVALID);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][(r * NT + n) * 4 + i][lane] = acc[r][n][i];
  __syncthreads();

  // (token, column) values: 128 NT of them, item = ((r NT + n) 2 + i) 32 + lane
  constexpr int kItems = R * NT * 2 * 32;
  constexpr int kPer = (kItems + kFewWarps * 32 - 1) / (kFewWarps * 32);
  float h[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int item = static_cast<int>(threadIdx.x) + k * kFewWarps * 32;
    h[k] = 0.0f;
    if (item < kItems) {
      const int l = item & 31, i = (item >> 5) & 1, rn = item >> 6;
      const int m = 8 * (rn % NT) + 2 * (l & 3) + i, c = c0 + 8 * (rn / NT) + (l >> 2);
      float g = 0.0f, u = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        g += red[w][rn * 4 + i][l];
        u += red[w][rn * 4 + 2 + i][l];
      }
      if (m < p.M) {
        h[k] = silu(g) * u;
        if (p.out.gu) {
          uint16_t *row = static_cast<uint16_t *>(p.out.gu) + static_cast<int64_t>(m) * p.out.ld_gu;
          row[c] = bf16_bits(g);
          row[F + c] = bf16_bits(u);
        }
        if (p.out.h)
          static_cast<uint16_t *>(p.out.h)[static_cast<int64_t>(m) * p.out.ldh + c] =
              bf16_bits(h[k]);
        // magnitudes order as their bits do
        if (p.out.q) atomicMax(&tok_amax[m], __float_as_int(fabsf(h[k])));
      }
    }
  }
  if (!p.out.q) return;  // the same in every CTA of the cluster
  __syncthreads();
  cluster_wait();  // every CTA of the cluster has started
  const uint32_t rank = cluster_ctarank();
  for (int i = threadIdx.x; i < 8 * 8 * NT; i += kFewWarps * 32)
    st_cluster_f32(smem_u32(&cl_amax[rank][i >> 3]), static_cast<uint32_t>(i & 7),
                   __int_as_float(tok_amax[i >> 3]));
  cluster_sync_all();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int item = static_cast<int>(threadIdx.x) + k * kFewWarps * 32;
    if (item >= kItems) continue;
    const int l = item & 31, i = (item >> 5) & 1, rn = item >> 6;
    const int mt = 8 * (rn % NT) + 2 * (l & 3) + i, c = 8 * (rn / NT) + (l >> 2);
    if (mt >= p.M) continue;
    float amax = cl_amax[0][mt];
#pragma unroll
    for (int j = 1; j < 8; ++j) amax = fmaxf(amax, cl_amax[j][mt]);
    float sc, inv;
    group_scale(amax, p.out.pow2 != 0, sc, inv);
    p.out.q[static_cast<int64_t>(mt) * p.out.ldq + c0 + c] =
        static_cast<uint8_t>(pack_e4m3x2(__fmul_rn(h[k], inv), 0.0f) & 0xFFu);
    if (rank == 0 && c == 0) p.out.s[static_cast<int64_t>(nb) * p.out.ld_s + mt] = sc;
  }
}

template <bool kPow2>
fp8q_status launch_few(const GluIn &in, const GluOut &out, cudaStream_t s) {
  FewArgs a{};
  a.a = static_cast<const uint8_t *>(in.a);
  a.lda = in.lda;
  a.sa = in.sa;
  a.ld_sa = in.ld_sa;
  a.b = static_cast<const uint8_t *>(in.b);
  a.ldb = in.ldb;
  a.sb = in.sb;
  a.ld_sb = in.ld_sb;
  a.M = static_cast<int>(in.M);
  a.num_kb = static_cast<int>(in.K / 128);
  a.out = out;
  const dim3 grid(static_cast<unsigned>(in.F / 16)), block(kFewWarps * 32);
  switch ((in.M + 7) / 8) {
    case 1: return launch_on(glu_few_tokens_kernel<1, kPow2>, grid, block, 0, s, a);
    case 2: return launch_on(glu_few_tokens_kernel<2, kPow2>, grid, block, 0, s, a);
    case 3: return launch_on(glu_few_tokens_kernel<3, kPow2>, grid, block, 0, s, a);
    default: return launch_on(glu_few_tokens_kernel<4, kPow2>, grid, block, 0, s, a);
  }
}

bool valid_mode(int m) { return m == FP8Q_SCALE_FP32 || m == FP8Q_SCALE_POW2; }

fp8q_status glu_entry(const GluIn &in, const GluOut &o, int scale_mode, bool pow2, bool grouped,
                      void *stream) {
  if (!valid_mode(scale_mode)) return FP8Q_ERR_INVALID;
  if (grouped && (in.G < 1 || in.G > 1024)) return FP8Q_ERR_SHAPE;
  if (in.M < 0 || in.F < 0 || in.K < 0 || in.K % 128 != 0 || in.F % 128 != 0)
    return FP8Q_ERR_SHAPE;
  if (in.M >= (1ll << 31) - 256 || in.K >= (1ll << 31) || in.F >= (1ll << 30) ||
      2 * in.F * in.G >= (1ll << 31) - 256)
    return FP8Q_ERR_SHAPE;
  if (in.ld_sa < in.M || (o.h && o.ldh < in.F) || (o.gu && o.ld_gu < 2 * in.F) ||
      (o.q && (o.ldq < in.F || o.ld_s < in.M)))
    return FP8Q_ERR_SHAPE;
  if (in.M == 0 || in.F == 0) return FP8Q_OK;
  if (!o.h && !o.gu && !o.q) return FP8Q_ERR_INVALID;
  if ((o.q == nullptr) != (o.s == nullptr)) return FP8Q_ERR_INVALID;
  if (grouped && !in.offs) return FP8Q_ERR_INVALID;
  if (in.K > 0) {
    if (in.lda < in.K || in.ldb < in.K || (!grouped && in.ld_sb < in.K / 128))
      return FP8Q_ERR_SHAPE;
    if (!in.a || !in.b || !in.sa || !in.sb) return FP8Q_ERR_INVALID;
    if (!aligned16(in.a) || !aligned16(in.b) || in.lda % 16 || in.ldb % 16 || !aligned4(in.sa) ||
        !aligned4(in.sb))
      return FP8Q_ERR_ALIGN;
  }
  if ((o.h && (!aligned16(o.h) || o.ldh % 8)) || (o.gu && (!aligned16(o.gu) || o.ld_gu % 8)) ||
      (o.q && (!aligned16(o.q) || o.ldq % 16 || !aligned4(o.s))) ||
      (grouped && !aligned4(in.offs)))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;
  auto s = static_cast<cudaStream_t>(stream);
  if (!grouped && in.M <= kFewTokens)
    return pow2 ? launch_few<true>(in, o, s) : launch_few<false>(in, o, s);
  return pow2 && in.K > 0 ? gemm_mx_glu(in, o, s) : gemm_glu(in, o, s);
}

GluIn glu_in(const void *a, int64_t lda, const float *sa, int64_t ld_sa, const void *b,
             int64_t ldb, const float *sb, int64_t ld_sb, const int32_t *offs, int G, int64_t M,
             int64_t F, int64_t K) {
  GluIn in{};
  in.a = a;
  in.lda = lda;
  in.sa = sa;
  in.ld_sa = ld_sa;
  in.b = b;
  in.ldb = ldb;
  in.sb = sb;
  in.ld_sb = ld_sb;
  in.offs = offs;
  in.G = G;
  in.M = M;
  in.F = F;
  in.K = K;
  return in;
}

GluOut glu_out(void *h, int64_t ldh, void *gu, int64_t ld_gu, void *q, int64_t ldq, float *s,
               int64_t ld_s, int scale_mode, int64_t F) {
  GluOut o{};
  o.h = h;
  o.ldh = ldh;
  o.gu = gu;
  o.ld_gu = ld_gu;
  o.q = static_cast<uint8_t *>(q);
  o.ldq = ldq;
  o.s = s;
  o.ld_s = ld_s;
  o.pow2 = scale_mode == FP8Q_SCALE_POW2;
  o.F = static_cast<int>(F);
  return o;
}

// ------------------------------------------------------------------ backward
// Memory bound: dh, g and u are read once (6 bytes per element of h) and every
// requested result is written from the same registers.
//  - A cluster of kCl CTAs covers a tile of 128 tokens x 128 columns of h, each
//    CTA 128 / kCl columns; a thread holds 4 tokens x 8 columns of dg, du and h
//    (16-byte loads, whole token rows of a CTA's columns per instruction).
//  - 1x128 max-abs (dg and du, per token): shuffles over a token's threads,
//    then one value per token and CTA to every CTA of the cluster through
//    distributed shared memory.  128x1 max-abs (dg, du, h, per column):
//    shuffles over a warp's tokens, then an atomic max on the values' bits in
//    shared memory (magnitudes order as their bits do; the result does not
//    depend on the order).
//  - One thread per group turns a max-abs into its scale, so that the two IEEE
//    divisions are done once per group.
//  - The transposed codes pass through shared memory: a thread's 4 tokens of a
//    column are one 32-bit word; word w of column row r sits at w ^ f(r), which
//    spreads a warp's words over all banks on the way in and keeps 16-byte
//    units whole on the way out, where eight lanes write a column's 128 bytes.
constexpr int kCl = 2;
constexpr int kChan = 128 / kCl;               // columns of h per CTA
constexpr int kBwdThreads = 4 * kChan;         // 32 token quads x kChan / 8 column octets
constexpr int kLW = kChan / 8;                 // lanes across a token row
constexpr int kRowsPerWarp = 32 / kLW;         // token quads per warp
static_assert(kCl == 2, "the swizzle below keeps 16-byte units whole for two CTAs per tile");

struct BwdArgs {
  const uint16_t *dh;
  int64_t ld_dh;
  const uint16_t *gu;
  int64_t ld_gu;
  uint16_t *d;
  int64_t ld_d;
  uint8_t *q;
  int64_t ldq;
  float *s;
  int64_t ld_s;
  uint8_t *qT;
  int64_t ldqT;
  float *sT;
  int64_t ld_sT;
  uint8_t *hT;
  int64_t ld_hT;
  float *shT;
  int64_t ld_shT;
  int64_t T, F;
  int pow2;
};

__device__ __forceinline__ uint32_t xpose_word(uint32_t r, uint32_t w) {
  return r * 32u + (w ^ (static_cast<uint32_t>(kRowsPerWarp) * ((r >> 3) % kLW)));
}

template <bool kRows, bool kCols, bool kH>
__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kBwdThreads, 512 / kBwdThreads)
    swiglu_bwd_kernel(const BwdArgs p) {
  constexpr int kColArrays = (kCols ? 2 : 0) + (kH ? 1 : 0);  // dg, du | h
  constexpr int kH0 = kCols ? 2 : 0;                          // h's place among them
  __shared__ float row_amax[kRows ? kCl : 1][2][128];         // [CTA of the cluster][dg, du][token]
  __shared__ float row_inv[2][128];
  __shared__ __align__(16) uint32_t col_bits[3][kChan];
  __shared__ __align__(16) float col_inv[3][kChan];
  __shared__ __align__(16) uint32_t xpose[kColArrays > 0 ? kColArrays : 1][kColArrays > 0 ? kChan * 32 : 4];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l8 = lane % kLW;                               // column octet
  const int quad = warp * kRowsPerWarp + lane / kLW;       // token quad
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * 128;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kChan;
  const int64_t c = c0 + 8 * l8;
  const uint32_t rank = cluster_ctarank();
  if (kRows) cluster_arrive_relaxed();
  if (kColArrays > 0) {
    for (int i = tid; i < kColArrays * kChan; i += kBwdThreads) (&col_bits[0][0])[i] = 0u;
    __syncthreads();
  }

  uint4 rd[4], rg[4], ru[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + 4 * quad + i;
    rd[i] = rg[i] = ru[i] = make_uint4(0, 0, 0, 0);
    if (t < p.T) {
      rd[i] = ld_stream_v4(p.dh + t * p.ld_dh + c);
      rg[i] = ld_stream_v4(p.gu + t * p.ld_gu + c);
      ru[i] = ld_stream_v4(p.gu + t * p.ld_gu + p.F + c);
    }
  }
  float dg[4][8], du[4][8], h[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t wd[4] = {rd[i].x, rd[i].y, rd[i].z, rd[i].w};
    const uint32_t wg[4] = {rg[i].x, rg[i].y, rg[i].z, rg[i].w};
    const uint32_t wu[4] = {ru[i].x, ru[i].y, ru[i].z, ru[i].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = j & 1 ? bf16_hi(wd[j / 2]) : bf16_lo(wd[j / 2]);
      const float g = j & 1 ? bf16_hi(wg[j / 2]) : bf16_lo(wg[j / 2]);
      const float u = j & 1 ? bf16_hi(wu[j / 2]) : bf16_lo(wu[j / 2]);
      const float sg = __fdividef(1.0f, 1.0f + __expf(-g));
      const float sl = g * sg;
      du[i][j] = y * sl;
      dg[i][j] = y * u * fmaf(sl, 1.0f - sg, sg);
      if (kH) h[i][j] = sl * u;
    }
    if (p.d) {
      const int64_t t = t0 + 4 * quad + i;
      if (t < p.T) {
        uint16_t *dst = p.d + t * p.ld_d + c;
        *reinterpret_cast<uint4 *>(dst) =
            make_uint4(bf16x2_bits(dg[i][0], dg[i][1]), bf16x2_bits(dg[i][2], dg[i][3]),
                       bf16x2_bits(dg[i][4], dg[i][5]), bf16x2_bits(dg[i][6], dg[i][7]));
        *reinterpret_cast<uint4 *>(dst + p.F) =
            make_uint4(bf16x2_bits(du[i][0], du[i][1]), bf16x2_bits(du[i][2], du[i][3]),
                       bf16x2_bits(du[i][4], du[i][5]), bf16x2_bits(du[i][6], du[i][7]));
      }
    }
  }
  if (!kRows && kColArrays == 0) return;

  // ---- max-abs of the groups
  if (kRows) {
    cluster_wait();  // every CTA of the cluster has started
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a = fmaxf(a, fabsf(dg[i][j]));
        b = fmaxf(b, fabsf(du[i][j]));
      }
#pragma unroll
      for (int o = kLW / 2; o > 0; o >>= 1) {
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
      }
      if (l8 < kCl) {  // lane l8 of a token serves CTA l8
        st_cluster_f32(smem_u32(&row_amax[rank][0][4 * quad + i]), static_cast<uint32_t>(l8), a);
        st_cluster_f32(smem_u32(&row_amax[rank][1][4 * quad + i]), static_cast<uint32_t>(l8), b);
      }
    }
  }
  if (kColArrays > 0) {
#pragma unroll
    for (int k = 0; k < kColArrays; ++k) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a = fmaxf(a, fabsf(kH && k == kH0 ? h[i][j] : k == 0 ? dg[i][j] : du[i][j]));
#pragma unroll
        for (int o = kLW; o < 32; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        // the warp's token quads share the atomics: quad (j mod kRowsPerWarp)
        if (lane / kLW == j % kRowsPerWarp)
          atomicMax(&col_bits[k][8 * l8 + j], __float_as_uint(a));
      }
    }
  }
  if (kRows) cluster_sync_all();
  else __syncthreads();

  // ---- scales, one group per thread
  if (kRows) {
    for (int i = tid; i < 256; i += kBwdThreads) {
      const int k = i >> 7, t = i & 127;
      float a = row_amax[0][k][t];
#pragma unroll
      for (int j = 1; j < kCl; ++j) a = fmaxf(a, row_amax[j][k][t]);
      float sc, inv;
      group_scale(a, p.pow2 != 0, sc, inv);
      row_inv[k][t] = inv;
      if (rank == 0 && t0 + t < p.T)
        p.s[(k * (p.F / 128) + c0 / 128) * p.ld_s + t0 + t] = sc;
    }
  }
  if (kColArrays > 0) {
    for (int i = tid; i < kColArrays * kChan; i += kBwdThreads) {
      const int k = i / kChan, cc = i % kChan;
      float sc, inv;
      group_scale(__uint_as_float(col_bits[k][cc]), p.pow2 != 0, sc, inv);
      col_inv[k][cc] = inv;
      if (kH && k == kH0) p.shT[(t0 / 128) * p.ld_shT + c0 + cc] = sc;
      else p.sT[(t0 / 128) * p.ld_sT + k * p.F + c0 + cc] = sc;
    }
  }
  __syncthreads();

  // ---- codes
  if (kRows) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tl = 4 * quad + i;
      if (t0 + tl < p.T) {
        uint8_t *dst = p.q + (t0 + tl) * p.ldq + c;
        const float a = row_inv[0][tl], b = row_inv[1][tl];
        const uint64_t a2 = pack_f32x2(a, a), b2 = pack_f32x2(b, b);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 x = unpack_f32x2(fmul2(pack_f32x2(dg[i][4 * e], dg[i][4 * e + 1]), a2));
          const float2 y = unpack_f32x2(fmul2(pack_f32x2(dg[i][4 * e + 2], dg[i][4 * e + 3]), a2));
          w[e] = pack_e4m3x4(x.x, x.y, y.x, y.y);
          const float2 v = unpack_f32x2(fmul2(pack_f32x2(du[i][4 * e], du[i][4 * e + 1]), b2));
          const float2 z = unpack_f32x2(fmul2(pack_f32x2(du[i][4 * e + 2], du[i][4 * e + 3]), b2));
          w[2 + e] = pack_e4m3x4(v.x, v.y, z.x, z.y);
        }
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(dst + p.F) = make_uint2(w[2], w[3]);
      }
    }
  }
  if (kColArrays > 0) {
#pragma unroll
    for (int k = 0; k < kColArrays; ++k) {
      float inv[8];
      *reinterpret_cast<float4 *>(&inv[0]) = *reinterpret_cast<const float4 *>(&col_inv[k][8 * l8]);
      *reinterpret_cast<float4 *>(&inv[4]) =
          *reinterpret_cast<const float4 *>(&col_inv[k][8 * l8 + 4]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = kH && k == kH0 ? h[i][j] : k == 0 ? dg[i][j] : du[i][j];
        const uint64_t i2 = pack_f32x2(inv[j], inv[j]);
        const float2 x = unpack_f32x2(fmul2(pack_f32x2(v[0], v[1]), i2));
        const float2 y = unpack_f32x2(fmul2(pack_f32x2(v[2], v[3]), i2));
        xpose[k][xpose_word(8 * l8 + j, quad)] = pack_e4m3x4(x.x, x.y, y.x, y.y);
      }
    }
    __syncthreads();
    // eight lanes write the 128 tokens of a column
    for (int i = tid; i < kColArrays * kChan * 8; i += kBwdThreads) {
      const int k = i / (kChan * 8), r = (i >> 3) % kChan, ch = i & 7;
      const uint4 v = *reinterpret_cast<const uint4 *>(&xpose[k][xpose_word(r, 4 * ch)]);
      uint8_t *dst = kH && k == kH0
                         ? p.hT + (c0 + r) * p.ld_hT + t0 + 16 * ch
                         : p.qT + (k * p.F + c0 + r) * p.ldqT + t0 + 16 * ch;
      *reinterpret_cast<uint4 *>(dst) = v;
    }
  }
}

template <bool kRows, bool kCols>
fp8q_status launch_bwd(const BwdArgs &a, dim3 grid, cudaStream_t s) {
  return a.hT ? launch_on(swiglu_bwd_kernel<kRows, kCols, true>, grid, dim3(kBwdThreads), 0, s, a)
              : launch_on(swiglu_bwd_kernel<kRows, kCols, false>, grid, dim3(kBwdThreads), 0, s, a);
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_gemm_swiglu(const void *a, int64_t lda, const float *sa, int64_t ld_sa,
                                        const void *b, int64_t ldb, const float *sb, int64_t ld_sb,
                                        void *h, int64_t ldh, void *gu, int64_t ld_gu, void *q,
                                        int64_t ldq, float *s, int64_t ld_s, int scale_mode,
                                        int64_t M, int64_t F, int64_t K, void *stream) {
  return glu_entry(glu_in(a, lda, sa, ld_sa, b, ldb, sb, ld_sb, nullptr, 1, M, F, K),
                   glu_out(h, ldh, gu, ld_gu, q, ldq, s, ld_s, scale_mode, F), scale_mode, false,
                   false, stream);
}

extern "C" fp8q_status fp8q_gemm_swiglu_pow2(const void *a, int64_t lda, const float *sa,
                                             int64_t ld_sa, const void *b, int64_t ldb,
                                             const float *sb, int64_t ld_sb, void *h, int64_t ldh,
                                             void *gu, int64_t ld_gu, void *q, int64_t ldq,
                                             float *s, int64_t ld_s, int scale_mode, int64_t M,
                                             int64_t F, int64_t K, void *stream) {
  return glu_entry(glu_in(a, lda, sa, ld_sa, b, ldb, sb, ld_sb, nullptr, 1, M, F, K),
                   glu_out(h, ldh, gu, ld_gu, q, ldq, s, ld_s, scale_mode, F), scale_mode, true,
                   false, stream);
}

extern "C" fp8q_status fp8q_grouped_gemm_swiglu(const void *a, int64_t lda, const float *sa,
                                                int64_t ld_sa, const void *b, int64_t ldb,
                                                const float *sb, const int32_t *offs, int G,
                                                void *h, int64_t ldh, void *gu, int64_t ld_gu,
                                                void *q, int64_t ldq, float *s, int64_t ld_s,
                                                int scale_mode, int64_t M, int64_t F, int64_t K,
                                                void *stream) {
  return glu_entry(glu_in(a, lda, sa, ld_sa, b, ldb, sb, K / 128, offs, G, M, F, K),
                   glu_out(h, ldh, gu, ld_gu, q, ldq, s, ld_s, scale_mode, F), scale_mode, false,
                   true, stream);
}

extern "C" fp8q_status fp8q_grouped_gemm_swiglu_pow2(
    const void *a, int64_t lda, const float *sa, int64_t ld_sa, const void *b, int64_t ldb,
    const float *sb, const int32_t *offs, int G, void *h, int64_t ldh, void *gu, int64_t ld_gu,
    void *q, int64_t ldq, float *s, int64_t ld_s, int scale_mode, int64_t M, int64_t F, int64_t K,
    void *stream) {
  return glu_entry(glu_in(a, lda, sa, ld_sa, b, ldb, sb, K / 128, offs, G, M, F, K),
                   glu_out(h, ldh, gu, ld_gu, q, ldq, s, ld_s, scale_mode, F), scale_mode, true,
                   true, stream);
}

extern "C" fp8q_status fp8q_swiglu_bwd(const void *dh, int64_t ld_dh, const void *gu,
                                       int64_t ld_gu, void *d, int64_t ld_d, void *q, int64_t ldq,
                                       float *s, int64_t ld_s, void *qT, int64_t ldqT, float *sT,
                                       int64_t ld_sT, void *hT, int64_t ld_hT, float *shT,
                                       int64_t ld_shT, int64_t T, int64_t F, int scale_mode,
                                       void *stream) {
  if (!valid_mode(scale_mode)) return FP8Q_ERR_INVALID;
  if (T < 0 || F < 0 || F % 128 != 0 || F > (1ll << 30) || T > 65535ll * 128) return FP8Q_ERR_SHAPE;
  if ((qT || hT) && T % 128 != 0) return FP8Q_ERR_SHAPE;
  if (ld_dh < F || ld_gu < 2 * F || (d && ld_d < 2 * F) || (q && (ldq < 2 * F || ld_s < T)) ||
      (qT && (ldqT < T || ld_sT < 2 * F)) || (hT && (ld_hT < T || ld_shT < F)))
    return FP8Q_ERR_SHAPE;
  if (T == 0 || F == 0) return FP8Q_OK;
  if (!dh || !gu || (!d && !q && !qT && !hT)) return FP8Q_ERR_INVALID;
  if (!q != !s || !qT != !sT || !hT != !shT) return FP8Q_ERR_INVALID;
  if (!aligned16(dh) || !aligned16(gu) || ld_dh % 8 || ld_gu % 8 ||
      (d && (!aligned16(d) || ld_d % 8)) || (q && (!aligned16(q) || ldq % 16 || !aligned4(s))) ||
      (qT && (!aligned16(qT) || ldqT % 16 || !aligned4(sT))) ||
      (hT && (!aligned16(hT) || ld_hT % 16 || !aligned4(shT))))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;
  BwdArgs a{};
  a.dh = static_cast<const uint16_t *>(dh);
  a.ld_dh = ld_dh;
  a.gu = static_cast<const uint16_t *>(gu);
  a.ld_gu = ld_gu;
  a.d = static_cast<uint16_t *>(d);
  a.ld_d = ld_d;
  a.q = static_cast<uint8_t *>(q);
  a.ldq = ldq;
  a.s = s;
  a.ld_s = ld_s;
  a.qT = static_cast<uint8_t *>(qT);
  a.ldqT = ldqT;
  a.sT = sT;
  a.ld_sT = ld_sT;
  a.hT = static_cast<uint8_t *>(hT);
  a.ld_hT = ld_hT;
  a.shT = shT;
  a.ld_shT = ld_shT;
  a.T = T;
  a.F = F;
  a.pow2 = scale_mode == FP8Q_SCALE_POW2;
  const dim3 grid(static_cast<unsigned>(F / kChan), static_cast<unsigned>((T + 127) / 128));
  auto st = static_cast<cudaStream_t>(stream);
  if (q) return qT ? launch_bwd<true, true>(a, grid, st) : launch_bwd<true, false>(a, grid, st);
  return qT ? launch_bwd<false, true>(a, grid, st) : launch_bwd<false, false>(a, grid, st);
}
