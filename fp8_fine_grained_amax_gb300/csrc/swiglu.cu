// swiglu.cu -- the gated feed-forward block (SwiGLU) around the FP8 GEMMs:
// argument checks of the forward calls, the forward kernel for few tokens, and
// the backward pass down to the gradients of the two projections' outputs.
//
//   forward   g = X Wg^T, u = X Wu^T (per-128-K-group scales, FP32 sums),
//             h = silu(g) * u,  silu(g) = g s,  s = 1 / (1 + exp(-g))
//   backward  du = dh g s,  dg = dh u s (1 + g (1 - s))
//
// Larger forward passes (few_tokens() below has the rule) and all of experts run
// on the tensor-core GEMMs of gemm.cu / gemm_mx.cu with the gated epilogue of
// fp8q_glu.cuh.
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

int *glu_status_word() {
  void *p = nullptr;
  return cudaGetSymbolAddress(&p, g_glu_status) == cudaSuccess ? static_cast<int *>(p) : nullptr;
}

namespace {

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t *>(&b);
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&p);
}

// Wait for a phase for at most 1 s regardless of any abort (own copies only).
__device__ __forceinline__ void mbar_wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > 1000000000ull) return;
}

// One FP32 value into the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster_f32(uint32_t local_addr, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa_shared(local_addr, rank)), "f"(v)
               : "memory");
}

// ------------------------------------------------------------------ few tokens
// With few tokens the block only streams its weights (2 F K bytes), and the
// 256-row tiles of the GEMMs would leave most SMs idle.  Here the weights are
// the MMA's M side and the tokens its N side: a CTA takes 64 columns of h (64
// gate rows and the 64 up rows of the same columns: one 128-row operand), N
// tokens, and one of S parts of the K-groups; a cluster of 2 S CTAs covers the
// 1x128 group of h (two column halves).  S is the most, up to four, that keeps
// every CTA resident at once (two per SM): all of them then stream until the
// end, where a second wave would leave SMs idle.
//   warp 0     TMA producer: weights and tokens per K-group into rings of 180,
//              160 or 144 KB per SM (two CTAs; 16, 32, 64 tokens; 160, 128 or 96
//              KB of it weights), so much on its way being what streaming at the
//              memory's rate needs
//   warp 1     MMA issuer: per K-group 4 x tcgen05.mma (M = 128, N tokens,
//              K = 32) into one of four TMEM buffers
//   warps 2-5  fold: each thread one weight row, acc += P * sa * sb in FP32,
//              the tokens' scales broadcast through shared memory
// Then the K parts are summed: each CTA sends its sums of the S-th part of the
// tokens to the CTA that finishes them (distributed shared memory, every sum
// has its own place, added in K order), which gates them; for the codes the two
// column halves of a group exchange one max-abs per token.
constexpr int kFewThreads = 192;
constexpr int kFewBufs = 4;        // TMEM buffers

template <int N, int S>
struct Few {
  static constexpr uint32_t kWBytes = 128 * 128, kXBytes = N * 128;
  // ring depth: what two CTAs per SM leave room for (three shallower ones
  // measured slower: 24 tokens of 7168 x 7168 28.6 us, against 24.5)
  static constexpr int kStages = N == 16 ? 5 : N == 32 ? 4 : 3;
  static constexpr int kPerSm = 2;
  static constexpr int kShare = N / S;  // tokens finished by a CTA
  static constexpr uint32_t kRecv = S * kShare * 128 * 4;
  static constexpr uint32_t kCols = kFewBufs * N;
  static constexpr size_t kSmem = 1024 + kStages * (kWBytes + kXBytes) + kRecv;
  static_assert(kPerSm * (kSmem + 4096) <= 227 * 1024, "shared memory");
  static_assert(kPerSm * kCols <= 512, "tensor memory");
};

struct FewArgs {
  const float *sa;
  int64_t ld_sa;
  const float *sb;
  int64_t ld_sb;
  int M, num_kb;
  GluOut out;
  uint64_t timeout_ns;
};

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

template <int N, int S, bool kPow2>
__global__ void __cluster_dims__(2 * S, 1, 1)
    __launch_bounds__(kFewThreads, Few<N, S>::kPerSm)
        glu_few_tokens_kernel(const __grid_constant__ CUtensorMap tmW,
                              const __grid_constant__ CUtensorMap tmX, const FewArgs p) {
  using C = Few<N, S>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], tfull[kFewBufs], tempty[kFewBufs], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(16) float s_sa[4][2][N];          // per fold warp, double-buffered
  __shared__ float s_amax[2][C::kShare];               // [column half][token]
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sW = smem_u32(smem), sX = sW + C::kStages * C::kWBytes;
  float *recv = reinterpret_cast<float *>(smem + C::kStages * (C::kWBytes + C::kXBytes));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_flag = &s_abort;
  const int rank = static_cast<int>(cluster_ctarank());
  const int half = rank / S, part = rank % S;  // column half, K part
  const int group = static_cast<int>(blockIdx.x) / (2 * S);
  const int F = p.out.F, c0 = group * 128 + half * 64;   // first column of h
  const int m0 = static_cast<int>(blockIdx.y) * N;       // first token
  const int per = (p.num_kb + S - 1) / S;
  const int kb0 = min(part * per, p.num_kb), kb1 = min(kb0 + per, p.num_kb);

  cluster_arrive_relaxed();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < kFewBufs; ++i) {
      mbar_init(smem_u32(&tfull[i]), 1);
      mbar_init(smem_u32(&tempty[i]), 4);
    }
    mbar_init(smem_u32(&drain), 1);
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), C::kCols);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  wait_for_previous_kernel();
  let_next_kernel_start();

  if (warp == 0) {
    if (lane == 0) {
      uint32_t armed = 0, armed_phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int st = (kb - kb0) % C::kStages;
        const uint32_t phase = static_cast<uint32_t>((kb - kb0) / C::kStages) & 1u;
        ok = mbar_wait_bounded(smem_u32(&empty[st]), phase ^ 1, abort_flag, &g_glu_status,
                               p.timeout_ns, FP8Q_ERR_TIMEOUT);
        if (!ok) break;
        const uint32_t fb = smem_u32(&full[st]);
        mbar_arrive_expect_tx(fb, C::kWBytes + C::kXBytes);
        tma_load_2d(sW + st * C::kWBytes, &tmW, fb, kb * 128, c0);
        tma_load_2d(sW + st * C::kWBytes + C::kWBytes / 2, &tmW, fb, kb * 128, F + c0);
        tma_load_2d(sX + st * C::kXBytes, &tmX, fb, kb * 128, m0);
        armed |= 1u << st;
        armed_phase = (armed_phase & ~(1u << st)) | (phase << st);
      }
      if (!ok)  // copies in flight land before the CTA's shared memory goes
        for (int i = 0; i < C::kStages; ++i)
          if (armed & (1u << i)) mbar_wait_drain(smem_u32(&full[i]), (armed_phase >> i) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true, issued = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int i = kb - kb0, st = i % C::kStages, buf = i % kFewBufs;
        ok = mbar_wait_bounded(smem_u32(&tempty[buf]),
                               (static_cast<uint32_t>(i / kFewBufs) & 1u) ^ 1u, abort_flag,
                               &g_glu_status, p.timeout_ns, FP8Q_ERR_TIMEOUT) &&
             mbar_wait_bounded(smem_u32(&full[st]), static_cast<uint32_t>(i / C::kStages) & 1u,
                               abort_flag, &g_glu_status, p.timeout_ns, FP8Q_ERR_TIMEOUT);
        if (!ok) break;
        tc_fence_after();
        const uint64_t wd = smem_desc_sw128(sW + st * C::kWBytes);
        const uint64_t xd = smem_desc_sw128(sX + st * C::kXBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8f6f4(tmem + buf * N, wd + 2 * k, xd + 2 * k, idesc_e4m3_f32(128, N),
                     k > 0 ? 1u : 0u);
        mma_commit(smem_u32(&empty[st]));
        mma_commit(smem_u32(&tfull[buf]));
        issued = true;
      }
      if (!ok && issued) {  // MMAs in flight finish before TMEM is freed
        mma_commit(smem_u32(&drain));
        mbar_wait_drain(smem_u32(&drain), 0);
      }
    }
  } else {
    const int fw = warp & 3;  // TMEM lane quarter: weight rows 32 fw .. + 31: gate for fw < 2, then up
    const float *sb = p.sb + static_cast<int64_t>(group + (fw < 2 ? 0 : F / 128)) * p.ld_sb;
    constexpr int kPer = (N + 31) / 32;  // token scales per lane
    uint64_t acc[N / 2];  // tokens 2i, 2i + 1
#pragma unroll
    for (int i = 0; i < N / 2; ++i) acc[i] = 0ull;
    bool bad = false;
    float x_nx[kPer], w_nx = 0.0f;
    auto load = [&](int kb) {
      w_nx = __ldg(sb + kb);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int m = m0 + lane + 32 * i;
        x_nx[i] = lane + 32 * i < N && m < p.M
                      ? __ldg(p.sa + static_cast<int64_t>(kb) * p.ld_sa + m)
                      : 1.0f;
      }
    };
    if (kb0 < kb1) load(kb0);
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      const int i = kb - kb0, buf = i % kFewBufs;
      float w = w_nx, x[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] = x_nx[j];
      if (kb + 1 < kb1) load(kb + 1);
      if (kPow2) {
        w = pow2_of(w, bad);
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[j] = pow2_of(x[j], bad);
      }
      // last read two groups ago, before the previous __syncwarp
      float *sx = s_sa[fw][i & 1];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (lane + 32 * j < N) sx[lane + 32 * j] = w * x[j];
      __syncwarp();
      const bool got = mbar_wait_bounded(smem_u32(&tfull[buf]),
                                         static_cast<uint32_t>(i / kFewBufs) & 1u, abort_flag,
                                         &g_glu_status, p.timeout_ns, FP8Q_ERR_TIMEOUT);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(fw * 32) << 16) + buf * N;
#pragma unroll
      for (int c = 0; c < N / 16; ++c) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(taddr + 16 * c, r);
        tmem_wait_ld_tied(r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 sc = ld_shared_v4(smem_u32(sx + 16 * c + 4 * j));
          ffma2(acc[8 * c + 2 * j], pack_u32x2(r[4 * j], r[4 * j + 1]), pack_u32x2(sc.x, sc.y));
          ffma2(acc[8 * c + 2 * j + 1], pack_u32x2(r[4 * j + 2], r[4 * j + 3]),
                pack_u32x2(sc.z, sc.w));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&tempty[buf]));
    }
    if (kPow2 && __any_sync(0xffffffffu, bad) && lane == 0)
      atomicCAS(&g_glu_status, 0, FP8Q_ERR_INVALID);
    tc_fence_before();
    __syncwarp();
    cluster_wait();  // every CTA of the cluster has started
    // token n's sums go to the CTA that finishes it, at [K part][token][row]
    const uint32_t mine = smem_u32(recv) + static_cast<uint32_t>(
        (part * C::kShare * 128 + fw * 32 + lane) * 4);
#pragma unroll
    for (int d = 0; d < S; ++d) {
      const uint32_t dst = mapa_shared(mine, static_cast<uint32_t>(half * S + d));
#pragma unroll
      for (int j = 0; j < C::kShare; ++j) {
        const int n = d * C::kShare + j;
        if (m0 + n < p.M) {
          const float2 v = unpack_f32x2(acc[n / 2]);
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + j * 512), "f"(n & 1 ? v.y : v.x)
                       : "memory");
        }
      }
    }
  }
  if (warp < 2) {
    __syncwarp();
    cluster_wait();
  }
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }

  // ---- this CTA's part of the tokens: 64 columns of h, two per lane
  constexpr int kWarps = kFewThreads / 32;
  constexpr int kTok = (C::kShare + kWarps - 1) / kWarps;  // tokens per warp
  float h[kTok][2];
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    const int j = warp + kWarps * k, m = m0 + part * C::kShare + j;
    h[k][0] = h[k][1] = 0.0f;
    if (j >= C::kShare || m >= p.M) continue;  // warp-uniform
    float2 gv = make_float2(0.0f, 0.0f), uv = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const float *src = recv + (s * C::kShare + j) * 128 + lane;
      gv.x += src[0];
      gv.y += src[32];
      uv.x += src[64];
      uv.y += src[96];
    }
    const float2 hv = unpack_f32x2(gate2(pack_f32x2(gv.x, gv.y), pack_f32x2(uv.x, uv.y)));
    h[k][0] = hv.x;
    h[k][1] = hv.y;
    float amax = fmaxf(fabsf(hv.x), fabsf(hv.y));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = lane + 32 * e;
      const float g = e ? gv.y : gv.x, u = e ? uv.y : uv.x;
      if (p.out.gu) {
        uint16_t *row = static_cast<uint16_t *>(p.out.gu) + static_cast<int64_t>(m) * p.out.ld_gu;
        row[c0 + col] = bf16_bits(g);
        row[F + c0 + col] = bf16_bits(u);
      }
      if (p.out.h)
        static_cast<uint16_t *>(p.out.h)[static_cast<int64_t>(m) * p.out.ldh + c0 + col] =
            bf16_bits(h[k][e]);
    }
    if (p.out.q) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (lane < 2)  // to both column halves of the group
        st_cluster_f32(smem_u32(&s_amax[half][j]), static_cast<uint32_t>(lane * S + part),
                       amax);
    }
  }
  if (!p.out.q) return;  // the same in every CTA of the cluster
  cluster_sync_all();
#pragma unroll
  for (int k = 0; k < kTok; ++k) {
    const int j = warp + kWarps * k, m = m0 + part * C::kShare + j;
    if (j >= C::kShare || m >= p.M) continue;
    float sc, inv;
    group_scale(fmaxf(s_amax[0][j], s_amax[1][j]), p.out.pow2 != 0, sc, inv);
    uint8_t *row = p.out.q + static_cast<int64_t>(m) * p.out.ldq + c0;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      row[lane + 32 * e] =
          static_cast<uint8_t>(pack_e4m3x2(__fmul_rn(h[k][e], inv), 0.0f) & 0xFFu);
    if (half == 0 && lane == 0) p.out.s[static_cast<int64_t>(group) * p.out.ld_s + m] = sc;
  }
}

template <int N, int S, bool kPow2>
fp8q_status launch_few(const GluIn &in, const GluOut &out, cudaStream_t s) {
  using C = Few<N, S>;
  auto kern = glu_few_tokens_kernel<N, S, kPow2>;
  static bool attr_set[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(C::kSmem)) != cudaSuccess)
        return FP8Q_ERR_CUDA;
      attr_set[dev] = true;
    }
  }
  // K == 0: no loads happen; describe a dummy 1 x 128 tensor so the maps are valid
  const bool k0 = in.K == 0;
  const void *any = out.h ? out.h : out.gu ? out.gu : out.q;
  CUtensorMap tw, tx;
  if (!make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, k0 ? any : in.b, k0 ? 1 : 2 * in.F,
                    k0 ? 128 : in.K, k0 ? 128 : in.ldb, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, k0 ? any : in.a, k0 ? 1 : in.M,
                    k0 ? 128 : in.K, k0 ? 128 : in.lda, 128, N, CU_TENSOR_MAP_SWIZZLE_128B))
    return FP8Q_ERR_CUDA;
  FewArgs a{};
  a.sa = in.sa;
  a.ld_sa = in.ld_sa;
  a.sb = in.sb;
  a.ld_sb = in.ld_sb;
  a.M = static_cast<int>(in.M);
  a.num_kb = static_cast<int>(in.K / 128);
  a.out = out;
  a.timeout_ns = wait_timeout_ns().load();
  const dim3 grid(static_cast<unsigned>(in.F / 128 * 2 * S),
                  static_cast<unsigned>((in.M + N - 1) / N));
  return launch_dependent(kern, grid, dim3(kFewThreads), C::kSmem, s, tw, tx, a);
}

template <int S, bool kPow2>
fp8q_status launch_few(const GluIn &in, const GluOut &out, cudaStream_t s) {
  return in.M <= 16   ? launch_few<16, S, kPow2>(in, out, s)
         : in.M <= 32 ? launch_few<32, S, kPow2>(in, out, s)
                      : launch_few<64, S, kPow2>(in, out, s);
}
template <bool kPow2>
fp8q_status launch_few(const GluIn &in, const GluOut &out, int sm_count, cudaStream_t s) {
  const int64_t ctas = in.F / 64 * ((in.M + 63) / 64), room = 2 * static_cast<int64_t>(sm_count);
  return 4 * ctas <= room   ? launch_few<4, kPow2>(in, out, s)
         : 2 * ctas <= room ? launch_few<2, kPow2>(in, out, s)
                            : launch_few<1, kPow2>(in, out, s);
}

// Up to 64 tokens, and for more while blocks of 64 tokens times blocks of 64
// columns are at most 128: the blocks share the weights through L2, and the GEMMs'
// tiles take the time of a whole K loop however few they are.  K = 7168, both
// sides measured (few-token kernel / tiles): F = 2048, 256 tokens (128 blocks)
// 21 / 31 us, 384 tokens (192) 37 / 33; F = 640, 512 tokens (80) 18 / 31, 1024
// tokens (160) 32 / 31; F = 7168, 192 tokens (336) 62 / 36; K = 1024, F = 7168,
// 128 tokens 12 / 9.
bool few_tokens(const GluIn &in) {
  return in.M <= 64 || in.F / 64 * ((in.M + 63) / 64) <= 128;
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
  if (!grouped && few_tokens(in))
    return pow2 ? launch_few<true>(in, o, dev.sm_count, s)
                : launch_few<false>(in, o, dev.sm_count, s);
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
// requested result is written from the same registers.  The kernel is
// persistent, two CTAs of 256 threads per SM, and TMA brings in the next tile
// while this one is turned into codes.
//  - A cluster of two CTAs covers a tile of 128 tokens x 128 columns of h, each
//    CTA 64 columns; a thread holds 4 tokens x 8 columns of dg, du and h as
//    packed FP32 pairs (96 registers; two-lane multiplies, three-input maxima).
//  - 1x128 max-abs (dg and du, per token): a halving exchange over a token's
//    eight threads (each ends with one of the eight maxima), then one value per
//    token and CTA to both CTAs by st.async, which completes on the receiver's
//    mbarrier: a cluster barrier would make every step wait for all of its
//    global stores (46 us against 36 at 8192 x 2048).
//  - 128x1 max-abs (dg, du, h, per column): each thread's four tokens go to shared
//    memory, and one thread per column takes the maximum of the 32 token quads.
//  - One thread per group turns a max-abs into its scale, so that the two IEEE
//    divisions are done once per group.
//  - The transposed codes pass through shared memory: a thread's 4 tokens of a
//    column are one 32-bit word; word w of column row r sits at w ^ f(r), which
//    spreads a warp's words over all banks on the way in and keeps 16-byte
//    units whole on the way out, where eight lanes write a column's 128 bytes.
// An abandoned wait only stops the copies and the stores; every thread still
// walks the loop and its CTA barriers to the end.
constexpr int kChan = 64;                      // columns of h per CTA
constexpr int kBwdThreads = 256;               // 32 token quads x 8 column octets
constexpr int kBwdCtasPerSm = 2;
constexpr uint32_t kRawBytes = 128 * kChan * 2;  // one input's tile of a CTA
constexpr uint32_t kXposeBytes = kChan * 128;    // one transposed tile of codes
constexpr uint32_t kPartBytes = 32 * kChan * 4;  // one array's column maxima by token quad

struct BwdArgs {
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
  int ncb, ntb;  // 128-wide column blocks, token blocks
  int pow2;
  uint64_t timeout_ns;
};

__device__ __forceinline__ uint32_t xpose_word(uint32_t r, uint32_t w) {
  return r * 32u + (w ^ (4u * ((r >> 3) & 7u)));
}
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) {
  return pack_f32x2(bf16_lo(w), bf16_hi(w));
}

// One FP32 value into CTA `rank`'s shared memory; its four bytes count towards
// the mbarrier at the same offset there as `local_bar` here.
__device__ __forceinline__ void st_async_f32(uint32_t local_addr, uint32_t local_bar, uint32_t rank,
                                             float v) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
          mapa_shared(local_addr, rank)),
      "r"(__float_as_uint(v)), "r"(mapa_shared(local_bar, rank))
      : "memory");
}

template <bool kRows, bool kCols, bool kH>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kBwdThreads, kBwdCtasPerSm)
    swiglu_bwd_kernel(const __grid_constant__ CUtensorMap tmD,
                      const __grid_constant__ CUtensorMap tmG, const BwdArgs p) {
  constexpr int kColArrays = (kCols ? 2 : 0) + (kH ? 1 : 0);  // dg, du | h
  constexpr int kH0 = kCols ? 2 : 0;                          // h's place among them
  extern __shared__ uint8_t dsm_raw[];
  uint8_t *raw = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint32_t *xpose = reinterpret_cast<uint32_t *>(raw + 3 * kRawBytes);
  // column maxima [token quad][array][position]; position 32 i + 4 l + e holds
  // column 8 l + 4 i + e, so that the eight lanes of a quad store whole rows
  float *col_part = reinterpret_cast<float *>(raw + 3 * kRawBytes + kColArrays * kXposeBytes);
  constexpr int kPartRow = (kColArrays > 0 ? kColArrays : 1) * kChan;
  // by step parity: the other CTA is at most one step ahead of what is read here,
  // since it needs all of this CTA's values of a step to go on
  __shared__ float row_amax[2][2][2][128];  // [step parity][CTA of the cluster][dg, du][token]
  __shared__ float row_inv[2][128];
  __shared__ __align__(16) float col_inv[3][kChan];
  __shared__ uint64_t full, rows_in[2];
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int l8 = lane & 7;                     // column octet
  const int quad = 4 * warp + (lane >> 3);     // token quad
  const uint32_t rank = cluster_ctarank();
  // tile t = (token block t / ncb, column block t % ncb), column blocks fastest;
  // this cluster takes every (gridDim.x / 2)-th, walked incrementally
  const uint32_t ncb = static_cast<uint32_t>(p.ncb), ntb = static_cast<uint32_t>(p.ntb);
  const uint32_t clusters = gridDim.x >> 1, id = blockIdx.x >> 1;
  const uint32_t dcb = clusters % ncb, dtb = clusters / ncb;
  uint32_t cb = id % ncb, tb = id / ncb;
  auto step = [&]() {
    cb += dcb;
    tb += dtb;
    if (cb >= ncb) {
      cb -= ncb;
      ++tb;
    }
  };
  auto issue = [&](uint32_t cbn, uint32_t tbn) {
    const uint32_t bar = smem_u32(&full), dst = smem_u32(raw);
    const int32_t c = static_cast<int32_t>(cbn * 128u + rank * kChan);
    const int32_t t = static_cast<int32_t>(tbn * 128u);
    mbar_arrive_expect_tx(bar, 3 * kRawBytes);
    tma_load_2d(dst, &tmD, bar, c, t);
    tma_load_2d(dst + kRawBytes, &tmG, bar, c, t);
    tma_load_2d(dst + 2 * kRawBytes, &tmG, bar, static_cast<int32_t>(p.F) + c, t);
  };
  bool pending = false;  // thread 0: a copy is on its way
  if (tid == 0) {
    abort_flag = 0;
    mbar_init(smem_u32(&full), 1);
    mbar_init(smem_u32(&rows_in[0]), 1);
    mbar_init(smem_u32(&rows_in[1]), 1);
    fence_barrier_init();
  }
  wait_for_previous_kernel();
  if (tid == 0 && tb < ntb) {
    issue(cb, tb);
    pending = true;
  }
  // barriers initialised in both CTAs before either sends
  if (kRows) cluster_sync_all();
  else __syncthreads();

  const uint64_t one2 = pack_f32x2(1.0f, 1.0f), neg2 = pack_f32x2(-1.0f, -1.0f);
  bool ok = true;
  for (uint32_t it = 0; tb < ntb; ++it) {
    const int64_t t0 = static_cast<int64_t>(tb) * 128;
    const int64_t c0 = static_cast<int64_t>(cb) * 128 + rank * kChan;
    const int64_t c = c0 + 8 * l8;
    const bool got = mbar_wait_bounded(smem_u32(&full), it & 1u, &abort_flag, &g_glu_status,
                                       p.timeout_ns, FP8Q_ERR_TIMEOUT);
    ok = ok && __all_sync(0xffffffffu, got);
    if (tid == 0 && ok) pending = false;

    // ---- dg, du, h of 4 tokens x 8 columns, as pairs of neighbouring columns
    uint64_t dg[4][4], du[4][4], h[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t src = smem_u32(raw) + static_cast<uint32_t>(4 * quad + i) * 128u + 16u * l8;
      const uint4 vd = ld_shared_v4(src), vg = ld_shared_v4(src + kRawBytes),
                  vu = ld_shared_v4(src + 2 * kRawBytes);
      const uint32_t wd[4] = {vd.x, vd.y, vd.z, vd.w}, wg[4] = {vg.x, vg.y, vg.z, vg.w},
                     wu[4] = {vu.x, vu.y, vu.z, vu.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t y = bf16_pair(wd[k]), g = bf16_pair(wg[k]), u = bf16_pair(wu[k]);
        const uint64_t s = sigmoid2(g);
        const uint64_t sl = fmul2(g, s);  // silu(g)
        du[i][k] = fmul2(y, sl);
        dg[i][k] = fmul2(fmul2(y, u), fma2(sl, fma2(s, neg2, one2), s));
        if (kH) h[i][k] = fmul2(sl, u);
      }
    }
    if (p.d && ok) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + 4 * quad + i;
        if (t < p.T) {
          uint16_t *dst = p.d + t * p.ld_d + c;
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 a = unpack_f32x2(dg[i][k]), b = unpack_f32x2(du[i][k]);
            w[k] = bf16x2_bits(a.x, a.y);
            w[4 + k] = bf16x2_bits(b.x, b.y);
          }
          *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4 *>(dst + p.F) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }

    // ---- max-abs of the groups
    if (kRows) {
      if (tid == 0) mbar_arrive_expect_tx(smem_u32(&rows_in[it & 1]), 2 * 256 * 4);
      float m[8];  // token i of this thread's four: dg at 2i, du at 2i + 1
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = unpack_f32x2(dg[i][k]), y = unpack_f32x2(du[i][k]);
          a = max3_abs(a, x.x, x.y);
          b = max3_abs(b, y.x, y.y);
        }
        m[2 * i] = a;
        m[2 * i + 1] = b;
      }
      // halving exchange over the eight lanes of the quad: lane l ends with the
      // maximum of m[l] over the lanes
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        const bool up = (l8 & o) != 0;
#pragma unroll
        for (int k = 0; k < o; ++k) {
          const float keep = up ? m[k + o] : m[k], give = up ? m[k] : m[k + o];
          m[k] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
      }
      const uint32_t at = smem_u32(&row_amax[it & 1][rank][l8 & 1][4 * quad + (l8 >> 1)]);
      st_async_f32(at, smem_u32(&rows_in[it & 1]), 0, m[0]);
      st_async_f32(at, smem_u32(&rows_in[it & 1]), 1, m[0]);
    }
#pragma unroll
    for (int k = 0; k < kColArrays; ++k) {
      float m[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = unpack_f32x2(kH && k == kH0 ? h[i][j] : k == 0 ? dg[i][j] : du[i][j]);
        m[2 * j] = max3_abs(max3_abs(v[0].x, v[1].x, v[2].x), v[3].x, 0.0f);
        m[2 * j + 1] = max3_abs(max3_abs(v[0].y, v[1].y, v[2].y), v[3].y, 0.0f);
      }
      float4 *dst = reinterpret_cast<float4 *>(col_part + quad * kPartRow + k * kChan) + l8;
      dst[0] = make_float4(m[0], m[1], m[2], m[3]);
      dst[8] = make_float4(m[4], m[5], m[6], m[7]);
    }
    __syncthreads();
    // every thread has read the raw tile (and used what it read): the next one
    // may come
    const uint32_t cbc = cb;
    step();
    if (tid == 0 && ok && tb < ntb) {
      issue(cb, tb);
      pending = true;
    }
    if (!kRows && kColArrays == 0) continue;

    // ---- scales, one group per thread at a time
    if (kColArrays > 0 && tid < kColArrays * kChan) {
      const int k = tid / kChan, pos = tid % kChan;
      const int cc = 8 * ((pos & 31) >> 2) + 4 * (pos >> 5) + (pos & 3);
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        a = max3_abs(a, col_part[i * kPartRow + tid], col_part[(i + 1) * kPartRow + tid]);
      float sc, inv;
      group_scale(a, p.pow2 != 0, sc, inv);
      col_inv[k][cc] = inv;
      if (ok) {
        if (kH && k == kH0) p.shT[(t0 / 128) * p.ld_shT + c0 + cc] = sc;
        else p.sT[(t0 / 128) * p.ld_sT + k * p.F + c0 + cc] = sc;
      }
    }
    if (kRows) {
      const bool in = mbar_wait_bounded(smem_u32(&rows_in[it & 1]), (it >> 1) & 1u, &abort_flag,
                                        &g_glu_status, p.timeout_ns, FP8Q_ERR_TIMEOUT);
      ok = __all_sync(0xffffffffu, in) && ok;
      const int k = tid >> 7, t = tid & 127;
      const float a = fmaxf(row_amax[it & 1][0][k][t], row_amax[it & 1][1][k][t]);
      float sc, inv;
      group_scale(a, p.pow2 != 0, sc, inv);
      row_inv[k][t] = inv;
      if (rank == 0 && ok && t0 + t < p.T)
        p.s[(static_cast<int64_t>(k) * p.ncb + cbc) * p.ld_s + t0 + t] = sc;
    }
    __syncthreads();

    // ---- codes
    if (kRows && ok) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tl = 4 * quad + i;
        if (t0 + tl < p.T) {
          uint8_t *dst = p.q + (t0 + tl) * p.ldq + c;
          const float a = row_inv[0][tl], b = row_inv[1][tl];
          const uint64_t a2 = pack_f32x2(a, a), b2 = pack_f32x2(b, b);
          *reinterpret_cast<uint2 *>(dst) =
              make_uint2(codes4(fmul2(dg[i][0], a2), fmul2(dg[i][1], a2)),
                         codes4(fmul2(dg[i][2], a2), fmul2(dg[i][3], a2)));
          *reinterpret_cast<uint2 *>(dst + p.F) =
              make_uint2(codes4(fmul2(du[i][0], b2), fmul2(du[i][1], b2)),
                         codes4(fmul2(du[i][2], b2), fmul2(du[i][3], b2)));
        }
      }
    }
    if (kColArrays > 0) {
#pragma unroll
      for (int k = 0; k < kColArrays; ++k) {
        const ulonglong2 i01 = *reinterpret_cast<const ulonglong2 *>(&col_inv[k][8 * l8]);
        const ulonglong2 i23 = *reinterpret_cast<const ulonglong2 *>(&col_inv[k][8 * l8 + 4]);
        const uint64_t inv[4] = {i01.x, i01.y, i23.x, i23.y};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i] = unpack_f32x2(
                fmul2(kH && k == kH0 ? h[i][j] : k == 0 ? dg[i][j] : du[i][j], inv[j]));
          uint32_t *row = xpose + k * (kXposeBytes / 4);
          row[xpose_word(8 * l8 + 2 * j, quad)] = codes4(v[0].x, v[1].x, v[2].x, v[3].x);
          row[xpose_word(8 * l8 + 2 * j + 1, quad)] = codes4(v[0].y, v[1].y, v[2].y, v[3].y);
        }
      }
      __syncthreads();
      // eight lanes write the 128 tokens of a column
      if (ok) {
#pragma unroll
        for (int k = 0; k < kColArrays; ++k)
#pragma unroll
          for (int i = 0; i < kChan * 8 / kBwdThreads; ++i) {
            const int r = (tid >> 3) + 32 * i, ch = tid & 7;
            const uint4 v = *reinterpret_cast<const uint4 *>(
                &xpose[k * (kXposeBytes / 4) + xpose_word(r, 4 * ch)]);
            uint8_t *dst = kH && k == kH0 ? p.hT + (c0 + r) * p.ld_hT + t0 + 16 * ch
                                          : p.qT + (k * p.F + c0 + r) * p.ldqT + t0 + 16 * ch;
            *reinterpret_cast<uint4 *>(dst) = v;
          }
      }
    }
  }
  let_next_kernel_start();
  if (kRows) cluster_sync_all();  // the other CTA no longer sends here
  // a copy still in flight after an abandoned wait lands before the CTA's shared
  // memory goes
  if (tid == 0 && pending) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
}

template <bool kRows, bool kCols, bool kH>
fp8q_status launch_bwd(const CUtensorMap &tmD, const CUtensorMap &tmG, const BwdArgs &a,
                       cudaStream_t s) {
  auto kern = swiglu_bwd_kernel<kRows, kCols, kH>;
  constexpr size_t smem =
      128 + 3 * kRawBytes + ((kCols ? 2 : 0) + (kH ? 1 : 0)) * (kXposeBytes + kPartBytes);
  static bool attr_set[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FP8Q_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem)) != cudaSuccess)
        return FP8Q_ERR_CUDA;
      attr_set[dev] = true;
    }
  }
  DeviceInfo info;
  if (fp8q_status st = device_info(info)) return st;
  const int64_t tiles = static_cast<int64_t>(a.ncb) * a.ntb;
  const int64_t room = static_cast<int64_t>(info.sm_count) * kBwdCtasPerSm / 2;
  return launch_dependent(kern, dim3(static_cast<unsigned>(2 * (tiles < room ? tiles : room))),
                          dim3(kBwdThreads), smem, s, tmD, tmG, a);
}

template <bool kRows, bool kCols>
fp8q_status launch_bwd(const CUtensorMap &tmD, const CUtensorMap &tmG, const BwdArgs &a,
                       cudaStream_t s) {
  return a.hT ? launch_bwd<kRows, kCols, true>(tmD, tmG, a, s)
              : launch_bwd<kRows, kCols, false>(tmD, tmG, a, s);
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
  a.ncb = static_cast<int>(F / 128);
  a.ntb = static_cast<int>((T + 127) / 128);
  a.timeout_ns = wait_timeout_ns().load();
  CUtensorMap tmD, tmG;
  if (!make_tmap_2d(&tmD, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dh, T, F, ld_dh * 2, kChan, 128,
                    CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tmap_2d(&tmG, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, gu, T, 2 * F, ld_gu * 2, kChan, 128,
                    CU_TENSOR_MAP_SWIZZLE_NONE))
    return FP8Q_ERR_CUDA;
  auto st = static_cast<cudaStream_t>(stream);
  if (q)
    return qT ? launch_bwd<true, true>(tmD, tmG, a, st) : launch_bwd<true, false>(tmD, tmG, a, st);
  return qT ? launch_bwd<false, true>(tmD, tmG, a, st) : launch_bwd<false, false>(tmD, tmG, a, st);
}
