// fp8q_glu.cuh -- the gated feed-forward block's outputs: h = silu(g) * u from
// the two projections g and u, shared by the tensor-core GEMMs (gemm.cu,
// gemm_mx.cu) and the few-token kernel (swiglu.cu).
//
// A tensor-core tile of the gated GEMM covers 128 columns of h.  Its 256 rows
// of B are interleaved 64 at a time -- 64 gate rows, the 64 up rows of the same
// columns, the next 64 gate rows, their up rows -- so that an epilogue warp,
// which reads 128 consecutive accumulator columns, holds g and u of the same
// 64 columns of h in the same threads: the activation and the product need no
// exchange.  A 1x128 group of h is two such warps wide; they exchange one
// max-abs per row through shared memory.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fp8q.h"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"

namespace fp8q {

// Where the results go; a null pointer leaves that result out.
struct GluOut {
  void *h;       // BF16 [M][ldh]
  int64_t ldh;
  void *gu;      // BF16 [M][ld_gu]: g in columns [0, F), u in [F, 2F)
  int64_t ld_gu;
  uint8_t *q;    // E4M3 [M][ldq], 1x128 codes of h
  int64_t ldq;
  float *s;      // FP32 scale of (m, group) at s[group * ld_s + m]
  int64_t ld_s;
  int pow2;      // scale mode of q, s
  int F;
};

// Operands of the gated GEMM; offs is null for the dense form (G = 1).
struct GluIn {
  const void *a;
  int64_t lda;
  const float *sa;
  int64_t ld_sa;
  const void *b;
  int64_t ldb;
  const float *sb;
  int64_t ld_sb;
  const int32_t *offs;
  int G;
  int64_t M, F, K;
};

// Tensor-core forms, defined in gemm.cu (FP32 scales, any K) and gemm_mx.cu
// (power-of-two scales, K > 0).  Arguments are already checked.
fp8q_status gemm_glu(const GluIn &in, const GluOut &out, cudaStream_t s);
fp8q_status gemm_mx_glu(const GluIn &in, const GluOut &out, cudaStream_t s);

// 1 / (1 + exp(-g)) of a pair, by the hardware's exp2 and reciprocal (a few FP32
// ulps and |g| ulps of the exponent's product, far below the rounding of any
// output).  exp(-g) = inf for g < -88 gives 0, where the exact value is below
// 1e-37.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g) {
  const float2 x = unpack_f32x2(fmul2(g, pack_f32x2(-1.4426950408889634f, -1.4426950408889634f)));
  const float2 d =
      unpack_f32x2(fadd2(pack_f32x2(ex2_ftz(x.x), ex2_ftz(x.y)), pack_f32x2(1.0f, 1.0f)));
  return pack_f32x2(rcp_ftz(d.x), rcp_ftz(d.y));
}
// silu(g) * u of a pair.
__device__ __forceinline__ uint64_t gate2(uint64_t g, uint64_t u) {
  return fmul2(fmul2(g, sigmoid2(g)), u);
}

// Row max-abs exchange between the two epilogue warps of a 128-column group.
struct GluExchange {
  alignas(8) uint64_t bar[4];  // one per TMEM lane quarter, two arrivals each
  float amax[2][8][32];        // [use parity][epilogue warp][row]
};
__device__ __forceinline__ void glu_exchange_init(GluExchange &x) {
  for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&x.bar[i]), 2);
}

// Tensor maps of the results: gu and h in boxes of 64 columns (128-byte swizzle),
// q in boxes of 64 columns (64-byte swizzle), 32 rows each.
struct GluMaps {
  CUtensorMap gu, h, q;
};
// Results that are left out keep a copy of `any`.
inline bool make_glu_maps(GluMaps &m, const CUtensorMap &any, const GluIn &in, const GluOut &out) {
  m = GluMaps{any, any, any};
  return (!out.gu ||
          make_tmap_2d(&m.gu, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out.gu, in.M, 2 * in.F,
                       out.ld_gu * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B)) &&
         (!out.h || make_tmap_2d(&m.h, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out.h, in.M, in.F,
                                 out.ldh * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B)) &&
         (!out.q || make_tmap_2d(&m.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, out.q, in.M, in.F, out.ldq,
                                 64, 32, CU_TENSOR_MAP_SWIZZLE_64B));
}

// Eight packed pairs -> 16 BF16 values (32 bytes) as two 16-byte units.
__device__ __forceinline__ uint4 bf16_unit(const uint64_t *v) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack_f32x2(v[e]);
    __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
    w[e] = *reinterpret_cast<uint32_t *>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 64 columns of this lane's row (32 pairs) into a 32-row x 128-byte box.
__device__ __forceinline__ void stage_box(uint32_t box, const uint64_t *v, int lane) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    st_shared_v4(box + lane * 128 + 16 * (k ^ (lane & 7)), bf16_unit(v + 4 * k));
}
// 64 columns of this lane's row to global memory, 64 bytes of each row at a time.
__device__ __forceinline__ void store_rows(uint32_t buf, const uint64_t *v, void *c, int64_t ldc,
                                           int row0, int row_end, int col0, int n, int lane) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint4 u[4] = {bf16_unit(v + 16 * b), bf16_unit(v + 16 * b + 4), bf16_unit(v + 16 * b + 8),
                        bf16_unit(v + 16 * b + 12)};
    warp_store_block64<2, false>(buf, u, c, ldc, row0, row_end, col0 + 32 * b, n, lane);
  }
}

// Store the results of one warp's 32 rows x 64 columns of h.  acc: this
// thread's row, 64 gate values then 64 up values as packed FP32 pairs.  buf:
// the warp's staging buffer (8 KB, 1024-byte aligned).  Whole blocks leave as TMA
// tensor stores that drain while the next tile is folded (8192 x 2048 x 7168 with
// gu and codes: 213 us, 220 with coalesced stores).  tma: this block may leave
// that way (warp-uniform; the maps clip at the tensor's last row only).  uses counts this warp's exchanges.  Returns false
// when a bounded wait gave up.  All branches are warp-uniform and the same for
// the two warps of a group.
__device__ __forceinline__ bool glu_store(uint64_t (&acc)[64], const GluOut &o, const GluMaps *maps,
                                          bool tma, uint32_t buf, int row0, int row_end, int col0,
                                          int ew, int lane, GluExchange &x, uint32_t &uses,
                                          volatile int *abort_flag, int *status_word,
                                          uint64_t timeout_ns) {
  // the last tile's stores have read the buffer
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
  if (o.gu) {
    if (tma) {
      stage_box(buf, acc, lane);
      stage_box(buf + 4096, acc + 32, lane);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        const uint64_t pol = l2_evict_first_policy();
        tma_store_2d_hint(&maps->gu, buf, col0, row0, pol);
        tma_store_2d_hint(&maps->gu, buf + 4096, o.F + col0, row0, pol);
        bulk_commit_group();
      }
    } else {
      store_rows(buf, acc, o.gu, o.ld_gu, row0, row_end, col0, o.F, lane);
      store_rows(buf, acc + 32, o.gu, o.ld_gu, row0, row_end, o.F + col0, 2 * o.F, lane);
    }
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    acc[i] = gate2(acc[i], acc[32 + i]);
    const float2 v = unpack_f32x2(acc[i]);
    amax = max3_abs(amax, v.x, v.y);
  }
  if (!o.h && !o.q) return true;
  if (o.q) {
    // this warp's maxima are on their way while h is stored; the buffer of this
    // parity was last read two uses ago, before the partner arrived for the
    // previous use
    x.amax[uses & 1u][ew][lane] = amax;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&x.bar[ew & 3]));
  }
  // gu's stores have read the buffer
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
  if (o.h) {
    if (tma) stage_box(buf, acc, lane);
    else store_rows(buf, acc, o.h, o.ldh, row0, row_end, col0, o.F, lane);
  }
  if (o.q) {
    const uint32_t par = uses & 1u;
    const bool got = mbar_wait_bounded(smem_u32(&x.bar[ew & 3]), par, abort_flag, status_word,
                                       timeout_ns, FP8Q_ERR_TIMEOUT);
    if (!__all_sync(0xffffffffu, got)) return false;
    ++uses;
    amax = fmaxf(amax, x.amax[par][ew ^ 4][lane]);
    float sc, inv;
    group_scale(amax, o.pow2 != 0, sc, inv);
    const uint64_t inv2 = pack_f32x2(inv, inv);
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = codes4(fmul2(acc[8 * k + 2 * e], inv2), fmul2(acc[8 * k + 2 * e + 1], inv2));
      v[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (tma) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        st_shared_v4(buf + 4096 + lane * 64 + 16 * (k ^ ((lane >> 1) & 3)), v[k]);
    } else {
      warp_store_block64<1, false>(buf, v, o.q, o.ldq, row0, row_end, col0, o.F, lane);
    }
    if (ew < 4 && row0 + lane < row_end)
      o.s[static_cast<int64_t>(col0 / 128) * o.ld_s + row0 + lane] = sc;
  }
  if (tma) {
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      const uint64_t pol = l2_evict_first_policy();
      if (o.h) tma_store_2d_hint(&maps->h, buf, col0, row0, pol);
      if (o.q) tma_store_2d_hint(&maps->q, buf + 4096, col0, row0, pol);
      bulk_commit_group();
    }
  }
  return true;
}

}  // namespace fp8q
