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

// Store the results of one warp's 32 rows x 64 columns of h.  acc: this
// thread's row, 64 gate values then 64 up values as packed FP32 pairs.  buf:
// the warp's 2 KB staging buffer.  uses counts this warp's exchanges.  Returns
// false when a bounded wait gave up.  All branches are warp-uniform and the
// same for the two warps of a group.
__device__ __forceinline__ bool glu_store(uint64_t (&acc)[64], const GluOut &o, uint32_t buf,
                                          int row0, int row_end, int col0, int ew, int lane,
                                          GluExchange &x, uint32_t &uses, volatile int *abort_flag,
                                          int *status_word, uint64_t timeout_ns) {
  if (o.gu) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // 32 columns (64 bytes) at a time: gate, gate, up, up
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_f32x2(acc[16 * b + 4 * k + e]);
          __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
          w[e] = *reinterpret_cast<uint32_t *>(&p);
        }
        v[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      warp_store_block64<2, false>(buf, v, o.gu, o.ld_gu, row0, row_end,
                                   (b >> 1) * o.F + col0 + 32 * (b & 1), 2 * o.F, lane);
    }
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    acc[i] = gate2(acc[i], acc[32 + i]);
    const float2 v = unpack_f32x2(acc[i]);
    amax = max3_abs(amax, v.x, v.y);
  }
  if (o.h) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_f32x2(acc[16 * b + 4 * k + e]);
          __nv_bfloat162 p = __floats2bfloat162_rn(f.x, f.y);
          w[e] = *reinterpret_cast<uint32_t *>(&p);
        }
        v[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      warp_store_block64<2, false>(buf, v, o.h, o.ldh, row0, row_end, col0 + 32 * b, o.F, lane);
    }
  }
  if (o.q) {
    // the buffer of this parity was last read two uses ago, before the partner
    // arrived for the previous use
    const uint32_t par = uses & 1u;
    const int quarter = ew & 3;
    x.amax[par][ew][lane] = amax;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&x.bar[quarter]));
    const bool got = mbar_wait_bounded(smem_u32(&x.bar[quarter]), par, abort_flag, status_word,
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
    warp_store_block64<1, false>(buf, v, o.q, o.ldq, row0, row_end, col0, o.F, lane);
    if (ew < 4 && row0 + lane < row_end)
      o.s[static_cast<int64_t>(col0 / 128) * o.ld_s + row0 + lane] = sc;
  }
  return true;
}

}  // namespace fp8q
