// fp8q_vec.cuh -- eight consecutive BF16 or FP32 values of a row or a list, as
// one thread moves them: 16-byte loads and stores and the conversions between; and a
// warp's sums.
#pragma once

#include <cstdint>

#include "fp8q.h"
#include "fp8q_ptx.cuh"

namespace fp8q {

enum Kind { kBf16 = FP8Q_OUT_BF16, kFp32 = FP8Q_OUT_FP32, kNone = 2 };

__host__ __device__ constexpr int size_of(int kind) { return kind == kBf16 ? 2 : 4; }
constexpr bool kind_ok(int kind) { return kind == kBf16 || kind == kFp32; }

// The same sum in all lanes.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(~0u, v); }

__device__ __forceinline__ float absmax8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) m = max3_abs(m, v[e], v[e + 1]);
  return m;
}

// Read once by one thread: not kept in L1.  (Not the read-only path: a result may
// be its own input, as when the residual stream is updated in place.)
__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void unpack8(const uint4 &a, const uint4 &b, float (&v)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}

// Eight consecutive values as FP32 (exact).
template <int kKind>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&v)[8]) {
  if constexpr (kKind == kBf16) {
    unpack8(ld_stream(static_cast<const uint16_t *>(base) + at), v);
  } else {
    const float *p = static_cast<const float *>(base) + at;
    const uint4 a = ld_stream(p), b = ld_stream(p + 4);
    unpack8(a, b, v);
  }
}
// The same from the weights, which every row reads again.
__device__ __forceinline__ void load8_w(const void *base, bool fp32, int at, float (&v)[8]) {
  if (fp32) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
    const uint4 a = p[0], b = p[1];
    unpack8(a, b, v);
  } else {
    unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at), v);
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight values rounded to nearest-even, or as they are.
template <int kKind>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&v)[8]) {
  if constexpr (kKind == kBf16) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) =
        make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  } else {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

}  // namespace fp8q
