// adamw.cu -- one AdamW step over a list of tensors:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)).
//
// Every value is read and written once: 28 bytes per value with FP32 parameters,
// gradients and moments, 16 with moments in 8 bits, 2 more for the BF16 copy.  It
// is bound by memory.  The list travels in the launch's parameters (no copy to the
// device, so a captured call holds it too); a CTA takes one chunk of values and finds
// its tensor by a binary search over the chunks' prefix sums.
//
// Moments in 8 bits: m and sqrt(v) as E4M3 with an FP32 scale per 128 values.  v
// itself spans the square of the gradients' range, which E4M3 (2^-9 to 448 below
// one scale) does not; its root spans the gradients' own.  A positive root is kept
// at or above the smallest code: rounded to zero it would leave |m| / eps as the
// step of a value whose gradients were small, not absent.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <vector>

#include "fp8q.h"
#include "fp8q_host.cuh"
#include "fp8q_ptx.cuh"
#include "fp8q_vec.cuh"

namespace fp8q {
namespace {

// Eight values per thread, one chunk per CTA, three CTAs per SM.  176 M values with
// moments in 8 bits: 467 us; CTAs of 256 threads 595, of 512 506 (496 held to 64
// registers), of 1024 657; two vectors per thread 556.  FP32 moments take 750 to 762 us
// in all of these, ten small tensors 8.6 to 9.3 (two vectors) and 10.7 (1024 threads).
constexpr int kThreads = 384;
constexpr int kChunk = kThreads * 8;
constexpr int kBatch = 128;  // tensors per launch

enum State { kStateBf16 = FP8Q_STATE_BF16, kStateFp32 = FP8Q_STATE_FP32, kStateE4m3 = FP8Q_STATE_E4M3 };

struct Tensor {
  void *p;
  const void *g;
  void *m, *v;
  float *ms, *vs;
  void *copy;
  int64_t n;
};

struct Batch {
  Tensor t[kBatch];
  int first[kBatch];  // first chunk of each tensor
  uint32_t wide[kBatch / 32];  // bit i: tensor i's addresses are all 16-byte aligned
  int count;
};

struct Args {
  float lr, wd, b1, omb1, b2, omb2, eps, ic1, isc2;
  float log_b1[2], log_b2[2];  // ln beta, high and low part, for a step in device memory
  const float *lr_dev, *grad_scale;
  const int64_t *step_dev;
};

// 1 - beta^t = -expm1(t ln beta), the product carried in two FP32 parts.
__device__ __forceinline__ float one_minus_power(const float (&log_b)[2], float t) {
  const float hi = t * log_b[0];
  if (!(hi > -100.0f)) return 1.0f;  // beta^t below 2^-144 (and beta = 0)
  const float lo = fmaf(t, log_b[0], -hi) + t * log_b[1];
  return -fmaf(expf(hi), lo, expm1f(hi));
}

// Element i of an array of `kind`.
template <int kKind>
__device__ __forceinline__ float get(const void *base, int64_t i) {
  if constexpr (kKind == kBf16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(base)[i]) << 16);
  else
    return static_cast<const float *>(base)[i];
}
template <int kKind>
__device__ __forceinline__ void put(void *base, int64_t i, float v) {
  if constexpr (kKind == kBf16)
    static_cast<uint16_t *>(base)[i] = static_cast<uint16_t>(bf16x2(v, 0.0f));
  else
    static_cast<float *>(base)[i] = v;
}

// Up to eight values from i on: all of them by wide loads, or the first `left`
// one by one (zeros behind).
template <int kKind>
__device__ __forceinline__ void get8(const void *base, int64_t i, bool wide, int left, float (&v)[8]) {
  if (wide) {
    load8<kKind>(base, i, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? get<kKind>(base, i + e) : 0.0f;
  }
}
template <int kKind>
__device__ __forceinline__ void put8(void *base, int64_t i, bool wide, int left, const float (&v)[8]) {
  if (wide) {
    store8<kKind>(base, i, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) put<kKind>(base, i + e, v[e]);
  }
}

__device__ __forceinline__ uint2 get_codes(const void *base, int64_t i, bool wide, int left) {
  const uint8_t *p = static_cast<const uint8_t *>(base) + i;
  if (wide) return *reinterpret_cast<const uint2 *>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) w[e >> 2] |= static_cast<uint32_t>(p[e]) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void put_codes(void *base, int64_t i, bool wide, int left, uint2 c) {
  uint8_t *p = static_cast<uint8_t *>(base) + i;
  if (wide) {
    *reinterpret_cast<uint2 *>(p) = c;
  } else {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
  }
}
// Four pairs of values: two-lane FP32 arithmetic (each lane rounded as by itself).
using Pairs = uint64_t[4];
__device__ __forceinline__ void pack(const float (&v)[8], Pairs &p) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = pack_f32x2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void unpack(const Pairs &p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_f32x2(p[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint64_t both(float v) { return pack_f32x2(v, v); }

// The sum of two products that are rounded before it: a packed addition is joined with
// a packed product into one rounding by the assembler, a scalar one is not.
__device__ __forceinline__ uint64_t sum2(uint64_t a, uint64_t b) {
  const float2 x = unpack_f32x2(a), y = unpack_f32x2(b);
  return pack_f32x2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

__device__ __forceinline__ void decode8(uint2 c, float s, Pairs &v) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t d = decode_e4m3x2(static_cast<uint16_t>(w[h >> 1] >> (16 * (h & 1))));
    v[h] = fmul2(pack_f32x2(f16_lo(d), f16_hi(d)), both(s));
  }
}
__device__ __forceinline__ float absmax8(const Pairs &p) {
  float v[8];
  unpack(p, v);
  return fp8q::absmax8(v);
}
__device__ __forceinline__ uint2 codes8(const Pairs &p) { return make_uint2(codes4(p[0], p[1]), codes4(p[2], p[3])); }

// Codes of groups of 128 values of m and of sqrt(v), 8 in each of 16 lanes; a scale:
// with a the max-abs (at least 2^-116) s = a * fl(1 / 448), codes
// E4M3(x * fl(448 * fl(1 / a))), one quotient where the quantisers' rule takes two.
// Their products with a stay at or below 448 (1 + 2^-22), which E4M3 rounds to 448.
// The lower eight lanes reduce m and take its scale, the upper eight the root's; s is
// each half's own.
__device__ __forceinline__ void encode(Pairs &m, Pairs &r, uint2 &cm, uint2 &cr, float &s) {
  const bool upper = threadIdx.x & 8;
  const float am = absmax8(m), ar = absmax8(r);
  float a = upper ? ar : am;
  a = fmaxf(a, __shfl_xor_sync(~0u, upper ? am : ar, 8));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
  a = fmaxf(a, 0x1p-116f);
  s = a * (1.0f / 448.0f);
  const float inv = __fdiv_rn(1.0f, a) * 448.0f, other = __shfl_xor_sync(~0u, inv, 8);
  const uint64_t im = both(upper ? other : inv), ir = both(upper ? inv : other), up = both(0x1p100f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = fmul2(m[i], im);
    // at least 2^-9 where the root, 2^-75 or more, is positive
    const float2 c = unpack_f32x2(fmul2(r[i], ir)), least = unpack_f32x2(fmul2(r[i], up));
    r[i] = pack_f32x2(fmaxf(c.x, fminf(least.x, 0x1p-9f)), fmaxf(c.y, fminf(least.y, 0x1p-9f)));
  }
  cm = codes8(m);
  cr = codes8(r);
}

// The codes of a root are steps of it, so it is the correctly rounded one; for the step
// alone an approximation to one unit in the last place does.
template <bool kExact>
__device__ __forceinline__ float root(float v) {
  if constexpr (kExact) return __fsqrt_rn(v);
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

template <int kP, int kG, int kS>
__global__ void __launch_bounds__(kThreads)
adamw_kernel(const __grid_constant__ Batch batch, const Args a) {
  wait_for_previous_kernel();
  const int chunk = blockIdx.x;
  int lo = 0, hi = batch.count - 1;  // the last tensor whose first chunk is at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (batch.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  const Tensor &t = batch.t[lo];
  const bool aligned = batch.wide[lo >> 5] >> (lo & 31) & 1;
  const int64_t i = static_cast<int64_t>(chunk - batch.first[lo]) * kChunk + threadIdx.x * 8;

  float lr = a.lr, ic1 = a.ic1, isc2 = a.isc2;
  if (a.lr_dev) lr = *a.lr_dev;
  if (a.step_dev) {
    const int64_t s = *a.step_dev;
    const float step = static_cast<float>(s < 1 ? 1 : s);
    ic1 = 1.0f / one_minus_power(a.log_b1, step);
    isc2 = 1.0f / sqrtf(one_minus_power(a.log_b2, step));
  }
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;

  constexpr bool kCodes = kS == kStateE4m3;
  const int64_t rest = t.n - i;
  const int left = rest < 8 ? static_cast<int>(rest < 0 ? 0 : rest) : 8;
  const bool wide = aligned && left == 8;
  Pairs p, g, m, v;
  float x[8];
  get8<kP>(t.p, i, wide, left, x);
  pack(x, p);
  get8<kG>(t.g, i, wide, left, x);
  pack(x, g);
  if constexpr (kCodes) {
    decode8(get_codes(t.m, i, wide, left), left ? t.ms[i >> 7] : 0.0f, m);
    decode8(get_codes(t.v, i, wide, left), left ? t.vs[i >> 7] : 0.0f, v);
  } else {
    get8<kS>(t.m, i, wide, left, x);
    pack(x, m);
    get8<kS>(t.v, i, wide, left, x);
    pack(x, v);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // each operation on the moments is rounded by itself, so that they are the same bits
    // in every compilation: a code is a step function of them
    const uint64_t d = fmul2(g[e], both(scale));
    const uint64_t v0 = kCodes ? fmul2(v[e], v[e]) : v[e];
    m[e] = sum2(fmul2(both(a.b1), m[e]), fmul2(both(a.omb1), d));
    v[e] = sum2(fmul2(both(a.b2), v0), fmul2(fmul2(both(a.omb2), d), d));
    const float2 s = unpack_f32x2(v[e]);
    const uint64_t r = pack_f32x2(root<kCodes>(s.x), root<kCodes>(s.y));
    const float2 den = unpack_f32x2(fma2(r, both(isc2), both(a.eps)));
    const float2 num = unpack_f32x2(fmul2(m[e], both(ic1)));
    const uint64_t step = pack_f32x2(__fdividef(num.x, den.x), __fdividef(num.y, den.y));
    p[e] = fma2(both(-lr), fma2(both(a.wd), p[e], step), p[e]);
    if (kCodes) v[e] = r;
  }
  unpack(p, x);
  put8<kP>(t.p, i, wide, left, x);
  if (t.copy) put8<kBf16>(t.copy, i, wide, left, x);
  if constexpr (kCodes) {
    uint2 cm, cr;
    float s;
    encode(m, v, cm, cr, s);
    put_codes(t.m, i, wide, left, cm);
    put_codes(t.v, i, wide, left, cr);
    // the group may end before the upper lanes' own values do
    const int64_t group = i >> 7;
    if ((threadIdx.x & 7) == 0 && group * 128 < t.n) (threadIdx.x & 8 ? t.vs : t.ms)[group] = s;
  } else {
    unpack(m, x);
    put8<kS>(t.m, i, wide, left, x);
    unpack(v, x);
    put8<kS>(t.v, i, wide, left, x);
  }
}

using Launch = fp8q_status (*)(const Batch &, const Args &, unsigned, cudaStream_t);
template <int kP, int kG, int kS>
fp8q_status launch(const Batch &b, const Args &a, unsigned chunks, cudaStream_t s) {
  return launch_dependent(adamw_kernel<kP, kG, kS>, dim3(chunks), dim3(kThreads), 0, s, b, a);
}
constexpr Launch kLaunch[2][2][3] = {
    {{launch<kBf16, kBf16, kStateBf16>, launch<kBf16, kBf16, kStateFp32>, launch<kBf16, kBf16, kStateE4m3>},
     {launch<kBf16, kFp32, kStateBf16>, launch<kBf16, kFp32, kStateFp32>, launch<kBf16, kFp32, kStateE4m3>}},
    {{launch<kFp32, kBf16, kStateBf16>, launch<kFp32, kBf16, kStateFp32>, launch<kFp32, kBf16, kStateE4m3>},
     {launch<kFp32, kFp32, kStateBf16>, launch<kFp32, kFp32, kStateFp32>, launch<kFp32, kFp32, kStateE4m3>}}};

uintptr_t address(const void *p) { return reinterpret_cast<uintptr_t>(p); }

// Whether two of the tensors' written ranges have a byte in common.
bool overlap(const fp8q_adamw_tensor *t, int64_t count, int p_size, int s_size) {
  std::vector<std::pair<uintptr_t, uintptr_t>> r;
  r.reserve(static_cast<size_t>(3 * count));
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const auto n = static_cast<uintptr_t>(t[i].n);
    r.emplace_back(address(t[i].p), address(t[i].p) + n * p_size);
    r.emplace_back(address(t[i].m), address(t[i].m) + n * s_size);
    r.emplace_back(address(t[i].v), address(t[i].v) + n * s_size);
  }
  std::sort(r.begin(), r.end());
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].first < r[i - 1].second) return true;
  return false;
}

fp8q_status adamw(const fp8q_adamw_tensor *tensors, int64_t count, int p_dtype, int g_dtype,
                  int state_kind, double lr, double beta1, double beta2, double eps,
                  double weight_decay, int64_t step, const float *lr_dev, const int64_t *step_dev,
                  const float *grad_scale, cudaStream_t stream) {
  const int p_size = p_dtype == kBf16 ? 2 : 4, g_size = g_dtype == kBf16 ? 2 : 4;
  const int s_size = state_kind == kStateE4m3 ? 1 : state_kind == kStateBf16 ? 2 : 4;
  const bool codes = state_kind == kStateE4m3;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    const fp8q_adamw_tensor &t = tensors[i];
    if (t.n < 0 || t.n > (int64_t{1} << 42) - total) return FP8Q_ERR_SHAPE;
    total += t.n;
  }
  for (int64_t i = 0; i < count; ++i) {
    const fp8q_adamw_tensor &t = tensors[i];
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (codes && (!t.m_scale || !t.v_scale)))
      return FP8Q_ERR_INVALID;
    if (address(t.p) % p_size || address(t.g) % g_size || address(t.m) % s_size ||
        address(t.v) % s_size || address(t.copy) % 2 ||
        (codes && (!aligned4(t.m_scale) || !aligned4(t.v_scale))))
      return FP8Q_ERR_ALIGN;
  }
  if (total == 0) return FP8Q_OK;
  if (overlap(tensors, count, p_size, s_size)) return FP8Q_ERR_INVALID;
  DeviceInfo dev;
  if (fp8q_status st = device_info(dev)) return st;

  Args a{};
  a.lr = static_cast<float>(lr);
  a.wd = static_cast<float>(weight_decay);
  a.b1 = static_cast<float>(beta1);
  a.omb1 = static_cast<float>(1.0 - beta1);
  a.b2 = static_cast<float>(beta2);
  a.omb2 = static_cast<float>(1.0 - beta2);
  a.eps = eps > 0.0 ? std::max(static_cast<float>(eps), FLT_MIN) : 0.0f;
  if (!step_dev) {
    a.ic1 = static_cast<float>(1.0 / (1.0 - std::pow(beta1, static_cast<double>(step))));
    a.isc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  }
  const double log_b[2] = {std::log(beta1), std::log(beta2)};
  for (int k = 0; k < 2; ++k) {
    float *to = k ? a.log_b2 : a.log_b1;
    to[0] = static_cast<float>(log_b[k]);
    to[1] = static_cast<float>(log_b[k] - static_cast<double>(to[0]));
  }
  a.lr_dev = lr_dev;
  a.step_dev = step_dev;
  a.grad_scale = grad_scale;

  const Launch go = kLaunch[p_dtype][g_dtype][state_kind];
  Batch b;
  int64_t chunks = 0;
  b.count = 0;
  const auto flush = [&]() {
    if (b.count == 0) return FP8Q_OK;
    const fp8q_status st = go(b, a, static_cast<unsigned>(chunks), stream);
    b.count = 0;
    chunks = 0;
    return st;
  };
  for (int64_t i = 0; i < count; ++i) {
    const fp8q_adamw_tensor &t = tensors[i];
    if (t.n == 0) continue;
    if (b.count == kBatch)
      if (fp8q_status st = flush()) return st;
    if (b.count % 32 == 0) b.wide[b.count / 32] = 0;
    const uintptr_t all = address(t.p) | address(t.g) | address(t.m) | address(t.v) | address(t.copy);
    if (all % 16 == 0) b.wide[b.count / 32] |= 1u << (b.count % 32);
    b.t[b.count] = {t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.copy, t.n};
    b.first[b.count++] = static_cast<int>(chunks);
    chunks += (t.n + kChunk - 1) / kChunk;
  }
  return flush();
}

}  // namespace
}  // namespace fp8q

extern "C" fp8q_status fp8q_adamw(const fp8q_adamw_tensor *tensors, int64_t count, int p_dtype,
                                  int g_dtype, int state_kind, double lr, double beta1,
                                  double beta2, double eps, double weight_decay, int64_t step,
                                  const float *lr_dev, const int64_t *step_dev,
                                  const float *grad_scale, void *stream) {
  using namespace fp8q;
  if ((p_dtype != kBf16 && p_dtype != kFp32) || (g_dtype != kBf16 && g_dtype != kFp32) ||
      state_kind < kStateBf16 || state_kind > kStateE4m3)
    return FP8Q_ERR_INVALID;
  const auto is_value = [](double v) { return std::fabs(v) <= static_cast<double>(FLT_MAX); };
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) ||
      !is_value(eps) || !is_value(lr) || !is_value(weight_decay) || (!step_dev && step < 1))
    return FP8Q_ERR_INVALID;
  if (count < 0) return FP8Q_ERR_SHAPE;
  if (count == 0) return FP8Q_OK;
  if (!tensors) return FP8Q_ERR_INVALID;
  if (!aligned4(lr_dev) || (reinterpret_cast<uintptr_t>(step_dev) & 7) || !aligned4(grad_scale))
    return FP8Q_ERR_ALIGN;
  try {
    return adamw(tensors, count, p_dtype, g_dtype, state_kind, lr, beta1, beta2, eps, weight_decay,
                 step, lr_dev, step_dev, grad_scale, static_cast<cudaStream_t>(stream));
  } catch (const std::exception &) {  // the list of ranges did not fit the host's memory
    return FP8Q_ERR_CUDA;
  }
}
