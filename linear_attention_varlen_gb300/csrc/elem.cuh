// Elements in memory (bf16, fp16, fp32) and the fp32 values they stand for; the activation SiLU and its slope.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace gdn {

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}

// K consecutive elements as they lie in memory
template <typename T, int K>
struct alignas(sizeof(T) * K > 16 ? 16 : sizeof(T) * K) Pack {
  T t[K];
};
// Elements p[0 .. K - 1], of which the first `n` exist (zero behind them). kVec: p is aligned to the pack, and n is
// K or 0.
template <typename T, int K, bool kVec>
__device__ __forceinline__ Pack<T, K> load_pack(const T* p, int n) {
  Pack<T, K> r;
  if (kVec && n >= K) {
    r = *reinterpret_cast<const Pack<T, K>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < K; ++i) r.t[i] = i < n ? p[i] : from_float<T>(0.f);
  }
  return r;
}
template <typename T, int K, bool kVec>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, K>& r, int n) {
  if (kVec && n >= K) {
    *reinterpret_cast<Pack<T, K>*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (i < n) p[i] = r.t[i];
  }
}

// 2^x, relative error about 2^-22
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504088896340736f;

// 1 / x within one unit
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-x): exact at the ends (0, 1), NaN stays NaN
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + exp2_approx(-kLog2e * x)); }
// x sigmoid(x); its limit 0 for x = -inf
__device__ __forceinline__ float silu_of(float x, float sig) { return sig == 0.f ? 0.f : x * sig; }
// d silu / dx = sig (1 + x (1 - sig)); its limits 0 and 1 at the infinities
__device__ __forceinline__ float silu_slope(float x, float sig) {
  return sig == 0.f || sig == 1.f ? sig : sig * fmaf(x, 1.f - sig, 1.f);
}

// log(1 + e^r) = max(r, 0) + log1p(e^-|r|), with log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3, by its series
// 2 s (1 + s^2 / 3 + s^4 / 5 + ...), cut where the next term is below 2^-25 of the sum. Relative error about 2^-21 (the
// exponential's, and its argument's rounding); NaN stays NaN.
__device__ __forceinline__ float softplus(float r) {
  const float e = exp2_approx(-kLog2e * fabsf(r));
  const float s = e * rcp_approx(2.f + e), q = s * s;
  float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
  p = fmaf(p, q, 1.f / 9.f);
  p = fmaf(p, q, 1.f / 7.f);
  p = fmaf(p, q, 1.f / 5.f);
  p = fmaf(p, q, 1.f / 3.f);
  const float t = s + s;
  return fmaxf(r, 0.f) + fmaf(t * q, p, t);
}

}  // namespace gdn
