// What the state-space block's kernels share: elements in memory (bf16, fp16, fp32) and the fp32 values they stand for,
// asynchronous copies, SiLU, its slope and softplus in packed pairs, how documents fork and share pool entries.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "bw_prims.cuh"

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
// Its elements to p[0 .. n - 1]. kVec: p is aligned to the pack, and n is K or 0.
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

// Asynchronous copies of 16 bytes into shared memory.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(bw::smem_u32(dst)), "l"(src) : "memory");
}
// 16 bytes, or zeros
__device__ __forceinline__ void cp_async16_if(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(bw::smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

// How documents hang together. A fork starts where an earlier document ends, its source. Forks of documents that are no
// forks (and, in reverse, sources whose forks have none) need but one step behind the rest; deeper ones go in order.
enum { kDocFork = 1, kDocSource = 2, kDocDeepFork = 4, kDocDeepSource = 8 };
// Where a document comes in three steps over all of them: 0, 1, or 2 (one after the other).
__device__ __forceinline__ int fork_step(int kind) { return kind & kDocDeepFork ? 2 : kind & kDocFork ? 1 : 0; }
__device__ __forceinline__ int source_step(int kind) { return kind & kDocDeepSource ? 2 : kind & kDocSource ? 1 : 0; }
// kind[0 .. N - 1] by one CTA, from an init_idx that has been checked; returns (to every thread) whether some are deep.
__device__ __forceinline__ bool fork_kinds(const int32_t* init_idx, int N, int n_init, int32_t* kind) {
  for (int i = threadIdx.x; i < N; i += blockDim.x) kind[i] = 0;
  __syncthreads();
  if (!init_idx) return false;
  for (int i = threadIdx.x; i < N; i += blockDim.x)
    if (init_idx[i] >= n_init) {
      atomicOr(&kind[i], kDocFork);
      atomicOr(&kind[init_idx[i] - n_init], kDocSource);
    }
  __syncthreads();
  int deep = 0;
  for (int i = threadIdx.x; i < N; i += blockDim.x)
    if (init_idx[i] >= n_init) {
      const int j = init_idx[i] - n_init;
      if (__ldcg(&kind[j]) & kDocFork) atomicOr(&kind[i], kDocDeepFork), deep = 1;
      if (__ldcg(&kind[i]) & kDocSource) atomicOr(&kind[j], kDocDeepSource), deep = 1;
    }
  return __syncthreads_or(deep);
}

// Documents that start from the same entry of a pool, as chains in their order: link[d] = {the next one or -1, whether d
// is the first}. One warp a document, warp `warp` of `warps`.
__device__ __forceinline__ void link_pool_starts(const int32_t* init_idx, int N, int n_init, int2* link, int64_t warp, int64_t warps) {
  const int lane = threadIdx.x & 31;
  for (int64_t d = warp; d < N; d += warps) {
    const int e = init_idx ? init_idx[d] : -1;
    int next = -1, first = e >= 0 && e < n_init;
    if (first) {
      for (int64_t i = d - 32; first && i > -32; i -= 32)  // earlier documents, the nearest first
        first = !__any_sync(0xffffffffu, i + lane >= 0 && init_idx[max(i + lane, (int64_t)0)] == e);
      for (int64_t i = d + 1; next < 0 && i < N; i += 32) {
        const unsigned m = __ballot_sync(0xffffffffu, i + lane < N && init_idx[min(i + lane, (int64_t)N - 1)] == e);
        if (m) next = (int)i + __ffs(m) - 1;
      }
    }
    if (lane == 0) link[d] = make_int2(next, first);
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
// 16 bytes of elements, kept as words until they are used: pair i of them, and its place taken by two values rounded.
struct alignas(16) Words {
  uint32_t w[4];
};
template <typename T>
constexpr int kPairs = 8 / (int)sizeof(T);
template <typename T>
__device__ __forceinline__ uint64_t pair_of(const uint32_t* w, int i) {
  if constexpr (sizeof(T) == 4) {
    return bw::f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    return bw::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(w + i));
    return bw::f2_pack(f.x, f.y);
  }
}
template <typename T>
__device__ __forceinline__ uint64_t pair_of(const Words& r, int i) {
  return pair_of<T>(r.w, i);
}
template <typename T>
__device__ __forceinline__ void set_pair(uint32_t* w, int i, uint64_t v) {
  if constexpr (sizeof(T) == 4) {
    w[2 * i] = __float_as_uint(bw::f2_lo(v));
    w[2 * i + 1] = __float_as_uint(bw::f2_hi(v));
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    w[i] = bw::pack_bf16x2(bw::f2_lo(v), bw::f2_hi(v));
  } else {
    const __half2 h = __floats2half2_rn(bw::f2_lo(v), bw::f2_hi(v));
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ void set_pair(Words& r, int i, uint64_t v) {
  set_pair<T>(r.w, i, v);
}
template <typename T>
__device__ __forceinline__ void set_element(uint32_t* w, int i, T v) {  // into zeros
  if constexpr (sizeof(T) == 4)
    w[i] = __float_as_uint(v);
  else
    w[i / 2] |= (uint32_t) * reinterpret_cast<const uint16_t*>(&v) << (i % 2 * 16);
}
// K consecutive elements as words, of which the first `n` exist (zero behind them). kVec: p is aligned to them, and n is
// K or 0.
template <typename T, int K>
struct alignas(sizeof(T) * K > 16 ? 16 : sizeof(T) * K) Bits {
  uint32_t w[sizeof(T) * K / 4];
};
template <typename T, int K, bool kVec>
__device__ __forceinline__ Bits<T, K> load_bits(const T* p, int n) {
  Bits<T, K> r{};
  if constexpr (kVec) {
    if (n > 0) r = *reinterpret_cast<const Bits<T, K>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (i < n) set_element<T>(r.w, i, p[i]);
  }
  return r;
}
// Nothing is made of the words before this point: loads that stand above are all under way when the first is waited for.
template <typename T, int K>
__device__ __forceinline__ void hold(Bits<T, K>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) * K / 4); ++i) asm volatile("" : "+r"(r.w[i]));
}
__device__ __forceinline__ void hold(float& v) { asm volatile("" : "+f"(v)); }
__device__ __forceinline__ void hold(float4& v) { asm volatile("" : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w)); }
template <typename T>
__device__ __forceinline__ T element_of(const Words& r, int i) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(r.w[i]);
  } else {
    const uint16_t h = (uint16_t)(r.w[i / 2] >> (i % 2 * 16));
    return *reinterpret_cast<const T*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ void set_element(Words& r, int i, T v) {
  set_element<T>(r.w, i, v);
}

// Pairs of the same in packed arithmetic.
__device__ __forceinline__ uint64_t f2_dup(float v) { return bw::f2_pack(v, v); }
__device__ __forceinline__ uint64_t exp2_pair(uint64_t x) { return bw::f2_pack(exp2_approx(bw::f2_lo(x)), exp2_approx(bw::f2_hi(x))); }
__device__ __forceinline__ uint64_t rcp_pair(uint64_t x) { return bw::f2_pack(rcp_approx(bw::f2_lo(x)), rcp_approx(bw::f2_hi(x))); }
// 1 / (1 + e^-x), as close as the softplus below: exact at the ends (0, 1), NaN stays NaN
__device__ __forceinline__ uint64_t sigmoid_pair(uint64_t x) {
  return rcp_pair(bw::f2_add(exp2_pair(bw::f2_mul(x, f2_dup(-kLog2e))), f2_dup(1.f)));
}
__device__ __forceinline__ float at_least(float x, float lo) {  // NaN stays NaN
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(lo));
  return y;
}
// x sigmoid(x); from -128 down that is 0, and x is held there so that -inf gives 0 too
__device__ __forceinline__ uint64_t silu_pair(uint64_t x) {
  x = bw::f2_pack(at_least(bw::f2_lo(x), -128.f), at_least(bw::f2_hi(x), -128.f));
  return bw::f2_mul(x, sigmoid_pair(x));
}
// d silu / dx = sig (1 + x (1 - sig)), x held within its limits' reach
__device__ __forceinline__ uint64_t silu_slope_pair(uint64_t x, uint64_t sig) {
  float lo, hi;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(lo) : "f"(at_least(bw::f2_lo(x), -128.f)), "f"(128.f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(hi) : "f"(at_least(bw::f2_hi(x), -128.f)), "f"(128.f));
  const uint64_t rest = bw::f2_fma(sig, f2_dup(-1.f), f2_dup(1.f));
  return bw::f2_mul(sig, bw::f2_fma(bw::f2_pack(lo, hi), rest, f2_dup(1.f)));
}
// log(1 + e^r) = max(r, 0) + log1p(e^-|r|), with log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3, and the rest of
// artanh(s) / s = 1 + s^2 p(s^2) by the cubic p nearest to 1/3 + q / 5 + q^2 / 7 + ... on [0, 1/9] (relative error of the
// sum 6e-9). About 2^-21 in all from r = -5 on (the exponential's 2^-22, and its argument's rounding); further down, where
// the sum is e^r, that rounding alone is |r| 2^-24 (2^-19 at -30). NaN stays NaN.
__device__ __forceinline__ uint64_t softplus_pair(uint64_t r) {
  const float lo = bw::f2_lo(r), hi = bw::f2_hi(r);
  const uint64_t e = bw::f2_pack(exp2_approx(-kLog2e * fabsf(lo)), exp2_approx(-kLog2e * fabsf(hi)));
  const uint64_t s = bw::f2_mul(e, rcp_pair(bw::f2_add(e, f2_dup(2.f)))), q = bw::f2_mul(s, s), t = bw::f2_add(s, s);
  uint64_t p = bw::f2_fma(q, f2_dup(0.139937878f), f2_dup(0.140037894f));
  p = bw::f2_fma(p, q, f2_dup(0.200105488f));
  p = bw::f2_fma(p, q, f2_dup(0.333332121f));
  return bw::f2_add(bw::f2_pack(fmaxf(lo, 0.f), fmaxf(hi, 0.f)), bw::f2_fma(bw::f2_mul(t, q), p, t));
}

}  // namespace gdn
