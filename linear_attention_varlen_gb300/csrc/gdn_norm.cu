// Root-mean-square norm with the residual's addition, and its backward (sm_103a). Per row of D:
//     h = x + r,  y = w h rs,  rs = (mean(h^2) + eps)^{-1/2}
// h is rounded once to the inputs' type for the residual stream; y is formed from the fp32 sum and
// rounded once, to the inputs' type or to e4m3 with a scale amax / 448 for the row or for each 128
// columns (448 is e4m3's largest value; a row or group of zeros takes scale 1). Backward, from the h
// the forward left:
//     dx = rs w dy - h rs^3 mean(w dy h) + dh,   dw = sum over rows of dy h rs.
//
// Both read each input once and write each output once and do a few operations an element: they are
// bound by HBM traffic. A thread holds 8 consecutive elements a vector in registers, in fp32; a row
// of up to 1024 elements is one warp's, a longer one a CTA's.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_host.h"

namespace gdn {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kNormMaxD = 32768;
constexpr int kRowThreads = 512;  // most threads to a row
constexpr int kGroup = 128;  // columns to one scale
constexpr int kWarpRows = 4;  // rows of a CTA whose warps own a row each

// ------------------------------------------------------------------------------ elements

template <typename T>
struct Vec8;  // 8 elements as raw bits
template <>
struct Vec8<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Vec8<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Vec8<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// columns c .. c + 7 of a row of D elements (zero past its end); kVec: the row is aligned and D a multiple of 8
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* row, int c, int D, float* f) {
  if constexpr (kVec) {
    if (c < D) {
      alignas(16) T t[8];
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(row + c)[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = Vec8<T>::get(t[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < D ? Vec8<T>::get(row[c + i]) : 0.f;
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* row, int c, int D, const float* f) {
  if constexpr (kVec) {
    if (c < D) {
      alignas(16) T t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = Vec8<T>::put(f[i]);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        reinterpret_cast<uint4*>(row + c)[i] = reinterpret_cast<const uint4*>(t)[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) row[c + i] = Vec8<T>::put(f[i]);
  }
}
template <bool kVec>
__device__ __forceinline__ void load_w8(const void* w, int dtype, int c, int D, float* f) {
  if (dtype == GDN_DTYPE_BF16)
    load8<__nv_bfloat16, kVec>(static_cast<const __nv_bfloat16*>(w), c, D, f);
  else if (dtype == GDN_DTYPE_FP16)
    load8<__half, kVec>(static_cast<const __half*>(w), c, D, f);
  else
    load8<float, kVec>(static_cast<const float*>(w), c, D, f);
}

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum (or maximum) over the threads of a row: a warp, or the CTA through `s` (33 floats).
template <bool kWarp>
__device__ __forceinline__ float row_sum(float x, float* s) {
  x = warp_sum(x);
  if constexpr (kWarp) return x;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (lane == 0) s[wid] = x;
  __syncthreads();
  float t = lane < nw ? s[lane] : 0.f;
  t = warp_sum(t);
  __syncthreads();
  return t;
}
template <bool kWarp>
__device__ __forceinline__ float row_max(float x, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  if constexpr (kWarp) return x;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (lane == 0) s[wid] = x;
  __syncthreads();
  float t = lane < nw ? s[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, o));
  __syncthreads();
  return t;
}

// ------------------------------------------------------------------------------ forward

struct NormFwdParams {
  const void *x, *r, *w;
  void *h, *y;
  float* scales;
  int64_t T;
  int D, w_dtype, quant;
  float eps;
};

template <typename T, int kNv, bool kWarp, bool kVec>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kRowThreads) norm_fwd_kernel(const __grid_constant__ NormFwdParams p) {
  __shared__ float s_red[33];
  const int tpr = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarp ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.T) return;
  const T* x = static_cast<const T*>(p.x) + row * p.D;
  float v[kNv][8];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < kNv; ++j) load8<T, kVec>(x, (t + j * tpr) * 8, p.D, v[j]);
  if (p.r) {
    const T* r = static_cast<const T*>(p.r) + row * p.D;
    T* h = static_cast<T*>(p.h) + row * p.D;
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
      float u[8];
      load8<T, kVec>(r, (t + j * tpr) * 8, p.D, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] += u[i];
    }
#pragma unroll
    for (int j = 0; j < kNv; ++j) store8<T, kVec>(h, (t + j * tpr) * 8, p.D, v[j]);
  }
#pragma unroll
  for (int j = 0; j < kNv; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[j][i], v[j][i], ss);
  const float rs = rsqrtf(row_sum<kWarp>(ss, s_red) / (float)p.D + p.eps);
#pragma unroll
  for (int j = 0; j < kNv; ++j) {
    float w[8];
    load_w8<kVec>(p.w, p.w_dtype, (t + j * tpr) * 8, p.D, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rs * w[i];
  }
  if (p.quant == GDN_QUANT_NONE) {
    T* y = static_cast<T*>(p.y) + row * p.D;
#pragma unroll
    for (int j = 0; j < kNv; ++j) store8<T, kVec>(y, (t + j * tpr) * 8, p.D, v[j]);
    return;
  }
  float am[kNv];
#pragma unroll
  for (int j = 0; j < kNv; ++j) {
    am[j] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) am[j] = max_nan(am[j], fabsf(v[j][i]));
  }
  if (p.quant == GDN_QUANT_ROW) {
    float m = am[0];
#pragma unroll
    for (int j = 1; j < kNv; ++j) m = max_nan(m, am[j]);
    m = row_max<kWarp>(m, s_red);
#pragma unroll
    for (int j = 0; j < kNv; ++j) am[j] = m;
    if (t == 0) p.scales[row] = m > 0.f ? m / kE4m3Max : 1.f;
  } else {
    const int groups = (p.D + kGroup - 1) / kGroup;
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) am[j] = max_nan(am[j], __shfl_xor_sync(0xffffffffu, am[j], o));
      const int g = (t + j * tpr) / 16;
      if ((t & 15) == 0 && g < groups) p.scales[row * groups + g] = am[j] > 0.f ? am[j] / kE4m3Max : 1.f;
    }
  }
  uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.D;
#pragma unroll
  for (int j = 0; j < kNv; ++j) {
    const float sc = am[j] > 0.f ? am[j] / kE4m3Max : 1.f;
    alignas(8) __nv_fp8x2_storage_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[j][2 * i] / sc, v[j][2 * i + 1] / sc), __NV_SATFINITE, __NV_E4M3);
    const int c = (t + j * tpr) * 8;
    if constexpr (kVec) {
      if (c < p.D) *reinterpret_cast<uint2*>(y + c) = *reinterpret_cast<const uint2*>(b);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < p.D) y[c + i] = reinterpret_cast<const uint8_t*>(b)[i];
    }
  }
}

// ------------------------------------------------------------------------------ backward

struct NormBwdParams {
  const void *h, *w, *dy, *dh;
  void* dx;
  float *part, *dw;
  int64_t T;
  int D, w_dtype, parts;
  float eps;
};

// Each CTA takes rows blockIdx.x, + gridDim.x, ... (a warp-row CTA kWarpRows at a time) and keeps
// the weight gradient's part of its own columns in registers; the parts are summed in a fixed order.
template <typename T, int kNv, bool kWarp, bool kVec>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kRowThreads) norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float s_red[33], s_red2[33];
  const int tpr = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first = kWarp ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = kWarp ? (int64_t)gridDim.x * kWarpRows : gridDim.x;
  float w[kNv][8], dw[kNv][8];
#pragma unroll
  for (int j = 0; j < kNv; ++j) {
    load_w8<kVec>(p.w, p.w_dtype, (t + j * tpr) * 8, p.D, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }
  for (int64_t row = first; row < p.T; row += step) {
    const T* h = static_cast<const T*>(p.h) + row * p.D;
    const T* dy = static_cast<const T*>(p.dy) + row * p.D;
    T* dx = static_cast<T*>(p.dx) + row * p.D;
    float hv[kNv][8], gv[kNv][8];
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
      load8<T, kVec>(h, (t + j * tpr) * 8, p.D, hv[j]);
      load8<T, kVec>(dy, (t + j * tpr) * 8, p.D, gv[j]);
    }
#pragma unroll
    for (int j = 0; j < kNv; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(hv[j][i], hv[j][i], ss);
        sg = fmaf(hv[j][i] * w[j][i], gv[j][i], sg);
      }
    ss = row_sum<kWarp>(ss, s_red);
    sg = row_sum<kWarp>(sg, s_red2);
    const float rs = rsqrtf(ss / (float)p.D + p.eps);
    const float c = rs * rs * rs * (sg / (float)p.D);
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
      float o[8], e[8];
      if (p.dh) load8<T, kVec>(static_cast<const T*>(p.dh) + row * p.D, (t + j * tpr) * 8, p.D, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[j][i] = fmaf(gv[j][i] * rs, hv[j][i], dw[j][i]);
        o[i] = fmaf(rs * w[j][i], gv[j][i], -c * hv[j][i]);
        if (p.dh) o[i] += e[i];
      }
      store8<T, kVec>(dx, (t + j * tpr) * 8, p.D, o);
    }
  }
  const int64_t part = kWarp ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
#pragma unroll
  for (int j = 0; j < kNv; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = (t + j * tpr) * 8 + i;
      if (c < p.D) p.part[part * p.D + c] = dw[j][i];
    }
}

// dw: 32 columns to a CTA, 8 warps sum every eighth part, then the warps' sums in order
__global__ void __launch_bounds__(256) norm_dw_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < p.D)
    for (int i = wid; i < p.parts; i += 8) a += p.part[(size_t)i * p.D + c];
  s[wid][lane] = a;
  __syncthreads();
  if (wid == 0 && c < p.D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += s[i][lane];
    p.dw[c] = a;
  }
}

// ------------------------------------------------------------------------------ host

struct NormShape {
  bool warp;
  int threads, nv;  // threads to a row and vectors of 8 to a thread
};
// A row of up to 1024 elements is one warp's (4 vectors a thread); a longer one takes a CTA of
// D / 16 threads (2 vectors each), from 128 up to 512, then more vectors.
NormShape norm_shape(int D) {
  const int vecs = (D + 7) / 8;
  if (vecs <= 128) return {true, 32, vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4};
  int threads = 128;
  while (threads < kRowThreads && threads * 2 < vecs) threads *= 2;
  int nv = 2;
  while (threads * nv < vecs) nv *= 2;
  return {false, threads, nv};
}
int norm_parts(int64_t T, int D, int sms) {
  const NormShape s = norm_shape(D);
  const int64_t rows = s.warp ? (T + kWarpRows - 1) / kWarpRows : T;
  const int64_t most = (int64_t)sms * (s.warp ? 8 : 2048 / s.threads > 4 ? 4 : 2048 / s.threads);
  return (int)(rows < most ? (rows < 1 ? 1 : rows) : most);  // CTAs
}

bool al(const void* p, uintptr_t b) { return (reinterpret_cast<uintptr_t>(p) % b) == 0; }
size_t esize(int dtype) { return dtype == GDN_DTYPE_FP32 ? 4 : 2; }
bool dtype_ok(int d) { return d == GDN_DTYPE_BF16 || d == GDN_DTYPE_FP16 || d == GDN_DTYPE_FP32; }

int check_device(const void* anchor, const void* const* ptrs, int n, DeviceGuard& guard, int* sms) {
  int dev = 0;
  if (device_of(anchor, ptrs, n, &dev) != kOk) return GDN_ERR_INVALID_ARG;
  if (!guard.set(dev)) return GDN_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return GDN_ERR_CUDA;
  return (major == 10 && minor == 3) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

template <typename T, bool kVec, typename F>
void by_shape(const NormShape& s, F&& f) {
  // f(kNv, kWarp) as integral constants
  using std::integral_constant;
  if (s.warp) {
    if (s.nv == 1)
      f(integral_constant<int, 1>{}, integral_constant<bool, true>{});
    else if (s.nv == 2)
      f(integral_constant<int, 2>{}, integral_constant<bool, true>{});
    else
      f(integral_constant<int, 4>{}, integral_constant<bool, true>{});
  } else {
    if (s.nv == 2)
      f(integral_constant<int, 2>{}, integral_constant<bool, false>{});
    else if (s.nv == 4)
      f(integral_constant<int, 4>{}, integral_constant<bool, false>{});
    else
      f(integral_constant<int, 8>{}, integral_constant<bool, false>{});
  }
}

template <typename T, bool kVec>
void launch_fwd(const NormFwdParams& p, cudaStream_t st) {
  const NormShape s = norm_shape(p.D);
  by_shape<T, kVec>(s, [&](auto nv, auto warp) {
    const unsigned grid = (unsigned)(warp ? (p.T + kWarpRows - 1) / kWarpRows : p.T);
    norm_fwd_kernel<T, nv, warp, kVec><<<grid, warp ? 32 * kWarpRows : s.threads, 0, st>>>(p);
  });
}
template <typename T, bool kVec>
void launch_bwd(const NormBwdParams& p, int ctas, cudaStream_t st) {
  const NormShape s = norm_shape(p.D);
  by_shape<T, kVec>(s, [&](auto nv, auto warp) {
    norm_bwd_kernel<T, nv, warp, kVec><<<ctas, warp ? 32 * kWarpRows : s.threads, 0, st>>>(p);
  });
}

}  // namespace
}  // namespace gdn

extern "C" int gdn_rmsnorm_fwd(const void* x, const void* residual, const void* w, int64_t T, int D, int dtype,
                               int w_dtype, float eps, void* residual_out, void* y, int quant, float* scales,
                               gdn_stream_t stream) {
  using namespace gdn;
  if (!dtype_ok(dtype) || !dtype_ok(w_dtype)) return GDN_ERR_UNSUPPORTED;
  if (D > kNormMaxD) return GDN_ERR_UNSUPPORTED;
  if (T < 0 || T > (int64_t)INT32_MAX || D < 1 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (quant != GDN_QUANT_NONE && quant != GDN_QUANT_ROW && quant != GDN_QUANT_GROUP) return GDN_ERR_INVALID_ARG;
  if (T == 0) return GDN_OK;
  if (!x || !w || !y || (residual != nullptr) != (residual_out != nullptr)) return GDN_ERR_INVALID_ARG;
  if ((quant != GDN_QUANT_NONE) != (scales != nullptr)) return GDN_ERR_INVALID_ARG;
  const uintptr_t e = esize(dtype);
  if (!al(x, e) || !al(residual, e) || !al(residual_out, e) || !al(w, esize(w_dtype)) || !al(scales, 4) ||
      (quant == GDN_QUANT_NONE && !al(y, e)))
    return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {residual, w, residual_out, y, scales};
  DeviceGuard guard;
  int sms = 0;
  const int rc = check_device(x, ptrs, 5, guard, &sms);
  if (rc != GDN_OK) return rc;
  const NormFwdParams p{x, residual, w, residual_out, y, scales, T, D, w_dtype, quant, eps};
  const bool vec = D % 8 == 0 && al(x, 16) && al(residual, 16) && al(residual_out, 16) && al(w, 16) &&
                   al(y, quant == GDN_QUANT_NONE ? 16 : 8);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == GDN_DTYPE_BF16)
    vec ? launch_fwd<__nv_bfloat16, true>(p, st) : launch_fwd<__nv_bfloat16, false>(p, st);
  else if (dtype == GDN_DTYPE_FP16)
    vec ? launch_fwd<__half, true>(p, st) : launch_fwd<__half, false>(p, st);
  else
    vec ? launch_fwd<float, true>(p, st) : launch_fwd<float, false>(p, st);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" size_t gdn_rmsnorm_workspace_size(int64_t T, int D) {
  if (T < 0 || T > (int64_t)INT32_MAX || D < 1 || D > gdn::kNormMaxD) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    sms = 152;
  }
  const size_t parts = (size_t)gdn::norm_parts(T, D, sms) * (gdn::norm_shape(D).warp ? gdn::kWarpRows : 1);
  return parts * D * sizeof(float);
}

extern "C" int gdn_rmsnorm_bwd(const void* h, const void* w, const void* dy, const void* dh, int64_t T, int D,
                               int dtype, int w_dtype, float eps, void* dx, float* dw, void* workspace,
                               size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  if (!dtype_ok(dtype) || !dtype_ok(w_dtype)) return GDN_ERR_UNSUPPORTED;
  if (D > kNormMaxD) return GDN_ERR_UNSUPPORTED;
  if (T < 0 || T > (int64_t)INT32_MAX || D < 1 || !(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  if (!w || !dw || !workspace || (T > 0 && (!h || !dy || !dx))) return GDN_ERR_INVALID_ARG;
  const uintptr_t e = esize(dtype);
  if (!al(h, e) || !al(dy, e) || !al(dh, e) || !al(dx, e) || !al(w, esize(w_dtype)) || !al(dw, 4) || !al(workspace, 256))
    return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {h, w, dy, dh, dx, dw};
  DeviceGuard guard;
  int sms = 0;
  const int rc = check_device(workspace, ptrs, 6, guard, &sms);
  if (rc != GDN_OK) return rc;
  const int ctas = norm_parts(T, D, sms);
  const int parts = ctas * (norm_shape(D).warp ? kWarpRows : 1);
  if (ws_bytes < (size_t)parts * D * sizeof(float)) return GDN_ERR_WORKSPACE;
  const NormBwdParams p{h, w, dy, dh, dx, static_cast<float*>(workspace), dw, T, D, w_dtype, parts, eps};
  const bool vec = D % 8 == 0 && al(h, 16) && al(dy, 16) && al(dh, 16) && al(dx, 16) && al(w, 16);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == GDN_DTYPE_BF16)
    vec ? launch_bwd<__nv_bfloat16, true>(p, ctas, st) : launch_bwd<__nv_bfloat16, false>(p, ctas, st);
  else if (dtype == GDN_DTYPE_FP16)
    vec ? launch_bwd<__half, true>(p, ctas, st) : launch_bwd<__half, false>(p, ctas, st);
  else
    vec ? launch_bwd<float, true>(p, ctas, st) : launch_bwd<float, false>(p, ctas, st);
  norm_dw_kernel<<<(D + 31) / 32, 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
