// Single-token step of the decayed linear attention over a pool of states (sm_103a): for sequence b,
// value head h (key head h / (H_v / H_k)) and S = pool[state_idx[b], h], in fp32
//     S = e^{g_h} S + k v^T (stored back),  o = scale S^T q.
// It is the chunked forward on a document of one token that starts from the pool entry.
//
// The step reads and writes each state once (128 KB a sequence and head) and does 5 operations an
// element: it is bound by HBM traffic. One CTA of 256 threads per (sequence, head): thread t holds
// rows 16 (t / 32) .. +15 at columns 4 (t % 32) .. +3 in registers, so a warp reads 512 contiguous
// bytes a row and all 64 KB are in flight at once; the sum over rows goes through 4 KB of shared memory.
// 200 sequences of 64 heads (1.68 GB read and written) take 244 us, 6.9 TB/s; one sequence of 8 heads 4.4 us, a
// launch and the latency of one read.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_host.h"

namespace gdn {
namespace {

constexpr int kStepThreads = 256;

struct LaStepParams {
  const uint16_t *q, *k, *v;
  int64_t stride_q, stride_k, stride_v;  // elements between sequences
  const float* log_decay;
  const int32_t* state_idx;
  float* pool;
  uint16_t* out;
  int32_t* status;
  int n_pool, Hk, Hv;
  float scale;
};

template <bool kF16>
__device__ __forceinline__ float from16(uint16_t b) {
  if constexpr (kF16)
    return __half2float(__ushort_as_half(b));
  else
    return __bfloat162float(__ushort_as_bfloat16(b));
}
template <bool kF16>
__device__ __forceinline__ uint16_t to16(float x) {
  if constexpr (kF16)
    return __half_as_ushort(__float2half_rn(x));
  else
    return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

template <bool kF16>
__global__ void __launch_bounds__(kStepThreads) la_step_kernel(const __grid_constant__ LaStepParams p) {
  const int b = blockIdx.x / p.Hv, h = blockIdx.x % p.Hv, hk = h / (p.Hv / p.Hk);
  const int t = threadIdx.x, cg = t & 31, rg = t >> 5;
  __shared__ float s_k[kDim], s_q[kDim];
  __shared__ float4 s_red[8][32];
  const int x = p.state_idx[b];
  uint16_t* orow = p.out + ((size_t)b * p.Hv + h) * kDim;
  if (x < 0 || x >= p.n_pool) {  // skipped, reported
    if (t < kDim) orow[t] = 0;
    if (t == 0 && p.status) atomicCAS(p.status, 0, kErrInvalid);
    return;
  }
  float* S = p.pool + ((size_t)x * p.Hv + h) * kDim * kDim + (size_t)(16 * rg) * kDim + 4 * cg;
  float4 st[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) st[i] = *reinterpret_cast<const float4*>(S + (size_t)i * kDim);
  const float lam = expf(p.log_decay[h]);
  if (t < kDim)
    s_k[t] = from16<kF16>(p.k[(size_t)b * p.stride_k + hk * kDim + t]);
  else
    s_q[t - kDim] = from16<kF16>(p.q[(size_t)b * p.stride_q + hk * kDim + t - kDim]) * p.scale;
  float4 v4;
  {
    const ushort4 raw = *reinterpret_cast<const ushort4*>(p.v + (size_t)b * p.stride_v + h * kDim + 4 * cg);
    v4 = make_float4(from16<kF16>(raw.x), from16<kF16>(raw.y), from16<kF16>(raw.z), from16<kF16>(raw.w));
  }
  __syncthreads();
  float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float kr = s_k[16 * rg + i], qr = s_q[16 * rg + i];
    st[i].x = fmaf(kr, v4.x, lam * st[i].x);
    st[i].y = fmaf(kr, v4.y, lam * st[i].y);
    st[i].z = fmaf(kr, v4.z, lam * st[i].z);
    st[i].w = fmaf(kr, v4.w, lam * st[i].w);
    *reinterpret_cast<float4*>(S + (size_t)i * kDim) = st[i];
    oo.x = fmaf(qr, st[i].x, oo.x);
    oo.y = fmaf(qr, st[i].y, oo.y);
    oo.z = fmaf(qr, st[i].z, oo.z);
    oo.w = fmaf(qr, st[i].w, oo.w);
  }
  s_red[rg][cg] = oo;
  __syncthreads();
  if (t < kDim) {
    float o = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) o += reinterpret_cast<const float*>(&s_red[r][0])[t];
    orow[t] = to16<kF16>(o);
  }
}

}  // namespace
}  // namespace gdn

extern "C" int gdn_la_decode_step(const void* q, const void* k, const void* v, const float* log_decay, int B, int H_k,
                                  int H_v, int head_dim, int dtype, const int64_t* strides, const int32_t* state_idx,
                                  float* state_pool, int n_pool, float scale, void* out, int32_t* status,
                                  gdn_stream_t stream) {
  using namespace gdn;
  if (head_dim != kDim) return GDN_ERR_UNSUPPORTED;
  if (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_FP16) return GDN_ERR_UNSUPPORTED;
  if (B < 0 || H_k < 1 || H_v < 1 || H_v % H_k != 0 || n_pool < 0 || scale != scale) return GDN_ERR_INVALID_ARG;
  if ((int64_t)B * H_v > (int64_t)INT32_MAX) return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  if (!q || !k || !v || !log_decay || !state_idx || !state_pool || !out || n_pool == 0) return GDN_ERR_INVALID_ARG;
  int64_t st[3];
  const int heads[3] = {H_k, H_k, H_v};
  for (int i = 0; i < 3; ++i) {
    st[i] = strides && strides[i] ? strides[i] : (int64_t)heads[i] * kDim;
    if (st[i] < (int64_t)heads[i] * kDim || st[i] % 8 != 0) return GDN_ERR_INVALID_ARG;
  }
  auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al16(q) || !al16(k) || !al16(v) || !al16(out) || !al16(state_pool)) return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, log_decay, state_idx, out, status};
  int dev = 0;
  if (device_of(state_pool, ptrs, (int)(sizeof(ptrs) / sizeof(ptrs[0])), &dev) != kOk) return GDN_ERR_INVALID_ARG;
  DeviceGuard guard;
  if (!guard.set(dev)) return GDN_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (major != 10 || minor != 3) return GDN_ERR_UNSUPPORTED;
  const LaStepParams p{static_cast<const uint16_t*>(q),
                       static_cast<const uint16_t*>(k),
                       static_cast<const uint16_t*>(v),
                       st[0],
                       st[1],
                       st[2],
                       log_decay,
                       state_idx,
                       state_pool,
                       static_cast<uint16_t*>(out),
                       status,
                       n_pool,
                       H_k,
                       H_v,
                       scale};
  const unsigned grid = (unsigned)(B * H_v);
  if (dtype == GDN_DTYPE_FP16)
    la_step_kernel<true><<<grid, kStepThreads, 0, (cudaStream_t)stream>>>(p);
  else
    la_step_kernel<false><<<grid, kStepThreads, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
