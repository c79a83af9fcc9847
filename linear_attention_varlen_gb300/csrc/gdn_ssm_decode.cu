// Single-token step of the selective scan over a pool of states (sm_103a): for sequence b and h = pool[state_idx[b]],
// in fp32, per channel and state
//     dt = softplus(raw + dt_bias),  h = exp(dt a) h + dt x b (stored back),  y = sum_s c h + skip x,  out = y silu(z).
// It is the scan on a document of one token that starts from the pool entry.
//
// The step reads and writes each state once and does seven operations an element: it is bound by HBM traffic. Four
// states of a channel to a thread; kRows sequences at once, so that a thread's decays are read once for them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gdn.h"
#include "elem.cuh"
#include "gdn_common.cuh"
#include "gdn_host.h"
#include "gdn_ssm.h"

namespace gdn {
namespace {

constexpr int kStepThreads = 256;

struct SsmStepParams {
  const void *x, *dt, *z, *b, *c;
  int64_t sx, sdt, sz, sb, sc;  // elements between sequences
  const float *a, *skip, *dt_bias;
  const int32_t* state_idx;
  float* pool;
  void* out;
  int32_t* status;
  int B, C, S, G, n_pool, softplus;
};

template <typename T, int kSp, int kRows, bool kVec>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(const __grid_constant__ SsmStepParams p) {
  constexpr int kQ = kSp / 4;
  const int q = threadIdx.x % kQ, c = blockIdx.x * (kStepThreads / kQ) + threadIdx.x / kQ;
  if (c >= p.C) return;  // whole channels leave
  const unsigned team = ((kQ == 32 ? 0u : 1u << kQ) - 1u) << ((threadIdx.x & 31) / kQ * kQ);
  const int g = c / (p.C / p.G), n = min(4, p.S - 4 * q);
  const auto A = load_pack<float, 4, kVec>(p.a + (int64_t)c * p.S + 4 * q, n);
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.skip ? p.skip[c] : 0.f;
  const int b0 = blockIdx.y * kRows;
  Pack<float, 4> h[kRows];
  int entry[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    entry[r] = b0 + r < p.B ? p.state_idx[b0 + r] : -1;
    if (entry[r] >= p.n_pool) entry[r] = -1;
  }
  // every load first
  Pack<T, 4> bm[kRows], cm[kRows];
  T x[kRows], dt[kRows], z[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t b = b0 + r;
    const bool live = entry[r] >= 0;
    h[r] = load_pack<float, 4, kVec>(p.pool + ((int64_t)max(entry[r], 0) * p.C + c) * p.S + 4 * q, live ? n : 0);
    x[r] = dt[r] = z[r] = from_float<T>(0.f);
    if (live) {
      x[r] = static_cast<const T*>(p.x)[b * p.sx + c];
      dt[r] = static_cast<const T*>(p.dt)[b * p.sdt + c];
      if (p.z) z[r] = static_cast<const T*>(p.z)[b * p.sz + c];
    }
    bm[r] = load_pack<T, 4, kVec>(static_cast<const T*>(p.b) + b * p.sb + g * p.S + 4 * q, live ? n : 0);
    cm[r] = load_pack<T, 4, kVec>(static_cast<const T*>(p.c) + b * p.sc + g * p.S + 4 * q, live ? n : 0);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t b = b0 + r;
    if (b >= p.B) break;
    T* out = static_cast<T*>(p.out) + b * p.C + c;
    if (entry[r] < 0) {  // skipped, reported
      if (q == 0) *out = from_float<T>(0.f);
      if (threadIdx.x == 0 && p.status) atomicCAS(p.status, 0, kErrInvalid);
      continue;
    }
    const float raw = to_float(dt[r]) + bias, delta = p.softplus ? softplus(raw) : raw, u = delta * to_float(x[r]);
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < n) {
        h[r].t[i] = fmaf(exp2_approx(delta * (kLog2e * A.t[i])), h[r].t[i], u * to_float(bm[r].t[i]));
        y = fmaf(to_float(cm[r].t[i]), h[r].t[i], y);
      }
    }
    store_pack<float, 4, kVec>(p.pool + ((int64_t)entry[r] * p.C + c) * p.S + 4 * q, h[r], n);
#pragma unroll
    for (int o = 1; o < kQ; o <<= 1) y += __shfl_xor_sync(team, y, o);
    if (q == 0) {
      y = fmaf(skip, to_float(x[r]), y);
      if (p.z) {
        const float zv = to_float(z[r]);
        y *= silu_of(zv, sigmoid(zv));
      }
      *out = from_float<T>(y);
    }
  }
}

template <typename T, int kSp>
void launch_step(const SsmStepParams& p, bool vec, cudaStream_t s) {
  constexpr int kPer = kStepThreads / (kSp / 4);
  const unsigned gx = (unsigned)((p.C + kPer - 1) / kPer);
  if (p.B == 1) {
    if (vec)
      ssm_step_kernel<T, kSp, 1, true><<<dim3(gx, 1), kStepThreads, 0, s>>>(p);
    else
      ssm_step_kernel<T, kSp, 1, false><<<dim3(gx, 1), kStepThreads, 0, s>>>(p);
  } else {
    const unsigned gy = (unsigned)((p.B + 3) / 4);
    if (vec)
      ssm_step_kernel<T, kSp, 4, true><<<dim3(gx, gy), kStepThreads, 0, s>>>(p);
    else
      ssm_step_kernel<T, kSp, 4, false><<<dim3(gx, gy), kStepThreads, 0, s>>>(p);
  }
}

template <typename T>
void launch_step_of(const SsmStepParams& p, bool vec, cudaStream_t s) {
  switch (ssm_padded(p.S)) {
    case 8: return launch_step<T, 8>(p, vec, s);
    case 16: return launch_step<T, 16>(p, vec, s);
    case 32: return launch_step<T, 32>(p, vec, s);
    default: return launch_step<T, 64>(p, vec, s);
  }
}

}  // namespace
}  // namespace gdn

extern "C" int gdn_ssm_decode_step(const void* x, const void* dt, const void* z, const float* a, const void* b,
                                   const void* c, const float* skip, const float* dt_bias, int B, int C, int S, int G,
                                   int dtype, const int64_t* strides, int dt_softplus, const int32_t* state_idx,
                                   float* state_pool, int n_pool, void* out, int32_t* status, gdn_stream_t stream) {
  using namespace gdn;
  if (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_FP16 && dtype != GDN_DTYPE_FP32) return GDN_ERR_UNSUPPORTED;
  if (B < 0 || C < 1 || S < 1 || S > kSsmMaxState || G < 1 || C % G != 0 || n_pool < 0) return GDN_ERR_INVALID_ARG;
  if (B > 4 * 65535 || (int64_t)C * S > ((int64_t)1 << 28)) return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  if (!x || !dt || !a || !b || !c || !state_idx || !state_pool || !out || n_pool == 0) return GDN_ERR_INVALID_ARG;
  const int64_t rows[5] = {C, C, C, (int64_t)G * S, (int64_t)G * S};
  int64_t st[5];
  for (int i = 0; i < 5; ++i) {
    st[i] = strides && strides[i] ? strides[i] : rows[i];
    if (st[i] < rows[i] || st[i] > ((int64_t)1 << 40)) return GDN_ERR_INVALID_ARG;
  }
  const int es = dtype == GDN_DTYPE_FP32 ? 4 : 2;
  auto al = [](const void* q, uintptr_t n) { return reinterpret_cast<uintptr_t>(q) % n == 0; };
  for (const void* q : {x, dt, z, b, c, (const void*)out})
    if (!al(q, es)) return GDN_ERR_INVALID_ARG;
  for (const void* q : {(const void*)a, (const void*)skip, (const void*)dt_bias, (const void*)state_idx, (const void*)state_pool,
                        (const void*)status})
    if (!al(q, 4)) return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {x, dt, z, a, b, c, skip, dt_bias, state_idx, out, status};
  int dev = 0;
  if (device_of(state_pool, ptrs, (int)(sizeof(ptrs) / sizeof(ptrs[0])), &dev) != kOk) return GDN_ERR_INVALID_ARG;
  DeviceGuard guard;
  if (!guard.set(dev)) return GDN_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (major != 10 || minor != 3) return GDN_ERR_UNSUPPORTED;
  const SsmStepParams p{x, dt, z, b, c, st[0], st[1], st[2], st[3], st[4], a, skip, dt_bias, state_idx, state_pool, out, status,
                        B, C, S, G, n_pool, dt_softplus != 0};
  const bool vec = S % 4 == 0 && al(a, 16) && al(state_pool, 16) && al(b, 4 * es) && al(c, 4 * es) && st[3] % 4 == 0 && st[4] % 4 == 0;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == GDN_DTYPE_BF16)
    launch_step_of<__nv_bfloat16>(p, vec, s);
  else if (dtype == GDN_DTYPE_FP16)
    launch_step_of<__half>(p, vec, s);
  else
    launch_step_of<float>(p, vec, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
