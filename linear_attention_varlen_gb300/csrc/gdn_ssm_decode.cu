// Single-token step of the selective scan over a pool of states (sm_103a): for sequence b and h = pool[state_idx[b]],
// in fp32, per channel and state
//     dt = softplus(raw + dt_bias),  h = exp(dt a) h + dt x b (stored back),  y = sum_s c h + skip x,  out = y silu(z).
// It is the scan on a document of one token that starts from the pool entry.
//
// The step reads and writes each state once and does seven operations an element: it is bound by HBM traffic as long as
// what is done for each channel stays small beside it, and that all loads are under way before the first is waited for
// (67 us without that). A thread takes four states of two channels of one sequence, in packed pairs.
// Measured: 200 sequences of 8192 channels of 16 states 42 us (223 MB, 5.3 TB/s); one sequence of 2048 channels 2 us.
// Several sequences to a CTA, one after the other or the next one's loads ahead, took 70 to 115 us.
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

constexpr int kStepThreads = 128;

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

// kVec: states, maps and pairs of channels are aligned.
template <typename T, int kSp, bool kVec>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(const __grid_constant__ SsmStepParams p) {
  using bw::f2_fma;
  using bw::f2_hi;
  using bw::f2_lo;
  using bw::f2_mul;
  using bw::f2_pack;
  constexpr int kQ = kSp / 4;
  const int q = threadIdx.x % kQ, pair = blockIdx.x * (kStepThreads / kQ) + threadIdx.x / kQ;
  const int Cg = p.C / p.G, g = blockIdx.z, cg = 2 * pair;
  if (cg >= Cg) return;  // whole teams leave
  const unsigned team = ((1u << kQ) - 1u) << ((threadIdx.x & 31) / kQ * kQ);
  const int two = cg + 1 < Cg ? 1 : 0, n = min(4, p.S - 4 * q);
  const int64_t b = blockIdx.y;
  const int k = 1 + two;  // channels
  const int64_t c0 = (int64_t)g * Cg;
  int entry = p.state_idx[b];
  Bits<float, 4> h[2], A[2];
#pragma unroll
  for (int d = 0; d < 2; ++d) A[d] = load_bits<float, 4, kVec>(p.a + c0 * p.S + (cg * p.S + 4 * q) + d * p.S, d < k ? n : 0);
  auto bm = load_bits<T, 4, kVec>(static_cast<const T*>(p.b) + (b * p.sb + (int64_t)g * p.S) + 4 * q, n);
  auto cm = load_bits<T, 4, kVec>(static_cast<const T*>(p.c) + (b * p.sc + (int64_t)g * p.S) + 4 * q, n);
  auto xr = load_bits<T, 2, kVec>(static_cast<const T*>(p.x) + (b * p.sx + c0) + cg, k);
  auto dr = load_bits<T, 2, kVec>(static_cast<const T*>(p.dt) + (b * p.sdt + c0) + cg, k);
  auto zr = load_bits<T, 2, kVec>(static_cast<const T*>(p.z) + (b * p.sz + c0) + cg, p.z ? k : 0);
  Bits<float, 2> bias = load_bits<float, 2, false>(p.dt_bias + c0 + cg, p.dt_bias ? k : 0);
  Bits<float, 2> skip = load_bits<float, 2, false>(p.skip + c0 + cg, p.skip ? k : 0);
  T* out = static_cast<T*>(p.out) + (b * p.C + c0) + cg;
  if (entry < 0 || entry >= p.n_pool) {  // skipped, reported
    if (q == 0) store_pack<T, 2, kVec>(out, Pack<T, 2>{}, k);
    if (threadIdx.x == 0 && p.status) atomicCAS(p.status, 0, kErrInvalid);
    return;
  }
  float* state = p.pool + ((int64_t)entry * p.C + c0) * p.S + (cg * p.S + 4 * q);
#pragma unroll
  for (int d = 0; d < 2; ++d) h[d] = load_bits<float, 4, kVec>(state + d * p.S, d < k ? n : 0);
  hold(h[0]), hold(h[1]), hold(A[0]), hold(A[1]), hold(bm), hold(cm), hold(xr), hold(dr), hold(zr), hold(bias), hold(skip);
  uint64_t delta = bw::f2_add(pair_of<T>(dr.w, 0), pair_of<float>(bias.w, 0));
  if (p.softplus) delta = softplus_pair(delta);
  const uint64_t x = pair_of<T>(xr.w, 0), u = f2_mul(delta, x);
  float y[2];
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const uint64_t dd = f2_dup((d ? f2_hi(delta) : f2_lo(delta)) * kLog2e), uu = f2_dup(d ? f2_hi(u) : f2_lo(u));
    uint64_t y2 = 0;
    Pack<float, 4> r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t e = exp2_pair(f2_mul(dd, pair_of<float>(A[d].w, i)));
      const uint64_t v = f2_fma(e, pair_of<float>(h[d].w, i), f2_mul(uu, pair_of<T>(bm.w, i)));
      y2 = f2_fma(pair_of<T>(cm.w, i), v, y2);
      r.t[2 * i] = f2_lo(v), r.t[2 * i + 1] = f2_hi(v);
    }
    y[d] = bw::f2_sum(y2);
    store_pack<float, 4, kVec>(state + d * p.S, r, d < k ? n : 0);
  }
#pragma unroll
  for (int o = 1; o < kQ; o <<= 1) {
    y[0] += __shfl_xor_sync(team, y[0], o);
    y[1] += __shfl_xor_sync(team, y[1], o);
  }
  if (q == 0) {
    uint64_t r = f2_fma(pair_of<float>(skip.w, 0), x, f2_pack(y[0], y[1]));
    if (p.z) r = f2_mul(r, silu_pair(pair_of<T>(zr.w, 0)));
    Pack<T, 2> o;
    o.t[0] = from_float<T>(f2_lo(r)), o.t[1] = from_float<T>(f2_hi(r));
    store_pack<T, 2, kVec>(out, o, k);
  }
}

template <typename T, int kSp>
void launch_step(const SsmStepParams& p, bool vec, cudaStream_t s) {
  constexpr int kPer = kStepThreads / (kSp / 4);
  const int pairs = (p.C / p.G + 1) / 2;
  const dim3 grid((unsigned)((pairs + kPer - 1) / kPer), (unsigned)p.B, (unsigned)p.G);
  if (vec)
    ssm_step_kernel<T, kSp, true><<<grid, kStepThreads, 0, s>>>(p);
  else
    ssm_step_kernel<T, kSp, false><<<grid, kStepThreads, 0, s>>>(p);
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
  if (B > 65535 || G > 65535 || (int64_t)C * S > ((int64_t)1 << 28)) return GDN_ERR_INVALID_ARG;
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
  bool vec = S % 4 == 0 && C / G % 2 == 0 && al(a, 16) && al(state_pool, 16) && al(b, 4 * es) && al(c, 4 * es) &&
             st[3] % 4 == 0 && st[4] % 4 == 0;
  for (const void* q : {x, dt, z, (const void*)out}) vec = vec && al(q, 2 * es);
  for (int i = 0; i < 3; ++i) vec = vec && (st[i] % 2 == 0 || (i == 2 && !z));
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == GDN_DTYPE_BF16)
    launch_step_of<__nv_bfloat16>(p, vec, s);
  else if (dtype == GDN_DTYPE_FP16)
    launch_step_of<__half>(p, vec, s);
  else
    launch_step_of<float>(p, vec, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
