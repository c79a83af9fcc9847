// Root-mean-square norm of each group of columns with its gate, and its backward (sm_103a). Per row and group of n
// consecutive columns (a head, or the whole row), with gate = silu(z):
//     norm first: u = x,       y = w u rs gate          rs = (mean(u^2) + eps)^{-1/2}
//     gate first: u = x gate,  y = w u rs
// backward with dn = dy gate (norm first) or dy (gate first), hat = u rs, g = w dn:
//     du = rs (g - hat mean(g hat)),  dw = sum over rows (and groups, where they share w) of dn hat
//     norm first: dx = du, dz = dy hat w silu'(z);   gate first: dx = du gate, dz = du x silu'(z)
//
// Both read each input once and write each output once: bound by HBM traffic. A team of threads (a power of two: part
// of a warp, a warp or a CTA) takes one group of columns down the rows with its weights, and in the backward their
// gradient, in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gdn.h"
#include "bw_prims.cuh"
#include "elem.cuh"
#include "gdn_common.cuh"
#include "gdn_host.h"

namespace gdn {
namespace {

constexpr int kMaxGroup = 16384;
constexpr int kWarpTeamThreads = 256;  // threads of a CTA whose teams lie within a warp
constexpr int kMaxTeam = 512;

struct GnormHeader {
  int32_t status;
  int32_t pad[63];
};

struct GnormParams {
  const void *x, *z, *dy, *w;
  int64_t sx, sz, sdy;  // elements between rows
  void *y, *dx, *dz;
  float *part, *dw;
  GnormHeader* hd;
  int64_t T, rows;  // rows; teams to a group of columns
  int D, group, ng, w_dtype, shared, gate_first;
  float eps;
};

__device__ __forceinline__ float load_w(const void* w, int dtype, int64_t i) {
  if (dtype == GDN_DTYPE_BF16) return to_float(static_cast<const __nv_bfloat16*>(w)[i]);
  if (dtype == GDN_DTYPE_FP16) return to_float(static_cast<const __half*>(w)[i]);
  return static_cast<const float*>(w)[i];
}

// A thread's share of a group: kNv vectors of 16 bytes, vector v of the team's lane at column (v L + lane) K (kVec), or
// the same number of elements one at a time, a team's lanes side by side.
template <typename T>
constexpr int kElems = 16 / (int)sizeof(T);

template <typename T, int kNv, bool kVec>
struct Share {
  static constexpr int K = kElems<T>;
  int lane, L, n;
  __device__ __forceinline__ int col(int v, int i) const { return kVec ? (v * L + lane) * K + i : (v * K + i) * L + lane; }
  __device__ __forceinline__ Pack<T, K> load(const T* p, int v, bool live) const {
    Pack<T, K> r{};
    if constexpr (kVec) {
      if (live && col(v, 0) < n) r = *reinterpret_cast<const Pack<T, K>*>(p + col(v, 0));
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (live && col(v, i) < n) r.t[i] = p[col(v, i)];
    }
    return r;
  }
  __device__ __forceinline__ void store(T* p, int v, const Pack<T, K>& r) const {
    if constexpr (kVec) {
      if (col(v, 0) < n) *reinterpret_cast<Pack<T, K>*>(p + col(v, 0)) = r;
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (col(v, i) < n) p[col(v, i)] = r.t[i];
    }
  }
};

// Sums over the team; every thread of it gets them. `buf` has room for two rows of a CTA's warps, used in turn, so that
// one barrier a row is enough.
template <int kN>
__device__ __forceinline__ void team_sum(float (&v)[kN], int L, float (*buf)[kN][kMaxTeam / 32], int& turn) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= L) break;
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (L <= 32) return;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, W = L >> 5;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) buf[turn][i][wid] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float s = lane < W ? buf[turn][i][lane] : 0.f;
#pragma unroll
    for (int o = 1; o < kMaxTeam / 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    v[i] = __shfl_sync(0xffffffffu, s, 0);
  }
  turn ^= 1;
}

// L threads to a team; a CTA of blockDim.x / L teams (one, where a team is more than a warp).
template <typename T, int kNv, bool kVec>
__global__ void __launch_bounds__(kMaxTeam) gnorm_fwd_kernel(const __grid_constant__ GnormParams p, int L) {
  constexpr int K = kElems<T>;
  __shared__ float buf[2][1][kMaxTeam / 32];
  int turn = 0;
  const int64_t team = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L;
  const int grp = (int)(team % p.ng);
  const int64_t row0 = team / p.ng;
  const Share<T, kNv, kVec> sh{(int)(threadIdx.x % L), L, p.group};
  float w[kNv][K];
#pragma unroll
  for (int v = 0; v < kNv; ++v)
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int c = sh.col(v, i);
      w[v][i] = c < p.group ? load_w(p.w, p.w_dtype, p.shared ? c : (int64_t)grp * p.group + c) : 0.f;
    }
  const int64_t trips = (p.T + p.rows - 1) / p.rows;  // the same for every team: the sums take whole warps
  const float inv = 1.f / (float)p.group;
  for (int64_t k = 0; k < trips; ++k) {
    const int64_t row = row0 + k * p.rows;
    const bool live = row0 < p.rows && row < p.T;
    const int64_t at = (int64_t)grp * p.group;
    Pack<T, K> xr[kNv], zr[kNv];
#pragma unroll
    for (int v = 0; v < kNv; ++v) {
      xr[v] = sh.load(static_cast<const T*>(p.x) + row * p.sx + at, v, live);
      zr[v] = sh.load(static_cast<const T*>(p.z) + row * p.sz + at, v, live);
    }
    float sum[1] = {0.f};
#pragma unroll
    for (int v = 0; v < kNv; ++v)
#pragma unroll
      for (int i = 0; i < K; ++i) {
        float u = to_float(xr[v].t[i]);
        if (p.gate_first) {
          const float z = to_float(zr[v].t[i]);
          u *= silu_of(z, sigmoid(z));
        }
        sum[0] = fmaf(u, u, sum[0]);
      }
    team_sum(sum, L, buf, turn);
    const float rs = 1.f / sqrtf(fmaf(sum[0], inv, p.eps));
    if (!live) continue;
#pragma unroll
    for (int v = 0; v < kNv; ++v) {
      Pack<T, K> o;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float z = to_float(zr[v].t[i]);
        o.t[i] = from_float<T>(to_float(xr[v].t[i]) * silu_of(z, sigmoid(z)) * (rs * w[v][i]));
      }
      sh.store(static_cast<T*>(p.y) + row * p.D + at, v, o);
    }
  }
}

// Up to 16 elements a thread, the row stays in registers between the sums and the gradients, and the weights for all
// rows; longer shares are read again (from L2).
template <typename T, int kNv, bool kVec>
__global__ void __launch_bounds__(kMaxTeam) gnorm_bwd_kernel(const __grid_constant__ GnormParams p, int L) {
  constexpr int K = kElems<T>;
  constexpr bool kKeep = kNv * K <= 16;
  __shared__ float buf[2][2][kMaxTeam / 32];
  int turn = 0;
  const int64_t team = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L;
  const int grp = (int)(team % p.ng);
  const int64_t row0 = team / p.ng;
  const Share<T, kNv, kVec> sh{(int)(threadIdx.x % L), L, p.group};
  const int64_t wat = p.shared ? 0 : (int64_t)grp * p.group;
  float wk[kKeep ? kNv : 1][K], dw[kNv][K];
  auto weight = [&](int v, int i) {
    const int c = sh.col(v, i);
    return c < p.group ? load_w(p.w, p.w_dtype, wat + c) : 0.f;
  };
#pragma unroll
  for (int v = 0; v < kNv; ++v)
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if constexpr (kKeep) wk[v][i] = weight(v, i);
      dw[v][i] = 0.f;
    }
  auto wt = [&](int v, int i) {
    if constexpr (kKeep)
      return wk[v][i];
    else
      return weight(v, i);
  };
  const int64_t trips = (p.T + p.rows - 1) / p.rows;
  const float inv = 1.f / (float)p.group;
  const int64_t at = (int64_t)grp * p.group;
  for (int64_t k = 0; k < trips; ++k) {
    const int64_t row = row0 + k * p.rows;
    const bool live = row0 < p.rows && row < p.T;
    const T *xp = static_cast<const T*>(p.x) + row * p.sx + at, *zp = static_cast<const T*>(p.z) + row * p.sz + at,
            *gp = static_cast<const T*>(p.dy) + row * p.sdy + at;
    Pack<T, K> xr[kNv], zr[kNv], gr[kNv];
    auto fetch = [&](int v, bool l) {
      xr[v] = sh.load(xp, v, l);
      zr[v] = sh.load(zp, v, l);
      gr[v] = sh.load(gp, v, l);
    };
    if constexpr (kKeep) {
#pragma unroll
      for (int v = 0; v < kNv; ++v) fetch(v, live);
    }
    float sum[2] = {0.f, 0.f};  // of u^2 and of u w dn
#pragma unroll
    for (int v = 0; v < kNv; ++v) {
      if constexpr (!kKeep) fetch(v, live);
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float x = to_float(xr[v].t[i]), z = to_float(zr[v].t[i]), gate = silu_of(z, sigmoid(z));
        const float xg = x * gate, u = p.gate_first ? xg : x;
        sum[0] = fmaf(u, u, sum[0]);
        sum[1] = fmaf(xg * wt(v, i), to_float(gr[v].t[i]), sum[1]);  // u dn is x gate dy either way
      }
    }
    team_sum(sum, L, buf, turn);
    const float rs = 1.f / sqrtf(fmaf(sum[0], inv, p.eps)), mean = sum[1] * inv * rs;  // of g hat
    if (!live) continue;
#pragma unroll
    for (int v = 0; v < kNv; ++v) {
      if constexpr (!kKeep) fetch(v, true);
      Pack<T, K> dx, dz;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const float x = to_float(xr[v].t[i]), z = to_float(zr[v].t[i]), dy = to_float(gr[v].t[i]);
        const float sig = sigmoid(z), gate = silu_of(z, sig), slope = silu_slope(z, sig);
        const float hat = (p.gate_first ? x * gate : x) * rs, dn = p.gate_first ? dy : dy * gate;
        const float w = wt(v, i), du = rs * fmaf(w, dn, -hat * mean);
        dw[v][i] = fmaf(dn, hat, dw[v][i]);
        dx.t[i] = from_float<T>(p.gate_first ? du * gate : du);
        dz.t[i] = from_float<T>((p.gate_first ? du * x : dy * hat * w) * slope);
      }
      sh.store(static_cast<T*>(p.dx) + row * p.D + at, v, dx);
      sh.store(static_cast<T*>(p.dz) + row * p.D + at, v, dz);
    }
  }
  if (row0 < p.rows) {
#pragma unroll
    for (int v = 0; v < kNv; ++v)
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int c = sh.col(v, i);
        if (c < p.group) p.part[row0 * p.D + at + c] = dw[v][i];
      }
  }
}

// dw over the teams of rows (and over the groups, where they share it), in a fixed order: 32 columns a CTA, each summed
// by eight threads.
__global__ void __launch_bounds__(256) gnorm_sum_kernel(const __grid_constant__ GnormParams p) {
  __shared__ float s[8][33];
  bw::griddep_wait();
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, n = p.shared ? p.group : p.D;
  const int64_t parts = p.shared ? p.rows * p.ng : p.rows;  // a shared weight's parts lie `group` apart
  float v = 0.f;
  if (c < n)
    for (int64_t k = r; k < parts; k += 8) v += p.part[k * n + c];
  s[r][lane] = v;
  __syncthreads();
  if (r == 0 && c < n) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][lane];
    p.dw[c] = v;
    if (c == 0) p.hd->status = 0;
  }
}

// ------------------------------------------------------------------------------ host

struct Shape {
  int L, nv, vec, threads;
  int64_t rows, ctas;
};

int next_pow2(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// The team for a group of `n` elements: one vector a thread while a warp holds the group, then two while a CTA does.
// Rows off alignment keep to one, which leaves registers for their addresses.
Shape shape_of(int n, int64_t T, int ng, int es, bool vec, int sms, int threads_per_sm) {
  Shape s{};
  const int K = 16 / es, nvec = (n + K - 1) / K;
  s.vec = vec;
  int L = next_pow2(nvec);
  if (L > 32 && vec) L /= 2;
  if (L > kMaxTeam) L = kMaxTeam;
  s.L = L;
  s.nv = next_pow2((nvec + L - 1) / L);
  s.threads = L > 32 ? L : kWarpTeamThreads;
  const int64_t teams = (int64_t)sms * threads_per_sm / L;  // resident
  int64_t rows = (teams + ng - 1) / ng;
  s.rows = rows < 1 ? 1 : rows > T ? T : rows;
  s.ctas = (s.rows * ng * L + s.threads - 1) / s.threads;
  return s;
}

bool al(const void* p, uintptr_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

int check(GnormParams* p, int dtype, bool bwd, bool* vec) {
  for (int d : {dtype, p->w_dtype})
    if (d != GDN_DTYPE_BF16 && d != GDN_DTYPE_FP16 && d != GDN_DTYPE_FP32) return GDN_ERR_UNSUPPORTED;
  if (p->T < 0 || p->D < 1 || p->group < 1 || p->D % p->group != 0) return GDN_ERR_INVALID_ARG;
  if (p->group > kMaxGroup) return GDN_ERR_UNSUPPORTED;
  if (p->T > ((int64_t)1 << 40) / p->D || !(p->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  for (int64_t* s : {&p->sx, &p->sz, &p->sdy}) {
    if (*s == 0) *s = p->D;
    if (*s < p->D || *s > ((int64_t)1 << 40)) return GDN_ERR_INVALID_ARG;
  }
  if (!p->w || (p->T > 0 && (!p->x || !p->z || (bwd ? !p->dy || !p->dx || !p->dz : !p->y)))) return GDN_ERR_INVALID_ARG;
  const int es = dtype == GDN_DTYPE_FP32 ? 4 : 2, K = 16 / es;
  bool v = p->group % K == 0;
  for (int64_t s : {p->sx, p->sz, p->sdy}) v = v && s % K == 0;
  for (const void* q : {p->x, p->z, p->dy, (const void*)p->y, (const void*)p->dx, (const void*)p->dz}) {
    if (!al(q, es)) return GDN_ERR_INVALID_ARG;
    v = v && al(q, 16);
  }
  if (!al(p->w, p->w_dtype == GDN_DTYPE_FP32 ? 4 : 2)) return GDN_ERR_INVALID_ARG;
  p->ng = p->D / p->group;
  *vec = v;
  return GDN_OK;
}

int check_device(const void* anchor, const void* const* ptrs, int n, DeviceGuard& guard, int* sms) {
  int dev = 0;
  if (device_of(anchor, ptrs, n, &dev) != kOk) return GDN_ERR_INVALID_ARG;
  if (!guard.set(dev)) return GDN_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return GDN_ERR_CUDA;
  return major == 10 && minor == 3 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

template <typename F>
void by_type(int dtype, F f) {
  if (dtype == GDN_DTYPE_BF16)
    f(__nv_bfloat16{});
  else if (dtype == GDN_DTYPE_FP16)
    f(__half{});
  else
    f(float{});
}
template <int kN>
struct Int {
  static constexpr int value = kN;
};
template <typename T, typename F>
void by_share(int nv, F f) {
  if (nv == 1) return f(Int<1>{});
  if (nv == 2) return f(Int<2>{});
  if (nv == 4) return f(Int<4>{});
  if constexpr (sizeof(T) == 4) f(Int<8>{});  // kMaxGroup / kElems / kMaxTeam vectors at most
}

constexpr int kFwdThreads = 1536, kBwdThreads = 640;  // resident threads to an SM that the grids are made for

// The most rows of parts that any shape of the backward writes: what a team of the smallest size would.
size_t part_bytes(int64_t T, int D, int group, int es, int sms) {
  return (size_t)shape_of(group, T, D / group, es, true, sms, kBwdThreads).rows * D * sizeof(float);  // the smaller team
}
constexpr int kSms = 152;  // of the GPU this library is built for

}  // namespace
}  // namespace gdn

extern "C" int gdn_gated_rmsnorm_fwd(const void* x, int64_t x_stride, const void* z, int64_t z_stride, const void* w,
                                     int64_t T, int D, int group, int shared_w, int first, int dtype, int w_dtype, float eps,
                                     void* y, gdn_stream_t stream) {
  using namespace gdn;
  if (first != GDN_GATE_AFTER_NORM && first != GDN_GATE_BEFORE_NORM) return GDN_ERR_UNSUPPORTED;
  GnormParams p{};
  p.x = x, p.z = z, p.w = w, p.y = y, p.sx = x_stride, p.sz = z_stride, p.T = T, p.D = D, p.group = group;
  p.w_dtype = w_dtype, p.shared = shared_w != 0, p.gate_first = first == GDN_GATE_BEFORE_NORM, p.eps = eps;
  bool vec = false;
  int rc = check(&p, dtype, false, &vec), sms = 0;
  if (rc != GDN_OK || T == 0) return rc;
  const void* ptrs[] = {x, z, w};
  DeviceGuard guard;
  if ((rc = check_device(y, ptrs, 3, guard, &sms)) != GDN_OK) return rc;
  const Shape s = shape_of(group, T, p.ng, dtype == GDN_DTYPE_FP32 ? 4 : 2, vec, sms, kFwdThreads);
  p.rows = s.rows;
  by_type(dtype, [&](auto t) {
    using T_ = decltype(t);
    by_share<T_>(s.nv, [&](auto n) {
      constexpr int kNv = decltype(n)::value;
      if (vec)
        gnorm_fwd_kernel<T_, kNv, true><<<(unsigned)s.ctas, s.threads, 0, (cudaStream_t)stream>>>(p, s.L);
      else
        gnorm_fwd_kernel<T_, kNv, false><<<(unsigned)s.ctas, s.threads, 0, (cudaStream_t)stream>>>(p, s.L);
    });
  });
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" size_t gdn_gated_rmsnorm_workspace_size(int64_t T, int D, int group, int dtype) {
  using namespace gdn;
  if (T < 0 || D < 1 || group < 1 || group > kMaxGroup || D % group != 0 || T > ((int64_t)1 << 40) / D) return 0;
  return sizeof(GnormHeader) + part_bytes(T, D, group, dtype == GDN_DTYPE_FP32 ? 4 : 2, kSms);
}

extern "C" int gdn_gated_rmsnorm_bwd(const void* x, int64_t x_stride, const void* z, int64_t z_stride, const void* w,
                                     const void* dy, int64_t dy_stride, int64_t T, int D, int group, int shared_w, int first,
                                     int dtype, int w_dtype, float eps, void* dx, void* dz, float* dw, void* workspace,
                                     size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  if (first != GDN_GATE_AFTER_NORM && first != GDN_GATE_BEFORE_NORM) return GDN_ERR_UNSUPPORTED;
  GnormParams p{};
  p.x = x, p.z = z, p.w = w, p.dy = dy, p.sx = x_stride, p.sz = z_stride, p.sdy = dy_stride, p.T = T, p.D = D;
  p.group = group, p.w_dtype = w_dtype, p.shared = shared_w != 0, p.gate_first = first == GDN_GATE_BEFORE_NORM, p.eps = eps;
  p.dx = dx, p.dz = dz, p.dw = dw;
  bool vec = false;
  int rc = check(&p, dtype, true, &vec), sms = 0;
  if (rc != GDN_OK) return rc;
  if (!dw || !al(dw, 4) || !workspace || !al(workspace, 256)) return GDN_ERR_INVALID_ARG;
  if (ws_bytes < gdn_gated_rmsnorm_workspace_size(T, D, group, dtype)) return GDN_ERR_WORKSPACE;
  const void* ptrs[] = {x, z, w, dy, dx, dz, dw};
  DeviceGuard guard;
  if ((rc = check_device(workspace, ptrs, 7, guard, &sms)) != GDN_OK) return rc;
  p.hd = static_cast<GnormHeader*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sizeof(GnormHeader));
  const Shape s = shape_of(group, T, p.ng, dtype == GDN_DTYPE_FP32 ? 4 : 2, vec, kSms, kBwdThreads);
  p.rows = s.rows;
  if (T > 0)
    by_type(dtype, [&](auto t) {
      using T_ = decltype(t);
      by_share<T_>(s.nv, [&](auto n) {
        constexpr int kNv = decltype(n)::value;
        if (vec)
          gnorm_bwd_kernel<T_, kNv, true><<<(unsigned)s.ctas, s.threads, 0, (cudaStream_t)stream>>>(p, s.L);
        else
          gnorm_bwd_kernel<T_, kNv, false><<<(unsigned)s.ctas, s.threads, 0, (cudaStream_t)stream>>>(p, s.L);
      });
    });
  launch_early(gnorm_sum_kernel, dim3((unsigned)(((p.shared ? group : D) + 31) / 32)), 256, 0, (cudaStream_t)stream, p);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
