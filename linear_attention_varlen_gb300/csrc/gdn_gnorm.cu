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
// gradient, in registers, the next rows' vectors on their way into each thread's own places in shared memory. The gate is
// formed once, in packed pairs. Measured (device time, bf16):
//     forward, 16384 x 64 groups of 128     120 us (805 MB, 6.7 TB/s; 179 us with loads at their use)
//     backward, 32768 x 2048                112 us (671 MB, 6.0 TB/s; 207 us), the sum over the teams 8
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

using bw::f2_fma;
using bw::f2_hi;
using bw::f2_lo;
using bw::f2_mul;
using bw::f2_pack;
using bw::f2_sum;

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
  __device__ __forceinline__ Words load(const T* p, int v, bool live) const {
    Words r{};
    if constexpr (kVec) {
      if (live && col(v, 0) < n) r = *reinterpret_cast<const Words*>(p + col(v, 0));
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (live && col(v, i) < n) set_element<T>(r, i, p[col(v, i)]);
    }
    return r;
  }
  __device__ __forceinline__ void store(T* p, int v, const Words& r) const {
    if constexpr (kVec) {
      if (col(v, 0) < n) *reinterpret_cast<Words*>(p + col(v, 0)) = r;
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (col(v, i) < n) p[col(v, i)] = element_of<T>(r, i);
    }
  }
};

// The next rows' vectors of a thread's share on their way into its own places in shared memory: kN tensors, kStages rows.
template <int kN, int kNv, int kStages>
struct Ring {
  static constexpr int bytes(int threads) { return kN * kNv * kStages * 16 * threads; }
  int pitch, row, put, take;  // bytes between a thread's vectors, and between rows; places of the next rows
  __device__ __forceinline__ Ring() : pitch(16 * (int)blockDim.x), row(kN * kNv * pitch), put(16 * (int)threadIdx.x), take(put) {}
  __device__ __forceinline__ Words* at(int place, int tensor, int v) const {
    extern __shared__ __align__(16) uint8_t ring[];
    return reinterpret_cast<Words*>(ring + place + (tensor * kNv + v) * pitch);
  }
  __device__ __forceinline__ void step(int& place) const {
    place += row;
    if (place >= kStages * row) place -= kStages * row;
  }
};

// Sums over the team; every thread of it gets them, added up in the same order. `buf` has room for two rows of a CTA's
// warps, used in turn, so that one barrier a row is enough.
template <int kN>
struct alignas(4 * kN) Sums {
  float v[kN];
};
template <int kN>
__device__ __forceinline__ void team_sum(float (&v)[kN], int L, Sums<kN> (*buf)[kMaxTeam / 32], int& turn) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= L) break;
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  if (L <= 32) return;
  const int W = L >> 5;
  if ((threadIdx.x & 31) == 0) {
    Sums<kN> s;
#pragma unroll
    for (int i = 0; i < kN; ++i) s.v[i] = v[i];
    buf[turn][threadIdx.x >> 5] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int w = 0; w < W; ++w) {
    const Sums<kN> s = buf[turn][w];
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += s.v[i];
  }
  turn ^= 1;
}

// Rows in flight for a thread, this one's included (0: read when they are needed). With four in the forward the same
// bytes came at 5.5 TB/s instead of 6.2: the reads and writes under way lie further apart.
template <typename T, int kNv, bool kVec>
__host__ __device__ constexpr int fwd_stages() {
  return !kVec || kNv > 2 ? 0 : 2;
}
template <typename T, int kNv, bool kVec>
__host__ __device__ constexpr int bwd_stages() {
  return !kVec ? 0 : kNv == 1 ? 3 : kNv == 2 ? 2 : 0;
}

// L threads to a team; a CTA of blockDim.x / L teams (one, where a team is more than a warp). Either order's output is
// x gate rs w; they differ in whose squares rs has. Rows ahead are on their way into
// shared memory.
template <typename T, int kNv, bool kVec, bool kGateFirst>
__global__ void __launch_bounds__(kMaxTeam) gnorm_fwd_kernel(const __grid_constant__ GnormParams p, int L) {
  constexpr int P = kPairs<T>, kStages = fwd_stages<T, kNv, kVec>();
  Ring<2, kNv, kStages> ring;
  __shared__ Sums<1> buf[2][kMaxTeam / 32];
  int turn = 0;
  const int64_t team = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L;
  const int64_t row0 = team / p.ng, at = (team - row0 * p.ng) * p.group;
  const Share<T, kNv, kVec> sh{(int)(threadIdx.x % L), L, p.group};
  uint64_t w[kNv][P];
#pragma unroll
  for (int v = 0; v < kNv; ++v)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = sh.col(v, 2 * i + j);
        f[j] = c < p.group ? load_w(p.w, p.w_dtype, p.shared ? c : at + c) : 0.f;
      }
      w[v][i] = f2_pack(f[0], f[1]);
    }
  const int trips = (int)((p.T + p.rows - 1) / p.rows);  // the same for every team: the sums take whole warps
  const float inv = 1.f / (float)p.group;
  const T *x = static_cast<const T*>(p.x) + row0 * p.sx + at, *z = static_cast<const T*>(p.z) + row0 * p.sz + at;
  T* y = static_cast<T*>(p.y) + row0 * p.D + at;
  const int64_t dx = p.rows * p.sx, dz = p.rows * p.sz, dy = p.rows * p.D;
  // rows behind the last one (and those of threads behind the last team) are left out
  const int mine = row0 < p.rows && row0 < p.T ? (int)((p.T - row0 + p.rows - 1) / p.rows) : 0;
  bool in[kNv];
#pragma unroll
  for (int v = 0; v < kNv; ++v) in[v] = sh.col(v, 0) < p.group;
  // x and z: the row that comes next
  auto issue = [&](int k) {
    if (k < mine) {
#pragma unroll
      for (int v = 0; v < kNv; ++v)
        if (in[v]) {
          cp_async16(ring.at(ring.put, 0, v), x + sh.col(v, 0));
          cp_async16(ring.at(ring.put, 1, v), z + sh.col(v, 0));
        }
    }
    cp_async_commit();
    x += dx, z += dz;
    ring.step(ring.put);
  };
  if constexpr (kStages > 0) {
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k);
  }
  for (int k = 0; k < trips; ++k) {
    if constexpr (kStages > 0) {
      issue(k + kStages - 1);
      cp_async_wait<(kStages > 0 ? kStages - 1 : 0)>();
    }
    uint64_t xg[kNv][P], sum2 = 0;
#pragma unroll
    for (int v = 0; v < kNv; ++v) {
      Words xr{}, zr{};
      if constexpr (kStages > 0) {
        if (k < mine && in[v]) xr = *ring.at(ring.take, 0, v), zr = *ring.at(ring.take, 1, v);
      } else {
        xr = sh.load(x, v, k < mine);
        zr = sh.load(z, v, k < mine);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t u = pair_of<T>(xr, i);
        xg[v][i] = f2_mul(u, silu_pair(pair_of<T>(zr, i)));
        sum2 = kGateFirst ? f2_fma(xg[v][i], xg[v][i], sum2) : f2_fma(u, u, sum2);
      }
    }
    if constexpr (kStages > 0)
      ring.step(ring.take);
    else
      x += dx, z += dz;
    float sum[1] = {f2_sum(sum2)};
    team_sum(sum, L, buf, turn);
    const uint64_t rs = f2_dup(rsqrtf(fmaf(sum[0], inv, p.eps)));
    if (k < mine) {
#pragma unroll
      for (int v = 0; v < kNv; ++v) {
        Words o;
#pragma unroll
        for (int i = 0; i < P; ++i) set_pair<T>(o, i, f2_mul(xg[v][i], f2_mul(rs, w[v][i])));
        sh.store(y, v, o);
      }
    }
    y += dy;
  }
}

// Either order: the sum of u w dn and dw are those of x gate w dy and x gate dy rs. Up to eight elements a thread, the
// weights and the row stay in registers; longer shares take both again. Rows ahead are on their way into shared memory
// where that holds enough of them, else a row's second reading comes from L2. kRegs: teams of less than a warp have more
// rows under way with fewer registers (8192 x 64 groups of 128: 5.1 against 4.7 TB/s with 128), the others rather not
// (32768 x 2048: 4.9 against 5.6).
template <typename T, int kNv, bool kVec, bool kGateFirst, int kRegs>
__global__ void __maxnreg__(kRegs) gnorm_bwd_kernel(const __grid_constant__ GnormParams p, int L) {
  constexpr int K = kElems<T>, P = kPairs<T>;
  constexpr bool kKeep = kNv * K <= 8;
  constexpr int kStages = bwd_stages<T, kNv, kVec>();
  Ring<3, kNv, kStages> ring;
  __shared__ Sums<2> buf[2][kMaxTeam / 32];
  int turn = 0;
  const int64_t team = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / L;
  const int64_t row0 = team / p.ng, at = (team - row0 * p.ng) * p.group;
  const Share<T, kNv, kVec> sh{(int)(threadIdx.x % L), L, p.group};
  uint64_t wk[kKeep ? kNv : 1][P] = {}, dw[kNv][P];
  auto weight = [&](int v, int i) {
    float f[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = sh.col(v, 2 * i + j);
      f[j] = c < p.group ? load_w(p.w, p.w_dtype, p.shared ? c : at + c) : 0.f;
    }
    return f2_pack(f[0], f[1]);
  };
  auto wt = [&](int v, int i) {
    if constexpr (kKeep)
      return wk[v][i];
    else
      return weight(v, i);
  };
#pragma unroll
  for (int v = 0; v < kNv; ++v)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if constexpr (kKeep) wk[v][i] = weight(v, i);
      dw[v][i] = 0;
    }
  const int trips = (int)((p.T + p.rows - 1) / p.rows);
  const float inv = 1.f / (float)p.group;
  const T *x = static_cast<const T*>(p.x) + row0 * p.sx + at, *z = static_cast<const T*>(p.z) + row0 * p.sz + at,
          *g = static_cast<const T*>(p.dy) + row0 * p.sdy + at;
  const int64_t ex = p.rows * p.sx, ez = p.rows * p.sz, eg = p.rows * p.sdy, eo = p.rows * p.D;
  T *dxp = static_cast<T*>(p.dx) + row0 * p.D + at, *dzp = static_cast<T*>(p.dz) + row0 * p.D + at;
  const int mine = row0 < p.rows && row0 < p.T ? (int)((p.T - row0 + p.rows - 1) / p.rows) : 0;
  bool in[kNv];
#pragma unroll
  for (int v = 0; v < kNv; ++v) in[v] = sh.col(v, 0) < p.group;
  // x, z and g: the row that comes next
  constexpr int kHold = kKeep ? kNv : 1;
  auto issue = [&](int k) {
    if (k < mine) {
#pragma unroll
      for (int v = 0; v < kNv; ++v)
        if (in[v]) {
          cp_async16(ring.at(ring.put, 0, v), x + sh.col(v, 0));
          cp_async16(ring.at(ring.put, 1, v), z + sh.col(v, 0));
          cp_async16(ring.at(ring.put, 2, v), g + sh.col(v, 0));
        }
    }
    cp_async_commit();
    x += ex, z += ez, g += eg;
    ring.step(ring.put);
  };
  if constexpr (kStages > 0) {
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) issue(k);
  }
  for (int k = 0; k < trips; ++k) {
    Words xr[kHold], zr[kHold], gr[kHold];
    uint64_t sig[kHold][P], sq = 0, dot = 0;
    auto sums = [&](int v, int hold) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t u = pair_of<T>(xr[hold], i), zz = pair_of<T>(zr[hold], i);
        sig[hold][i] = sigmoid_pair(zz);
        const uint64_t zc = f2_pack(at_least(f2_lo(zz), -128.f), at_least(f2_hi(zz), -128.f));
        const uint64_t xg = f2_mul(u, f2_mul(zc, sig[hold][i]));
        sq = kGateFirst ? f2_fma(xg, xg, sq) : f2_fma(u, u, sq);
        dot = f2_fma(f2_mul(xg, wt(v, i)), pair_of<T>(gr[hold], i), dot);
      }
    };
    if constexpr (kStages > 0) {
      issue(k + kStages - 1);
      cp_async_wait<(kStages > 0 ? kStages - 1 : 0)>();
    }
    auto fetch = [&](int v, int hold, bool live) {
      if constexpr (kStages > 0) {
        xr[hold] = zr[hold] = gr[hold] = Words{};
        if (live && in[v]) xr[hold] = *ring.at(ring.take, 0, v), zr[hold] = *ring.at(ring.take, 1, v), gr[hold] = *ring.at(ring.take, 2, v);
      } else {
        xr[hold] = sh.load(x, v, live);
        zr[hold] = sh.load(z, v, live);
        gr[hold] = sh.load(g, v, live);
      }
    };
#pragma unroll
    for (int v = 0; v < kNv; ++v) {
      fetch(v, kKeep ? v : 0, k < mine);
      sums(v, kKeep ? v : 0);
    }
    float sum[2] = {f2_sum(sq), f2_sum(dot)};
    team_sum(sum, L, buf, turn);
    const float r = rsqrtf(fmaf(sum[0], inv, p.eps));
    const uint64_t rs = f2_dup(r), mean = f2_dup(-sum[1] * inv * r * r);  // - rs mean(g hat)
    if (k < mine) {
#pragma unroll
      for (int v = 0; v < kNv; ++v) {
        const int hold = kKeep ? v : 0;
        if constexpr (!kKeep) fetch(v, 0, true);
        Words dx, dz;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t xx = pair_of<T>(xr[hold], i), zz = pair_of<T>(zr[hold], i), dy = pair_of<T>(gr[hold], i);
          const uint64_t sg = kKeep ? sig[hold][i] : sigmoid_pair(zz);
          const uint64_t zc = f2_pack(at_least(f2_lo(zz), -128.f), at_least(f2_hi(zz), -128.f));
          const uint64_t gate = f2_mul(zc, sg), slope = silu_slope_pair(zz, sg), xg = f2_mul(xx, gate);
          const uint64_t ry = f2_mul(rs, dy), wv = wt(v, i);
          dw[v][i] = f2_fma(ry, xg, dw[v][i]);
          const uint64_t wr = f2_mul(ry, wv);  // rs w dy
          if constexpr (kGateFirst) {
            const uint64_t du = f2_fma(f2_mul(xg, rs), mean, wr);
            set_pair<T>(dx, i, f2_mul(du, gate));
            set_pair<T>(dz, i, f2_mul(f2_mul(du, xx), slope));
          } else {
            const uint64_t hat = f2_mul(xx, rs);
            set_pair<T>(dx, i, f2_fma(hat, mean, f2_mul(wr, gate)));
            set_pair<T>(dz, i, f2_mul(f2_mul(wr, xx), slope));
          }
        }
        sh.store(dxp, v, dx);
        sh.store(dzp, v, dz);
      }
    }
    dxp += eo, dzp += eo;
    if constexpr (kStages > 0)
      ring.step(ring.take);
    else
      x += ex, z += ez, g += eg;
  }
  if (row0 < p.rows) {
#pragma unroll
    for (int v = 0; v < kNv; ++v)
#pragma unroll
      for (int i = 0; i < K; ++i) {
        const int c = sh.col(v, i);
        if (c < p.group) p.part[row0 * p.D + at + c] = i % 2 ? f2_hi(dw[v][i / 2]) : f2_lo(dw[v][i / 2]);
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
#pragma unroll 8
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

// The team for a group of `n` elements: one vector a thread as long as a CTA holds the group.
Shape shape_of(int n, int64_t T, int ng, int es, bool vec, int sms, int threads_per_sm) {
  Shape s{};
  const int K = 16 / es, nvec = (n + K - 1) / K;
  s.vec = vec;
  int L = next_pow2(nvec);
  if (L > kMaxTeam) L = kMaxTeam;
  s.L = L;
  s.nv = next_pow2((nvec + L - 1) / L);
  s.threads = L > 32 ? L : kWarpTeamThreads;
  const int64_t teams = (int64_t)sms * threads_per_sm / L;  // resident
  const int64_t rows = teams / ng;  // no more than are resident: a few more would take a second turn
  s.rows = rows < 1 ? 1 : rows;
  if (s.rows > T) s.rows = T;  // none for no rows: the sum of dw takes what the teams wrote
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

// Shared memory beyond the default limit.
template <typename K>
bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 40 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

constexpr int kFwdThreads = 1024, kBwdThreads = 512;  // resident threads to an SM that the grids are made for

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
  bool ok = true;
  by_type(dtype, [&](auto t) {
    using T_ = decltype(t);
    by_share<T_>(s.nv, [&](auto n) {
      constexpr int kNv = decltype(n)::value;
      auto* kernel = p.gate_first ? (vec ? gnorm_fwd_kernel<T_, kNv, true, true> : gnorm_fwd_kernel<T_, kNv, false, true>)
                                  : (vec ? gnorm_fwd_kernel<T_, kNv, true, false> : gnorm_fwd_kernel<T_, kNv, false, false>);
      const size_t ring = vec ? Ring<2, kNv, fwd_stages<T_, kNv, true>()>::bytes(s.threads) : 0;
      ok = allow_smem(kernel, ring);
      if (ok) kernel<<<(unsigned)s.ctas, s.threads, ring, (cudaStream_t)stream>>>(p, s.L);
    });
  });
  return ok && cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
  bool ok = true;
  if (T > 0)
    by_type(dtype, [&](auto t) {
      using T_ = decltype(t);
      by_share<T_>(s.nv, [&](auto n) {
        constexpr int kNv = decltype(n)::value;
        auto pick = [&](auto regs) {
          constexpr int kRegs = decltype(regs)::value;
          return p.gate_first
                     ? (vec ? gnorm_bwd_kernel<T_, kNv, true, true, kRegs> : gnorm_bwd_kernel<T_, kNv, false, true, kRegs>)
                     : (vec ? gnorm_bwd_kernel<T_, kNv, true, false, kRegs> : gnorm_bwd_kernel<T_, kNv, false, false, kRegs>);
        };
        auto* kernel = pick(Int<128>{});
        if constexpr (kNv == 1) {
          if (s.L < 32) kernel = pick(Int<96>{});
        }
        const size_t ring = vec ? Ring<3, kNv, bwd_stages<T_, kNv, true>()>::bytes(s.threads) : 0;
        ok = allow_smem(kernel, ring);
        if (ok) kernel<<<(unsigned)s.ctas, s.threads, ring, (cudaStream_t)stream>>>(p, s.L);
      });
    });
  launch_early(gnorm_sum_kernel, dim3((unsigned)(((p.shared ? group : D) + 31) / 32)), 256, 0, (cudaStream_t)stream, p);
  return ok && cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
