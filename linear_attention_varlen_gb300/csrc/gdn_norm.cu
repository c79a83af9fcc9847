// Root-mean-square norm with the residual's addition, and its backward (sm_103a). Per row of D:
//     h = x + r,  y = w h rs,  rs = (mean(h^2) + eps)^{-1/2}
// h is rounded once to the inputs' type for the residual stream; y is formed from the fp32 sum and
// rounded once, to the inputs' type or to e4m3 with a scale amax / 448 for the row or for each 128
// columns (448 is e4m3's largest value; a row or group of zeros takes scale 1). Backward, from the h
// the forward left:
//     dx = rs w dy - h rs^3 mean(w dy h) + dh,   dw = sum over rows of dy h rs.
//
// Both read each input once and write each output once and do a few operations an element: they are
// bound by HBM traffic, as long as the arithmetic stays small beside it (pairs of elements in packed fp32,
// no division an element) and enough bytes are in flight: by many resident rows in the forward, by bulk copies
// into rings of row buffers in the backward, whose registers hold the weight gradient. A thread holds 8
// consecutive elements a vector. Measured (device time):
//     forward, bf16, 16384 x 8192, residual, e4m3 by groups     177 us   944 MB    5.3 TB/s
//     forward, bf16, 65536 x 1024, residual (x itself)           66 us   403 MB    6.1 TB/s
//     backward, bf16, 65536 x 1024, with dh                      88 us   537 MB    6.1 TB/s
//     backward, fp32, 777 x 1001 (rows off alignment)            15 us, of it 4 the sum over the parts
// The 8-bit forward issues an instruction in 56 % of the cycles and waits for its loads in most others (three CTAs of
// 512 threads to an SM is what the registers allow); small calls are bound by their launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/gdn.h"
#include "bw_prims.cuh"
#include "gdn_common.cuh"
#include "gdn_host.h"

namespace gdn {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kNormMaxD = 32768;
constexpr int kRowThreads = 512;  // most threads to a row
constexpr int kGroup = 128;       // columns to one scale
constexpr int kWarpRows = 8;      // rows of a CTA whose warps own a row each

// ------------------------------------------------------------------------------ elements

__device__ __forceinline__ float elem(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem(float v) { return v; }
template <typename T>
__device__ __forceinline__ T round_to(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 round_to<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half round_to<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float round_to<float>(float v) {
  return v;
}

// 8 elements as they lie in memory
template <typename T>
struct alignas(16) Raw8 {
  T t[8];
};
// Words w[0 .. kN + 3] moved down by `bytes` (below 16, a multiple of sizeof(T), the same for the warp): the first
// kN are valid.
template <typename T, int kN>
__device__ __forceinline__ void shift_words(uint32_t* w, uint32_t bytes) {
  if (bytes & 8) {
#pragma unroll
    for (int i = 0; i < kN + 2; ++i) w[i] = w[i + 2];
  }
  if (bytes & 4) {
#pragma unroll
    for (int i = 0; i < kN + 1; ++i) w[i] = w[i + 1];
  }
  if (sizeof(T) == 2 && (bytes & 2)) {
#pragma unroll
    for (int i = 0; i < kN; ++i) w[i] = __byte_perm(w[i], w[i + 1], 0x5432);
  }
}

// Columns c .. c + 7 of a row of D elements (zero past its end) of a tensor that lies in [lo, hi). kVec: rows are
// aligned and D a multiple of 8. Other rows are read in whole 16-byte pieces too, the ones that cover the
// columns, and moved into place: element by element a warp's lanes lie 8 elements apart, and each of the eight loads
// touches every sector of the range (forward of 65536 x 1023: 365 us in fp32 and 265 us in bf16, now 160 us and
// 158 us; aligned 130 us and 66 us). Only a piece that sticks out of the tensor is read by elements.
template <typename T, bool kVec>
__device__ __forceinline__ Raw8<T> load8(const T* row, int c, int D, const T* lo, const T* hi) {
  constexpr int kP = sizeof(T) / 2;  // pieces to 8 elements
  Raw8<T> r;
  uint4* q = reinterpret_cast<uint4*>(r.t);
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kP; ++i) q[i] = c < D ? reinterpret_cast<const uint4*>(row + c)[i] : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < kP; ++i) q[i] = make_uint4(0, 0, 0, 0);
    if (c >= D) return r;
    const uintptr_t a = reinterpret_cast<uintptr_t>(row + c), a0 = a & ~(uintptr_t)15;
    const uint32_t m = (uint32_t)(a - a0);
    if (a0 >= reinterpret_cast<uintptr_t>(lo) && a0 + 16 * (kP + (m ? 1 : 0)) <= reinterpret_cast<uintptr_t>(hi)) {
      uint32_t w[4 * kP + 4];
#pragma unroll
      for (int i = 0; i < kP + 1; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (i < kP || m) x = reinterpret_cast<const uint4*>(a0)[i];
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
      }
      shift_words<T, 4 * kP>(w, m);
#pragma unroll
      for (int i = 0; i < kP; ++i) q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      if (c + 8 > D) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i >= D) r.t[i] = round_to<T>(0.f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < D) r.t[i] = row[c + i];
    }
  }
  return r;
}
// The same columns written, by whole warps whose lanes hold consecutive vectors. In rows that are not aligned a lane
// writes the aligned pieces that begin inside its own vector, with the next lane's first elements; what no lane of
// the warp can write whole (its first and last piece, a row's end) goes element by element.
template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* row, int c, int D, const uint64_t* f) {  // four pairs of fp32
  constexpr int kP = sizeof(T) / 2;
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2 && !std::is_same_v<T, __half>) {
      reinterpret_cast<uint32_t*>(r.t)[i] = bw::pack_bf16x2(bw::f2_lo(f[i]), bw::f2_hi(f[i]));
    } else if constexpr (sizeof(T) == 2) {
      reinterpret_cast<__half2*>(r.t)[i] = __floats2half2_rn(bw::f2_lo(f[i]), bw::f2_hi(f[i]));
    } else {
      r.t[2 * i] = bw::f2_lo(f[i]);
      r.t[2 * i + 1] = bw::f2_hi(f[i]);
    }
  }
  const uint4* q = reinterpret_cast<const uint4*>(r.t);
  if constexpr (kVec) {
    if (c < D) {
#pragma unroll
      for (int i = 0; i < kP; ++i) reinterpret_cast<uint4*>(row + c)[i] = q[i];
    }
  } else {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row + c), a0 = a & ~(uintptr_t)15;
    const uint32_t m = (uint32_t)(a - a0);  // the same in every lane
    bool whole[kP + 1];                     // pieces 0 (the lane before writes it) to kP
    const int lane = threadIdx.x & 31, head = (16 - (int)m) / (int)sizeof(T);  // elements of piece 0
    constexpr int kE = 16 / sizeof(T);
    whole[0] = m == 0 ? c + kE <= D : lane > 0 && c + head <= D;
#pragma unroll
    for (int i = 1; i <= kP; ++i) whole[i] = m == 0 ? c + kE * (i + 1) <= D : (i < kP || lane < 31) && c + head + kE * i <= D;
    if (m == 0) {
#pragma unroll
      for (int i = 0; i < kP; ++i)
        if (whole[i]) reinterpret_cast<uint4*>(a0)[i] = q[i];
    } else {
      uint32_t w[4 * kP + 4];
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        w[4 * i] = q[i].x;
        w[4 * i + 1] = q[i].y;
        w[4 * i + 2] = q[i].z;
        w[4 * i + 3] = q[i].w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * kP + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
      shift_words<T, 4 * kP>(w, 16 - m);
#pragma unroll
      for (int i = 0; i < kP; ++i)
        if (whole[i + 1])
          reinterpret_cast<uint4*>(a0)[i + 1] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    bool all = true;
#pragma unroll
    for (int i = 0; i <= kP; ++i) all = all && (whole[i] || (m == 0 && i == kP));
    if (!all) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t at = (m + i * (uint32_t)sizeof(T)) >> 4;
        const bool done = at == 0 ? whole[0] : at == 1 ? whole[1] : whole[kP];
        if (c + i < D && !done) row[c + i] = r.t[i];
      }
    }
  }
}
// eight bytes, the same way in pieces of eight
template <bool kVec>
__device__ __forceinline__ void store8_bytes(uint8_t* row, int c, int D, uint64_t v) {
  if constexpr (kVec) {
    if (c < D) *reinterpret_cast<uint64_t*>(row + c) = v;
  } else {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row + c), a0 = a & ~(uintptr_t)7;
    const int m = (int)(a - a0), lane = threadIdx.x & 31, head = 8 - m;
    const bool first = m == 0 ? c + 8 <= D : lane > 0 && c + head <= D, last = m != 0 && lane < 31 && c + head + 8 <= D;
    if (m == 0) {
      if (first) *reinterpret_cast<uint64_t*>(a0) = v;
    } else {
      const uint64_t next = __shfl_down_sync(0xffffffffu, v, 1);
      if (last) *reinterpret_cast<uint64_t*>(a0 + 8) = v >> (8 * head) | next << (8 * m);
    }
    if (!first || (m != 0 && !last)) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < D && !(m + i < 8 ? first : last)) row[c + i] = (uint8_t)(v >> (8 * i));
    }
  }
}
template <bool kVec>
__device__ __forceinline__ void load_w8(const void* w, int dtype, int c, int D, float* f) {
  auto get = [&](auto* p) {
    const auto r = load8<std::remove_const_t<std::remove_pointer_t<decltype(p)>>, kVec>(p, c, D, p, p + D);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = elem(r.t[i]);
  };
  if (dtype == GDN_DTYPE_BF16)
    get(static_cast<const __nv_bfloat16*>(w));
  else if (dtype == GDN_DTYPE_FP16)
    get(static_cast<const __half*>(w));
  else
    get(static_cast<const float*>(w));
}

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sums of two values (or a maximum, kMax, of one) over the threads of a row: a warp, or the CTA through the
// 16 pairs of `s`. The caller alternates between buffers: one barrier is enough.
template <bool kWarp, bool kMax = false>
__device__ __forceinline__ float2 row_reduce(float2 x, float2* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, x.x, o);
    x.x = kMax ? max_nan(x.x, a) : x.x + a;
    if constexpr (!kMax) x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
  }
  if constexpr (kWarp) return x;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (lane == 0) s[wid] = x;
  __syncthreads();
  x = s[lane & 15];
  if ((lane & 15) >= nw) x = make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, x.x, o);
    x.x = kMax ? max_nan(x.x, a) : x.x + a;
    if constexpr (!kMax) x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
  }
  return x;
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
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kNv == 1 ? 256 : kRowThreads, kNv == 1 ? 6 : kNv == 2 ? 3 : 1)
    norm_fwd_kernel(const __grid_constant__ NormFwdParams p) {
  __shared__ float2 s_red[2][16];
  const int tpr = kWarp ? 32 : blockDim.x, t = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = kWarp ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= p.T) return;
  uint64_t v[kNv][4];  // pairs of fp32
  uint64_t ss = 0;
  const bool res = p.r != nullptr;
  {
    const T *xs = static_cast<const T*>(p.x), *rr = static_cast<const T*>(p.r);
    Raw8<T> x[kNv], r[kNv];
#pragma unroll
    for (int j = 0; j < kNv; ++j) x[j] = load8<T, kVec>(xs + row * p.D, (t + j * tpr) * 8, p.D, xs, xs + p.T * p.D);
    if (res) {
#pragma unroll
      for (int j = 0; j < kNv; ++j) r[j] = load8<T, kVec>(rr + row * p.D, (t + j * tpr) * 8, p.D, rr, rr + p.T * p.D);
    }
#pragma unroll
    for (int j = 0; j < kNv; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[j][i] = bw::f2_pack(elem(x[j].t[2 * i]), elem(x[j].t[2 * i + 1]));
        if (res) v[j][i] = bw::f2_add(v[j][i], bw::f2_pack(elem(r[j].t[2 * i]), elem(r[j].t[2 * i + 1])));
        ss = bw::f2_fma(v[j][i], v[j][i], ss);
      }
  }
  if (res) {
    T* h = static_cast<T*>(p.h) + row * p.D;
#pragma unroll
    for (int j = 0; j < kNv; ++j) store8<T, kVec>(h, (t + j * tpr) * 8, p.D, v[j]);
  }
  const float rs = rsqrtf(row_reduce<kWarp>(make_float2(bw::f2_sum(ss), 0.f), s_red[0]).x / (float)p.D + p.eps);
  const uint64_t rs2 = bw::f2_pack(rs, rs);
#pragma unroll
  for (int j = 0; j < kNv; ++j) {
    float w[8];
    load_w8<kVec>(p.w, p.w_dtype, (t + j * tpr) * 8, p.D, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[j][i] = bw::f2_mul(bw::f2_mul(v[j][i], rs2), bw::f2_pack(w[2 * i], w[2 * i + 1]));
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
    for (int i = 0; i < 4; ++i) am[j] = max_nan(max_nan(am[j], fabsf(bw::f2_lo(v[j][i]))), fabsf(bw::f2_hi(v[j][i])));
  }
  if (p.quant == GDN_QUANT_ROW) {
    float m = am[0];
#pragma unroll
    for (int j = 1; j < kNv; ++j) m = max_nan(m, am[j]);
    m = row_reduce<kWarp, true>(make_float2(m, 0.f), s_red[1]).x;
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
    // One reciprocal for the thread's elements, not of the stored scale (a division later) but within two units of its
    // reciprocal, far below a step of e4m3; scales so small that it would overflow are taken up by 2^100 first.
    const bool tiny = am[j] < 1e-27f;
    if (tiny) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = bw::f2_mul(v[j][i], bw::f2_pack(0x1p100f, 0x1p100f));
    }
    float inv;
    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(am[j] * (tiny ? 0x1p100f / kE4m3Max : 1.f / kE4m3Max)));
    if (!(am[j] > 0.f)) inv = 1.f;
    const uint64_t inv2 = bw::f2_pack(inv, inv);
    alignas(8) __nv_fp8x2_storage_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t z = bw::f2_mul(v[j][i], inv2);
      b[i] = __nv_cvt_float2_to_fp8x2(make_float2(bw::f2_lo(z), bw::f2_hi(z)), __NV_SATFINITE, __NV_E4M3);
    }
    store8_bytes<kVec>(y, (t + j * tpr) * 8, p.D, *reinterpret_cast<const uint64_t*>(b));
  }
}

// ------------------------------------------------------------------------------ backward

struct NormBwdParams {
  const void *h, *w, *dy, *dh;
  void* dx;
  float *part, *dw;
  int32_t *status, *flags;  // of the call, and of each CTA with rings (null where there are none)
  int64_t T, withheld;      // withheld: the row that a test leaves out (-1 = none)
  long long budget;         // limit of a wait, clock cycles
  int D, w_dtype, parts;
  float eps;
};

// A CTA's sixteen warps are teams of kTeam; each walks rows of its own and keeps the weight gradient's part of
// its columns in registers. Aligned rows (kRing) come through a ring of row buffers in shared memory that bulk
// copies fill ahead of the team: the next rows are always in flight, at no cost in registers. Other rows are read
// from memory as they come, with the same thread for the same columns, so that the results are the same bits. A
// team reads a row twice: for the two sums, and for the outputs. The wait for a row is bounded: a team whose row does
// not come writes nothing more, lets its copies in flight land (again bounded) and leaves; the CTA's flag tells.
constexpr int kBwdWarps = 16;
constexpr uint32_t kBwdRing = 196608;  // bytes of the rings of a CTA

template <typename T, int kNv, int kTeam, bool kRing>
__global__ void __launch_bounds__(32 * kBwdWarps, 1) norm_bwd_team_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int kTeams = kBwdWarps / kTeam;
  bw::griddep_launch_dependents();  // the sum over the parts may take its place, and waits there
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t s_full[kTeams][8];
  __shared__ float2 s_red[kTeams][2][kTeam];
  __shared__ int s_abort[kTeams];
  const int team = threadIdx.x / (32 * kTeam), t = threadIdx.x % (32 * kTeam), lane = t & 31, wt = t >> 5;
  const int tensors = p.dh ? 3 : 2;
  const uint32_t row_bytes = (uint32_t)p.D * sizeof(T), stage_bytes = row_bytes * tensors;
  const int stages = kRing ? min(8, (int)(kBwdRing / kTeams / stage_bytes)) : 1;
  uint8_t* mine = ring + (size_t)team * stages * stage_bytes;
  const T* src[3] = {static_cast<const T*>(p.h), static_cast<const T*>(p.dy), static_cast<const T*>(p.dh)};
  const int64_t first = (int64_t)blockIdx.x * kTeams + team, step = (int64_t)gridDim.x * kTeams, n = p.T * p.D;
  if (kRing && t == 0) {
    for (int i = 0; i < stages; ++i) bw::mbar_init(&s_full[team][i], 1);
    s_abort[team] = 0;
    bw::fence_mbar_init();
  }
  auto team_sync = [&]() {
    if constexpr (kTeam == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kTeam) : "memory");
  };
  auto fetch = [&](int64_t row, int st) {
    if (row == p.withheld) return;
    bw::mbar_arrive_expect_tx(&s_full[team][st], stage_bytes);
    for (int k = 0; k < tensors; ++k)
      bw::bulk_load(mine + st * stage_bytes + k * row_bytes, src[k] + row * p.D, row_bytes, &s_full[team][st]);
  };
  if (kRing && t == 0)
    for (int i = 0; i < stages && first + i * step < p.T; ++i) fetch(first + i * step, i);
  float dw[kNv][8];
  Raw8<T> w[kNv];  // the weight in the rows' type where it has it, else read from memory for each row
  const bool same = p.w_dtype == (sizeof(T) == 4 ? GDN_DTYPE_FP32 : std::is_same_v<T, __half> ? GDN_DTYPE_FP16 : GDN_DTYPE_BF16);
#pragma unroll
  for (int j = 0; j < kNv; ++j) {
    const T* pw = static_cast<const T*>(p.w);
    if (same) w[j] = load8<T, kRing>(pw, (t + j * 32 * kTeam) * 8, p.D, pw, pw + p.D);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }
  auto weight = [&](int j, float* f) {
    if (same) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = elem(w[j].t[i]);
    } else {
      load_w8<kRing>(p.w, p.w_dtype, (t + j * 32 * kTeam) * 8, p.D, f);
    }
  };
  team_sync();
  int st = 0, turn = 0;
  uint32_t phase = 0;
  for (int64_t row = first; row < p.T; row += step, turn ^= 1) {
    const T *h = src[0] + row * p.D, *g = src[1] + row * p.D, *e = src[2] + row * p.D;
    if constexpr (kRing) {
      if (!bw::mbar_wait(&s_full[team][st], phase, p.budget)) *static_cast<volatile int*>(&s_abort[team]) = 1;
      const uint8_t* b = mine + st * stage_bytes;
      h = reinterpret_cast<const T*>(b);
      g = reinterpret_cast<const T*>(b + row_bytes);
      e = reinterpret_cast<const T*>(b + 2 * row_bytes);
    }
    float2 sum = make_float2(0.f, 0.f);
    // Rows that had to be moved into place stay in registers where two vectors of each fit (65536 x 1023 fp32: 213 us
    // against 259); with four, in 16 bits, that spills (288 us against 257).
    constexpr bool kKeep = !kRing && kNv <= 2;
    Raw8<T> hs[kKeep ? kNv : 1], gs[kKeep ? kNv : 1];
    if constexpr (kKeep) {
#pragma unroll
      for (int j = 0; j < kNv; ++j) {
        const int c = (t + j * 32 * kTeam) * 8;
        hs[j] = load8<T, false>(h, c, p.D, src[0], src[0] + n);
        gs[j] = load8<T, false>(g, c, p.D, src[1], src[1] + n);
      }
    }
    auto again = [&](int k, const T* from, const Raw8<T>* kept, int j, int c) {
      if constexpr (kKeep)
        return kept[j];
      else
        return load8<T, kRing>(from, c, p.D, src[k], src[k] + n);
    };
    {
      uint64_t s1 = 0, s2 = 0;
#pragma unroll
      for (int j = 0; j < kNv; ++j) {
        const int c = (t + j * 32 * kTeam) * 8;
        const Raw8<T> hr = again(0, h, hs, j, c), gr = again(1, g, gs, j, c);
        float wf[8];
        weight(j, wf);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t hv = bw::f2_pack(elem(hr.t[2 * i]), elem(hr.t[2 * i + 1]));
          s1 = bw::f2_fma(hv, hv, s1);
          s2 = bw::f2_fma(bw::f2_mul(hv, bw::f2_pack(wf[2 * i], wf[2 * i + 1])),
                          bw::f2_pack(elem(gr.t[2 * i]), elem(gr.t[2 * i + 1])), s2);
        }
      }
      sum = make_float2(bw::f2_sum(s1), bw::f2_sum(s2));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
    }
    if constexpr (kTeam > 1) {
      if (lane == 0) s_red[team][turn][wt] = sum;
      team_sync();
      sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kTeam; ++k) {
        const float2 x = s_red[team][turn][k];
        sum.x += x.x;
        sum.y += x.y;
      }
    } else if constexpr (kRing) {
      __syncwarp();
    }
    // Whether some thread's wait ran out: the team has met since, and none is at the next row's before all have read it.
    if constexpr (kRing) {
      if (*static_cast<volatile int*>(&s_abort[team])) {
        if (t == 0)
          for (int i = 0; i < stages && row + i * step < p.T; ++i) {
            const bool wrap = st + i >= stages;
            bw::mbar_wait(&s_full[team][wrap ? st + i - stages : st + i], phase ^ (wrap ? 1 : 0), p.budget);
          }
        break;
      }
    }
    const float rs = rsqrtf(sum.x / (float)p.D + p.eps);
    const float cc = -rs * rs * rs * (sum.y / (float)p.D);
    const uint64_t rs2 = bw::f2_pack(rs, rs), c2 = bw::f2_pack(cc, cc);
    T* dx = static_cast<T*>(p.dx) + row * p.D;
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
      const int c = (t + j * 32 * kTeam) * 8;
      const Raw8<T> hr = again(0, h, hs, j, c), gr = again(1, g, gs, j, c);
      Raw8<T> er;
      if (p.dh) er = load8<T, kRing>(e, c, p.D, src[2], src[2] + n);
      float wf[8];
      weight(j, wf);
      uint64_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t hv = bw::f2_pack(elem(hr.t[2 * i]), elem(hr.t[2 * i + 1]));
        const uint64_t gv = bw::f2_mul(bw::f2_pack(elem(gr.t[2 * i]), elem(gr.t[2 * i + 1])), rs2);
        const uint64_t d = bw::f2_fma(gv, hv, bw::f2_pack(dw[j][2 * i], dw[j][2 * i + 1]));
        dw[j][2 * i] = bw::f2_lo(d);
        dw[j][2 * i + 1] = bw::f2_hi(d);
        o[i] = bw::f2_fma(bw::f2_pack(wf[2 * i], wf[2 * i + 1]), gv, bw::f2_mul(c2, hv));
        if (p.dh) o[i] = bw::f2_add(o[i], bw::f2_pack(elem(er.t[2 * i]), elem(er.t[2 * i + 1])));
      }
      store8<T, kRing>(dx, c, p.D, o);
    }
    if constexpr (kRing) {
      team_sync();  // the buffer has been read
      if (t == 0 && row + stages * step < p.T) {
        bw::fence_proxy_async_smem();
        fetch(row + stages * step, st);
      }
      if (++st == stages) {
        st = 0;
        phase ^= 1;
      }
    }
  }
  // the CTA's part: its teams', summed in their order through the rings (every copy has landed and been read)
  __syncthreads();
  if (kRing && threadIdx.x == 0) {
    int bad = 0;
#pragma unroll
    for (int k = 0; k < kTeams; ++k) bad |= s_abort[k];
    p.flags[blockIdx.x] = bad;
  }
  float* s_dw = reinterpret_cast<float*>(ring);
  const int pad = (p.D + 7) & ~7;
#pragma unroll
  for (int j = 0; j < kNv; ++j) {
    const int c = (t + j * 32 * kTeam) * 8;
    if (c < p.D) {
      float4* d = reinterpret_cast<float4*>(s_dw + team * pad + c);
      d[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
      d[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.D; c += 32 * kBwdWarps) {
    float a = s_dw[c];
#pragma unroll
    for (int k = 1; k < kTeams; ++k) a += s_dw[k * pad + c];
    p.part[(int64_t)blockIdx.x * p.D + c] = a;
  }
}

// Rows too long for a team's registers and ring (above 16384 elements, 8192 in fp32): one a CTA at a time, rows
// blockIdx.x, + gridDim.x, ..., read twice (with the row kept in registers 8 vectors a thread spilled more; as it is, the
// instances of eight vectors spill 16 bytes in 16 bits and 96 in fp32). 0.9 to 1.8 TB/s.
template <typename T, int kNv>
__global__ void __launch_bounds__(kRowThreads, 1) norm_bwd_long_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float2 s_red[2][16];
  bw::griddep_launch_dependents();
  const int tpr = blockDim.x, t = threadIdx.x;
  const T *hs = static_cast<const T*>(p.h), *gs = static_cast<const T*>(p.dy), *es = static_cast<const T*>(p.dh);
  const int64_t n = p.T * p.D;
  float dw[kNv][8];
#pragma unroll
  for (int j = 0; j < kNv; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, turn ^= 1) {
    const T *h = hs + row * p.D, *g = gs + row * p.D, *e = es ? es + row * p.D : nullptr;
    T* dx = static_cast<T*>(p.dx) + row * p.D;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
      const int at = (t + j * tpr) * 8;
      const Raw8<T> hr = load8<T, false>(h, at, p.D, hs, hs + n), gr = load8<T, false>(g, at, p.D, gs, gs + n);
      float w[8];
      load_w8<false>(p.w, p.w_dtype, at, p.D, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hv = elem(hr.t[i]);
        sum.x = fmaf(hv, hv, sum.x);
        sum.y = fmaf(hv * w[i], elem(gr.t[i]), sum.y);
      }
    }
    sum = row_reduce<false>(sum, s_red[turn]);
    const float rs = rsqrtf(sum.x / (float)p.D + p.eps);
    const float c = rs * rs * rs * (sum.y / (float)p.D);
#pragma unroll
    for (int j = 0; j < kNv; ++j) {
      const int at = (t + j * tpr) * 8;
      const Raw8<T> hr = load8<T, false>(h, at, p.D, hs, hs + n), gr = load8<T, false>(g, at, p.D, gs, gs + n);
      float w[8], o[8];
      load_w8<false>(p.w, p.w_dtype, at, p.D, w);
      Raw8<T> er;
      if (e) er = load8<T, false>(e, at, p.D, es, es + n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hv = elem(hr.t[i]), gv = elem(gr.t[i]) * rs;
        dw[j][i] = fmaf(gv, hv, dw[j][i]);
        o[i] = fmaf(w[i], gv, -c * hv);
        if (e) o[i] += elem(er.t[i]);
      }
      uint64_t o2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o2[i] = bw::f2_pack(o[2 * i], o[2 * i + 1]);
      store8<T, false>(dx, at, p.D, o2);
    }
  }
#pragma unroll
  for (int j = 0; j < kNv; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = (t + j * tpr) * 8 + i;
      if (c < p.D) p.part[(int64_t)blockIdx.x * p.D + c] = dw[j][i];
    }
}

// dw: 32 columns to a CTA, 32 warps sum every 32nd part, then the warps' sums in order. The first CTA also makes the
// call's status of the flags.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float s[32][33];
  bw::griddep_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < p.D)
#pragma unroll 4
    for (int i = wid; i < p.parts; i += 32) a += p.part[(size_t)i * p.D + c];
  s[wid][lane] = a;
  int bad = 0;
  if (blockIdx.x == 0 && p.flags)
    for (int i = threadIdx.x; i < p.parts; i += 1024) bad |= p.flags[i];
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = bad ? kErrTimeout : kOk;
  if (wid == 0 && c < p.D) {
#pragma unroll
    for (int i = 1; i < 32; ++i) a += s[i][lane];
    p.dw[c] = a;
  }
}

// ------------------------------------------------------------------------------ host

struct NormShape {
  bool warp;
  int threads, nv;  // threads to a row and vectors of 8 to a thread
};
// Up to 256 elements a row is one warp's; up to 2048 a CTA's with one vector a thread; longer ones take
// two or more vectors a thread and at most 512 threads.
NormShape norm_shape(int D) {
  const int vecs = (D + 7) / 8;
  if (vecs <= 32) return {true, 32, 1};
  int nv = 1;
  while (vecs > nv * (nv == 1 ? 256 : kRowThreads)) nv *= 2;
  return {false, ((vecs + nv - 1) / nv + 31) / 32 * 32, nv};
}
// The backward's teams of warps: the fewest whose vectors (at most four a thread, two in fp32) cover the row;
// their rings then hold two rows at least. 0 where a row is too long for that.
int norm_team(int D, size_t esize) {
  for (int team = 1; team <= kBwdWarps; team *= 2)
    if (team * 256 * (esize == 4 ? 2 : 4) >= D) return team;
  return 0;
}
static_assert(kBwdRing / kBwdWarps >= 2 * 3 * 1024 * 2, "two rows of three tensors a warp");
// CTAs of the backward, each with a part of the weight's gradient
int norm_parts(int64_t T, int D, size_t esize, int sms) {
  const int team = norm_team(D, esize), per = team ? kBwdWarps / team : 1;  // rows at a time
  const int64_t rows = (T + per - 1) / per;
  return (int)(rows < sms ? (rows < 1 ? 1 : rows) : sms);
}

// Workspace: the status word, the CTAs' flags, their parts of the weight's gradient.
constexpr size_t kNormHeader = 256;
size_t norm_parts_at(int parts) { return kNormHeader + align_up(parts * sizeof(int32_t), 256); }
size_t norm_ws_bytes(int parts, int D) { return norm_parts_at(parts) + (size_t)parts * D * sizeof(float); }

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

// f(kNv, kWarp) as integral constants
template <typename F>
void by_shape(const NormShape& s, F&& f) {
  using std::integral_constant;
  if (s.warp)
    f(integral_constant<int, 1>{}, integral_constant<bool, true>{});
  else if (s.nv == 1)
    f(integral_constant<int, 1>{}, integral_constant<bool, false>{});
  else if (s.nv == 2)
    f(integral_constant<int, 2>{}, integral_constant<bool, false>{});
  else if (s.nv == 4)
    f(integral_constant<int, 4>{}, integral_constant<bool, false>{});
  else
    f(integral_constant<int, 8>{}, integral_constant<bool, false>{});
}

template <typename T, bool kVec>
void launch_fwd(const NormFwdParams& p, cudaStream_t st) {
  const NormShape s = norm_shape(p.D);
  by_shape(s, [&](auto nv, auto warp) {
    const unsigned grid = (unsigned)(warp ? (p.T + kWarpRows - 1) / kWarpRows : p.T);
    norm_fwd_kernel<T, nv, warp, kVec><<<grid, warp ? 32 * kWarpRows : s.threads, 0, st>>>(p);
  });
}
template <typename T, int kNv, int kTeam>
bool launch_team(const NormBwdParams& p, bool ring, int dev, cudaStream_t st) {
  if (!ring) {
    // the teams' parts are summed in shared memory: 16 rows of at most 1024 floats, whatever the team
    const size_t smem = (size_t)(kBwdWarps / kTeam) * ((p.D + 7) & ~7) * sizeof(float);
    static PerDevice set;
    if (smem > 48000 && !set.done(dev)) {
      if (cudaFuncSetAttribute(norm_bwd_team_kernel<T, kNv, kTeam, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kBwdWarps * 1024 * (int)sizeof(float)) != cudaSuccess)
        return false;
      set.mark(dev);
    }
    norm_bwd_team_kernel<T, kNv, kTeam, false><<<p.parts, 32 * kBwdWarps, smem, st>>>(p);
    return true;
  }
  static PerDevice set;
  if (!set.done(dev)) {
    if (cudaFuncSetAttribute(norm_bwd_team_kernel<T, kNv, kTeam, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kBwdRing) != cudaSuccess)
      return false;
    set.mark(dev);
  }
  norm_bwd_team_kernel<T, kNv, kTeam, true><<<p.parts, 32 * kBwdWarps, kBwdRing, st>>>(p);
  return true;
}
// vectors a thread: as the row needs in a team of one warp, the most in larger ones
template <typename T>
bool launch_bwd(const NormBwdParams& p, bool ring, int dev, cudaStream_t st) {
  constexpr int kMost = sizeof(T) == 4 ? 2 : 4;
  const int team = norm_team(p.D, sizeof(T));
  switch (team) {
    case 1:
      return p.D <= 256   ? launch_team<T, 1, 1>(p, ring, dev, st)
             : p.D <= 512 ? launch_team<T, 2, 1>(p, ring, dev, st)
                          : launch_team<T, kMost, 1>(p, ring, dev, st);
    case 2:
      return launch_team<T, kMost, 2>(p, ring, dev, st);
    case 4:
      return launch_team<T, kMost, 4>(p, ring, dev, st);
    case 8:
      return launch_team<T, kMost, 8>(p, ring, dev, st);
    case 16:
      return launch_team<T, kMost, 16>(p, ring, dev, st);
  }
  // 1024 vectors at least (fp32; 2048 else): 512 threads with the fewest vectors each that cover the row
  const int nv = (p.D + 8 * kRowThreads - 1) / (8 * kRowThreads);
  if (nv <= 4)
    norm_bwd_long_kernel<T, 4><<<p.parts, kRowThreads, 0, st>>>(p);
  else
    norm_bwd_long_kernel<T, 8><<<p.parts, kRowThreads, 0, st>>>(p);
  return true;
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

extern "C" size_t gdn_rmsnorm_workspace_size(int64_t T, int D, int dtype) {
  if (!gdn::dtype_ok(dtype) || T < 0 || T > (int64_t)INT32_MAX || D < 1 || D > gdn::kNormMaxD) return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    sms = 152;
  }
  return gdn::norm_ws_bytes(gdn::norm_parts(T, D, gdn::esize(dtype), sms), D);
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
  const int parts = norm_parts(T, D, e, sms);
  if (ws_bytes < norm_ws_bytes(parts, D)) return GDN_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool vec = D % 8 == 0 && al(h, 16) && al(dy, 16) && al(dh, 16) && al(dx, 16) && al(w, 16);
  const bool ring = vec && norm_team(D, e) != 0;
  const TestWithhold test = test_withhold();
  const NormBwdParams p{h,
                        w,
                        dy,
                        dh,
                        dx,
                        reinterpret_cast<float*>(ws + norm_parts_at(parts)),
                        dw,
                        reinterpret_cast<int32_t*>(ws),
                        ring ? reinterpret_cast<int32_t*>(ws + kNormHeader) : nullptr,
                        T,
                        test.copy,
                        test.budget,
                        D,
                        w_dtype,
                        parts,
                        eps};
  cudaStream_t st = (cudaStream_t)stream;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  const bool ok = dtype == GDN_DTYPE_BF16   ? launch_bwd<__nv_bfloat16>(p, ring, dev, st)
                  : dtype == GDN_DTYPE_FP16 ? launch_bwd<__half>(p, ring, dev, st)
                                            : launch_bwd<float>(p, ring, dev, st);
  if (!ok) return GDN_ERR_CUDA;
  launch_early(norm_dw_kernel, dim3((D + 31) / 32), 1024, 0, st, p);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
