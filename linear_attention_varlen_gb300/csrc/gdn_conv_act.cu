// Width-4 causal depthwise convolution with its activation over packed documents, forward and backward, and its step
// for single tokens (sm_103a). Per channel c and document with inputs x[0 .. n-1], as in the convolution without one:
//     E = (start[0], start[1], start[2], x[0], ..., x[n-1]),  u[p] = bias[c] + sum_m w[c][m] E[p + m],
//     y[p] = silu(u[p]),  tail = (E[n], E[n+1], E[n+2]);
// backward du = dy silu'(u), dE[e] = sum_m w[c][m] du[e - m] (+ dtail), dw[c][m] = sum_p du[p] E[p + m],
// dbias = sum_p du[p]. u is formed again from x: nothing but the inputs is kept between the two directions.
//
// All of it is bound by memory traffic: each input is read once, each output written once, but for the three rows
// before a block of tokens (and the three behind it in the backward). A thread takes four channels, in packed pairs, down
// the tokens of a block, the window of three inputs in registers; four rows at a time are worked on while the next four
// are on their way. Four rows of one document go without a look at its bounds.
// Measured (device time, bf16): 32768 x 2048 51 us (269 MB, 5.2 TB/s); backward of 16384 x 4096 101 us (537 MB, 5.3 TB/s; sixteen
// warps an SM, twenty spill: 200 us), sum over its blocks 6, tails 12; step of 200 x 8192 in fp16 7.5 us
// one after the other, 9.5 with cold caches. Eight channels to a thread without packed pairs took 79 and 227 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/gdn.h"
#include "bw_prims.cuh"
#include "elem.cuh"
#include "gdn_common.cuh"
#include "gdn_host.h"

namespace gdn {
namespace {

constexpr int kActThreads = 128;
constexpr int kFwdTokens = 32;                   // tokens to a block
constexpr int kBwdThreads = 64;
// Tokens to a block of the backward: few enough for small calls to spread, else 124. Blocks a power of two of rows
// apart meet in memory: 64 took 128, 96 took 126 and 124 took 116 us at 16384 x 4096.
constexpr int kBwdShort = 60, kBwdLong = 124;
// the fewest tokens that go in long blocks: eight CTAs of them to each SM
inline int64_t bwd_long_from(int C) {
  const int64_t cb = (C / 4 + kBwdThreads - 1) / kBwdThreads;
  return kBwdLong * ((8 * 152 + cb - 1) / cb);
}
constexpr int kRows = 4;                         // rows at a time
constexpr int kCh = 4, kPr = kCh / 2;             // channels of a thread, and their pairs

using bw::f2_add;
using bw::f2_fma;
using bw::f2_hi;
using bw::f2_lo;
using bw::f2_mul;
using bw::f2_pack;

struct ActHeader {
  int32_t status, deep;
  int32_t pad[62];
};

struct ActParams {
  const void *x, *dy;
  int64_t sx, sdy;  // elements between tokens
  const float *w, *bias;
  const int32_t *cu, *init_idx;
  const void* conv_init;
  int N, T, C, n_init, silu, n_tb, tokens;
  void *y, *tail;
  const float* dtail;  // given gradient of the tails
  float *dx, *dw, *dbias, *dinit;
  ActHeader* hd;
  float *dstart, *part;
  int32_t* kind;
  int2* link;
};

struct ActLayout {
  size_t header, kind, dstart, part, link, total;
  int n_tb, tokens;
};
inline ActLayout act_layout(int N, int T, int C, bool bwd) {
  ActLayout L{};
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t at = o;
    o = align_up(o + b, 256);
    return at;
  };
  L.tokens = !bwd ? kFwdTokens : T >= bwd_long_from(C) ? kBwdLong : kBwdShort;
  L.n_tb = (T + L.tokens - 1) / L.tokens;
  L.header = take(sizeof(ActHeader));
  if (bwd) {
    L.dstart = take((size_t)N * 3 * C * 4);     // gradient at each document's start
    L.kind = take(sizeof(int32_t) * N);
    // dw, dbias of each block of tokens: [block][5][C]. Room for those of any call of no more tokens, which may have more
    // (short) blocks, so that the size grows with T.
    const int64_t room = std::max<int64_t>(L.n_tb, (std::min<int64_t>(T, bwd_long_from(C) - 1) + kBwdShort - 1) / kBwdShort);
    L.part = take((size_t)room * C * 5 * 4);
    L.link = take(sizeof(int2) * N);            // documents of the same pool entry
  }
  L.total = o;
  return L;
}

// Row e (of three) in front of document d, and row k of its tail: an input, an entry of the pool, or null for zero.
// A fork's start is the tail of an earlier document, so the walk ends.
template <typename T>
__device__ __forceinline__ const T* start_row(const ActParams& p, int d, int e) {
  for (;;) {
    const int s = p.init_idx ? p.init_idx[d] : -1;
    if (s < 0) return nullptr;
    if (s < p.n_init) return static_cast<const T*>(p.conv_init) + ((int64_t)s * 3 + e) * p.C;
    d = s - p.n_init;
    e += p.cu[d + 1] - p.cu[d];
    if (e >= 3) return static_cast<const T*>(p.x) + ((int64_t)p.cu[d] + e - 3) * p.sx;
  }
}

__device__ __forceinline__ int doc_at(const int32_t* cu, int N, int t) {  // the document that holds token t
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Four channels as they lie in memory.
template <typename T>
struct alignas(sizeof(T) * kCh) Raw4 {
  uint32_t w[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw4<T> row_or_zero(const T* row, int c) {
  Raw4<T> r{};
  if (row) r = *reinterpret_cast<const Raw4<T>*>(row + c);
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw4<T>& r, uint64_t* f) {
#pragma unroll
  for (int i = 0; i < kPr; ++i) f[i] = pair_of<T>(r.w, i);
}

// Block 0 checks cu_seqlens and init_idx. The others (backward with a pool): which documents share an entry, and the
// entries' gradients set to zero.
__global__ void __launch_bounds__(256) act_check_kernel(const __grid_constant__ ActParams p) {
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (blockIdx.x > 0) {
    const int64_t n = (int64_t)p.n_init * 3 * p.C, step = (int64_t)(gridDim.x - 1) * 256;
    const int64_t i0 = (int64_t)(blockIdx.x - 1) * 256 + threadIdx.x;
    link_pool_starts(p.init_idx, p.N, p.n_init, p.link, i0 / 32, step / 32);
    for (int64_t i = i0; i < n; i += step) p.dinit[i] = 0.f;
    return;
  }
  __shared__ int s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.N; i += 256) {
    const int b = p.cu[i], e = p.cu[i + 1], x = p.init_idx ? p.init_idx[i] : -1;
    if (b < 0 || e < b || e > p.T || (i == 0 && b != 0) || (i == p.N - 1 && e != p.T) || x < -1 || (x >= p.n_init && x - p.n_init >= i))
      s_bad = 1;
  }
  __syncthreads();
  const bool deep = !s_bad && p.kind && fork_kinds(p.init_idx, p.N, p.n_init, p.kind);
  if (threadIdx.x == 0) {
    p.hd->deep = deep;
    p.hd->status = s_bad ? kErrInvalid : 0;
  }
}

struct Taps {
  uint64_t w[4][kPr], bias[kPr];
  __device__ __forceinline__ Taps(const float* wp, const float* bp, int c) {
    float4 v[kCh];
#pragma unroll
    for (int i = 0; i < kCh; ++i) v[i] = *reinterpret_cast<const float4*>(wp + (int64_t)(c + i) * 4);
#pragma unroll
    for (int i = 0; i < kPr; ++i) {
      w[0][i] = f2_pack(v[2 * i].x, v[2 * i + 1].x), w[1][i] = f2_pack(v[2 * i].y, v[2 * i + 1].y);
      w[2][i] = f2_pack(v[2 * i].z, v[2 * i + 1].z), w[3][i] = f2_pack(v[2 * i].w, v[2 * i + 1].w);
      bias[i] = bp ? f2_pack(bp[c + 2 * i], bp[c + 2 * i + 1]) : 0;
    }
  }
  // u of the fourth of four consecutive inputs
  __device__ __forceinline__ uint64_t dot(int i, uint64_t a, uint64_t b, uint64_t c, uint64_t d) const {
    return f2_fma(w[3][i], d, f2_fma(w[2][i], c, f2_fma(w[1][i], b, f2_fma(w[0][i], a, bias[i]))));
  }
};

// Blocks of kFwdTokens tokens, then one block for each document's tail.
template <typename T>
__global__ void __launch_bounds__(kActThreads) act_fwd_kernel(const __grid_constant__ ActParams p) {
  using P = Raw4<T>;
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (p.hd->status != 0) return;
  const int c = (blockIdx.y * kActThreads + threadIdx.x) * kCh;
  if (c >= p.C) return;
  if ((int)blockIdx.x >= p.n_tb) {
    const int d = blockIdx.x - p.n_tb, n = p.cu[d + 1] - p.cu[d];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const T* row = n + k >= 3 ? static_cast<const T*>(p.x) + ((int64_t)p.cu[d] + n + k - 3) * p.sx : start_row<T>(p, d, n + k);
      *reinterpret_cast<P*>(static_cast<T*>(p.tail) + ((int64_t)d * 3 + k) * p.C + c) = row_or_zero<T>(row, c);
    }
    return;
  }
  const int t0 = blockIdx.x * kFwdTokens, t1 = min(t0 + kFwdTokens, p.T);
  const T* x = static_cast<const T*>(p.x) + c;
  T* y = static_cast<T*>(p.y) + c;
  P next[kRows];
  auto fetch = [&](int t) {
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (t + k < t1) next[k] = *reinterpret_cast<const P*>(x + (int64_t)(t + k) * p.sx);
  };
  fetch(t0);
  const Taps taps(p.w, p.bias, c);
  int d = doc_at(p.cu, p.N, t0), end = p.cu[d + 1];
  uint64_t win[3][kPr];  // the three inputs before the token
  auto window = [&](int t) {
    const int at = t - p.cu[d];
#pragma unroll
    for (int k = 0; k < 3; ++k)
      unpack(row_or_zero<T>(at + k >= 3 ? static_cast<const T*>(p.x) + ((int64_t)t + k - 3) * p.sx : start_row<T>(p, d, at + k), c),
             win[k]);
  };
  auto put = [&](int t, const uint64_t* u) {
    P o;
#pragma unroll
    for (int i = 0; i < kPr; ++i) set_pair<T>(o.w, i, p.silu ? silu_pair(u[i]) : u[i]);
    *reinterpret_cast<P*>(y + (int64_t)t * p.C) = o;
  };
  window(t0);
  for (int ta = t0; ta < t1; ta += kRows) {
    P r[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) r[k] = next[k];
    fetch(ta + kRows);
    if (ta + kRows <= t1 && ta + kRows <= end) {
      uint64_t e[kRows + 3][kPr];
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < kPr; ++i) e[k][i] = win[k][i];
#pragma unroll
      for (int k = 0; k < kRows; ++k) unpack(r[k], e[k + 3]);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        uint64_t u[kPr];
#pragma unroll
        for (int i = 0; i < kPr; ++i) u[i] = taps.dot(i, e[k][i], e[k + 1][i], e[k + 2][i], e[k + 3][i]);
        put(ta + k, u);
      }
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < kPr; ++i) win[k][i] = e[kRows + k][i];
      continue;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int t = ta + k;
      if (t >= t1) break;
      if (t >= end) {
        while (p.cu[d + 1] <= t) ++d;
        end = p.cu[d + 1];
        window(t);
      }
      uint64_t cur[kPr], u[kPr];
      unpack(r[k], cur);
#pragma unroll
      for (int i = 0; i < kPr; ++i) {
        u[i] = taps.dot(i, win[0][i], win[1][i], win[2][i], cur[i]);
        win[0][i] = win[1][i];
        win[1][i] = win[2][i];
        win[2][i] = cur[i];
      }
      put(t, u);
    }
  }
}

// Blocks of p.tokens tokens. du runs up the tokens once; the gradient of an input is complete three tokens later, so a
// block goes three tokens beyond its own (as far as its last document) and leaves dw and dbias of those to the next.
template <typename T>
__global__ void __launch_bounds__(kBwdThreads) act_bwd_kernel(const __grid_constant__ ActParams p) {
  using P = Raw4<T>;
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (p.hd->status != 0) return;
  const int c = (blockIdx.y * kBwdThreads + threadIdx.x) * kCh;
  if (c >= p.C) return;
  const int t0 = blockIdx.x * p.tokens, t1 = min(t0 + p.tokens, p.T), stop = min(p.T, t1 + 3);
  const T *x = static_cast<const T*>(p.x) + c, *dy = static_cast<const T*>(p.dy) + c;
  P xn[kRows], gn[kRows];
  auto fetch = [&](int t) {
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (t + k < stop) {
        xn[k] = *reinterpret_cast<const P*>(x + (int64_t)(t + k) * p.sx);
        gn[k] = *reinterpret_cast<const P*>(dy + (int64_t)(t + k) * p.sdy);
      }
  };
  fetch(t0);
  const Taps taps(p.w, p.bias, c);
  uint64_t win[3][kPr], pend[3][kPr], dw[5][kPr];
#pragma unroll
  for (int i = 0; i < kPr; ++i) {
#pragma unroll
    for (int m = 0; m < 5; ++m) dw[m][i] = 0;
    pend[0][i] = pend[1][i] = pend[2][i] = 0;
  }
  int d = doc_at(p.cu, p.N, t0), begin = p.cu[d], end = p.cu[d + 1];
  auto window = [&](int t) {
    const int at = t - begin;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      unpack(row_or_zero<T>(at + k >= 3 ? static_cast<const T*>(p.x) + ((int64_t)t + k - 3) * p.sx : start_row<T>(p, d, at + k), c),
             win[k]);
  };
  auto slope = [&](uint64_t u) { return silu_slope_pair(u, sigmoid_pair(u)); };
  auto write = [&](float* to, const uint64_t* g) {
    *reinterpret_cast<float4*>(to + c) = make_float4(f2_lo(g[0]), f2_hi(g[0]), f2_lo(g[1]), f2_hi(g[1]));
  };
  // the gradient of E[e] of document d, complete: an input of this block, or a row of the document's start
  auto emit = [&](int e, const uint64_t* g) {
    if (e < 3) {
      if (begin >= t0) write(p.dstart + ((int64_t)d * 3 + e) * p.C, g);
    } else if (begin + e - 3 >= t0 && begin + e - 3 < t1) {
      write(p.dx + ((int64_t)begin + e - 3) * p.C, g);
    }
  };
  window(t0);
  for (int ta = t0; ta < stop; ta += kRows) {
    P xr[kRows], gr[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) xr[k] = xn[k], gr[k] = gn[k];
    fetch(ta + kRows);
    if (ta + kRows <= t1 && ta + kRows <= end && ta - 3 >= t0 && ta - 3 >= begin) {
      uint64_t e[kRows + 3][kPr], g[kRows + 3][kPr];
#pragma unroll
      for (int i = 0; i < kPr; ++i) {
#pragma unroll
        for (int k = 0; k < 3; ++k) e[k][i] = win[k][i], g[k][i] = pend[k][i];
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        unpack(xr[k], e[k + 3]);
        uint64_t du[kPr];
        unpack(gr[k], du);
#pragma unroll
        for (int i = 0; i < kPr; ++i) {
          if (p.silu) du[i] = f2_mul(du[i], slope(taps.dot(i, e[k][i], e[k + 1][i], e[k + 2][i], e[k + 3][i])));
#pragma unroll
          for (int m = 0; m < 4; ++m) dw[m][i] = f2_fma(du[i], e[k + m][i], dw[m][i]);
          dw[4][i] = f2_add(dw[4][i], du[i]);
#pragma unroll
          for (int m = 0; m < 3; ++m) g[k + m][i] = f2_fma(taps.w[m][i], du[i], g[k + m][i]);
          g[k + 3][i] = f2_mul(taps.w[3][i], du[i]);
        }
        write(p.dx + (int64_t)(ta + k - 3) * p.C, g[k]);
      }
#pragma unroll
      for (int i = 0; i < kPr; ++i) {
#pragma unroll
        for (int k = 0; k < 3; ++k) win[k][i] = e[kRows + k][i], pend[k][i] = g[kRows + k][i];
      }
      continue;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int t = ta + k;
      if (t >= stop) break;
      if (t >= end) {
        if (t >= t1) break;  // behind the block only the rest of its last document counts
#pragma unroll
        for (int m = 0; m < 3; ++m) emit(end - begin + m, pend[m]);
        while (p.cu[d + 1] <= t) ++d;
        begin = p.cu[d];
        end = p.cu[d + 1];
        window(t);
#pragma unroll
        for (int i = 0; i < kPr; ++i) pend[0][i] = pend[1][i] = pend[2][i] = 0;
      }
      uint64_t cur[kPr], du[kPr], done[kPr];
      unpack(xr[k], cur);
      unpack(gr[k], du);
#pragma unroll
      for (int i = 0; i < kPr; ++i) {
        if (p.silu) du[i] = f2_mul(du[i], slope(taps.dot(i, win[0][i], win[1][i], win[2][i], cur[i])));
        if (t < t1) {
          dw[0][i] = f2_fma(du[i], win[0][i], dw[0][i]);
          dw[1][i] = f2_fma(du[i], win[1][i], dw[1][i]);
          dw[2][i] = f2_fma(du[i], win[2][i], dw[2][i]);
          dw[3][i] = f2_fma(du[i], cur[i], dw[3][i]);
          dw[4][i] = f2_add(dw[4][i], du[i]);
        }
        done[i] = f2_fma(taps.w[0][i], du[i], pend[0][i]);
        pend[0][i] = f2_fma(taps.w[1][i], du[i], pend[1][i]);
        pend[1][i] = f2_fma(taps.w[2][i], du[i], pend[2][i]);
        pend[2][i] = f2_mul(taps.w[3][i], du[i]);
        win[0][i] = win[1][i];
        win[1][i] = win[2][i];
        win[2][i] = cur[i];
      }
      emit(t - begin, done);
    }
  }
  if (end <= stop) {  // the document ended within reach: its last inputs are complete
#pragma unroll
    for (int m = 0; m < 3; ++m) emit(end - begin + m, pend[m]);
  }
#pragma unroll
  for (int m = 0; m < 5; ++m) write(p.part + ((int64_t)blockIdx.x * 5 + m) * p.C, dw[m]);
}

// dw[.][m], or dbias (m = 4), m = blockIdx.y, over the blocks of tokens in a fixed order: 32 channels a CTA, each summed
// by eight threads.
__global__ void __launch_bounds__(256) act_sum_kernel(const __grid_constant__ ActParams p) {
  __shared__ float s[8][32];
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (p.hd->status != 0) return;
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, m = blockIdx.y;
  float v = 0.f;
  if (c < p.C) {
#pragma unroll 8
    for (int b = r; b < p.n_tb; b += 8) v += p.part[((int64_t)b * 5 + m) * p.C + c];
  }
  s[r][lane] = v;
  __syncthreads();
  if (r == 0 && c < p.C) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][lane];
    if (m < 4)
      p.dw[(int64_t)c * 4 + m] = v;
    else if (p.dbias)
      p.dbias[c] = v;
  }
}

// The tails' gradients, given ones and those of forks, into the inputs they copy or on into the document's start. One
// thread to a channel and the documents of blockIdx.y, in three steps as the scan's (kStep).
template <int kStep>
__global__ void __launch_bounds__(256) act_ends_kernel(const __grid_constant__ ActParams p) {
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (p.hd->status != 0 || (kStep == 2 && !p.hd->deep)) return;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.C) return;
  const int step = gridDim.y, d0 = blockIdx.y;
  for (int d = d0 + (p.N - 1 - d0) / step * step; d >= 0; d -= step) {
    if (source_step(p.kind[d]) != kStep) continue;
    const int t0 = p.cu[d], n = p.cu[d + 1] - t0;
    float* start = p.dstart + (int64_t)d * 3 * p.C + c;
    float g[3], v[3];
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      g[e] = n > 0 ? start[(int64_t)e * p.C] : 0.f;
      v[e] = p.dtail ? p.dtail[((int64_t)d * 3 + e) * p.C + c] : 0.f;
    }
    if (kStep > 0) {
      constexpr int kAhead = 8;
      for (int f0 = d + 1; f0 < p.N; f0 += kAhead) {
        float f[kAhead][3];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const bool mine = f0 + j < p.N && p.init_idx[f0 + j] == p.n_init + d;
#pragma unroll
          for (int e = 0; e < 3; ++e) f[j][e] = mine ? p.dstart[((int64_t)(f0 + j) * 3 + e) * p.C + c] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int e = 0; e < 3; ++e) v[e] += f[j][e];
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (n + k >= 3) {
        if (p.dtail || kStep > 0) p.dx[((int64_t)t0 + n + k - 3) * p.C + c] += v[k];
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (e == n + k) g[e] += v[k];
      }
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) start[(int64_t)e * p.C] = g[e];
  }
}

// The gradients of the pool entries that some document starts from: their documents' start gradients, in order.
__global__ void __launch_bounds__(256) act_pool_kernel(const __grid_constant__ ActParams p) {
  bw::griddep_wait();
  if (p.hd->status != 0) return;
  const int64_t row = 3 * (int64_t)p.C;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.N * row; i += (int64_t)gridDim.x * 256) {
    int d = (int)(i / row);
    if (!p.link[d].y) continue;
    const int64_t r = i - d * row, e = p.init_idx[d];
    float v = 0.f;
    for (; d >= 0; d = p.link[d].x) v += p.dstart[d * row + r];
    p.dinit[e * row + r] = v;
  }
}

struct StepParams {
  const void* x;
  int64_t sx;
  const float *w, *bias;
  const int32_t* idx;
  void *pool, *y;
  int32_t* status;
  int B, C, n_pool, silu;
};

template <typename T>
__global__ void __launch_bounds__(kActThreads) act_step_kernel(const __grid_constant__ StepParams p) {
  using P = Raw4<T>;
  const int64_t b = blockIdx.y;
  const int c = (blockIdx.x * kActThreads + threadIdx.x) * kCh, e = p.idx[b];
  if (c >= p.C) return;
  P* out = reinterpret_cast<P*>(static_cast<T*>(p.y) + b * p.C + c);
  if (e < 0 || e >= p.n_pool) {  // skipped, reported
    *out = P{};
    if (threadIdx.x == 0 && p.status) atomicCAS(p.status, 0, kErrInvalid);
    return;
  }
  T* tail = static_cast<T*>(p.pool) + (int64_t)e * 3 * p.C + c;
  P r[4];
#pragma unroll
  for (int k = 0; k < 3; ++k) r[k] = *reinterpret_cast<const P*>(tail + (int64_t)k * p.C);
  r[3] = *reinterpret_cast<const P*>(static_cast<const T*>(p.x) + b * p.sx + c);
  const Taps taps(p.w, p.bias, c);
  P o;
#pragma unroll
  for (int i = 0; i < kPr; ++i) {
    const uint64_t u = taps.dot(i, pair_of<T>(r[0].w, i), pair_of<T>(r[1].w, i), pair_of<T>(r[2].w, i), pair_of<T>(r[3].w, i));
    set_pair<T>(o.w, i, p.silu ? silu_pair(u) : u);
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) *reinterpret_cast<P*>(tail + (int64_t)k * p.C) = r[k + 1];
  *out = o;
}

// ------------------------------------------------------------------------------ host

bool al(const void* p, uintptr_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }
int elem_size(int dtype) { return dtype == GDN_DTYPE_FP32 ? 4 : 2; }

int check_device(const void* anchor, const void* const* ptrs, int n, DeviceGuard& guard) {
  int dev = 0;
  if (device_of(anchor, ptrs, n, &dev) != kOk) return GDN_ERR_INVALID_ARG;
  if (!guard.set(dev)) return GDN_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return GDN_ERR_CUDA;
  return major == 10 && minor == 3 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

int check_kind(int dtype, int activation) {
  if (dtype != GDN_DTYPE_BF16 && dtype != GDN_DTYPE_FP16 && dtype != GDN_DTYPE_FP32) return GDN_ERR_UNSUPPORTED;
  return activation == GDN_ACT_NONE || activation == GDN_ACT_SILU ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// Block counts and the token loops' bounds stay within 31 bits.
bool sizes_ok(int N, int T, int C) {
  return N >= 1 && N <= (1 << 30) && T >= 0 && T <= INT32_MAX - 4096 && C >= 8 && C <= (1 << 23) && C % 8 == 0 &&
         (int64_t)T * C <= ((int64_t)1 << 40);
}

// The elements between two tokens: 0 = contiguous; rows start on 16 bytes.
bool stride_ok(int64_t* s, int C, int dtype) {
  if (*s == 0) *s = C;
  return *s >= C && *s <= ((int64_t)1 << 40) && *s * elem_size(dtype) % 16 == 0;
}

int check_packed(ActParams* p, int dtype, const void* workspace) {
  if (!sizes_ok(p->N, p->T, p->C) || p->n_init < 0) return GDN_ERR_INVALID_ARG;
  if (!p->cu || !p->w || !workspace || (p->T > 0 && !p->x) || (p->n_init > 0 && !p->conv_init)) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(&p->sx, p->C, dtype) || !stride_ok(&p->sdy, p->C, dtype)) return GDN_ERR_INVALID_ARG;
  if (!al(p->x, 16) || !al(p->dy, 16) || !al(p->w, 16) || !al(p->conv_init, 16) || !al(workspace, 256) || !al(p->bias, 4) ||
      !al(p->cu, 4) || !al(p->init_idx, 4))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
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

}  // namespace
}  // namespace gdn

extern "C" size_t gdn_conv_act_workspace_size(int N, int T, int C, int backward) {
  if (!gdn::sizes_ok(N, T, C)) return 0;
  return gdn::act_layout(N, T, C, backward != 0).total;
}

extern "C" int gdn_conv_act_fwd(const void* x, int64_t x_stride, const float* w, const float* bias,
                                const int32_t* cu_seqlens, int N, int T, int C, int dtype, int activation,
                                const int32_t* init_idx, const void* conv_init, int n_init, void* y, void* final_tail,
                                void* workspace, size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  int rc = check_kind(dtype, activation);
  if (rc != GDN_OK) return rc;
  ActParams p{};
  p.x = x, p.sx = x_stride, p.w = w, p.bias = bias, p.cu = cu_seqlens, p.init_idx = init_idx, p.conv_init = conv_init;
  p.N = N, p.T = T, p.C = C, p.n_init = n_init, p.silu = activation == GDN_ACT_SILU, p.y = y, p.tail = final_tail;
  if ((rc = check_packed(&p, dtype, workspace)) != GDN_OK) return rc;
  if (!final_tail || (T > 0 && !y) || !al(y, 16) || !al(final_tail, 16)) return GDN_ERR_INVALID_ARG;
  const ActLayout L = act_layout(N, T, C, false);
  if (ws_bytes < L.total) return GDN_ERR_WORKSPACE;
  const void* ptrs[] = {x, w, bias, cu_seqlens, init_idx, conv_init, y, final_tail};
  DeviceGuard guard;
  if ((rc = check_device(workspace, ptrs, (int)(sizeof(ptrs) / sizeof(ptrs[0])), guard)) != GDN_OK) return rc;
  p.hd = static_cast<ActHeader*>(workspace);
  p.n_tb = L.n_tb;
  p.tokens = L.tokens;
  cudaStream_t s = (cudaStream_t)stream;
  launch_early(act_check_kernel, dim3(1), 256, 0, s, p);
  by_type(dtype, [&](auto t) {
    using T_ = decltype(t);
    const unsigned cb = (unsigned)((C / kCh + kActThreads - 1) / kActThreads);
    launch_early(act_fwd_kernel<T_>, dim3((unsigned)(L.n_tb + N), cb), kActThreads, 0, s, p);
  });
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_conv_act_bwd(const void* x, int64_t x_stride, const float* w, const float* bias,
                                const int32_t* cu_seqlens, int N, int T, int C, int dtype, int activation,
                                const int32_t* init_idx, const void* conv_init, int n_init, const void* dy,
                                int64_t dy_stride, const float* dfinal_tail, float* dx, float* dw, float* dbias,
                                float* dconv_init, void* workspace, size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  int rc = check_kind(dtype, activation);
  if (rc != GDN_OK) return rc;
  ActParams p{};
  p.x = x, p.sx = x_stride, p.w = w, p.bias = bias, p.cu = cu_seqlens, p.init_idx = init_idx, p.conv_init = conv_init;
  p.N = N, p.T = T, p.C = C, p.n_init = n_init, p.silu = activation == GDN_ACT_SILU, p.dy = dy, p.sdy = dy_stride;
  p.dtail = dfinal_tail, p.dx = dx, p.dw = dw, p.dbias = dbias, p.dinit = dconv_init;
  if ((rc = check_packed(&p, dtype, workspace)) != GDN_OK) return rc;
  if (!dw || (T > 0 && (!dy || !dx)) || (n_init > 0 && !dconv_init)) return GDN_ERR_INVALID_ARG;
  if (!al(dx, 16) || !al(dw, 4) || !al(dbias, 4) || !al(dfinal_tail, 4) || !al(dconv_init, 4)) return GDN_ERR_INVALID_ARG;
  const ActLayout L = act_layout(N, T, C, true);
  if (ws_bytes < L.total) return GDN_ERR_WORKSPACE;
  const void* ptrs[] = {x, w, bias, cu_seqlens, init_idx, conv_init, dy, dfinal_tail, dx, dw, dbias, dconv_init};
  DeviceGuard guard;
  if ((rc = check_device(workspace, ptrs, (int)(sizeof(ptrs) / sizeof(ptrs[0])), guard)) != GDN_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.hd = reinterpret_cast<ActHeader*>(ws + L.header);
  p.dstart = reinterpret_cast<float*>(ws + L.dstart);
  p.kind = reinterpret_cast<int32_t*>(ws + L.kind);
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.link = reinterpret_cast<int2*>(ws + L.link);
  p.n_tb = L.n_tb;
  p.tokens = L.tokens;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t zeros = n_init > 0 ? ((int64_t)n_init * 3 * C + 32 * (int64_t)N + 1023) / 1024 : 0;  // blocks
  launch_early(act_check_kernel, dim3((unsigned)(1 + (zeros < 1024 ? zeros : 1024))), 256, 0, s, p);
  if (T > 0)
    by_type(dtype, [&](auto t) {
      using T_ = decltype(t);
      const unsigned cb = (unsigned)((C / kCh + kBwdThreads - 1) / kBwdThreads);
      launch_early(act_bwd_kernel<T_>, dim3((unsigned)L.n_tb, cb), kBwdThreads, 0, s, p);
    });
  launch_early(act_sum_kernel, dim3((unsigned)((C + 31) / 32), 5), 256, 0, s, p);
  const unsigned cb = (unsigned)((C + 255) / 256), db = (unsigned)(N < 64 ? N : 64);
  if (dfinal_tail || init_idx) launch_early(act_ends_kernel<0>, dim3(cb, db), 256, 0, s, p);
  if (init_idx && N > 1) launch_early(act_ends_kernel<1>, dim3(cb, db), 256, 0, s, p);
  if (init_idx && N > 2) launch_early(act_ends_kernel<2>, dim3(cb, 1), 256, 0, s, p);  // a fork of a fork is a third
  if (n_init > 0 && init_idx) {
    const int64_t blocks = ((int64_t)N * 3 * C + 255) / 256;
    launch_early(act_pool_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), 256, 0, s, p);
  }
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_conv_decode_step(const void* x, int64_t x_stride, const float* w, const float* bias, int B, int C,
                                    int dtype, int activation, const int32_t* state_idx, void* tail_pool, int n_pool,
                                    void* y, int32_t* status, gdn_stream_t stream) {
  using namespace gdn;
  int rc = check_kind(dtype, activation);
  if (rc != GDN_OK) return rc;
  if (B < 0 || B > 65535 || C < 8 || C > (1 << 23) || C % 8 != 0 || n_pool < 0) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(&x_stride, C, dtype)) return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  if (!x || !w || !state_idx || !tail_pool || !y || n_pool == 0) return GDN_ERR_INVALID_ARG;
  if (!al(x, 16) || !al(w, 16) || !al(tail_pool, 16) || !al(y, 16) || !al(bias, 4) || !al(state_idx, 4) || !al(status, 4))
    return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {x, w, bias, state_idx, y, status};
  DeviceGuard guard;
  if ((rc = check_device(tail_pool, ptrs, (int)(sizeof(ptrs) / sizeof(ptrs[0])), guard)) != GDN_OK) return rc;
  const StepParams p{x, x_stride, w, bias, state_idx, tail_pool, y, status, B, C, n_pool, activation == GDN_ACT_SILU};
  by_type(dtype, [&](auto t) {
    using T_ = decltype(t);
    const unsigned cb = (unsigned)((C / kCh + kActThreads - 1) / kActThreads);
    act_step_kernel<T_><<<dim3(cb, (unsigned)B), kActThreads, 0, (cudaStream_t)stream>>>(p);
  });
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
