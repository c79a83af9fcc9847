// Selective scan over packed documents, forward and backward (sm_103a). Per channel c with states s (group g of the
// maps b, c: channel / (channels / groups)):
//     dt = softplus(raw + dt_bias),  h_t = exp(dt_t a) h_{t-1} + dt_t x_t b_t,  y_t = sum_s c_t h_t + skip x_t,
//     out = y silu(z)
// with a decay for each channel and state and a step for each token and channel, so that a token's map has no
// low-rank form to put on the tensor cores: the walk is fp32 arithmetic, an exponential, two products and two
// multiply-adds for each token, channel and state.
//
// Documents are cut into segments so that a long one fills the GPU. The first walk leaves each segment's end state
// from zero and its summed time; the scan kernel makes start states of them (exp(a sum dt) carries a state across a
// segment); the second walk starts from those. A document of one segment is walked once. Backward, with k_t the
// gradient of h_t:
//     k_t = c_t dy_t + exp(dt_{t+1} a) k_{t+1},  dc = dy h,  db = dt x k,  du = sum_s k b  (u = dt x),
//     d dt = x du + sum_s a k exp(dt a) h_{t-1},  da = sum_t dt k exp(dt a) h_{t-1}
// the first walk also leaves the gradient of each segment's start state for a zero gradient behind it
// (sum_t exp(a (dt_1 + .. + dt_t)) c_t dy_t, formed forward in time) and the state at every 16th (8th) token, so that the
// walk in reverse needs no state but a tile's.
//
// What bounds it is its instructions, not memory: the recurrence alone, 32 exponentials and 48 packed products for a token
// of a warp's 64 channels and 16 states, takes 168 clocks of a scheduler (an exponential 4.4, a packed product with three
// operands 2.6) of the 243 and 356 that the two walks take, and what is done once for a token and channel takes as many
// instructions again. So that part is in packed pairs too and without branches, and the inputs come by asynchronous
// copies. No pipe is full, though: forward 61 to 64 % of the issue slots and 46 to 60 % of the FMA and exponential pipes are
// in use, in reverse 53, 46 and 29 %. With three warps to a scheduler (two in reverse, whose registers allow no more)
// instructions wait for the ones before. Measured (device time, bf16, 16 states):
//     32768 x 2048, one document      walks 203 + 298 us, planner and scan 21; its bytes once would take 81
//     9001 x 2048, 12 documents       walks 64 + 94 us
//     backward, 16384 x 2048          first walk 179 us, walk in reverse 594, planner, scan and sums 33; bytes once 71
//     backward, 1501 x 768 x 8 fp32   10 + 31 us, planner, scan and sums 30
//
// Every sum has a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gdn.h"
#include "bw_prims.cuh"
#include "elem.cuh"
#include "gdn_common.cuh"
#include "gdn_host.h"
#include "gdn_ssm.h"

namespace gdn {
namespace {

using bw::f2_fma;
using bw::f2_hi;
using bw::f2_lo;
using bw::f2_mul;
using bw::f2_pack;
using bw::f2_sum;

constexpr int kGradSub = 4;  // tokens whose states the backward's walk holds at once
constexpr int kPlanThreads = 1024;

struct SsmParams {
  const void *x, *dt, *z, *b, *c, *dout;
  int64_t sx, sdt, sz, sb, sc, sdo;  // elements between tokens
  const float *a, *skip, *dt_bias, *init;
  const int32_t *cu, *init_idx;
  int N, T, C, S, G, n_init, softplus, dtype;
  void* out;
  float* final_state;
  // backward
  const float* dfinal;
  void *dx, *ddt, *dz, *db, *dc;
  float *da, *dskip, *dbias, *dinit;
  // workspace
  SsmHeader* hd;
  SsmSeg* segs;
  int32_t *seg0, *kind;
  int2* link;
  float *maps, *slot, *sums, *slot_r, *ckpt, *csum, *dstart, *fin, *part_a, *part_c, *part_m;
  int64_t smax;
  int parts, seg_tokens, bwd, whole;
};

// ------------------------------------------------------------------------------ planner, maps in fp32

// A warp takes whole tokens, its lanes four states of a map each.
template <typename T>
__device__ void maps_to_float(const SsmParams& p, int block, int blocks) {
  const int Q = ssm_padded(p.S) / 4, row = p.G * 2 * Q;  // quads to a token
  const int lane = threadIdx.x & 31, per = row < 32 ? 32 / row : 1, sub = row < 32 ? lane / row : 0;
  const int64_t step = (int64_t)blocks * (blockDim.x / 32) * per;
  if (sub >= per) return;
  for (int64_t t = ((int64_t)block * (blockDim.x / 32) + (threadIdx.x >> 5)) * per + sub; t < p.T; t += step)
    for (int i = row < 32 ? lane - sub * row : lane; i < row; i += 32) {
      const int g = i / (2 * Q), r = i - g * 2 * Q, q = r < Q ? r : r - Q;
      const T* from = r < Q ? static_cast<const T*>(p.b) + t * p.sb : static_cast<const T*>(p.c) + t * p.sc;
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = 4 * q + k < p.S ? to_float(from[g * p.S + 4 * q + k]) : 0.f;
      *reinterpret_cast<float4*>(p.maps + (t * row + i) * 4) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// Block 0: checks cu_seqlens and init_idx and cuts the documents into segments of at most seg_tokens. The others:
// the maps b and c in fp32, [T][G][2][Sp], zero behind the last state; in the backward which documents share a pool entry,
// and the entries' gradients set to zero.
__global__ void __launch_bounds__(kPlanThreads) ssm_plan_kernel(const __grid_constant__ SsmParams p) {
  bw::griddep_wait();  // the call before on this stream may still read the workspace
  bw::griddep_launch_dependents();
  if (blockIdx.x > 0) {
    if (p.bwd && p.n_init > 0) {
      const int64_t n = (int64_t)p.n_init * p.C * p.S, step = (int64_t)(gridDim.x - 1) * blockDim.x;
      const int64_t i0 = (int64_t)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
      link_pool_starts(p.init_idx, p.N, p.n_init, p.link, i0 / 32, step / 32);
      for (int64_t i = i0; i < n; i += step) p.dinit[i] = 0.f;
    }
    if (p.dtype == GDN_DTYPE_BF16)
      maps_to_float<__nv_bfloat16>(p, blockIdx.x - 1, gridDim.x - 1);
    else if (p.dtype == GDN_DTYPE_FP16)
      maps_to_float<__half>(p, blockIdx.x - 1, gridDim.x - 1);
    else
      maps_to_float<float>(p, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  __shared__ int s_warp[32], s_base, s_bad, s_long, s_doc[kPlanThreads], s_at[kPlanThreads], s_k[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) s_base = s_bad = 0;
  __syncthreads();
  for (int i = tid; i < p.N; i += kPlanThreads) {
    const int b = p.cu[i], e = p.cu[i + 1], x = p.init_idx ? p.init_idx[i] : -1;
    if (b < 0 || e < b || e > p.T || (i == 0 && b != 0) || (i == p.N - 1 && e != p.T) || x < -1 || (x >= p.n_init && x - p.n_init >= i))
      s_bad = 1;
  }
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      p.hd->status = kErrInvalid;
      p.hd->n_segs = 0;
    }
    return;
  }
  const bool deep = fork_kinds(p.init_idx, p.N, p.n_init, p.kind);
  const uint32_t L = p.seg_tokens;  // a document's tokens and a segment's more can pass 31 bits, not 32
  for (int i0 = 0; i0 < p.N; i0 += kPlanThreads) {
    const int i = i0 + tid;
    const int k = i < p.N ? ((uint32_t)(p.cu[i + 1] - p.cu[i]) + L - 1) / L : 0;
    int upto = k;  // inclusive sum over the warp, then over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s_warp[wid] = upto;
    __syncthreads();
    if (wid == 0) {
      int v = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
      }
      s_warp[lane] = v;
    }
    __syncthreads();
    const int at = s_base + upto - k + (wid ? s_warp[wid - 1] : 0);
    // a document's segment j of k, equal ones in whole tiles
    auto cut = [&](int doc, int first, int j, int k) {
      const int t0 = p.cu[doc], src = p.init_idx ? p.init_idx[doc] : -1;
      const uint32_t n = p.cu[doc + 1] - t0, len = ((n + k - 1) / k + kSsmSegStep - 1) / kSsmSegStep * kSsmSegStep;
      const uint32_t from = min(n, j * len), to = min(n, (j + 1) * len);
      SsmSeg s;
      s.doc = doc;
      s.tok0 = t0 + (int)from;
      s.ntok = (int)(to - from);
      s.last = j == k - 1;
      s.src = j > 0 || src >= p.n_init ? -2 : src;
      s.need = p.bwd || j < k - 1 || (__ldcg(&p.kind[doc]) & kDocSource);
      s.pad[0] = s.pad[1] = 0;
      p.segs[first + j] = s;
    };
    if (tid == 0) s_long = 0;
    __syncthreads();
    if (i < p.N) {
      p.seg0[i] = at;
      if (k <= 8) {
        for (int j = 0; j < k; ++j) cut(i, at, j, k);
      } else {
        const int l = atomicAdd(&s_long, 1);  // in any order: their places are fixed
        s_doc[l] = i, s_at[l] = at, s_k[l] = k;
      }
    }
    __syncthreads();
    for (int l = 0; l < s_long; ++l)  // long ones by all threads
      for (int j = tid; j < s_k[l]; j += kPlanThreads) cut(s_doc[l], s_at[l], j, s_k[l]);
    __syncthreads();
    if (tid == 0) s_base += s_warp[31];
    __syncthreads();
  }
  if (tid == 0) {
    p.seg0[p.N] = s_base;
    p.hd->n_segs = s_base;
    p.hd->deep = deep;
    p.hd->status = 0;
  }
}

// ------------------------------------------------------------------------------ walks forward in time

enum { kWalkState = 0, kWalkOut = 1, kWalkGrad = 2 };

// Rows of a [T, C] tensor on their way into shared memory: the kN channels from `first` on, of up to kRows tokens one
// after the other, by asynchronous copies of 16 bytes from kThreads threads. kVec: everything is aligned to them, and a
// thread keeps its place. Other rows bring the pieces that cover the channels, and each row's place within its first
// piece is found again from its address; a piece that sticks out of the tensor is copied by elements. Rows behind the
// last one are zero.
template <typename T, int kN, int kRows, int kThreads, bool kVec>
struct Rows {
  static constexpr int K = 16 / (int)sizeof(T);
  static constexpr int kBytes = (kN * (int)sizeof(T) + 15) / 16 * 16 + (kVec ? 0 : 16);  // of a row in shared memory
  static constexpr int kPieces = kBytes / 16;
  static_assert(!kVec || kThreads % kPieces == 0);
  const T* src;  // channel `first` of token 0
  int64_t stride;
  const T *lo, *hi;
  int n, tid;  // channels that exist
  __device__ __forceinline__ Rows(const void* base, int64_t stride_, int64_t first, int n_, int T_, int C, int tid_)
      : stride(stride_), n(n_), tid(tid_) {
    lo = static_cast<const T*>(base);
    src = lo + first;
    hi = kVec ? nullptr : lo + (T_ - 1) * stride_ + C;
  }
  // tokens t .. t + rows - 1
  __device__ __forceinline__ void fetch(uint8_t* dst, int64_t t, int rows) const {
    if constexpr (kVec) {
      constexpr int kAbreast = kThreads / kPieces;  // rows that the threads take at once
      const int r0 = tid / kPieces, q = tid % kPieces;
      if (q * K >= n) return;
      const T* p = src + (t + r0) * stride + q * K;
#pragma unroll
      for (int i = 0; i < (kRows + kAbreast - 1) / kAbreast; ++i) {
        if (r0 + i * kAbreast < kRows) cp_async16_if(dst + tid * 16 + i * kThreads * 16, r0 + i * kAbreast < rows ? p : src, r0 + i * kAbreast < rows);
        p += kAbreast * stride;
      }
    } else {
      for (int i = tid; i < kRows * kPieces; i += kThreads) {
        const int r = i / kPieces, q = i - r * kPieces;
        uint8_t* to = dst + r * kBytes + q * 16;
        if (r >= rows) {
          *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
          continue;
        }
        const T* p = src + (t + r) * stride;
        const T* piece = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15) + q * K;
        if (piece >= p + n) continue;
        if (piece >= lo && piece + K <= hi) {
          cp_async16(to, piece);
        } else {
          for (int e = 0; e < K; ++e)
            if (piece + e >= p && piece + e < p + n) reinterpret_cast<T*>(to)[e] = piece[e];
        }
      }
    }
  }
  // channels c .. c + kK - 1 of row r, token t
  template <int kK>
  __device__ __forceinline__ Pack<T, kK> get(const uint8_t* from, int r, int64_t t, int c) const {
    const uint8_t* row = from + r * kBytes;
    Pack<T, kK> v;
    if constexpr (kVec) {
      v = *reinterpret_cast<const Pack<T, kK>*>(row + c * sizeof(T));
    } else {
      const uint32_t at = ((uint32_t)reinterpret_cast<uintptr_t>(src) + (uint32_t)(t * stride) * (uint32_t)sizeof(T)) & 15u;
#pragma unroll
      for (int i = 0; i < kK; ++i) v.t[i] = *reinterpret_cast<const T*>(row + at + (c + i) * sizeof(T));
    }
    return v;
  }
};

// Four states of channel c of an entry of [entries, C, S], zero behind the last one. `whole`: S is a multiple of four and
// the array lies on 16 bytes.
__device__ __forceinline__ float4 pool_quad(const float* pool, int64_t entry, int C, int S, int c, int q, int whole) {
  const float* h = pool + (entry * C + c) * S + 4 * q;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (whole) {
    if (4 * q < S) v = *reinterpret_cast<const float4*>(h);
  } else {
    if (4 * q < S) v.x = h[0];
    if (4 * q + 1 < S) v.y = h[1];
    if (4 * q + 2 < S) v.z = h[2];
    if (4 * q + 3 < S) v.w = h[3];
  }
  return v;
}
// The same for quads q0 .. q0 + kN - 1.
template <int kN>
__device__ __forceinline__ void pool_quads(float4* v, const float* pool, int64_t entry, int C, int S, int c, int q0, int whole) {
  if (whole) {
    const float4* h = reinterpret_cast<const float4*>(pool + (entry * C + c) * S) + q0;
#pragma unroll
    for (int q = 0; q < kN; ++q) v[q] = 4 * (q0 + q) < S ? h[q] : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
#pragma unroll
    for (int q = 0; q < kN; ++q) v[q] = pool_quad(pool, entry, C, S, c, q0 + q, 0);
  }
}
__device__ __forceinline__ void store_quad(float* pool, int64_t entry, int C, int S, int c, int q, float4 v, int whole) {
  float* h = pool + (entry * C + c) * S + 4 * q;
  if (whole) {
    if (4 * q < S) *reinterpret_cast<float4*>(h) = v;
  } else {
    if (4 * q < S) h[0] = v.x;
    if (4 * q + 1 < S) h[1] = v.y;
    if (4 * q + 2 < S) h[2] = v.z;
    if (4 * q + 3 < S) h[3] = v.w;
  }
}

// A warp walks one segment for 32 kDt / kNl channels: kNl lanes share a channel, each lane holds kNt states of kDt
// channels in registers, pairs of states in packed fp32. kWalkState leaves the end state from zero and the summed
// time; kWalkGrad also the states at each tile and the start state's gradient; kWalkOut the outputs. The inputs of kTb
// tokens are on their way into the warp's part of shared memory while the ones before are worked on (through registers
// the compiler waited for each at once: 2735 instead of 1000 us for 32768 tokens). All states of a channel in one lane
// leave nothing to be summed between lanes, and a token's maps serve two channels.
template <typename T, int kSp, int kMode, bool kVec>
struct WalkShape {
  static constexpr int kNl = kSp == 64 ? 2 : 1, kNt = kSp / kNl, kDt = kSp <= 16 ? 2 : 1, kCh = 32 / kNl * kDt;
  static constexpr int kTb = 8;
  using R = Rows<T, kCh, kTb, 32, kVec>;
  static constexpr int kTensors = kMode == kWalkState ? 2 : kMode == kWalkOut ? 3 : 4;
  static constexpr int kRowsBytes = kTb * R::kBytes, kMapBytes = kTb * 2 * kSp * 4;
  static constexpr int kStage = kTensors * kRowsBytes + kMapBytes;
  static constexpr int kSmem = kSsmWarps * 2 * kStage;
};

template <typename T, int kSp, int kMode, bool kVec>
__global__ void __launch_bounds__(32 * kSsmWarps, kMode == kWalkGrad ? 2 : 4)
    ssm_walk_kernel(const __grid_constant__ SsmParams p) {
  using W = WalkShape<T, kSp, kMode, kVec>;
  using R = typename W::R;
  constexpr int kNl = W::kNl, kNt = W::kNt, kDt = W::kDt, kCh = W::kCh, kTb = W::kTb;
  constexpr int kQt = kNt / 4, kQ = kSp / 4, kP = kNt / 2, kBatch = 2;
  constexpr bool kGate = kMode != kWalkState;  // z is read
  static_assert(kCh == ssm_walk_channels(kSp));
  extern __shared__ __align__(16) uint8_t raw_smem[];
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (p.hd->status != 0) return;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, nl = lane % kNl, dl = lane / kNl;
  uint8_t* ring = raw_smem + wid * 2 * W::kStage;
  const int Cg = p.C / p.G, nb = (Cg + kCh - 1) / kCh, blocks = nb * p.G;
  const int64_t items = (int64_t)p.hd->n_segs * blocks;
  const bool has_z = kGate && p.z != nullptr;
  for (int64_t item = (int64_t)blockIdx.x * kSsmWarps + wid; item < items; item += (int64_t)gridDim.x * kSsmWarps) {
    const int seg = (int)(item / blocks), blk = (int)(item % blocks), g = blk / nb;
    const SsmSeg sg = p.segs[seg];
    if (kMode == kWalkState && !sg.need) continue;
    const int cb = (blk % nb) * kCh, cg = cb + dl * kDt;  // the warp's first channel in its group, the lane's
    const int nch = max(0, min(kDt, Cg - cg));
    const int c0 = g * Cg + min(cg, Cg - 1);              // a channel that exists
    const int64_t first = (int64_t)g * Cg + cb;
    const int have = min(kCh, Cg - cb);
    const R rx(p.x, p.sx, first, have, p.T, p.C, lane), rd(p.dt, p.sdt, first, have, p.T, p.C, lane);
    const R rz(p.z, p.sz, first, have, p.T, p.C, lane), ro(p.dout, p.sdo, first, have, p.T, p.C, lane);
    auto fetch = [&](int i0, uint8_t* st) {  // the inputs of tokens i0 .. i0 + kTb - 1 of the segment
      const int64_t t = sg.tok0 + i0;
      const int rows = min(kTb, sg.ntok - i0);
      rx.fetch(st, t, rows);
      rd.fetch(st + W::kRowsBytes, t, rows);
      if constexpr (kGate) {
        if (has_z) rz.fetch(st + 2 * W::kRowsBytes, t, rows);
      }
      if constexpr (kMode == kWalkGrad) ro.fetch(st + 3 * W::kRowsBytes, t, rows);
      uint8_t* mp = st + W::kTensors * W::kRowsBytes;
      constexpr int kM = kSp / 2;  // pieces of a token's maps
      const float* from = p.maps + ((t + lane / kM) * p.G + g) * 2 * kSp + lane % kM * 4;
#pragma unroll
      for (int i = 0; i < kTb * kM / 32; ++i) {
        const bool live = i * 32 + lane < rows * kM;
        cp_async16_if(mp + (i * 32 + lane) * 16, live ? from : p.maps, live);
        from += (int64_t)(32 / kM) * p.G * 2 * kSp;
      }
      cp_async_commit();
    };
    fetch(0, ring);
    uint64_t A[kDt][kP], h[kDt][kP], ga[kMode == kWalkGrad ? kDt : 1][kP], pr[kMode == kWalkGrad ? kDt : 1][kP];
    float bias[kDt], skip[kDt], total[kDt];
    float4 av[kDt][kQt], hv[kDt][kQt];
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
      const int c = min(c0 + d, g * Cg + Cg - 1);
      bias[d] = p.dt_bias ? p.dt_bias[c] : 0.f;
      skip[d] = kMode == kWalkOut && p.skip ? p.skip[c] : 0.f;
      total[d] = 0.f;
      pool_quads<kQt>(av[d], p.a, 0, p.C, p.S, c, nl * kQt, p.whole);
      if constexpr (kMode == kWalkOut) {
        if (sg.src >= 0) {
          pool_quads<kQt>(hv[d], p.init, sg.src, p.C, p.S, c, nl * kQt, p.whole);
        } else {
#pragma unroll
          for (int q = 0; q < kQt; ++q)
            hv[d][q] = sg.src == -2 ? *reinterpret_cast<const float4*>(p.slot + (((int64_t)seg * kQ + nl * kQt + q) * p.C + c) * 4)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
#pragma unroll
    for (int d = 0; d < kDt; ++d)
#pragma unroll
      for (int q = 0; q < kQt; ++q) {
        hold(av[d][q]);
        if constexpr (kMode == kWalkOut)
          hold(hv[d][q]);
        else
          hv[d][q] = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = av[d][q], s = hv[d][q];
        A[d][2 * q] = f2_pack(a.x * kLog2e, a.y * kLog2e), A[d][2 * q + 1] = f2_pack(a.z * kLog2e, a.w * kLog2e);
        h[d][2 * q] = f2_pack(s.x, s.y), h[d][2 * q + 1] = f2_pack(s.z, s.w);
        if constexpr (kMode == kWalkGrad) {
          ga[d][2 * q] = ga[d][2 * q + 1] = 0;
          pr[d][2 * q] = pr[d][2 * q + 1] = f2_pack(1.f, 1.f);
        }
      }
    for (int i0 = 0, it = 0; i0 < sg.ntok; i0 += kTb, ++it) {
      if constexpr (kMode == kWalkGrad) {
        constexpr int kTile = ssm_tile(kSp);
        if (i0 % kTile == 0 && nch > 0) {
          const int64_t tile = sg.tok0 / kTile + seg + i0 / kTile;
#pragma unroll
          for (int d = 0; d < kDt; ++d) {
            if (d >= nch) break;
#pragma unroll
            for (int q = 0; q < kQt; ++q)
              *reinterpret_cast<float4*>(p.ckpt + ((tile * kQ + nl * kQt + q) * p.C + c0 + d) * 4) =
                  make_float4(f2_lo(h[d][2 * q]), f2_hi(h[d][2 * q]), f2_lo(h[d][2 * q + 1]), f2_hi(h[d][2 * q + 1]));
            if (nl == 0) p.csum[tile * p.C + c0 + d] = total[d];
          }
        }
      }
      uint8_t* st = ring + (it & 1) * W::kStage;
      if (i0 + kTb < sg.ntok) {
        fetch(i0 + kTb, ring + (~it & 1) * W::kStage);
        cp_async_wait<1>();
      } else {
        cp_async_wait<0>();
      }
      __syncwarp();
      const int rows = min(kTb, sg.ntok - i0);
      const float* maps = reinterpret_cast<const float*>(st + W::kTensors * W::kRowsBytes) + nl * kNt;
      // kBatch tokens at a time, without a branch, so that what belongs to different tokens can run side by side. Behind
      // the last token the inputs are zero and the step is held at zero: the state stays.
#pragma unroll 2
      for (int kb = 0; kb < rows; kb += kBatch) {
        constexpr int kN = kBatch * kDt;
        float x[kN], delta[kN], gate[kN];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int64_t t = sg.tok0 + i0 + kb + k;
          const auto xv = rx.template get<kDt>(st, kb + k, t, dl * kDt);
          const auto dv = rd.template get<kDt>(st + W::kRowsBytes, kb + k, t, dl * kDt);
#pragma unroll
          for (int d = 0; d < kDt; ++d) {
            x[k * kDt + d] = to_float(xv.t[d]);
            delta[k * kDt + d] = to_float(dv.t[d]) + bias[d];
            gate[k * kDt + d] = 1.f;
          }
          if constexpr (kGate) {
            const auto zv = rz.template get<kDt>(st + 2 * W::kRowsBytes, kb + k, t, dl * kDt);
#pragma unroll
            for (int d = 0; d < kDt; ++d) gate[k * kDt + d] = to_float(zv.t[d]);
          }
        }
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
          const uint64_t v = softplus_pair(f2_pack(delta[i], delta[i + 1]));
          delta[i] = kb + i / kDt >= rows ? 0.f : p.softplus ? f2_lo(v) : delta[i];
          delta[i + 1] = kb + (i + 1) / kDt >= rows ? 0.f : p.softplus ? f2_hi(v) : delta[i + 1];
          if constexpr (kGate) {
            const uint64_t w = silu_pair(f2_pack(gate[i], gate[i + 1]));
            gate[i] = has_z ? f2_lo(w) : 1.f, gate[i + 1] = has_z ? f2_hi(w) : 1.f;
          }
        }
        if constexpr (kMode == kWalkGrad) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const auto ov = ro.template get<kDt>(st + 3 * W::kRowsBytes, kb + k, sg.tok0 + i0 + kb + k, dl * kDt);
#pragma unroll
            for (int d = 0; d < kDt; ++d) gate[k * kDt + d] *= to_float(ov.t[d]);  // the gradient of y
          }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const float* mp = maps + (kb + k) * 2 * kSp;
          uint64_t dd[kDt], uu[kDt], gg[kDt], y2[kDt];
#pragma unroll
          for (int d = 0; d < kDt; ++d) {
            const int i = k * kDt + d;
            total[d] += delta[i];
            dd[d] = f2_dup(delta[i]);
            uu[d] = f2_dup(delta[i] * x[i]);
            gg[d] = f2_dup(gate[i]);
            y2[d] = 0;
          }
#pragma unroll
          for (int q = 0; q < kQt; ++q) {
            const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(mp + 4 * q);
            ulonglong2 cv;
            if (kMode != kWalkState) cv = *reinterpret_cast<const ulonglong2*>(mp + kSp + 4 * q);
#pragma unroll
            for (int d = 0; d < kDt; ++d) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint64_t arg = f2_mul(dd[d], A[d][2 * q + j]);
                const uint64_t e = exp2_pair(arg);
                h[d][2 * q + j] = f2_fma(e, h[d][2 * q + j], f2_mul(uu[d], j ? bv.y : bv.x));
                if constexpr (kMode == kWalkOut) y2[d] = f2_fma(h[d][2 * q + j], j ? cv.y : cv.x, y2[d]);
                if constexpr (kMode == kWalkGrad) {
                  pr[d][2 * q + j] = f2_mul(pr[d][2 * q + j], e);
                  ga[d][2 * q + j] = f2_fma(pr[d][2 * q + j], f2_mul(gg[d], j ? cv.y : cv.x), ga[d][2 * q + j]);
                }
              }
            }
          }
          if constexpr (kMode == kWalkOut) {
            Pack<T, kDt> r;
#pragma unroll
            for (int d = 0; d < kDt; ++d) {
              float y = f2_sum(y2[d]);
              if constexpr (kNl == 2) y += __shfl_xor_sync(0xffffffffu, y, 1);
              r.t[d] = from_float<T>(fmaf(skip[d], x[k * kDt + d], y) * gate[k * kDt + d]);
            }
            if (nl == 0 && nch > 0 && kb + k < rows)
              store_pack<T, kDt, kVec>(static_cast<T*>(p.out) + ((int64_t)sg.tok0 + i0 + kb + k) * p.C + c0, r, nch);
          }
        }
      }
      __syncwarp();  // the stage is free
    }
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll
    for (int d = 0; d < kDt; ++d) {
      if (d >= nch) break;
      if (kMode != kWalkOut && nl == 0) p.sums[(int64_t)seg * p.C + c0 + d] = total[d];
#pragma unroll
      for (int q = 0; q < kQt; ++q) {
        const int qq = nl * kQt + q;
        const float4 hv = make_float4(f2_lo(h[d][2 * q]), f2_hi(h[d][2 * q]), f2_lo(h[d][2 * q + 1]), f2_hi(h[d][2 * q + 1]));
        if constexpr (kMode == kWalkOut) {
          if (sg.last) store_quad(p.final_state, sg.doc, p.C, p.S, c0 + d, qq, hv, p.whole);
        } else {
          *reinterpret_cast<float4*>(p.slot + (((int64_t)seg * kQ + qq) * p.C + c0 + d) * 4) = hv;
        }
        if constexpr (kMode == kWalkGrad)
          *reinterpret_cast<float4*>(p.slot_r + (((int64_t)seg * kQ + qq) * p.C + c0 + d) * 4) = make_float4(
              f2_lo(ga[d][2 * q]), f2_hi(ga[d][2 * q]), f2_lo(ga[d][2 * q + 1]), f2_hi(ga[d][2 * q + 1]));
      }
    }
  }
}

// ------------------------------------------------------------------------------ scan over segments

constexpr int kScanThreads = 128, kScanAhead = 16;  // segments whose loads are in flight

__device__ __forceinline__ float4 carry(float4 a, float time, float4 h, float4 add) {
  return make_float4(fmaf(exp2_approx(a.x * time), h.x, add.x), fmaf(exp2_approx(a.y * time), h.y, add.y),
                     fmaf(exp2_approx(a.z * time), h.z, add.z), fmaf(exp2_approx(a.w * time), h.w, add.w));
}

// Start states of the segments from their end states, in place; final states of empty documents and of those that
// others fork from; in the backward the gradients behind the segments from those before them, and each document's
// start-state gradient. A thread takes four states of a channel through the documents of blockIdx.y. Three launches where
// documents may fork: kStep 0 for documents that need no other, 1 for those that need what 0 left, 2 for the rest in order.
template <int kStep>
__global__ void __launch_bounds__(kScanThreads) ssm_scan_kernel(const __grid_constant__ SsmParams p) {
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (p.hd->status != 0 || (kStep == 2 && !p.hd->deep)) return;
  const int Sp = ssm_padded(p.S), Q = Sp / 4;
  const int64_t i = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= (int64_t)Q * p.C) return;
  const int q = (int)(i / p.C), c = (int)(i % p.C), step = gridDim.y, d0 = blockIdx.y;
  const int64_t state = (int64_t)Q * p.C * 4;
  float4 a = pool_quad(p.a, 0, p.C, p.S, c, q, p.whole);
  a = make_float4(a.x * kLog2e, a.y * kLog2e, a.z * kLog2e, a.w * kLog2e);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fin = [&](int64_t d) { return reinterpret_cast<float4*>(p.fin + d * state + i * 4); };        // backward only
  auto dstart = [&](int64_t d) { return reinterpret_cast<float4*>(p.dstart + d * state + i * 4); };
  for (int d = d0; d < p.N; d += step) {
    const int kind = p.kind[d];
    if (fork_step(kind) != kStep) continue;
    const int s0 = p.seg0[d], s1 = p.seg0[d + 1];
    const int src = p.init_idx ? p.init_idx[d] : -1;
    const bool fork = kind & kDocFork, source = kind & kDocSource;
    if (!p.bwd && s1 - s0 == 1 && !fork && !source) continue;
    float4 h = zero;
    if (fork)
      h = p.bwd ? *fin(src - p.n_init) : pool_quad(p.final_state, src - p.n_init, p.C, p.S, c, q, p.whole);
    else if (src >= 0)
      h = pool_quad(p.init, src, p.C, p.S, c, q, p.whole);
    const int se = source ? s1 : s1 - 1;  // the last segment's end state is wanted for forks only
    for (int sb = s0; sb < s1; sb += kScanAhead) {
      float4 e[kScanAhead];
      float time[kScanAhead];
#pragma unroll
      for (int k = 0; k < kScanAhead; ++k)
        if (sb + k < se) {
          e[k] = *reinterpret_cast<const float4*>(p.slot + (sb + k) * state + i * 4);
          time[k] = p.sums[(int64_t)(sb + k) * p.C + c];
        }
#pragma unroll
      for (int k = 0; k < kScanAhead; ++k) {
        if (sb + k < s1) *reinterpret_cast<float4*>(p.slot + (sb + k) * state + i * 4) = h;
        if (sb + k < se) h = carry(a, time[k], h, e[k]);
      }
    }
    if (p.bwd) {
      if (source) *fin(d) = h;
    } else if (s1 == s0 || source) {
      store_quad(p.final_state, d, p.C, p.S, c, q, h, p.whole);
    }
  }
  if (!p.bwd) return;
  for (int d = d0 + (p.N - 1 - d0) / step * step; d >= 0; d -= step) {
    const int kind = p.kind[d];
    if (source_step(kind) != kStep) continue;
    const int s0 = p.seg0[d], s1 = p.seg0[d + 1];
    float4 k = p.dfinal ? pool_quad(p.dfinal, d, p.C, p.S, c, q, p.whole) : zero;
    if (kStep > 0)  // what its forks send back, in their order
      for (int f0 = d + 1; f0 < p.N; f0 += kScanAhead) {
        float4 e[kScanAhead];
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j)
          e[j] = f0 + j < p.N && p.init_idx[f0 + j] == p.n_init + d ? *dstart(f0 + j) : zero;
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j) k = make_float4(k.x + e[j].x, k.y + e[j].y, k.z + e[j].z, k.w + e[j].w);
      }
    for (int sb = s1 - 1; sb >= s0; sb -= kScanAhead) {
      float4 e[kScanAhead];
      float time[kScanAhead];
#pragma unroll
      for (int j = 0; j < kScanAhead; ++j)
        if (sb - j >= s0) {
          e[j] = *reinterpret_cast<const float4*>(p.slot_r + (sb - j) * state + i * 4);
          time[j] = p.sums[(int64_t)(sb - j) * p.C + c];
        }
#pragma unroll
      for (int j = 0; j < kScanAhead; ++j)
        if (sb - j >= s0) {
          *reinterpret_cast<float4*>(p.slot_r + (sb - j) * state + i * 4) = k;
          k = carry(a, time[j], k, e[j]);
        }
    }
    *dstart(d) = k;
  }
}

// ------------------------------------------------------------------------------ walk of the backward

// A CTA of four warps walks a segment in reverse, tile by tile, each warp for 4 * 32 / kNl channels: a lane holds four
// states of four channels, pairs of states in packed fp32, kNl = kSp / 4 lanes share a channel. Within a tile the states
// go forward again from the kept one, every fourth of them through shared memory; four tokens at a time come back in
// reverse. The sums over the states of a channel and over the warp's channels are made by halving: at each exchange
// between two lanes each keeps half of the values, so that a lane ends up with one channel's sums. The gradients of the
// tile's tokens are made of them at its end, four channels to a lane (token by token in the walk they took 200 of the
// kernel's 710 us at 16384 x 2048 x 16).
template <typename T, int kSp, bool kVec>
struct GradSmem {
  static constexpr int kNl = kSp / 4, kDl = 32 / kNl, kCh = 4 * kDl, kCtaCh = kSsmWarps * kCh;
  static constexpr int kTile = ssm_tile(kSp);
  static constexpr int kStages = sizeof(T) == 2 ? 2 : 1;  // two CTAs to an SM either way
  using R = Rows<T, kCtaCh, kTile, 32 * kSsmWarps, kVec>;
  uint8_t raw[kStages][4][kTile * R::kBytes];  // x, dt, z, dout
  float maps[kStages][kTile][2 * kSp];
  float part[kSsmWarps][kTile][2 * kSp];       // db and dc of each warp's channels
  float bias[kSsmWarps][kCh], skip[kSsmWarps][kCh];
  float delta[kSsmWarps][kTile][kCh];
  float u[kSsmWarps][kTile][kCh];   // then sum_s b k
  float dy[kSsmWarps][kTile][kCh];  // then sum_s a k exp(dt a) h_{t-1}
  float y[kSsmWarps][kTile][kCh];
  float4 keep[kSsmWarps][kTile / kGradSub][4][32];
};

// v[0 .. kN - 1] of two lanes that differ in `mask` become the sums of the first half in the one without the bit, of
// the second half in the other.
template <int kN>
__device__ __forceinline__ void halve(float* v, int mask, bool up) {
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) {
    const float send = up ? v[i] : v[i + kN / 2], keep = up ? v[i + kN / 2] : v[i];
    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
  }
}

template <typename T, int kSp, bool kVec>
__global__ void __launch_bounds__(32 * kSsmWarps, 2) ssm_grad_kernel(const __grid_constant__ SsmParams p) {
  using Smem = GradSmem<T, kSp, kVec>;
  using R = typename Smem::R;
  constexpr int kNl = Smem::kNl, kDl = Smem::kDl, kCh = Smem::kCh, kQ = kSp / 4, kTb = Smem::kTile, kStages = Smem::kStages;
  constexpr int kCl = kNl >= 4 ? 1 : 2;  // channels whose sums a lane ends up with
  extern __shared__ __align__(16) uint8_t raw_smem[];
  Smem& sm = *reinterpret_cast<Smem*>(raw_smem);
  bw::griddep_wait();
  bw::griddep_launch_dependents();
  if (p.hd->status != 0) return;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, nl = lane % kNl, dl = lane / kNl;
  const int Cg = p.C / p.G, blocks = p.parts * p.G;
  const int64_t items = (int64_t)p.hd->n_segs * blocks;
  const bool has_z = p.z != nullptr;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int seg = (int)(item / blocks), blk = (int)(item % blocks), g = blk / p.parts, part = blk % p.parts;
    const SsmSeg sg = p.segs[seg];
    const int ctab = part * Smem::kCtaCh, cb = ctab + wid * kCh;  // first channel in the group: the CTA's, the warp's
    const int nch = max(0, min(4, Cg - cb - 4 * dl));
    const int c0 = g * Cg + min(cb + 4 * dl, Cg - 1), cmax = g * Cg + Cg - 1;
    const int64_t first = (int64_t)g * Cg + ctab;
    const int have = min(Smem::kCtaCh, Cg - ctab);
    const int tid = threadIdx.x;
    const R rx(p.x, p.sx, first, have, p.T, p.C, tid), rd(p.dt, p.sdt, first, have, p.T, p.C, tid);
    const R rz(p.z, p.sz, first, have, p.T, p.C, tid), ro(p.dout, p.sdo, first, have, p.T, p.C, tid);
    auto fetch = [&](int tile) {
      const int st = tile % kStages, rows = min(kTb, sg.ntok - tile * kTb);
      const int64_t t = sg.tok0 + tile * kTb;
      rx.fetch(sm.raw[st][0], t, rows);
      rd.fetch(sm.raw[st][1], t, rows);
      if (has_z) rz.fetch(sm.raw[st][2], t, rows);
      ro.fetch(sm.raw[st][3], t, rows);
      for (int i = threadIdx.x; i < kTb * (kSp / 2); i += 32 * kSsmWarps) {  // zeros behind the last token
        const int k = i / (kSp / 2), r = i % (kSp / 2);
        cp_async16_if(&sm.maps[st][k][4 * r], p.maps + ((t + min(k, rows - 1)) * p.G + g) * 2 * kSp + 4 * r, k < rows);
      }
      cp_async_commit();
    };
    const int tiles = (sg.ntok + kTb - 1) / kTb;
    if (tiles > 0) fetch(tiles - 1);
    uint64_t A[4][2], K[4][2], dA[4][2];  // A in units of log2 e
    {
      float4 av[4], kv[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int c = min(c0 + d, cmax);
        pool_quads<1>(&av[d], p.a, 0, p.C, p.S, c, nl, p.whole);
        kv[d] = *reinterpret_cast<const float4*>(p.slot_r + (((int64_t)seg * kQ + nl) * p.C + c) * 4);
      }
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        hold(av[d]), hold(kv[d]);
        A[d][0] = f2_pack(av[d].x * kLog2e, av[d].y * kLog2e), A[d][1] = f2_pack(av[d].z * kLog2e, av[d].w * kLog2e);
        K[d][0] = f2_pack(kv[d].x, kv[d].y), K[d][1] = f2_pack(kv[d].z, kv[d].w);
        dA[d][0] = dA[d][1] = 0;
      }
    }
    for (int i = lane; i < kCh; i += 32) {
      const int c = g * Cg + min(cb + i, Cg - 1);
      sm.bias[wid][i] = p.dt_bias ? p.dt_bias[c] : 0.f;
      sm.skip[wid][i] = p.skip ? p.skip[c] : 0.f;
    }
    // for the steps and the gradients a lane takes four channels of every kNl-th token
    const int lq = lane % kDl, lt = lane / kDl, lcg = cb + 4 * lq, ln = max(0, min(4, Cg - lcg));
    uint64_t dskip[2] = {0, 0}, dbias[2] = {0, 0};
    for (int tile = tiles - 1; tile >= 0; --tile) {
      const int st = tile % kStages;
      const int64_t t0 = sg.tok0 + tile * kTb;
      const int nt = min(kTb, sg.ntok - tile * kTb);
      // the state before the tile: kept from zero, and what is left of the segment's start state
      uint64_t h[4][2];
      {
        const int64_t tl = sg.tok0 / kTb + seg + tile;
        float4 kept[4], start[4];
        float time[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int c = min(c0 + d, cmax);
          kept[d] = *reinterpret_cast<const float4*>(p.ckpt + ((tl * kQ + nl) * p.C + c) * 4);
          time[d] = p.csum[tl * p.C + c];
          if (sg.src >= 0)
            pool_quads<1>(&start[d], p.init, sg.src, p.C, p.S, c, nl, p.whole);
          else
            start[d] = sg.src == -2 ? *reinterpret_cast<const float4*>(p.slot + (((int64_t)seg * kQ + nl) * p.C + c) * 4)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        cp_async_wait<0>();
        __syncthreads();  // this tile has landed, and every warp is done with the one before
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          hold(kept[d]), hold(start[d]), hold(time[d]);
          const uint64_t t = f2_dup(time[d]);
          h[d][0] = f2_fma(exp2_pair(f2_mul(A[d][0], t)), f2_pack(start[d].x, start[d].y), f2_pack(kept[d].x, kept[d].y));
          h[d][1] = f2_fma(exp2_pair(f2_mul(A[d][1], t)), f2_pack(start[d].z, start[d].w), f2_pack(kept[d].z, kept[d].w));
        }
      }
      if (kStages == 2 && tile > 0) fetch(tile - 1);
      for (int k = lt; k < kTb; k += kNl) {  // behind the last token everything is zero
        const int64_t t = t0 + k;
        const int at = wid * kCh + 4 * lq;
        const auto xr = rx.template get<4>(sm.raw[st][0], k, t, at);
        const auto dr = rd.template get<4>(sm.raw[st][1], k, t, at);
        const auto zr = rz.template get<4>(sm.raw[st][2], k, t, at);
        const auto gr = ro.template get<4>(sm.raw[st][3], k, t, at);
        const float4 bi = *reinterpret_cast<const float4*>(&sm.bias[wid][4 * lq]);
        float dv[4] = {bi.x, bi.y, bi.z, bi.w}, uv[4], gv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) dv[j] += to_float(dr.t[j]);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const uint64_t v = softplus_pair(f2_pack(dv[j], dv[j + 1]));
          const uint64_t w = silu_pair(f2_pack(to_float(zr.t[j]), to_float(zr.t[j + 1])));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool live = k < nt && j + i < ln;
            dv[j + i] = !live ? 0.f : p.softplus ? (i ? f2_hi(v) : f2_lo(v)) : dv[j + i];
            uv[j + i] = live ? dv[j + i] * to_float(xr.t[j + i]) : 0.f;
            gv[j + i] = to_float(gr.t[j + i]);
            gv[j + i] = live ? (has_z ? gv[j + i] * (i ? f2_hi(w) : f2_lo(w)) : gv[j + i]) : 0.f;
          }
        }
        *reinterpret_cast<float4*>(&sm.delta[wid][k][4 * lq]) = make_float4(dv[0], dv[1], dv[2], dv[3]);
        *reinterpret_cast<float4*>(&sm.u[wid][k][4 * lq]) = make_float4(uv[0], uv[1], uv[2], uv[3]);
        *reinterpret_cast<float4*>(&sm.dy[wid][k][4 * lq]) = make_float4(gv[0], gv[1], gv[2], gv[3]);
      }
      __syncwarp();
      auto row4 = [&](const float* r, float* v) {
        const float4 f = *reinterpret_cast<const float4*>(r);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
      };
      // one token forward: h = e h + u b
      auto forward = [&](int k) {
        float dv[4], uv[4];
        row4(&sm.delta[wid][k][4 * dl], dv);
        row4(&sm.u[wid][k][4 * dl], uv);
        const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&sm.maps[st][k][4 * nl]);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint64_t dd = f2_dup(dv[d]), uu = f2_dup(uv[d]);
          h[d][0] = f2_fma(exp2_pair(f2_mul(dd, A[d][0])), h[d][0], f2_mul(uu, bv.x));
          h[d][1] = f2_fma(exp2_pair(f2_mul(dd, A[d][1])), h[d][1], f2_mul(uu, bv.y));
        }
      };
      const int subs = (nt + kGradSub - 1) / kGradSub;
      for (int s = 0; s < subs; ++s) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
          *reinterpret_cast<ulonglong2*>(&sm.keep[wid][s][d][lane]) = make_ulonglong2(h[d][0], h[d][1]);
        if (s + 1 < subs) {
#pragma unroll
          for (int k = 0; k < kGradSub; ++k) forward(kGradSub * s + k);
        }
      }
      for (int s = subs - 1; s >= 0; --s) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&sm.keep[wid][s][d][lane]);
          h[d][0] = f.x, h[d][1] = f.y;
        }
        uint64_t hb[kGradSub][4][2];  // states before each of these tokens
#pragma unroll
        for (int k = 0; k < kGradSub; ++k) {
#pragma unroll
          for (int d = 0; d < 4; ++d) hb[k][d][0] = h[d][0], hb[k][d][1] = h[d][1];
          forward(kGradSub * s + k);  // behind the last token dt, u, b and c are 0: the state stays
        }
#pragma unroll
        for (int k = kGradSub - 1; k >= 0; --k) {
          const int tk = kGradSub * s + k;
          float dv[4], uv[4], gv[4];
          row4(&sm.delta[wid][tk][4 * dl], dv);
          row4(&sm.u[wid][tk][4 * dl], uv);
          row4(&sm.dy[wid][tk][4 * dl], gv);
          const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&sm.maps[st][tk][4 * nl]);
          const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(&sm.maps[st][tk][kSp + 4 * nl]);
          uint64_t db[2] = {0, 0}, dc[2] = {0, 0};
          float v[12], w[8];  // of each channel the sums of K b, A (K e) h and c h; of each state those of u K and dy h
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint64_t dd = f2_dup(dv[d]), uu = f2_dup(uv[d]), gg = f2_dup(gv[d]);
            uint64_t du = 0, va = 0, yv = 0;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint64_t hn = k == kGradSub - 1 ? h[d][n] : hb[k == kGradSub - 1 ? k : k + 1][d][n], b = n ? bv.y : bv.x, c = n ? cv.y : cv.x;
              K[d][n] = f2_fma(gg, c, K[d][n]);
              yv = f2_fma(c, hn, yv);
              dc[n] = f2_fma(gg, hn, dc[n]);
              db[n] = f2_fma(uu, K[d][n], db[n]);
              du = f2_fma(b, K[d][n], du);
              K[d][n] = f2_mul(K[d][n], exp2_pair(f2_mul(dd, A[d][n])));
              const uint64_t kh = f2_mul(K[d][n], hb[k][d][n]);
              va = f2_fma(A[d][n], kh, va);
              dA[d][n] = f2_fma(dd, kh, dA[d][n]);
            }
            v[3 * d] = f2_sum(du), v[3 * d + 1] = f2_sum(va), v[3 * d + 2] = f2_sum(yv);
          }
          // over the states: the lane's channels at the end are those of ec
          if constexpr (kNl >= 4) {
            halve<12>(v, 2, nl & 2);
            halve<6>(v, 1, nl & 1);
#pragma unroll
            for (int o = 4; o < kNl; o <<= 1)
#pragma unroll
              for (int i = 0; i < 3; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
          } else {
            halve<12>(v, 1, nl & 1);
          }
          // over the channels: a lane keeps kW of the eight sums
          constexpr int kW = kDl >= 8 ? 1 : kDl == 4 ? 2 : 4;
          w[0] = f2_lo(db[0]), w[1] = f2_hi(db[0]), w[2] = f2_lo(db[1]), w[3] = f2_hi(db[1]);
          w[4] = f2_lo(dc[0]), w[5] = f2_hi(dc[0]), w[6] = f2_lo(dc[1]), w[7] = f2_hi(dc[1]);
          int at = 0;  // the first of them
          if constexpr (kDl >= 8) {
            halve<8>(w, 4 * kNl, dl & 4);
            halve<4>(w, 2 * kNl, dl & 2);
            halve<2>(w, kNl, dl & 1);
            if constexpr (kDl == 16) w[0] += __shfl_xor_sync(0xffffffffu, w[0], 8 * kNl);
            at = dl & 7;
          } else if constexpr (kDl == 4) {
            halve<8>(w, 2 * kNl, dl & 2);
            halve<4>(w, kNl, dl & 1);
            at = 2 * dl;
          } else {
            halve<8>(w, kNl, dl & 1);
            at = 4 * dl;
          }
          if (dl < 8) {
#pragma unroll
            for (int i = 0; i < kW; ++i) sm.part[wid][tk][(at + i) / 4 * kSp + 4 * nl + (at + i) % 4] = w[i];
          }
          __syncwarp();  // the token's u and dy have been read
          if (nl < 4) {
#pragma unroll
            for (int j = 0; j < kCl; ++j) {
              const int c = 4 * dl + (kCl == 1 ? (nl & 3) : 2 * nl + j);
              sm.u[wid][tk][c] = v[3 * j];
              sm.dy[wid][tk][c] = v[3 * j + 1];
              sm.y[wid][tk][c] = v[3 * j + 2];
            }
          }
        }
      }
      __syncwarp();
      for (int k = lt; k < nt; k += kNl) {
        const int64_t t = t0 + k, o = t * p.C + (int64_t)g * Cg + lcg;
        const int at = wid * kCh + 4 * lq;
        const auto xr = rx.template get<4>(sm.raw[st][0], k, t, at);
        const auto dr = rd.template get<4>(sm.raw[st][1], k, t, at);
        const auto zr = rz.template get<4>(sm.raw[st][2], k, t, at);
        const auto gr = ro.template get<4>(sm.raw[st][3], k, t, at);
        auto pairs = [&](const float* r) { return *reinterpret_cast<const ulonglong2*>(r + 4 * lq); };
        const ulonglong2 du = pairs(sm.u[wid][k]), va = pairs(sm.dy[wid][k]), yv = pairs(sm.y[wid][k]), de = pairs(sm.delta[wid][k]);
        const ulonglong2 bi = pairs(sm.bias[wid]), sk = pairs(sm.skip[wid]);
        Pack<T, 4> dx, dd, dz;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint64_t x = f2_pack(to_float(xr.t[2 * j]), to_float(xr.t[2 * j + 1]));
          const uint64_t z = f2_pack(to_float(zr.t[2 * j]), to_float(zr.t[2 * j + 1]));
          const uint64_t go = f2_pack(to_float(gr.t[2 * j]), to_float(gr.t[2 * j + 1]));
          const uint64_t raw = bw::f2_add(f2_pack(to_float(dr.t[2 * j]), to_float(dr.t[2 * j + 1])), j ? bi.y : bi.x);
          const uint64_t s = j ? sk.y : sk.x, sig = sigmoid_pair(z), sp = sigmoid_pair(raw);
          const uint64_t zc = f2_pack(at_least(f2_lo(z), -128.f), at_least(f2_hi(z), -128.f));
          const uint64_t dy = has_z ? f2_mul(go, f2_mul(zc, sig)) : go;
          const uint64_t a = f2_mul(go, f2_mul(f2_fma(s, x, j ? yv.y : yv.x), silu_slope_pair(z, sig)));
          const uint64_t b = f2_fma(j ? de.y : de.x, j ? du.y : du.x, f2_mul(s, dy));
          uint64_t c = f2_fma(x, j ? du.y : du.x, f2_mul(j ? va.y : va.x, f2_dup(1.f / kLog2e)));
          c = p.softplus ? f2_mul(c, sp) : c;
          dbias[j] = bw::f2_add(dbias[j], c);
          dskip[j] = f2_fma(dy, x, dskip[j]);
          dx.t[2 * j] = from_float<T>(f2_lo(b)), dx.t[2 * j + 1] = from_float<T>(f2_hi(b));
          dd.t[2 * j] = from_float<T>(f2_lo(c)), dd.t[2 * j + 1] = from_float<T>(f2_hi(c));
          dz.t[2 * j] = from_float<T>(f2_lo(a)), dz.t[2 * j + 1] = from_float<T>(f2_hi(a));
        }
        if (ln > 0) {
          store_pack<T, 4, kVec>(static_cast<T*>(p.dx) + o, dx, ln);
          store_pack<T, 4, kVec>(static_cast<T*>(p.ddt) + o, dd, ln);
          if (has_z) store_pack<T, 4, kVec>(static_cast<T*>(p.dz) + o, dz, ln);
        }
      }
      __syncthreads();
      if (kStages == 1 && tile > 0) fetch(tile - 1);
      for (int i = threadIdx.x; i < nt * (kSp / 2); i += 32 * kSsmWarps) {
        const int k = i / (kSp / 2), r = i % (kSp / 2);
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSsmWarps; ++w) {
          const float4 e = *reinterpret_cast<const float4*>(&sm.part[w][k][4 * r]);
          f = make_float4(f.x + e.x, f.y + e.y, f.z + e.z, f.w + e.w);
        }
        *reinterpret_cast<float4*>(p.part_m + (((int64_t)part * p.T + t0 + k) * p.G + g) * 2 * kSp + 4 * r) = f;
      }
    }
    __syncthreads();  // the next item's copies go where this one's tiles were
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (d < nch)
        *reinterpret_cast<float4*>(p.part_a + (((int64_t)seg * kQ + nl) * p.C + c0 + d) * 4) =
            make_float4(f2_lo(dA[d][0]), f2_hi(dA[d][0]), f2_lo(dA[d][1]), f2_hi(dA[d][1]));
    float sums[8] = {f2_lo(dskip[0]), f2_hi(dskip[0]), f2_lo(dskip[1]), f2_hi(dskip[1]),
                     f2_lo(dbias[0]), f2_hi(dbias[0]), f2_lo(dbias[1]), f2_hi(dbias[1])};
#pragma unroll
    for (int o = kDl; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], o);
    if (lt == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < ln) {
          const int64_t c = (int64_t)g * Cg + lcg + j;
          p.part_c[(int64_t)seg * 2 * p.C + c] = sums[j];
          p.part_c[((int64_t)seg * 2 + 1) * p.C + c] = sums[4 + j];
        }
    }
  }
}

// ------------------------------------------------------------------------------ sums of the backward

template <typename T>
__device__ void maps_grad(const SsmParams& p, int64_t i) {  // i over [T][G][2][S]
  const int Sp = ssm_padded(p.S);
  const int64_t tg = i >> 31 ? i / (2 * p.S) : (int64_t)((uint32_t)i / (uint32_t)(2 * p.S));
  const int r = (int)(i - tg * 2 * p.S), m = r >= p.S, s = m ? r - p.S : r;
  float v = 0.f;
#pragma unroll 8
  for (int k = 0; k < p.parts; ++k) v += p.part_m[((int64_t)k * p.T * p.G + tg) * 2 * Sp + m * Sp + s];
  static_cast<T*>(m ? p.dc : p.db)[tg * p.S + s] = from_float<T>(v);
}

// The sum of term(0) .. term(n - 1), eight threads (threadIdx.x / 32) to a result, in a fixed order; valid in the first.
template <typename V, typename F>
__device__ V sum_by_eight(int n, V zero, V (*s)[32], F term) {
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  V v = zero;
#pragma unroll 4
  for (int k = r; k < n; k += 8) v = v + term(k);
  __syncthreads();
  s[r][lane] = v;
  __syncthreads();
  if (r == 0) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v = v + s[k][lane];
  }
  return v;
}
struct Quad {
  float4 f;
  __device__ __forceinline__ Quad operator+(const Quad& o) const {
    return {make_float4(f.x + o.f.x, f.y + o.f.y, f.z + o.f.z, f.w + o.f.w)};
  }
};

// blockIdx.y 0: db and dc over the CTAs of the channels; 1: da over the segments; 2: dskip and ddt_bias; 3: the start
// states' gradients over the documents of each pool entry that some document starts from.
__global__ void __launch_bounds__(256) ssm_sum_kernel(const __grid_constant__ SsmParams p) {
  __shared__ Quad s_quad[8][32];
  __shared__ float s_one[8][32];
  bw::griddep_wait();
  if (p.hd->status != 0) return;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  const int64_t j0 = (int64_t)blockIdx.x * 32, jstep = (int64_t)gridDim.x * 32;
  const int lane = threadIdx.x & 31;
  const int Sp = ssm_padded(p.S), Q = Sp / 4, segs = p.hd->n_segs;
  const int64_t state = (int64_t)Q * p.C * 4;
  if (blockIdx.y == 0) {
    const int64_t n = (int64_t)p.T * p.G * 2 * p.S;
    for (int64_t i = i0; i < n; i += step) {
      if (p.dtype == GDN_DTYPE_BF16)
        maps_grad<__nv_bfloat16>(p, i);
      else if (p.dtype == GDN_DTYPE_FP16)
        maps_grad<__half>(p, i);
      else
        maps_grad<float>(p, i);
    }
  } else if (blockIdx.y == 1) {
    const int64_t n = (int64_t)Q * p.C;
    for (int64_t j = j0; j < n; j += jstep) {
      const int64_t i = min(j + lane, n - 1);
      const Quad v = sum_by_eight(segs, Quad{make_float4(0.f, 0.f, 0.f, 0.f)}, s_quad,
                                  [&](int s) { return Quad{*reinterpret_cast<const float4*>(p.part_a + s * state + i * 4)}; });
      if (threadIdx.x < 32 && j + lane < n) store_quad(p.da, 0, p.C, p.S, (int)(i % p.C), (int)(i / p.C), v.f, p.whole);
    }
  } else if (blockIdx.y == 2) {
    const int64_t n = 2 * (int64_t)p.C;
    for (int64_t j = j0; j < n; j += jstep) {
      const int64_t i = min(j + lane, n - 1);
      const float v = sum_by_eight(segs, 0.f, s_one, [&](int s) { return p.part_c[s * n + i]; });
      float* out = i < p.C ? p.dskip : p.dbias;
      if (threadIdx.x < 32 && j + lane < n && out) out[i % p.C] = v;
    }
  } else {
    const int64_t per = (int64_t)Q * p.C;
    for (int64_t i = i0; i < p.N * per; i += step) {
      int d = (int)(i / per);
      if (!p.link[d].y) continue;
      const int64_t e = p.init_idx[d], r = i - d * per;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (; d >= 0; d = p.link[d].x) {
        const float4 f = *reinterpret_cast<const float4*>(p.dstart + d * state + r * 4);
        v = make_float4(v.x + f.x, v.y + f.y, v.z + f.z, v.w + f.w);
      }
      store_quad(p.dinit, e, p.C, p.S, (int)(r % p.C), (int)(r / p.C), v, p.whole);
    }
  }
}

// ------------------------------------------------------------------------------ host

bool sizes_ok(int N, int T, int C, int S, int G) {
  return N >= 1 && N <= (1 << 30) && T >= 0 && T <= INT32_MAX - 4096 && C >= 1 && S >= 1 && S <= kSsmMaxState && G >= 1 && C % G == 0 &&
         (int64_t)T * C <= ((int64_t)1 << 40) && (int64_t)C * S <= ((int64_t)1 << 28) &&
         (int64_t)N * C <= ((int64_t)1 << 36);
}

struct SsmCall {
  const void *x, *dt, *z;
  const float* a;
  const void *b, *c;
  const float *skip, *dt_bias;
  const int32_t* cu;
  int N, T, C, S, G, dtype;
  const int64_t* strides;
  int softplus;
  const int32_t* init_idx;
  const float* init;
  int n_init;
  const void* dout;
  void* ws;
  size_t ws_bytes;
  bool bwd;
};

// outs: the first n_typed of the call's type, the others fp32 (dfinal_state, an input, among them).
int prepare(const SsmCall& c, const void* const* outs, int n_outs, int n_typed, SsmParams* p, SsmLayout* L, DeviceGuard& guard, int* sms) {
  if (c.dtype != GDN_DTYPE_BF16 && c.dtype != GDN_DTYPE_FP16 && c.dtype != GDN_DTYPE_FP32) return GDN_ERR_UNSUPPORTED;
  if (!sizes_ok(c.N, c.T, c.C, c.S, c.G) || c.n_init < 0) return GDN_ERR_INVALID_ARG;
  if (!c.a || !c.cu || !c.ws || (c.n_init > 0 && !c.init)) return GDN_ERR_INVALID_ARG;
  if (c.T > 0 && (!c.x || !c.dt || !c.b || !c.c || (c.bwd && !c.dout))) return GDN_ERR_INVALID_ARG;
  const int64_t rows[6] = {c.C, c.C, c.C, (int64_t)c.G * c.S, (int64_t)c.G * c.S, c.C};
  int64_t st[6];
  for (int i = 0; i < 6; ++i) {
    st[i] = c.strides && (i < 5 || c.bwd) && c.strides[i] ? c.strides[i] : rows[i];
    if (st[i] < rows[i] || st[i] > ((int64_t)1 << 40)) return GDN_ERR_INVALID_ARG;
  }
  const int es = c.dtype == GDN_DTYPE_FP32 ? 4 : 2;
  auto al = [](const void* q, uintptr_t n) { return reinterpret_cast<uintptr_t>(q) % n == 0; };
  for (const void* q : {c.x, c.dt, c.z, c.b, c.c, c.dout})
    if (!al(q, es)) return GDN_ERR_INVALID_ARG;
  for (const void* q : {(const void*)c.a, (const void*)c.skip, (const void*)c.dt_bias, (const void*)c.init, (const void*)c.cu,
                        (const void*)c.init_idx})
    if (!al(q, 4)) return GDN_ERR_INVALID_ARG;
  for (int i = 0; i < n_outs; ++i)
    if (!al(outs[i], i < n_typed ? es : 4)) return GDN_ERR_INVALID_ARG;
  if (!al(c.ws, 256)) return GDN_ERR_INVALID_ARG;
  *L = ssm_layout(c.N, c.T, c.C, c.S, c.G, c.bwd);
  if (c.ws_bytes < L->total) return GDN_ERR_WORKSPACE;
  const void* ptrs[24] = {c.x, c.dt, c.z, c.a, c.b, c.c, c.skip, c.dt_bias, c.cu, c.init_idx, c.init, c.dout};
  int n = 12;
  for (int i = 0; i < n_outs; ++i) ptrs[n++] = outs[i];
  int dev = 0;
  if (device_of(c.ws, ptrs, n, &dev) != kOk) return GDN_ERR_INVALID_ARG;
  if (!guard.set(dev)) return GDN_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (major != 10 || minor != 3) return GDN_ERR_UNSUPPORTED;
  *p = SsmParams{};
  p->x = c.x, p->dt = c.dt, p->z = c.z, p->b = c.b, p->c = c.c, p->dout = c.dout;
  p->sx = st[0], p->sdt = st[1], p->sz = st[2], p->sb = st[3], p->sc = st[4], p->sdo = st[5];
  p->a = c.a, p->skip = c.skip, p->dt_bias = c.dt_bias, p->init = c.init, p->cu = c.cu, p->init_idx = c.init_idx;
  p->N = c.N, p->T = c.T, p->C = c.C, p->S = c.S, p->G = c.G, p->n_init = c.n_init, p->softplus = c.softplus != 0;
  p->dtype = c.dtype;
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  p->hd = reinterpret_cast<SsmHeader*>(ws + L->header);
  p->segs = reinterpret_cast<SsmSeg*>(ws + L->segs);
  p->seg0 = reinterpret_cast<int32_t*>(ws + L->seg0);
  p->kind = reinterpret_cast<int32_t*>(ws + L->kind);
  p->maps = f(L->maps), p->slot = f(L->slot), p->sums = f(L->sums);
  if (c.bwd) {
    p->link = reinterpret_cast<int2*>(ws + L->link);
    p->slot_r = f(L->slot_r), p->ckpt = f(L->ckpt), p->csum = f(L->csum), p->dstart = f(L->dstart);
    p->fin = f(L->fin), p->part_a = f(L->part_a), p->part_c = f(L->part_c), p->part_m = f(L->part_m);
  }
  p->smax = L->smax;
  p->parts = L->parts;
  p->bwd = c.bwd;
  p->whole = c.S % 4 == 0 && al(c.a, 16) && al(c.init, 16);
  for (int i = 0; i < n_outs; ++i) p->whole = p->whole && al(outs[i], 16);
  p->seg_tokens = L->seg_tokens;
  return GDN_OK;
}

// Whether every row of every block of channels begins on 16 bytes.
bool vectors_ok(const SsmParams& p) {
  const int k = p.dtype == GDN_DTYPE_FP32 ? 4 : 8;
  if (p.C / p.G % k) return false;
  for (int64_t s : {p.sx, p.sdt, p.z ? p.sz : 0, p.dout ? p.sdo : 0})
    if (s % k) return false;
  for (const void* q : {p.x, p.dt, p.z, p.dout, (const void*)p.out, (const void*)p.dx, (const void*)p.ddt, (const void*)p.dz})
    if (reinterpret_cast<uintptr_t>(q) % 16) return false;
  return true;
}

// One attribute a kernel and device: shared memory beyond the default limit.
template <typename K>
bool allow_smem(K kernel, PerDevice& ready, int dev, size_t bytes) {
  if (bytes <= 48 * 1024 || ready.done(dev)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
  ready.mark(dev);
  return true;
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
template <typename F>
void by_state(int Sp, F f) {
  if (Sp == 8)
    f(Int<8>{});
  else if (Sp == 16)
    f(Int<16>{});
  else if (Sp == 32)
    f(Int<32>{});
  else
    f(Int<64>{});
}

template <typename T, int kSp, int kMode, bool kVec>
bool launch_walk_of(const SsmParams& p, unsigned grid, int dev, cudaStream_t s) {
  static PerDevice ready;
  constexpr size_t bytes = WalkShape<T, kSp, kMode, kVec>::kSmem;
  if (!allow_smem(ssm_walk_kernel<T, kSp, kMode, kVec>, ready, dev, bytes)) return false;
  launch_early(ssm_walk_kernel<T, kSp, kMode, kVec>, dim3(grid), 32 * kSsmWarps, bytes, s, p);
  return true;
}

template <int kMode>
bool launch_walk(const SsmParams& p, int sms, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const int Sp = ssm_padded(p.S), ch = ssm_walk_channels(Sp);
  const int64_t items = p.smax * p.G * ((p.C / p.G + ch - 1) / ch), ctas = (items + kSsmWarps - 1) / kSsmWarps;
  const unsigned grid = (unsigned)(ctas < 64 * sms ? ctas : 64 * sms);
  const bool vec = vectors_ok(p);
  bool ok = false;
  by_type(p.dtype, [&](auto t) {
    using T = decltype(t);
    by_state(Sp, [&](auto n) {
      constexpr int kSp = decltype(n)::value;
      ok = vec ? launch_walk_of<T, kSp, kMode, true>(p, grid, dev, s) : launch_walk_of<T, kSp, kMode, false>(p, grid, dev, s);
    });
  });
  return ok;
}

void launch_plan(const SsmParams& p, int sms, cudaStream_t s) {
  int64_t n = (int64_t)p.T * p.G * 2 * ssm_padded(p.S);
  if (p.bwd && p.n_init > 0) n += (int64_t)p.n_init * p.C * p.S + 32 * (int64_t)p.N;
  const int64_t blocks = (n + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  launch_early(ssm_plan_kernel, dim3((unsigned)(1 + (blocks < 2 * sms ? blocks : 2 * sms))), kPlanThreads, 0, s, p);
}

void launch_scan(const SsmParams& p, cudaStream_t s) {
  const unsigned gx = (unsigned)(((int64_t)ssm_padded(p.S) / 4 * p.C + kScanThreads - 1) / kScanThreads), gy = (unsigned)(p.N < 64 ? p.N : 64);
  launch_early(ssm_scan_kernel<0>, dim3(gx, gy), kScanThreads, 0, s, p);
  if (!p.init_idx) return;
  if (p.N > 1) launch_early(ssm_scan_kernel<1>, dim3(gx, gy), kScanThreads, 0, s, p);
  if (p.N > 2) launch_early(ssm_scan_kernel<2>, dim3(gx, 1), kScanThreads, 0, s, p);  // a fork of a fork is a third
}

template <typename T, int kSp, bool kVec>
bool launch_grad_of(const SsmParams& p, unsigned grid, int dev, cudaStream_t s) {
  static PerDevice ready;
  constexpr size_t bytes = sizeof(GradSmem<T, kSp, kVec>);
  if (!allow_smem(ssm_grad_kernel<T, kSp, kVec>, ready, dev, bytes)) return false;
  launch_early(ssm_grad_kernel<T, kSp, kVec>, dim3(grid), 32 * kSsmWarps, bytes, s, p);
  return true;
}

bool launch_grad(const SsmParams& p, int sms, cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const int64_t items = p.smax * p.G * p.parts;
  const unsigned grid = (unsigned)(items < 64 * sms ? items : 64 * sms);
  const bool vec = vectors_ok(p);
  bool ok = false;
  by_type(p.dtype, [&](auto t) {
    using T = decltype(t);
    by_state(ssm_padded(p.S), [&](auto n) {
      constexpr int kSp = decltype(n)::value;
      ok = vec ? launch_grad_of<T, kSp, true>(p, grid, dev, s) : launch_grad_of<T, kSp, false>(p, grid, dev, s);
    });
  });
  return ok;
}

}  // namespace
}  // namespace gdn

extern "C" size_t gdn_ssm_workspace_size(int N, int T, int C, int S, int G, int backward) {
  if (!gdn::sizes_ok(N, T, C, S, G)) return 0;
  return gdn::ssm_layout(N, T, C, S, G, backward != 0).total;
}

extern "C" int gdn_ssm_fwd(const void* x, const void* dt, const void* z, const float* a, const void* b, const void* c,
                           const float* skip, const float* dt_bias, const int32_t* cu_seqlens, int N, int T, int C, int S,
                           int G, int dtype, const int64_t* strides, int dt_softplus, const int32_t* init_idx,
                           const float* initial_state, int n_init, void* out, float* final_state, void* workspace,
                           size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  if (!final_state || (T > 0 && !out)) return GDN_ERR_INVALID_ARG;
  const SsmCall call{x,       dt,          z,        a,             b,      c,       skip,      dt_bias,  cu_seqlens, N, T, C, S, G, dtype,
                     strides, dt_softplus, init_idx, initial_state, n_init, nullptr, workspace, ws_bytes, false};
  const void* outs[] = {out, final_state};
  SsmParams p;
  SsmLayout L;
  DeviceGuard guard;
  int sms = 0;
  const int rc = prepare(call, outs, 2, 1, &p, &L, guard, &sms);
  if (rc != GDN_OK) return rc;
  p.out = out;
  p.final_state = final_state;
  cudaStream_t s = (cudaStream_t)stream;
  launch_plan(p, sms, s);
  if (T > 0 && !launch_walk<kWalkState>(p, sms, s)) return GDN_ERR_CUDA;
  launch_scan(p, s);
  if (T > 0 && !launch_walk<kWalkOut>(p, sms, s)) return GDN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_ssm_bwd(const void* x, const void* dt, const void* z, const float* a, const void* b, const void* c,
                           const float* skip, const float* dt_bias, const int32_t* cu_seqlens, int N, int T, int C, int S,
                           int G, int dtype, const int64_t* strides, int dt_softplus, const int32_t* init_idx,
                           const float* initial_state, int n_init, const void* dout, const float* dfinal_state, void* dx,
                           void* ddt, void* dz, float* da, void* db, void* dc, float* dskip, float* ddt_bias,
                           float* dinitial_state, void* workspace, size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  if (!da || (T > 0 && (!dx || !ddt || !db || !dc)) || (n_init > 0 && !dinitial_state)) return GDN_ERR_INVALID_ARG;
  if ((z != nullptr && T > 0 && !dz) || (skip != nullptr && !dskip) || (dt_bias != nullptr && !ddt_bias))
    return GDN_ERR_INVALID_ARG;
  const SsmCall call{x,       dt,          z,        a,             b,      c,    skip,      dt_bias,  cu_seqlens, N, T, C, S, G, dtype,
                     strides, dt_softplus, init_idx, initial_state, n_init, dout, workspace, ws_bytes, true};
  const void* outs[] = {dx, ddt, dz, db, dc, da, dskip, ddt_bias, dinitial_state, dfinal_state};
  SsmParams p;
  SsmLayout L;
  DeviceGuard guard;
  int sms = 0;
  const int rc = prepare(call, outs, 10, 5, &p, &L, guard, &sms);
  if (rc != GDN_OK) return rc;
  p.dfinal = dfinal_state;
  p.dx = dx, p.ddt = ddt, p.dz = dz, p.db = db, p.dc = dc;
  p.da = da, p.dskip = dskip, p.dbias = ddt_bias, p.dinit = dinitial_state;
  cudaStream_t s = (cudaStream_t)stream;
  launch_plan(p, sms, s);
  if (T > 0 && !launch_walk<kWalkGrad>(p, sms, s)) return GDN_ERR_CUDA;
  launch_scan(p, s);
  if (T > 0 && !launch_grad(p, sms, s)) return GDN_ERR_CUDA;
  launch_early(ssm_sum_kernel, dim3((unsigned)(4 * sms), n_init > 0 ? 4u : 3u), 256, 0, s, p);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
