// Decayed linear attention over packed documents (sm_103a): per value head h with lam = exp(g_h),
//     S_t = lam S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t.
//
// Chunks of 128 tokens. With S the state before a chunk of n tokens (t, s local):
//     o_t = scale (lam^{t+1} S^T q_t + sum_{s <= t} lam^{t-s} (q_t . k_s) v_s)
//     S'  = lam^n S + sum_s lam^{n-1-s} k_s v_s^T
// The gradients are the same recurrence with its tensors permuted (X = the state's gradient after
// the chunk):
//     dq_t = scale (lam^{t+1} S do_t + sum_{s <= t} lam^{t-s} (do_t . v_s) k_s)    (do, v, k), state S^T
//     dv_t = lam^{n-1-t} X^T k_t + scale sum_{i >= t} lam^{i-t} (k_t . q_i) do_i   (k, q, do), reversed
//     dk_t = lam^{n-1-t} X v_t   + scale sum_{i >= t} lam^{i-t} (v_t . do_i) q_i   (v, do, q), reversed
//     X'   = lam^n X + scale sum_i lam^{i+1} q_i do_i^T
// so one kernel serves the forward and, as three roles, the backward. With u the token's place in
// the role's own time (u = t, or n-1-t reversed) and a = 1 forward, 0 reversed, every role has row
// factors lam^{u+a} on its state term and weights lam^{n-a-u} on its key rows.
//
// Precision. The products' operands are bf16. The state is held in fp32 registers, and its update
// uses the weighted keys as a sum of two bf16 terms (relative error about 2^-17 an element), because
// the states are fp32 outputs. The map P is a sum of two bf16 terms too: a row may hold a single one
// of weight (the first tokens, a strong decay), and its rounding would double that of the output. The
// state that the queries read is rounded to bf16 once: each output averages 128 of those roundings.
//
// Row factors leave the products: the output is r_t (S^T q_t + sum_s P''_ts v_s) with r_t =
// max(lam^{u+a}, 2^-86) and P'' = P / r_t, so the query enters the state product as it was loaded.
// Below 2^-86 the state term is too large by at most that factor of the state, which is nothing
// fp32 or the bf16 output resolves.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_dev.cuh"
#include "gdn_host.h"
#include "gdn_la.h"
#include "tmap.h"

namespace gdn {
namespace {

using namespace bw;

constexpr int kLaThreads = 256;
constexpr float kLaLog2e = 1.44269504f;
constexpr float kLaCut = -86.f;  // log2 of the smallest row factor
constexpr uint32_t kTile = 32768;  // 128 x 128 bf16, two 64-column blocks

enum { kMapQ = 0, kMapK = 1, kMapV = 2, kMapDo = 3 };

struct LaRole {
  int mq, mk, mv;           // tensor maps of the role's query, key and value
  int div_q, div_k, div_v;  // value heads to one head of each
  int rev;                  // walks the document from its end
  int trans;                // its state is stored transposed
  float s_in, s_out;        // factors of the key rows (and P), and of the output
  void* out;                // [T, Hv, 128] bf16, or fp32 partials
  int out_f32;
  float* last;              // state after the document's last segment of this role: [N, Hv, 128, 128]
};

struct LaParams {
  CUtensorMap map[4];
  LaRole role[3];
  const float* log_decay;
  const float* start;   // pool of start states
  const float* dfinal;  // gradient of the final states, or null
  LaHeader* hd;
  LaSeg* segs;
  int32_t* seg0;
  int32_t* is_src;
  float *slot_f, *slot_r, *fin, *acc;
  const int32_t* cu;
  const int32_t* init_idx;
  int N, T, Hv, n_init, seg_chunks, bwd;
};

__device__ __forceinline__ void la_status(LaHeader* hd, int code) { atomicCAS(&hd->status, 0, code); }

// ---------------------------------------------------------------------------------------- plan

constexpr int kLaPlanThreads = 1024;

// One CTA: checks cu_seqlens and init_idx and cuts the documents into segments.
__global__ void __launch_bounds__(kLaPlanThreads) la_plan_kernel(const __grid_constant__ LaParams p) {
  griddep_wait();  // the previous call on this stream may still read the workspace
  griddep_launch_dependents();
  __shared__ int s_warp[32], s_base, s_bad, s_scan;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    s_base = 0;
    s_bad = 0;
    s_scan = 0;
  }
  for (int i = tid; i < p.N; i += kLaPlanThreads) p.is_src[i] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < p.N; i += kLaPlanThreads) {
    const int b = p.cu[i], e = p.cu[i + 1];
    if (b < 0 || e < b || e > p.T) bad = true;
    if (i == 0 && b != 0) bad = true;
    if (i == p.N - 1 && e != p.T) bad = true;
    if (p.init_idx) {
      const int x = p.init_idx[i];
      if (x < -1 || (x >= p.n_init && x - p.n_init >= i))
        bad = true;
      else if (x >= p.n_init)
        p.is_src[x - p.n_init] = 1;
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      p.hd->status = kErrInvalid;
      p.hd->n_segs = 0;
      p.hd->scan = 0;
    }
    return;
  }
  const int seg_tok = p.seg_chunks * kLaChunk;
  for (int i0 = 0; i0 < p.N; i0 += kLaPlanThreads) {
    const int i = i0 + tid;
    int b = 0, len = 0, cnt = 0;
    if (i < p.N) {
      b = p.cu[i];
      len = p.cu[i + 1] - b;
      cnt = (seg_tok && len > seg_tok) ? (len + seg_tok - 1) / seg_tok : 1;
    }
    int x = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += t;
    }
    if (lane == 31) s_warp[wid] = x;
    __syncthreads();
    if (wid == 0) {
      int t = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += u;
      }
      s_warp[lane] = t;
    }
    __syncthreads();
    const int base = s_base + (wid ? s_warp[wid - 1] : 0) + x - cnt;
    const int total = s_warp[31];
    if (i < p.N) {
      p.seg0[i] = base;
      const int idx = p.init_idx ? p.init_idx[i] : -1;
      const bool fork = idx >= p.n_init && idx >= 0, src = p.is_src[i] != 0;
      if (cnt > 1 || fork || src) s_scan = 1;
      for (int k = 0; k < cnt; ++k) {
        LaSeg s;
        s.doc = i;
        s.tok0 = b + k * seg_tok;
        s.ntok = cnt > 1 ? min(seg_tok, len - k * seg_tok) : len;
        s.k = k;
        s.nseg = cnt;
        s.src_fwd = (k > 0 || fork) ? -2 : idx;
        s.src_rev = (k < cnt - 1 || src) ? -2 : -1;
        s.need = ((k < cnt - 1 || src) ? 1 : 0) | ((k > 0 || fork) ? 2 : 0);
        p.segs[base + k] = s;
      }
    }
    __syncthreads();
    if (tid == 0) s_base += total;
    __syncthreads();
  }
  if (tid == 0) {
    p.seg0[p.N] = s_base;
    p.hd->status = kOk;
    p.hd->n_segs = s_base;
    p.hd->scan = s_scan;
  }
}

// ---------------------------------------------------------------------------------------- chunks

struct LaSmem {
  uint8_t q[kTile], k[kTile], v[kTile], s[kTile];
  float w[kLaChunk];     // weights of the key rows
  float col[kLaChunk];   // column factors of P''
  float rowe[kLaChunk];  // log2 of the row factors
  uint64_t bar_load, bar_mma;
  uint32_t tmem;
  int fail;
};

constexpr uint32_t kColQK = 0, kColO = 128, kColKV = 256, kColHi = 384, kColLo = 448;

__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* m, int head, int tok, uint64_t* bar) {
  tma_load_3d(dst, m, 0, head, tok, bar);
  tma_load_3d(static_cast<uint8_t*>(dst) + kTile / 2, m, 64, head, tok, bar);
}

// D (+)= A B over K = 128, A and B in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, bool b_mn, uint32_t idesc) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    umma_bf16(d, kmajor_step(a, kTile / 2, ks), b_mn ? mnmajor_step(b, ks) : kmajor_step(b, kTile / 2, ks), idesc,
              ks > 0);
}

// exp(g x) for a whole number x of steps, the product's rounding error carried along
__device__ __forceinline__ float decay_pow(float g, float x) {
  const float hi = g * x;
  const float lo = fmaf(g, x, -hi);
  const float e = expf(hi);
  return isfinite(lo) ? fmaf(e, lo, e) : e;
}

// Walks the chunks of one segment. kOut: the whole role (outputs and end state); otherwise only the
// segment's end state from zero, for the scan.
template <bool kOut>
__global__ void __launch_bounds__(kLaThreads, 1) la_chunk_kernel(const __grid_constant__ LaParams p) {
  extern __shared__ uint8_t raw[];
  LaSmem& sm = *reinterpret_cast<LaSmem*>(smem_align1024(raw));
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int quarter = wid & 3, ch = wid >> 2;  // tensor-memory lanes 32 quarter .. +31, columns 64 ch .. +63
  const int row = 32 * quarter + lane;
  griddep_wait();
  griddep_launch_dependents();
  const int sidx = blockIdx.x / p.Hv, h = blockIdx.x % p.Hv;
  if (sidx >= p.hd->n_segs) return;
  const LaRole& R = p.role[blockIdx.y];
  const LaSeg seg = p.segs[sidx];
  if (!kOut && !((seg.need >> R.rev) & 1)) return;
  if (wid == 0) {
    tmem_alloc(&sm.tmem, 512);
    if (lane == 0) {
      mbar_init(&sm.bar_load, 1);
      mbar_init(&sm.bar_mma, 1);
      fence_mbar_init();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm.tmem;
  const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);

  const float g = fmaxf(p.log_decay[h], -1e4f), g2 = g * kLaLog2e;
  const bool strong = g2 * kLaChunk < kLaCut;  // some row factor of a full chunk is below the cut
  const float a = R.rev ? 0.f : 1.f;
  const int hq = h / R.div_q, hk = h / R.div_k, hv = h / R.div_v;

  // the state: row `row`, columns 64 ch .. +63
  float S[64];
  const int src = R.rev ? seg.src_rev : seg.src_fwd;
  const float* sp = nullptr;
  if constexpr (kOut) {
    if (src == -2)
      sp = (R.rev ? p.slot_r : p.slot_f) + ((size_t)sidx * p.Hv + h) * kLaState;
    else if (R.rev)
      sp = p.dfinal ? p.dfinal + ((size_t)seg.doc * p.Hv + h) * kLaState : nullptr;
    else if (src >= 0)
      sp = p.start + ((size_t)src * p.Hv + h) * kLaState;
  }
  if (!sp) {
#pragma unroll
    for (int j = 0; j < 64; ++j) S[j] = 0.f;
  } else if (R.trans) {
#pragma unroll
    for (int j = 0; j < 64; ++j) S[j] = sp[(size_t)(64 * ch + j) * kDim + row];
  } else {
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      const float4 x = *reinterpret_cast<const float4*>(sp + (size_t)row * kDim + 64 * ch + j);
      S[j] = x.x;
      S[j + 1] = x.y;
      S[j + 2] = x.z;
      S[j + 3] = x.w;
    }
  }

  const uint32_t idesc_qk = idesc_bf16(128, 128, 0, 0), idesc_mn = idesc_bf16(128, 128, 0, 1);
  const uint64_t dq = kmajor_desc(smem_u32(sm.q), kTile / 2, 0), dk = kmajor_desc(smem_u32(sm.k), kTile / 2, 0);
  const uint64_t dv = mnmajor_desc(smem_u32(sm.v), kTile / 2, 0), ds = mnmajor_desc(smem_u32(sm.s), kTile / 2, 0);

  const int nch = (seg.ntok + kLaChunk - 1) / kLaChunk;
  uint32_t ph_load = 0, ph_mma = 0;
  bool ok = true;
  for (int c = 0; c < nch; ++c) {
    // chunks are cut from the segment's first token in both directions
    const int ci = R.rev ? nch - 1 - c : c;
    const int tok = seg.tok0 + ci * kLaChunk;
    const int n = min(kLaChunk, seg.ntok - ci * kLaChunk);
    if (tid == 0) {
      mbar_arrive_expect_tx(&sm.bar_load, (kOut ? 3 : 2) * kTile);
      if constexpr (kOut) load_tile(sm.q, &p.map[R.mq], hq, tok, &sm.bar_load);
      load_tile(sm.k, &p.map[R.mk], hk, tok, &sm.bar_load);
      load_tile(sm.v, &p.map[R.mv], hv, tok, &sm.bar_load);
    }
    if (tid < kLaChunk) {
      const int u = R.rev ? n - 1 - tid : tid;
      const bool in = tid < n;
      sm.w[tid] = in ? R.s_in * decay_pow(g, (float)(n - u) - a) : 0.f;
      if constexpr (kOut) {
        sm.col[tid] = in ? R.s_in * exp2f(-g2 * ((float)u + a)) : 0.f;
        sm.rowe[tid] = in ? fmaxf(g2 * ((float)u + a), kLaCut) : 0.f;
      }
    }
    const float lam_hi = expf(g * (float)n);
    if (!wait_all(&sm.bar_load, ph_load)) {
      ok = false;
      break;
    }
    ph_load ^= 1;
    // rows past the chunk belong to another document (or lie outside the tensor): zero them, so
    // that nothing they hold reaches the products
    if (n < kLaChunk) {
      for (int i = tid; i < (kLaChunk - n) * 16; i += kLaThreads) {
        const int r = n + i / 16, x = i % 16;
        *reinterpret_cast<uint4*>(sm.v + (x >> 3) * (kTile / 2) + r * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
    }
    // weighted keys, transposed (lane = key dimension), as hi + lo bf16
    {
      const uint8_t* kb = sm.k + (row >> 6) * (kTile / 2);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int t = 64 * ch + 32 * half + 2 * j;
          const float w0 = sm.w[t], w1 = sm.w[t + 1];
          float x0 = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(kb + sw128_off(t, row & 63)));
          float x1 = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(kb + sw128_off(t + 1, row & 63)));
          x0 = t < n ? x0 * w0 : 0.f;
          x1 = t + 1 < n ? x1 * w1 : 0.f;
          const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
          hi[j] = *reinterpret_cast<const uint32_t*>(&b);
          lo[j] = pack_bf16x2(x0 - __low2float(b), x1 - __high2float(b));
        }
        tmem_st16(tl + kColHi + 32 * ch + 16 * half, hi);
        tmem_st16(tl + kColLo + 32 * ch + 16 * half, lo);
      }
      tmem_st_wait();
    }
    if constexpr (kOut) {
      // the state as the queries' operand: row = key dimension, 64 value columns to a block
      uint8_t* sb = sm.s + ch * (kTile / 2);
#pragma unroll
      for (int j = 0; j < 64; j += 8)
        *reinterpret_cast<uint4*>(sb + sw128_off(row, j)) =
            make_uint4(pack_bf16x2(S[j], S[j + 1]), pack_bf16x2(S[j + 2], S[j + 3]), pack_bf16x2(S[j + 4], S[j + 5]),
                       pack_bf16x2(S[j + 6], S[j + 7]));
    }
    sync_generic_to_async();
    if (tid == 0) {
      if constexpr (kOut) {
        mma_ss(tm + kColQK, dq, dk, false, idesc_qk);
        mma_ss(tm + kColO, dq, ds, true, idesc_mn);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        umma_bf16_ts(tm + kColKV, tm + (i < 8 ? kColHi : kColLo) + 8 * (i & 7), mnmajor_step(dv, i & 7), idesc_mn, i > 0);
      umma_commit(&sm.bar_mma);
    }
    if (!wait_all(&sm.bar_mma, ph_mma)) {
      ok = false;
      break;
    }
    ph_mma ^= 1;
    tc_fence_after();
    if constexpr (kOut) {
      // P'': row = query token, columns = key tokens; bf16 over the fp32 columns this warp has read
      const int ut = R.rev ? n - 1 - row : row;
      const float re = sm.rowe[row];
      float x[64];
      tmem_ld32(tl + kColQK + 64 * ch, x);
      tmem_ld32(tl + kColQK + 64 * ch + 32, x + 32);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 64; ++j) {
        const int s = 64 * ch + j;
        const int us = R.rev ? n - 1 - s : s;
        const float f = strong ? R.s_in * exp2f(g2 * (float)(ut - us) - re) : sm.col[s];
        x[j] = (us <= ut && s < n) ? x[j] * f : 0.f;
      }
      // hi + lo, 32 columns each: a row may have a single term of weight, whose rounding nothing averages
      uint32_t hi[32], lo[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        hi[j] = *reinterpret_cast<const uint32_t*>(&b);
        lo[j] = pack_bf16x2(x[2 * j] - __low2float(b), x[2 * j + 1] - __high2float(b));
      }
      tmem_st16(tl + kColQK + 64 * ch, hi);
      tmem_st16(tl + kColQK + 64 * ch + 16, hi + 16);
      tmem_st16(tl + kColQK + 64 * ch + 32, lo);
      tmem_st16(tl + kColQK + 64 * ch + 48, lo + 16);
      tmem_st_wait();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int ks = i & 7;
          umma_bf16_ts(tm + kColO, tm + kColQK + 64 * (ks >> 2) + 32 * (i >> 3) + 8 * (ks & 3), mnmajor_step(dv, ks),
                       idesc_mn, 1);
        }
        umma_commit(&sm.bar_mma);
      }
    }
    // S = lam^n S + this chunk's part
    {
      const float hi = g * (float)n, lo = fmaf(g, (float)n, -hi);
      const float lam_lo = isfinite(lo) ? lam_hi * lo : 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[32];
        tmem_ld32(tl + kColKV + 64 * ch + 32 * half, x);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) S[32 * half + j] = fmaf(S[32 * half + j], lam_hi, fmaf(S[32 * half + j], lam_lo, x[j]));
      }
    }
    if constexpr (kOut) {
      if (!wait_all(&sm.bar_mma, ph_mma)) {
        ok = false;
        break;
      }
      ph_mma ^= 1;
      tc_fence_after();
      float x[64];
      tmem_ld32(tl + kColO + 64 * ch, x);
      tmem_ld32(tl + kColO + 64 * ch + 32, x + 32);
      tmem_ld_wait();
      const float f = R.s_out * exp2f(sm.rowe[row]);
      if (row < n) {
        const size_t at = ((size_t)(tok + row) * p.Hv + h) * kDim + 64 * ch;
        if (R.out_f32) {
          float* o = static_cast<float*>(R.out) + at;
#pragma unroll
          for (int j = 0; j < 64; j += 4)
            *reinterpret_cast<float4*>(o + j) = make_float4(x[j] * f, x[j + 1] * f, x[j + 2] * f, x[j + 3] * f);
        } else {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(R.out) + at;
#pragma unroll
          for (int j = 0; j < 64; j += 8)
            *reinterpret_cast<uint4*>(o + j) =
                make_uint4(pack_bf16x2(x[j] * f, x[j + 1] * f), pack_bf16x2(x[j + 2] * f, x[j + 3] * f),
                           pack_bf16x2(x[j + 4] * f, x[j + 5] * f), pack_bf16x2(x[j + 6] * f, x[j + 7] * f));
        }
      }
    }
    tc_fence_before();
    __syncthreads();
  }
  if (!ok) {
    if (tid == 0) la_status(p.hd, kErrTimeout);
  } else {
    float* dst = nullptr;
    if (!kOut)
      dst = (R.rev ? p.slot_r : p.slot_f) + ((size_t)sidx * p.Hv + h) * kLaState;
    else if (R.last && (R.rev ? seg.k == 0 : seg.k == seg.nseg - 1))
      dst = R.last + ((size_t)seg.doc * p.Hv + h) * kLaState;
    if (dst) {
#pragma unroll
      for (int j = 0; j < 64; j += 4)
        *reinterpret_cast<float4*>(dst + (size_t)row * kDim + 64 * ch + j) =
            make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
    }
  }
  __syncthreads();
  if (wid == 0) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------------------------------- scan

// Start states of the segments from their end states from zero, in place: one thread per head and
// four elements walks the documents in order (blockIdx.y = 1: the state gradients, from the end).
__global__ void __launch_bounds__(256) la_scan_kernel(const __grid_constant__ LaParams p) {
  griddep_wait();
  griddep_launch_dependents();
  if (!p.hd->scan) return;
  const int h = blockIdx.x / 16, e = ((blockIdx.x % 16) * 256 + threadIdx.x) * 4;
  const float g = fmaxf(p.log_decay[h], -1e4f);
  auto at = [&](float* base, int i) { return reinterpret_cast<float4*>(base + ((size_t)i * p.Hv + h) * kLaState + e); };
  auto cat = [&](const float* base, int i) {
    return *reinterpret_cast<const float4*>(base + ((size_t)i * p.Hv + h) * kLaState + e);
  };
  auto step = [&](float4& S, int n, const float4& b) {
    const float l = decay_pow(g, (float)n);
    S = make_float4(fmaf(S.x, l, b.x), fmaf(S.y, l, b.y), fmaf(S.z, l, b.z), fmaf(S.w, l, b.w));
  };
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  if (blockIdx.y == 0) {
    for (int d = 0; d < p.N; ++d) {
      const int s0 = p.seg0[d], s1 = p.seg0[d + 1];
      const int idx = p.init_idx ? p.init_idx[d] : -1;
      const bool fork = idx >= 0 && idx >= p.n_init, src = p.is_src[d] != 0;
      if (s1 - s0 == 1 && !fork && !src) continue;
      float4 S = fork ? *at(p.fin, idx - p.n_init) : idx >= 0 ? cat(p.start, idx) : zero;
      for (int s = s0; s < s1; ++s) {
        const int need = p.segs[s].need, n = p.segs[s].ntok;
        float4* slot = at(p.slot_f, s);
        const float4 b = (need & 1) ? *slot : zero;
        *slot = S;
        step(S, n, b);
      }
      if (src) *at(p.fin, d) = S;
    }
  } else {
    if (p.init_idx)
      for (int d = 0; d < p.N; ++d)
        if (p.is_src[d]) *at(p.acc, d) = zero;
    for (int d = p.N - 1; d >= 0; --d) {
      const int s0 = p.seg0[d], s1 = p.seg0[d + 1];
      const int idx = p.init_idx ? p.init_idx[d] : -1;
      const bool fork = idx >= 0 && idx >= p.n_init, src = p.is_src[d] != 0;
      if (s1 - s0 == 1 && !fork && !src) continue;
      float4 X = p.dfinal ? cat(p.dfinal, d) : zero;
      if (src) {
        const float4 b = *at(p.acc, d);
        X = make_float4(X.x + b.x, X.y + b.y, X.z + b.z, X.w + b.w);
      }
      for (int s = s1 - 1; s >= s0; --s) {
        const int need = p.segs[s].need, n = p.segs[s].ntok;
        float4* slot = at(p.slot_r, s);
        const float4 b = (need & 2) ? *slot : zero;
        *slot = X;
        step(X, n, b);
      }
      if (fork) {
        float4* acc = at(p.acc, idx - p.n_init);
        const float4 b = *acc;
        *acc = make_float4(X.x + b.x, X.y + b.y, X.z + b.z, X.w + b.w);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------- sums

// dq, dk of the shared key heads: the sum over each group's value heads, in their order
struct LaGroupParams {
  const float *part_q, *part_k;
  __nv_bfloat16 *dq, *dk;
  int64_t n4;  // T * Hk * 32
  int G;
};
__global__ void __launch_bounds__(256) la_group_sum_kernel(const __grid_constant__ LaGroupParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const float* src = blockIdx.y ? p.part_k : p.part_q;
  __nv_bfloat16* dst = blockIdx.y ? p.dk : p.dq;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.n4; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i >> 5;
    const int c = (int)(i & 31) * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < p.G; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(src + (row * p.G + j) * kDim + c);
      a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
    }
    *reinterpret_cast<uint2*>(dst + row * kDim + c) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

// gradient of each pool entry: the sum over the documents that start from it, in their order
struct LaInitParams {
  const float* dstart;
  const int32_t* init_idx;
  const LaHeader* hd;
  float* dinit;
  int N, Hv;
};
__global__ void __launch_bounds__(256) la_init_sum_kernel(const __grid_constant__ LaInitParams p) {
  griddep_wait();
  griddep_launch_dependents();
  if (p.hd->n_segs == 0) return;
  const int x = blockIdx.y;
  const size_t e = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4, per = (size_t)p.Hv * kLaState;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int d = 0; d < p.N; ++d) {
    if (p.init_idx == nullptr || p.init_idx[d] != x) continue;
    const float4 b = *reinterpret_cast<const float4*>(p.dstart + (size_t)d * per + e);
    a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
  }
  *reinterpret_cast<float4*>(p.dinit + (size_t)x * per + e) = a;
}

// ---------------------------------------------------------------------------------------- host

bool al(const void* p, uintptr_t b) { return (reinterpret_cast<uintptr_t>(p) % b) == 0; }

int sm_count(int dev) {
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 152;
  }
  return n;
}

bool la_sizes_ok(int N, int T, int H_k, int H_v) {
  return N >= 1 && T >= 0 && H_k >= 1 && H_v >= 1 && H_v % H_k == 0 && (int64_t)T * H_v * kDim <= ((int64_t)1 << 40) &&
         ((int64_t)N + T / kLaChunk) * H_v < (int64_t)INT32_MAX && H_v <= 4096;
}

struct LaCall {
  const void *q, *k, *v, *dout;
  const float* log_decay;
  const int32_t* cu;
  int N, T, Hk, Hv, head_dim;
  const int64_t* strides;
  const int32_t* init_idx;
  const float* initial_state;
  int n_init;
  float scale;
  void* ws;
  size_t ws_bytes;
  bool bwd;
};

PerDevice g_la_setup;

// Everything the two directions share: checks, the workspace's addresses, the tensor maps.
int la_prepare(const LaCall& c, const void* const* outs, int n_outs, LaParams* p, LaLayout* L, DeviceGuard& guard,
               int* num_sms) {
  if (c.head_dim != kDim) return GDN_ERR_UNSUPPORTED;
  if (!la_sizes_ok(c.N, c.T, c.Hk, c.Hv) || c.n_init < 0 || c.scale != c.scale) return GDN_ERR_INVALID_ARG;
  if (!c.log_decay || !c.cu || !c.ws || (c.n_init > 0 && !c.initial_state)) return GDN_ERR_INVALID_ARG;
  if (c.T > 0 && (!c.q || !c.k || !c.v || (c.bwd && !c.dout))) return GDN_ERR_INVALID_ARG;
  const void* in[4] = {c.q, c.k, c.v, c.dout};
  const int heads[4] = {c.Hk, c.Hk, c.Hv, c.Hv};
  int64_t stride[4];
  for (int i = 0; i < 4; ++i) {
    // the forward's array has no entry for dout
    const int64_t given = c.strides && (i < 3 || c.bwd) ? c.strides[i] : 0;
    stride[i] = given ? given : (int64_t)heads[i] * kDim;
    if (stride[i] < (int64_t)heads[i] * kDim || stride[i] % 8 != 0 || stride[i] >= ((int64_t)1 << 38))
      return GDN_ERR_INVALID_ARG;
    if (!al(in[i], 16)) return GDN_ERR_INVALID_ARG;
  }
  for (int i = 0; i < n_outs; ++i)
    if (!al(outs[i], 16)) return GDN_ERR_INVALID_ARG;
  if (!al(c.initial_state, 16) || !al(c.ws, 256)) return GDN_ERR_INVALID_ARG;
  const void* ptrs[16] = {c.q, c.k, c.v, c.dout, c.log_decay, c.cu, c.init_idx, c.initial_state};
  for (int i = 0; i < n_outs; ++i) ptrs[8 + i] = outs[i];
  int dev = 0;
  if (device_of(c.ws, ptrs, 8 + n_outs, &dev) != kOk) return GDN_ERR_INVALID_ARG;
  if (!guard.set(dev)) return GDN_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (major != 10 || minor != 3) return GDN_ERR_UNSUPPORTED;
  *num_sms = sm_count(dev);
  *L = la_layout(c.N, c.T, c.Hk, c.Hv, c.init_idx != nullptr, c.bwd, *num_sms);
  if (c.ws_bytes < L->total) return GDN_ERR_WORKSPACE;
  if (!g_la_setup.done(dev)) {
    const int smem = sizeof(LaSmem) + 1024;
    if (cudaFuncSetAttribute(la_chunk_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(la_chunk_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return GDN_ERR_CUDA;
    g_la_setup.mark(dev);
  }
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  *p = LaParams{};
  for (int i = 0; i < (c.bwd ? 4 : 3); ++i)
    if (c.T > 0 && !make_tmap_bf16_3d(&p->map[i], in[i], kDim, heads[i], c.T, kDim * 2, (uint64_t)stride[i] * 2, 64, 1,
                                      kLaChunk))
      return GDN_ERR_CUDA;
  p->log_decay = c.log_decay;
  p->start = c.initial_state;
  p->hd = reinterpret_cast<LaHeader*>(ws + L->header);
  p->segs = reinterpret_cast<LaSeg*>(ws + L->segs);
  p->seg0 = reinterpret_cast<int32_t*>(ws + L->seg0);
  p->is_src = reinterpret_cast<int32_t*>(ws + L->is_src);
  p->slot_f = reinterpret_cast<float*>(ws + L->slot_f);
  p->slot_r = reinterpret_cast<float*>(ws + L->slot_r);
  p->fin = reinterpret_cast<float*>(ws + L->fin);
  p->acc = reinterpret_cast<float*>(ws + L->acc);
  p->cu = c.cu;
  p->init_idx = c.init_idx;
  p->N = c.N;
  p->T = c.T;
  p->Hv = c.Hv;
  p->n_init = c.n_init;
  p->seg_chunks = L->seg_chunks;
  p->bwd = c.bwd;
  return GDN_OK;
}

void la_launch_chunks(const LaParams& p, const LaLayout& L, bool out, int roles, cudaStream_t s) {
  const dim3 grid((unsigned)(L.smax * p.Hv), roles);
  const size_t smem = sizeof(LaSmem) + 1024;
  if (out)
    launch_early(la_chunk_kernel<true>, grid, kLaThreads, smem, s, p);
  else
    launch_early(la_chunk_kernel<false>, grid, kLaThreads, smem, s, p);
}

// Plan, and, where documents are cut or may fork, the segments' start states.
void la_launch_starts(const LaParams& p, const LaLayout& L, const LaRole& fwd, const LaRole* rev, cudaStream_t s) {
  launch_early(la_plan_kernel, dim3(1), kLaPlanThreads, 0, s, p);
  if (!L.seg_chunks && !p.init_idx) return;
  LaParams a = p;
  a.role[0] = fwd;
  if (rev) a.role[1] = *rev;
  la_launch_chunks(a, L, false, rev ? 2 : 1, s);
  launch_early(la_scan_kernel, dim3(16 * p.Hv, rev ? 2 : 1), 256, 0, s, a);
}

}  // namespace
}  // namespace gdn

extern "C" size_t gdn_la_workspace_size(int N, int T, int H_k, int H_v, int has_init, int backward) {
  if (!gdn::la_sizes_ok(N, T, H_k, H_v)) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
  return gdn::la_layout(N, T, H_k, H_v, has_init != 0, backward != 0, gdn::sm_count(dev)).total;
}

extern "C" int gdn_la_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                          const int32_t* cu_seqlens, int N, int T, int H_k, int H_v, int head_dim,
                          const int64_t* strides, const int32_t* init_idx, const float* initial_state, int n_init,
                          float scale, void* out, float* final_state, void* workspace, size_t ws_bytes,
                          gdn_stream_t stream) {
  using namespace gdn;
  if (!final_state || (T > 0 && !out)) return GDN_ERR_INVALID_ARG;
  const LaCall c{q,       k,        v,             nullptr, log_decay, cu_seqlens, N,        T,    H_k, H_v, head_dim,
                 strides, init_idx, initial_state, n_init,  scale,     workspace,  ws_bytes, false};
  const void* outs[] = {out, final_state};
  LaParams p;
  LaLayout L;
  DeviceGuard guard;
  int sms = 0;
  const int rc = la_prepare(c, outs, 2, &p, &L, guard, &sms);
  if (rc != GDN_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  const int G = H_v / H_k;
  const LaRole fwd{kMapQ, kMapK, kMapV, G, G, 1, 0, 0, 1.f, scale, out, 0, final_state};
  la_launch_starts(p, L, fwd, nullptr, s);
  p.role[0] = fwd;
  la_launch_chunks(p, L, true, 1, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_la_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                          const int32_t* cu_seqlens, int N, int T, int H_k, int H_v, int head_dim,
                          const int64_t* strides, const int32_t* init_idx, const float* initial_state, int n_init,
                          float scale, const void* dout, const float* dfinal_state, void* dq, void* dk, void* dv,
                          float* dinitial_state, void* workspace, size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  if (T > 0 && (!dq || !dk || !dv)) return GDN_ERR_INVALID_ARG;
  if (n_init > 0 && !dinitial_state) return GDN_ERR_INVALID_ARG;
  const LaCall c{q,       k,        v,             dout,   log_decay, cu_seqlens, N,        T,   H_k, H_v, head_dim,
                 strides, init_idx, initial_state, n_init, scale,     workspace,  ws_bytes, true};
  const void* outs[] = {dq, dk, dv, dinitial_state, dfinal_state};
  LaParams p;
  LaLayout L;
  DeviceGuard guard;
  int sms = 0;
  const int rc = la_prepare(c, outs, 5, &p, &L, guard, &sms);
  if (rc != GDN_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int G = H_v / H_k;
  p.dfinal = dfinal_state;
  float* part_q = G > 1 ? reinterpret_cast<float*>(ws + L.part_q) : nullptr;
  float* part_k = G > 1 ? reinterpret_cast<float*>(ws + L.part_k) : nullptr;
  float* dstart = n_init > 0 && init_idx ? reinterpret_cast<float*>(ws + L.dstart) : nullptr;
  const LaRole fwd{kMapQ, kMapK, kMapV, G, G, 1, 0, 0, 1.f, scale, nullptr, 0, nullptr};
  const LaRole rdq{kMapDo, kMapV, kMapK, 1, 1, G, 0, 1, 1.f, scale, G > 1 ? (void*)part_q : dq, G > 1, nullptr};
  const LaRole rdv{kMapK, kMapQ, kMapDo, G, G, 1, 1, 0, scale, 1.f, dv, 0, dstart};
  const LaRole rdk{kMapV, kMapDo, kMapQ, 1, 1, G, 1, 1, scale, 1.f, G > 1 ? (void*)part_k : dk, G > 1, nullptr};
  la_launch_starts(p, L, fwd, &rdv, s);
  p.role[0] = rdq;
  p.role[1] = rdv;
  p.role[2] = rdk;
  la_launch_chunks(p, L, true, 3, s);
  if (G > 1 && T > 0) {
    const LaGroupParams gp{part_q, part_k, static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk),
                           (int64_t)T * H_k * 32, G};
    const int64_t blocks = (gp.n4 + 255) / 256;
    launch_early(la_group_sum_kernel, dim3((unsigned)(blocks < 16 * sms ? blocks : 16 * sms), 2), 256, 0, s, gp);
  }
  if (n_init > 0) {
    const LaInitParams ip{dstart, init_idx, p.hd, dinitial_state, N, H_v};
    launch_early(la_init_sum_kernel, dim3(16 * H_v, n_init), 256, 0, s, ip);
  }
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
