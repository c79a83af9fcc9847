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
// Precision. The products' operands are bf16. The state is held in fp32 registers and its update uses the weighted
// keys as a sum of bf16 terms: three (relative error 2.5e-8 an element) as long as the chunk's part reaches an fp32
// state among the outputs before it has decayed below 2^-10, else two (2.5e-6: far below the rounding of the bf16
// copy of the state that the queries read). The map P is a sum of two bf16 terms near its diagonal (in the 32 x 32
// blocks on it): a row may hold a single entry of weight there (the first tokens, a strong decay), and its rounding
// would double that of the output. The rest of P, and the state that the queries read, are rounded to bf16 once: an
// output averages many of those roundings. Gradients of shared keys are summed over the heads in fp32.
//
// Row factors leave the products: the output is r_t (S^T q_t + sum_s P''_ts v_s) with r_t = lam^{u+a} and
// P'' = P / r_t, so the query enters the state product as it was loaded. What is summed is then larger than the output
// by 1 / r_t. Heads whose r_t falls below 2^-24 within a chunk (log-decay below -0.13) take another way: P as it is
// (its weights are at most 1), and the state's term S^T q_t multiplied with its row factor in tensor memory, in fp32,
// before P V is added. So nothing is larger than 2^24 times the product it stands for, and every row factor is
// the decay's own down to fp32's end. (With one cut at 2^-86 for all heads, sums above 2^42 became infinite, and
// a row whose values were all zero kept 2^-86 of a state that had decayed further. With two such heads of eight
// the extra pass costs 3 %: 16384 tokens in 12 documents 72.5 -> 74.7 us, the backward of 65536 tokens 479 -> 492.)
//
// A call is a planner, a walk that leaves the end state of each segment of a cut document (from zero), a scan over
// them, the walk that forms the outputs, and in the backward the sums over shared heads. Measured on a GB300 (device
// time of each kernel, us; 128 dimensions, 2 key heads and 8 value heads):
//                                     planner  states  scan  outputs  sums
//     forward, 1 x 32768 tokens             6      26     8       44     -    (HBM floor 25 for all of it)
//     forward, 16384 tokens, 12 documents   6      21     8       42     -    (13)
//     backward, 65536 tokens, 4 documents   6      74    14      296    87    (79)
// The walks are bound by the chain of hand-overs between their warps, below; the sums by HBM traffic (6.9 TB/s).
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

constexpr float kLaLog2e = 1.44269504f;
constexpr float kLaCut = -24.f;  // log2 of the smallest row factor that leaves the products
constexpr uint32_t kTile = 32768;  // 128 x 128 bf16, two 64-column blocks

enum { kMapQ = 0, kMapK = 1, kMapV = 2, kMapDo = 3 };

struct LaRole {
  int mq, mk, mv, mo;       // tensor maps of the role's query, key, value and output
  int div_q, div_k, div_v;  // value heads to one head of each
  int rev;                  // walks the document from its end
  int trans;                // its state is stored transposed
  float s_in, s_out;        // factors of the key rows (and P), and of the output
  void* out;                // [T, Hv, 128] bf16, or fp32 partials
  int out_f32;
  float* last;              // state after the document's last segment of this role: [N, Hv, 128, 128]
};

struct LaParams {
  CUtensorMap map[4], map_out[3];
  LaRole role[3];
  int n_roles;
  const float* log_decay;
  const float* start;   // pool of start states
  const float* dfinal;  // gradient of the final states, or null
  LaHeader* hd;
  LaSeg* segs;    // the longest first
  int32_t* seg0;  // each document's first segment, documents in order
  int32_t* is_src;
  float *slot_f, *slot_r, *fin, *acc;
  float *end_fwd, *end_rev;  // final states, start-state gradients of the documents; null = not wanted
  const int32_t* cu;
  const int32_t* init_idx;
  int N, T, Hv, n_init, min_seg, num_sms, bwd;
  int withheld;      // tile of each walk's first CTA that a test leaves out (-1 = none)
  long long budget;  // limit of a wait, clock cycles
};

__device__ __forceinline__ void la_status(LaHeader* hd, int code) { atomicCAS(&hd->status, 0, code); }

// The head's log-decay, no lower than -10000 (whose exponential is zero as well). A NaN stays one, and with it every
// output of the head: a maximum would turn it into a decay that forgets everything.
__device__ __forceinline__ float la_decay(const LaParams& p, int h) {
  const float g = p.log_decay[h];
  return g < -1e4f ? -1e4f : g;
}

// ---------------------------------------------------------------------------------------- plan

constexpr int kLaPlanThreads = 1024;

// Time of a call with documents cut to segments of L chunks (0 = uncut), in chunks of the output walk. From the
// documents: chunks in all and in the cut ones, segments in all and in the cut ones, the longest segment.
// Measured: an item's start (its state, the first tiles, the pipeline's fill) costs about one chunk; a chunk of
// the states-only walk 0.6; a cut segment's slot, written, scanned in place and read, three; the two extra
// kernels four. Items are drawn longest first, so the last ones end about half a segment apart, unless all fit
// the SMs at once.
__device__ __forceinline__ float la_plan_cost(const LaParams& p, int chunks, int cut_chunks, int segs, int cut_segs,
                                              int longest) {
  const float roles = p.bwd ? 3.f : 1.f, passes = p.bwd ? 2.f : 1.f, sms = (float)p.num_sms, Hv = (float)p.Hv;
  auto walk = [&](float items, float work, float seg) {
    return items <= sms ? seg : fmaxf(work / sms + 0.5f * seg, seg);
  };
  float t = walk(roles * Hv * segs, roles * Hv * (chunks + (float)segs), longest + 1.f);
  if (cut_segs)
    t += 4.f + walk(passes * Hv * cut_segs, passes * Hv * (0.6f * cut_chunks + 3.f * cut_segs), 0.6f * longest + 3.f);
  return t;
}

// One CTA: checks cu_seqlens and init_idx, chooses the segments' length among 32 candidates (one to a warp) and
// cuts the documents into segments.
__global__ void __launch_bounds__(kLaPlanThreads) la_plan_kernel(const __grid_constant__ LaParams p) {
  griddep_wait();  // the previous call on this stream may still read the workspace
  griddep_launch_dependents();
  __shared__ int s_warp[32], s_base, s_bad, s_scan, s_len, s_hist[64];
  __shared__ float s_cost[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tid == 0) {
    s_base = 0;
    s_bad = 0;
    s_scan = 0;
  }
  if (tid < 64) s_hist[tid] = 0;
  if (p.init_idx)
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
      p.hd->n_starts = 0;
      p.hd->scan = 0;
    }
    return;
  }
  if (p.min_seg) {
    // candidates: 16 lengths spread over the logarithm, 15 from the one that gives an item to each SM, uncut
    const float all = (float)(p.T / kLaChunk + 1);
    int L = 0;
    if (wid < 16)
      L = (int)((float)p.min_seg * exp2f((float)wid / 16.f * log2f(fmaxf(1.f, all / (float)p.min_seg))));
    else if (wid < 31)
      L = (int)ceilf(all * (float)p.Hv * (p.bwd ? 3.f : 1.f) / (float)p.num_sms) + wid - 16;
    if (wid < 31) L = max(L, p.min_seg);
    int chunks = 0, cut_chunks = 0, segs = 0, cut_segs = 0, longest = 0;
    for (int i = lane; i < p.N; i += 32) {
      const int n = (p.cu[i + 1] - p.cu[i] + kLaChunk - 1) / kLaChunk;
      const bool cut = L && n > L;
      const int k = cut ? (n + L - 1) / L : 1;
      chunks += n;
      segs += k;
      if (cut) {
        cut_chunks += n;
        cut_segs += k;
      }
      longest = max(longest, cut ? L : n);
    }
    chunks = __reduce_add_sync(0xffffffffu, chunks);
    cut_chunks = __reduce_add_sync(0xffffffffu, cut_chunks);
    segs = __reduce_add_sync(0xffffffffu, segs);
    cut_segs = __reduce_add_sync(0xffffffffu, cut_segs);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
      s_cost[wid] = la_plan_cost(p, chunks, cut_chunks, segs, cut_segs, longest);
      s_warp[wid] = L;
    }
    __syncthreads();
    if (wid == 0) {
      float c = s_cost[lane];
      int best = lane;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float c2 = __shfl_xor_sync(0xffffffffu, c, o);
        const int b2 = __shfl_xor_sync(0xffffffffu, best, o);
        if (c2 < c || (c2 == c && b2 > best)) {  // uncut where it is no worse
          c = c2;
          best = b2;
        }
      }
      if (lane == 0) s_len = s_warp[best];
    }
    __syncthreads();
  } else if (tid == 0) {
    s_len = 0;
  }
  __syncthreads();
  const int seg_tok = s_len * kLaChunk;
  auto bucket = [](int tokens) { return 63 - min(63, (tokens + kLaChunk - 1) / kLaChunk); };
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
      if (cnt > 1 || (idx >= 0 && idx >= p.n_init) || (p.init_idx && p.is_src[i])) s_scan = 1;
      if (cnt > 1) atomicAdd(&s_hist[bucket(seg_tok)], cnt - 1);
      atomicAdd(&s_hist[bucket(len - (cnt - 1) * seg_tok)], 1);
    }
    __syncthreads();
    if (tid == 0) s_base += total;
    __syncthreads();
  }
  // the order in which items are drawn: by length, the longest first (a length's order among itself is free:
  // no result depends on it)
  if (wid == 0) {
    const int h0 = s_hist[2 * lane], h1 = s_hist[2 * lane + 1];
    int x = h0 + h1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += t;
    }
    s_hist[2 * lane] = x - h0 - h1;
    s_hist[2 * lane + 1] = x - h1;
  }
  __syncthreads();
  const int n_segs = s_base;
  for (int g = tid; g < n_segs; g += kLaPlanThreads) {
    int i = 0, hi = p.N;  // the document: the last one whose first segment is not after this one
    while (hi - i > 1) {
      const int mid = (i + hi) >> 1;
      (p.seg0[mid] <= g ? i : hi) = mid;
    }
    const int b = p.cu[i], len = p.cu[i + 1] - b;
    const int cnt = (seg_tok && len > seg_tok) ? (len + seg_tok - 1) / seg_tok : 1, k = g - p.seg0[i];
    const int idx = p.init_idx ? p.init_idx[i] : -1;
    const bool fork = idx >= p.n_init && idx >= 0, src = p.init_idx && p.is_src[i] != 0;
    LaSeg s;
    s.doc = i;
    s.tok0 = b + k * seg_tok;
    s.ntok = cnt > 1 ? min(seg_tok, len - k * seg_tok) : len;
    s.k = k;
    s.nseg = cnt;
    s.src_fwd = (k > 0 || fork) ? -2 : idx;
    s.slot = g;
    // a cut document's final state, and its start's gradient where one is wanted, come from the scan
    s.need = ((cnt > 1 || src) ? 1 : 0) | ((k > 0 || fork || (cnt > 1 && p.end_rev)) ? 2 : 0) | (src ? 4 : 0) |
             (fork ? 8 : 0) | ((k < cnt - 1 || src) ? 16 : 0);
    p.segs[atomicAdd(&s_hist[bucket(s.ntok)], 1)] = s;
  }
  if (tid == 0) {
    p.seg0[p.N] = n_segs;
    p.hd->status = kOk;
    p.hd->n_segs = n_segs;
    p.hd->n_starts = s_scan ? n_segs : 0;
    p.hd->scan = s_scan;
    p.hd->seg_chunks = s_len;
    p.hd->ticket[0] = 0;
    p.hd->ticket[1] = 0;
  }
}

// ---------------------------------------------------------------------------------------- chunks
//
// One persistent CTA per SM walks items (segment, role, head), chunk by chunk. Warps:
//   S (8): the state's update in registers, and its bf16 copy, the queries' operand
//   K (4, without outputs 8): the weighted keys into tensor memory, 32 tokens and 32 dimensions a warp at a time
//   P/O (8): the map from Q K^T, in place in tensor memory, and the outputs
//   then a warp for the copies and one that issues the products.
// Per chunk the products are Q K^T, Q S, K~^T V (two or three terms) and P V (two terms), each of 128^3: eight
// instructions of 64 cycles a term, about 3100 cycles (3600 with three terms), against about 2900 cycles of HBM traffic
// (80 KB at four value heads to a key head). A chunk takes about 5200 cycles in the forward and 6600 where the
// output is fp32 partial sums: the tensor pipe is busy 54 % of the time. What it waits for is the chain through the warps: Q K^T
// goes to P/O, whose map takes 1600 cycles, P V follows, and its result holds P/O for another 1000 (bf16) to 3000
// (fp32) before the next map; in the meantime the state goes through S and back as an operand. With all vector work
// taken out of it an earlier form of the backward walk still took 226 of its 313 us. Tried on earlier forms, and slower:
// outputs by other warps, 16 P/O warps, two issuing warps (56, 45 and 46 us against 44), partial sums stored from registers
// (349 us against 275), the heads of a group added up in place by one CTA (341 + 36 us against 275 + 87).
// The votes that make a wait's outcome the whole warp's cost 2 % (backward of 65536 tokens 492 -> 503 us).
//
// The states-only walk has one product (1024 or 1536 cycles a chunk) and takes 2200: its first chunks wait for HBM
// (every SM fills its ring at once), the later ones for the issuing warp.
//
// Tensor memory: K~^T V, Q K^T and P (in place: 16 key tokens' fp32 columns become 8 columns of the first
// bf16 term and 8 of the second), O, and the weighted keys (four stages of 32 tokens in
// two terms, or two in three; the states-only walk: two accumulators, four stages in three).

constexpr uint32_t kColKV = 0, kColQK = 128, kColO = 256;
constexpr int kSWarps = 8, kPoWarps = 8;

// Shared memory is seven tiles of 32 KB. The role's walk keeps a ring of five (a chunk's K, Q, V in this
// order: Q is done with first, after Q S, then K, then V), the state and the outputs on their way out;
// the states-only walk a ring of seven (K, V).
template <bool kOut>
struct LaShape {
  static constexpr uint32_t kSlots = kOut ? 5 : 7, kPerChunk = kOut ? 3 : 2, kTileV = kOut ? 2 : 1;
  // the states-only walk has room for two accumulators and a stage for each quarter of a chunk's keys
  static constexpr int kKv = kOut ? 1 : 2;
  static constexpr uint32_t kColKt = kOut ? 384 : 256;
  static constexpr int kKWarps = kOut ? 4 : 8, kPo0 = kSWarps + kKWarps, kTmaWarp = kPo0 + (kOut ? kPoWarps : 0), kMmaWarp = kTmaWarp + 1;
  static constexpr int kThreads = 32 * (kTmaWarp + 4);  // whole warpgroups, so that registers can move
  // registers of a thread at launch, and what the warpgroups of each role make of them
  static constexpr int kRegs = kOut ? 80 : 96, kRegsS = kOut ? 104 : 120, kRegsK = kOut ? 72 : 88, kRegsPo = 80,
                       kRegsRest = kOut ? 40 : 64;
  static_assert(2 * kRegsS + kKWarps / 4 * kRegsK + (kOut ? 2 * kRegsPo : 0) + kRegsRest == kThreads / 128 * kRegs,
                "the split is of what the block was launched with");
};

struct LaSmem {
  uint8_t tiles[5 * kTile];
  uint8_t s[kTile], o[kTile];  // the states-only walk's last two tiles
  uint4 w[2][kLaChunk / 2];  // weights of the keys, of a full chunk and of the item's last
  float col[kLaChunk];       // column factors of P''
  uint64_t full[7], free_[7], kt_ready[4], kt_free[4], kv_full[2], kv_free[2];
  uint64_t w_sync, col_sync, drain, item_full[2], item_free[2];
  uint64_t qk_full, p_ready[2], s_ready, qs_done, o_full, o_free;
  uint32_t tmem;
  int abort;
  long long budget;
  int item[2];  // what the copy warp has drawn
};
static_assert(sizeof(LaSmem) <= 232448, "227 KB of shared memory");

__device__ __forceinline__ void load_tile(void* dst, const CUtensorMap* m, int head, int tok, uint64_t* bar) {
  tma_load_3d(dst, m, 0, head, tok, bar);
  tma_load_3d(static_cast<uint8_t*>(dst) + kTile / 2, m, 64, head, tok, bar);
}

// exp(g x) for a whole number x of steps, the product's rounding error carried along
__device__ __forceinline__ float decay_pow(float g, float x) {
  const float hi = g * x;
  const float lo = fmaf(g, x, -hi);
  const float e = expf(hi);
  return isfinite(lo) ? fmaf(e, lo, e) : e;
}

// Bounded wait of one thread; false once any role of the CTA has given up.
__device__ __forceinline__ bool la_wait(uint64_t* bar, uint32_t parity, LaSmem& sm) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
    if (clock64() - t0 > sm.budget) {
      *reinterpret_cast<volatile int*>(&sm.abort) = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// The same of a whole warp: every lane has the same outcome, so that none leaves while others go on to an instruction
// of the warp (ldmatrix, the tensor-memory accesses) that expects them all.
__device__ __forceinline__ bool la_wait_warp(uint64_t* bar, uint32_t parity, LaSmem& sm) {
  if (all_ok(mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!all_ok(mbar_try_wait(bar, parity))) {
    if (!all_ok(!*reinterpret_cast<volatile int*>(&sm.abort) && clock64() - t0 <= sm.budget)) {
      *reinterpret_cast<volatile int*>(&sm.abort) = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// tmem_ld32 and its wait as one statement: nothing, not even a spill, can touch the registers in between
__device__ __forceinline__ void tmem_ld32_wait(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// 16 lanes x 16 columns: register 2i is row lane / 4, column 4i + lane % 4, register 2i + 1 row lane / 4 + 8
__device__ __forceinline__ void tmem_st16x128_x4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
  return f2_fma(b, f2_pack(-1.f, -1.f), a);
}
template <int kTo, int kFrom>
__device__ __forceinline__ void set_regs() {
  if constexpr (kTo > kFrom)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTo));
  else if constexpr (kTo < kFrom)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTo));
}
// Four lanes, a row each, four columns to a quad: lane i's quad k and lane k's quad i change places. Rows then leave
// in whole sectors, 64 bytes of a row at a time; a row to a lane, 16 bytes at a time, a state's 64 KB took about 6000
// cycles to write, longer than a chunk. (Reading a state that way as well made the registers spill: 20.6 us against
// 18.3 for 512 tokens, 277 against 269 for the backward's walk as they then were; the two halves of a sector meet in L1.)
__device__ __forceinline__ void swap_quads(float* x) {
  const bool b0 = threadIdx.x & 1, b1 = threadIdx.x & 2;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const float t = __shfl_xor_sync(0xffffffffu, b0 ? x[4 * k + c] : x[4 * k + 4 + c], 1);
      x[4 * k + c] = b0 ? t : x[4 * k + c];
      x[4 * k + 4 + c] = b0 ? x[4 * k + 4 + c] : t;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float t = __shfl_xor_sync(0xffffffffu, b1 ? x[4 * k + c] : x[4 * k + 8 + c], 2);
      x[4 * k + c] = b1 ? t : x[4 * k + c];
      x[4 * k + 8 + c] = b1 ? x[4 * k + 8 + c] : t;
    }
  }
}
// true in one lane of a converged warp, the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// the two bf16 of a word as fp32 (exact)
__device__ __forceinline__ uint64_t f2_of_bf16x2(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16x2_of(uint64_t v) { return pack_bf16x2(f2_lo(v), f2_hi(v)); }

// Columns of the weighted keys of quarter q. With outputs: four stages of two terms, or two of three.
template <bool kOut>
__device__ __forceinline__ uint32_t la_kt_col(int q, bool three) {
  return kOut ? (three ? 48u * (q & 1) : 32u * q) : 48u * q;
}

// Tile i (K 0; with outputs Q 1 and V 2, else V 1) of the CTA's x-th chunk in its ring.
template <bool kOut>
struct LaTile {
  uint32_t slot, use;
  __device__ __forceinline__ LaTile(uint32_t slot, uint32_t use) : slot(slot), use(use) {}
  static __device__ __forceinline__ LaTile of(uint32_t x, uint32_t i) {
    const uint32_t t = LaShape<kOut>::kPerChunk * x + i;
    return {t % LaShape<kOut>::kSlots, t / LaShape<kOut>::kSlots};
  }
  __device__ __forceinline__ uint8_t* at(LaSmem& sm) const { return sm.tiles + slot * kTile; }
  __device__ __forceinline__ bool wait_full(LaSmem& sm) const { return la_wait_warp(&sm.full[slot], use & 1, sm); }
};

struct LaItem;
__device__ __forceinline__ bool la_writes_end(const LaParams& p, const LaItem& it);
// One item of a CTA's walk and what its roles derive from it.
struct LaItem {
  LaSeg seg;
  int h, nch;
  int exact;  // chunks from this one on update the state with three terms
  bool strong;  // some row factor of a full chunk is below the cut
  const LaRole* R;
  __device__ __forceinline__ bool three(int c) const { return c >= exact; }
};
template <bool kOut>
__device__ __forceinline__ bool la_item(const LaParams& p, int roles, int i, LaItem& it) {
  it.h = i % p.Hv;
  const int r = (i / p.Hv) % roles;
  it.R = &p.role[r];
  it.seg = p.segs[i / (p.Hv * roles)];
  it.nch = (it.seg.ntok + kLaChunk - 1) / kLaChunk;
  const float g = -la_decay(p, it.h) * kLaChunk;  // decay of a chunk
  if (kOut) {
    // Three terms where the state itself is an output (of an uncut document; the scan gives a cut one's)
    // and this chunk's part of it is not below 2^-10 by then; else two, far below the rounding of the
    // state's bf16 copy that the queries read.
    it.strong = g * kLaLog2e > -kLaCut;
    it.exact = it.nch;
    if (la_writes_end(p, it))
      it.exact = it.nch - (g > 0.f ? (int)fminf(ceilf(7.f / g) + 1.f, (float)it.nch) : it.nch);
  } else {
    // Every chunk is walked, however deep its decay: what the later ones hold is not known beforehand, and where it
    // is smaller still (padding, values that fall in time), the early ones are the state.
    it.exact = it.nch;
    // three terms where the state reaches an output of the scan (the document's last state, or its start's
    // gradient where one is wanted, or a fork's) before it has decayed below 2^-10
    const bool fork = (it.seg.need >> 2 >> it.R->rev) & 1;
    if (fork || (it.R->rev ? p.end_rev : p.end_fwd) != nullptr) {
      const int between = it.R->rev ? it.seg.k : it.seg.nseg - 1 - it.seg.k;  // whole segments, one perhaps short
      const float away = fork ? 0.f : (float)(max(between - 1, 0) * p.hd->seg_chunks);
      it.exact = it.nch - (g > 0.f ? (int)fminf(fmaxf(ceilf(7.f / g) + 1.f - away, 0.f), (float)it.nch) : it.nch);
    }
  }
  return kOut || ((it.seg.need >> it.R->rev) & 1);
}
// whether the walk's last state goes to the role's output: an uncut document's, unless the scan has it
__device__ __forceinline__ bool la_writes_end(const LaParams& p, const LaItem& it) {
  return it.R->last != nullptr && it.seg.nseg == 1 && !((it.seg.need >> it.R->rev) & 1);
}
// chunk c of the item in its walking order: first token and count (cut from the segment's first token)
__device__ __forceinline__ int la_chunk_at(const LaItem& it, int c, int& n) {
  const int ci = it.R->rev ? it.nch - 1 - c : c;
  n = min(kLaChunk, it.seg.ntok - ci * kLaChunk);
  return it.seg.tok0 + ci * kLaChunk;
}

// kOut: the whole role (outputs and end state); otherwise only each segment's end state from zero,
// for the scan.
template <bool kOut>
__global__ void __launch_bounds__(LaShape<kOut>::kThreads, 1) la_chunk_kernel(const __grid_constant__ LaParams p) {
  using Sh = LaShape<kOut>;
  extern __shared__ __align__(1024) uint8_t raw[];
  if ((smem_u32(raw) & 1023u) != 0) {  // the swizzled tiles need it; no room is left to round up
    if (threadIdx.x == 0) la_status(p.hd, kErrCuda);
    return;
  }
  LaSmem& sm = *reinterpret_cast<LaSmem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (wid == Sh::kMmaWarp) tmem_alloc(&sm.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < 7; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.free_[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_free[i], Sh::kTmaWarp + 1);  // the other warps that work
      mbar_init(&sm.kv_free[i], kSWarps);
    }
    for (int i = 0; i < 4; ++i) {
      if (i < 2) mbar_init(&sm.p_ready[i], 4);
      mbar_init(&sm.kt_ready[i], 4);
      mbar_init(&sm.kt_free[i], 1);
    }
    mbar_init(&sm.w_sync, Sh::kKWarps);
    mbar_init(&sm.col_sync, kPoWarps);
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.qk_full, 1);
    mbar_init(&sm.qs_done, 1);
    mbar_init(&sm.s_ready, kSWarps);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, kPoWarps);
    sm.abort = 0;
    sm.budget = p.budget;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, sm.tmem, 0);
  griddep_wait();
  griddep_launch_dependents();
  const int roles = p.n_roles;
  const int n_items = (kOut ? p.hd->n_segs : p.hd->n_starts) * roles * p.Hv;
  // The next item of a warp's walk, as the copy warp has drawn it; false at the end (or after a failed wait).
  uint32_t items = 0;
  auto next_item = [&](LaItem& it) {
    for (;;) {
      const uint32_t slot = items & 1, use = items >> 1;
      if (!la_wait_warp(&sm.item_full[slot], use & 1, sm)) return false;
      const int i = *reinterpret_cast<volatile int*>(&sm.item[slot]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_free[slot]);
      ++items;
      if (i >= n_items) return false;
      if (la_item<kOut>(p, roles, i, it)) return true;
    }
  };
  uint32_t cc = 0;      // chunks this CTA has begun, over all its items
  uint32_t loaded = 0;  // tiles that the copy warp has asked for
  bool ok = true;
  LaItem it;

  if (wid < kSWarps) {
    // ------------------------------------------------------------------ state
    set_regs<Sh::kRegsS, Sh::kRegs>();
    const int quarter = wid & 3, ch = wid >> 2;  // tensor-memory lanes 32 quarter .. +31, columns 64 ch .. +63
    constexpr int kCols = 64;
    const int row = 32 * quarter + lane;
    const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
    float S[kCols];
    while (ok && next_item(it)) {
      const LaRole& R = *it.R;
      const float g = la_decay(p, it.h);
      const float* sp = nullptr;
      if constexpr (kOut) {
        const int src = it.seg.src_fwd;
        if (R.rev ? it.seg.need & 16 : src == -2)
          sp = (R.rev ? p.slot_r : p.slot_f) + ((size_t)it.seg.slot * p.Hv + it.h) * kLaState;
        else if (R.rev)
          sp = p.dfinal ? p.dfinal + ((size_t)it.seg.doc * p.Hv + it.h) * kLaState : nullptr;
        else if (src >= 0)
          sp = p.start + ((size_t)src * p.Hv + it.h) * kLaState;
      }
      if (!sp) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) S[j] = 0.f;
      } else if (R.trans) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) S[j] = sp[(size_t)(kCols * ch + j) * kDim + row];
      } else {
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
          const float4 x = *reinterpret_cast<const float4*>(sp + (size_t)row * kDim + kCols * ch + j);
          S[j] = x.x;
          S[j + 1] = x.y;
          S[j + 2] = x.z;
          S[j + 3] = x.w;
        }
      }
      float lam_hi = 1.f, lam_lo = 0.f;
      int n_state = -1;
      // the state as the queries' operand: row = key dimension, 64 value columns to a block
      auto publish = [&]() {
        if constexpr (kOut) {
          uint8_t* sb = sm.s + ch * (kTile / 2);
#pragma unroll
          for (int j = 0; j < kCols; j += 8)
            *reinterpret_cast<uint4*>(sb + sw128_off(row, j)) =
                make_uint4(pack_bf16x2(S[j], S[j + 1]), pack_bf16x2(S[j + 2], S[j + 3]),
                           pack_bf16x2(S[j + 4], S[j + 5]), pack_bf16x2(S[j + 6], S[j + 7]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_ready);
        }
      };
      if (it.nch > 0) publish();
      for (int c = 0; c < it.nch; ++c, ++cc) {
        if (!(ok = la_wait_warp(&sm.kv_full[cc % Sh::kKv], (cc / Sh::kKv) & 1, sm))) break;
        tc_fence_after();
        int n;
        la_chunk_at(it, c, n);
        if (n != n_state) {
          const float hi = g * (float)n, lo = fmaf(g, (float)n, -hi);
          lam_hi = expf(hi);
          lam_lo = isfinite(lo) ? lam_hi * lo : 0.f;
          n_state = n;
        }
        // S = lam^n S + this chunk's part
        const uint64_t lh = f2_pack(lam_hi, lam_hi), ll = f2_pack(lam_lo, lam_lo);
#pragma unroll
        for (int y = 0; y < kCols; y += 32) {
          float x[32];
          tmem_ld32_wait(tl + kColKV + 128 * (cc % Sh::kKv) + kCols * ch + y, x);
          if (y + 32 == kCols) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.kv_free[cc % Sh::kKv]);
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint64_t s2 = f2_pack(S[y + j], S[y + j + 1]);
            const uint64_t r = f2_fma(s2, lh, f2_fma(s2, ll, f2_pack(x[j], x[j + 1])));
            S[y + j] = f2_lo(r);
            S[y + j + 1] = f2_hi(r);
          }
        }
        // the copy of the state that the queries of this chunk read may go
        if constexpr (kOut)
          if (!(ok = la_wait_warp(&sm.qs_done, cc & 1, sm))) break;
        if (c + 1 < it.nch) publish();
      }
      if (!ok) break;
      float* dst = nullptr;
      if (!kOut)
        dst = (R.rev ? p.slot_r : p.slot_f) + ((size_t)it.seg.slot * p.Hv + it.h) * kLaState;
      else if (la_writes_end(p, it))
        dst = R.last + ((size_t)it.seg.doc * p.Hv + it.h) * kLaState;
      if (dst) {
        // where a lane's first four columns lie once each four lanes have exchanged theirs
        dst += (row & ~3) * kDim + kCols * ch + 4 * (lane & 3);
#pragma unroll
        for (int j = 0; j < kCols; j += 16) {
          swap_quads(S + j);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4*>(dst + k * kDim + j) =
                make_float4(S[j + 4 * k], S[j + 4 * k + 1], S[j + 4 * k + 2], S[j + 4 * k + 3]);
        }
      }
    }
  } else if (wid < Sh::kPo0) {
    // ------------------------------------------------------------------ keys
    set_regs<Sh::kRegsK, Sh::kRegs>();
    const int quarter = wid & 3, q0 = (wid - kSWarps) >> 2;  // dimensions 32 quarter .. +31; first quarter of the tokens
    constexpr int kQStep = Sh::kKWarps / 4;
    const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
    uint32_t w_phase = 0;
    bool was_three = false;  // terms of the chunk before
    auto sync_w = [&]() {  // these warps meet, with the limit of every other wait
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.w_sync);
      const bool met = la_wait_warp(&sm.w_sync, w_phase, sm);
      w_phase ^= 1;
      return met;
    };
    while (ok && next_item(it)) {
      const LaRole& R = *it.R;
      const float g = la_decay(p, it.h);
      const float a = R.rev ? 0.f : 1.f;
      // The weights, for full chunks and for the last one: in pairs of tokens, as fp32, and as bf16 of the
      // weight and of its rest.
      if (!(ok = sync_w())) break;  // every warp is done with the last item's
      if (const int e = tid - 32 * kSWarps; e < kLaChunk) {
        const int t = e & 63, n = e < 64 ? kLaChunk : it.seg.ntok - (it.nch - 1) * kLaChunk;
        float f[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int tok = 2 * t + z, u = R.rev ? n - 1 - tok : tok;
          f[z] = tok < n ? R.s_in * decay_pow(g, (float)(n - u) - a) : 0.f;
        }
        const uint32_t w1 = pack_bf16x2(f[0], f[1]);
        const uint64_t r = f2_sub(f2_pack(f[0], f[1]), f2_of_bf16x2(w1));
        sm.w[e >> 6][t] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), w1, bf16x2_of(r));
      }
      if (!(ok = sync_w())) break;
      for (int c = 0; ok && c < it.nch; ++c, ++cc) {
        // The chunk's weighted keys, 32 tokens (a quarter) and 32 dimensions a warp at a time, in two or three
        // bf16 terms.
        int n;
        la_chunk_at(it, c, n);
        const LaTile<kOut> tk = LaTile<kOut>::of(cc, 0);
        const bool three = it.three(c);
        if (!(ok = tk.wait_full(sm))) break;
        // rows past the chunk belong to another document (or lie outside the tensor): nothing they hold may
        // reach the products
        if (q0 == 0 && n < kLaChunk) {
          const LaTile<kOut> tv = LaTile<kOut>::of(cc, Sh::kTileV);
          if (!(ok = tv.wait_full(sm))) break;
          uint8_t* vt = tv.at(sm);
          for (int e = tid - 32 * kSWarps; e < (kLaChunk - n) * 16; e += 128) {
            const int r = n + e / 16, y = e % 16;
            *reinterpret_cast<uint4*>(vt + (y >> 3) * (kTile / 2) + r * 128 + (y & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        // this lane's row of the four 8 x 8 blocks that a load takes: 8 tokens (lane bit 4), 8 dimensions (bit 3)
        const int tok = ((lane >> 4) & 1) * 8 + (lane & 7), d8 = 4 * quarter + ((lane >> 3) & 1);
        const uint32_t kr = smem_u32(tk.at(sm)) + (d8 >> 3) * (kTile / 2) + tok * 128;
        const uint4* wt = &sm.w[n < kLaChunk][lane & 3];
        auto load = [&](int q, int hl, uint32_t* k) {  // 32 tokens, 16 dimensions
          const uint32_t ka = kr + q * 32 * 128 + ((((d8 + 2 * hl) ^ tok) & 7) << 4);
          ldsm_x4_trans(ka, k);
          ldsm_x4_trans(ka + 16 * 128, k + 4);
          if (n < kLaChunk) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int t = 32 * q + 8 * y + 2 * (lane & 3);
              const uint32_t keep = (t < n ? 0xffffu : 0u) | (t + 1 < n ? 0xffff0000u : 0u);
              k[2 * y] &= keep;
              k[2 * y + 1] &= keep;
            }
          }
        };
        // The stage's last reader: each quarter has its own, but for three terms with outputs, where the later
        // half takes the earlier one's place. The two layouts overlap, so next to three terms a chunk follows
        // the whole of the one before. (Every earlier phase of a barrier is over when it is waited for: this
        // warp has waited for it, or for a later product. So its parity cannot be mistaken.)
        auto stage_free = [&](int q) {
          bool got = true;
          if (kOut && three && q > 0) {
            if (q >= 2) got = la_wait_warp(&sm.kt_free[q - 2], cc & 1, sm);
          } else if (cc > 0) {
            got = la_wait_warp(&sm.kt_free[kOut && q == 0 && (three || was_three) ? 3 : q], (cc - 1) & 1, sm);
          }
          tc_fence_after();
          return got;
        };
        auto ready = [&](int q) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.kt_ready[q]);
        };
        if (three) {
          auto split = [&](int q, int hl, uint32_t* k1, uint32_t* k2, uint32_t* k3) {
            load(q, hl, k3);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint4 wy = wt[16 * q + 4 * y];
              const uint64_t f = f2_pack(__uint_as_float(wy.x), __uint_as_float(wy.y));
#pragma unroll
              for (int z = 2 * y; z < 2 * y + 2; ++z) {
                const uint64_t v = f2_mul(f2_of_bf16x2(k3[z]), f);
                k1[z] = bf16x2_of(v);
                const uint64_t r1 = f2_sub(v, f2_of_bf16x2(k1[z]));
                k2[z] = bf16x2_of(r1);
                k3[z] = bf16x2_of(f2_sub(r1, f2_of_bf16x2(k2[z])));
              }
            }
          };
          auto store = [&](int q, int hl, const uint32_t* k1, const uint32_t* k2, const uint32_t* k3) {
            const uint32_t tb = tl + Sh::kColKt + la_kt_col<kOut>(q, true) + ((uint32_t)(16 * hl) << 16);
            tmem_st16x128_x4(tb, k1);
            tmem_st16x128_x4(tb + 16, k2);
            tmem_st16x128_x4(tb + 32, k3);
          };
#pragma unroll 1
          for (int q = q0; q < 4; q += kQStep) {
            if constexpr (kOut) {
              // 16 dimensions (lanes) at a time: the loop stays rolled, since the roles' code together should
              // stay in the instruction cache; the first half is ready before the stage is waited for
#pragma unroll 1
              for (int hl = 0; hl < 2; ++hl) {
                uint32_t k1[8], k2[8], k3[8];
                split(q, hl, k1, k2, k3);
                if (hl == 0 && !(ok = stage_free(q))) break;
                store(q, hl, k1, k2, k3);
              }
              if (!ok) break;
            } else {  // all of it before the stage is waited for
              uint32_t k1[2][8], k2[2][8], k3[2][8];
              split(q, 0, k1[0], k2[0], k3[0]);
              split(q, 1, k1[1], k2[1], k3[1]);
              if (!(ok = stage_free(q))) break;
              store(q, 0, k1[0], k2[0], k3[0]);
              store(q, 1, k1[1], k2[1], k3[1]);
            }
            ready(q);
          }
        } else {
          // With w = w1 + w2 in bf16: k w1 rounded, then its exact error (16 bits in all) plus k w2. All of it is
          // done before the stage is waited for: the products of the chunk before decide how soon this chunk's
          // can follow.
#pragma unroll 1
          for (int q = q0; q < 4; q += kQStep) {
            uint32_t k[2][8], k1[2][8];
            load(q, 0, k[0]);
            load(q, 1, k[1]);
            const uint4* w = wt + 16 * q;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint2 wy = *reinterpret_cast<const uint2*>(&w[4 * y].z);
#pragma unroll
              for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                for (int z = 2 * y; z < 2 * y + 2; ++z) {
                  k1[hl][z] = bf2_mul(k[hl][z], wy.x);
                  k[hl][z] = bf2_fma(k[hl][z], wy.y, bf2_fma(k[hl][z], wy.x, k1[hl][z] ^ 0x80008000u));
                }
            }
            if (!(ok = stage_free(q))) break;
#pragma unroll
            for (int hl = 0; hl < 2; ++hl) {
              const uint32_t tb = tl + Sh::kColKt + la_kt_col<kOut>(q, false) + ((uint32_t)(16 * hl) << 16);
              tmem_st16x128_x4(tb, k1[hl]);
              tmem_st16x128_x4(tb + 16, k[hl]);
            }
            ready(q);
          }
        }
        was_three = three;
      }
    }
  } else if (kOut && wid < Sh::kTmaWarp) {
    // ------------------------------------------------------------------ map and outputs
    set_regs<Sh::kRegsPo, Sh::kRegs>();
    const int quarter = wid & 3, half = (wid - Sh::kPo0) >> 2;  // query rows 32 quarter .. +31, columns 64 half .. +63
    const int row = 32 * quarter + lane, ct = tid - 32 * Sh::kPo0;
    uint32_t col_phase = 0;
    auto sync_col = [&]() {  // the eight warps meet, with the limit of every other wait
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.col_sync);
      const bool met = la_wait_warp(&sm.col_sync, col_phase, sm);
      col_phase ^= 1;
      return met;
    };
    const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
    while (ok && next_item(it)) {
      const LaRole& R = *it.R;
      const float g2 = la_decay(p, it.h) * kLaLog2e;
      const bool strong = it.strong;
      const float a = R.rev ? 0.f : 1.f;
      int n_prev = -1, ut = 0;
      float re = 0.f, of = 0.f, rf = 1.f;  // of the row: log2 of its factor outside the products, of its output, of S^T q
      if (!(ok = sync_col())) break;  // every warp is done with the last item's
      if (ct < kLaChunk) sm.col[ct] = R.s_in * exp2f(-g2 * ((float)(R.rev ? kLaChunk - 1 - ct : ct) + a));
      if (!(ok = sync_col())) break;
      const uint32_t diag = R.rev ? 0xffffffffu << lane : (2u << lane) - 1u;  // the diagonal block's columns of this row
      for (int c = 0; c < it.nch; ++c, ++cc) {
        int n;
        const int tok = la_chunk_at(it, c, n);
        if (n != n_prev) {
          ut = R.rev ? n - 1 - row : row;
          const float e = row < n ? g2 * ((float)ut + a) : 0.f;
          re = strong ? 0.f : e;
          rf = strong ? exp2f(e) : 1.f;
          of = R.s_out * exp2f(re);
          n_prev = n;
        }
        if (!(ok = la_wait_warp(&sm.qk_full, cc & 1, sm))) break;
        tc_fence_after();
        // P'': row = query token; 16 key tokens' fp32 columns become 8 columns of each bf16 term
        float x[32];
#pragma unroll 1
        for (int jb = 2 * half; jb < 2 * half + 2; ++jb) {
          const uint32_t tq = tl + kColQK + 32 * jb;
          if (R.rev ? jb < quarter : jb > quarter) {
            uint32_t z[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = 0;
            tmem_st16(tq, z);
            tmem_st16(tq + 16, z);
          } else {
            tmem_ld32_wait(tq, x);
            if (strong || (R.rev && n < kLaChunk)) {
              // whole numbers of steps, exact in fp32, before the decay multiplies them
              const float base = (float)(R.rev ? ut - (n - 1) + 32 * jb : ut - 32 * jb), step = R.rev ? 1.f : -1.f;
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] *= R.s_in * ex2(g2 * fmaxf(fmaf(step, (float)j, base), 0.f) - re);
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&sm.col[32 * jb + j]);
                const uint64_t v0 = f2_mul(f2_pack(x[j], x[j + 1]), f2_pack(f.x, f.y));
                const uint64_t v1 = f2_mul(f2_pack(x[j + 2], x[j + 3]), f2_pack(f.z, f.w));
                x[j] = f2_lo(v0);
                x[j + 1] = f2_hi(v0);
                x[j + 2] = f2_lo(v1);
                x[j + 3] = f2_hi(v1);
              }
            }
            if (jb == quarter) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(diag & (1u << j))) x[j] = 0.f;
            }
            if (n < kLaChunk) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = 32 * jb + j < n ? x[j] : 0.f;
            }
#pragma unroll
            for (int k16 = 0; k16 < 2; ++k16) {
              uint32_t t[16];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                t[j] = pack_bf16x2(x[16 * k16 + 2 * j], x[16 * k16 + 2 * j + 1]);
                t[8 + j] = 0;
              }
              if (jb == quarter) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  t[8 + j] = bf16x2_of(f2_sub(f2_pack(x[16 * k16 + 2 * j], x[16 * k16 + 2 * j + 1]), f2_of_bf16x2(t[j])));
              }
              tmem_st16(tq + 16 * k16, t);
            }
          }
        }
        if (strong) {  // the state's term with its row's factor, before P V is added to it
          if (!(ok = la_wait_warp(&sm.qs_done, cc & 1, sm))) break;
          tc_fence_after();
#pragma unroll 1
          for (int jb = 0; jb < 4; ++jb) {
            const uint32_t to = tl + kColO + 64 * half + 16 * jb;
            uint32_t z[16];
            tmem_ld16_wait(to, z);
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = __float_as_uint(rf * __uint_as_float(z[j]));
            tmem_st16(to, z);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[half]);
        // The outputs leave through 4 KB of shared memory of the warp's own, as the tensor maps store them
        // (32 rows of 64 bf16, or of 32 fp32 partial sums at a time); rows of a ragged end go from registers.
        const bool whole = 32 * quarter + 32 <= n;
        uint8_t* stage = sm.o + (wid - Sh::kPo0) * (kTile / 8);
        const size_t at = ((size_t)(tok + row) * p.Hv + it.h) * kDim + 64 * half;
        if (lane == 0) bulk_wait_read_all();
        if (!(ok = la_wait_warp(&sm.o_full, cc & 1, sm))) break;
        tc_fence_after();
        __syncwarp();
        const uint64_t of2 = f2_pack(of, of);
#pragma unroll 1
        for (int jb = 0; jb < 2; ++jb) {
          tmem_ld32_wait(tl + kColO + 64 * half + 32 * jb, x);
          if (jb == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.o_free);
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint64_t v = f2_mul(f2_pack(x[j], x[j + 1]), of2);
            x[j] = f2_lo(v);
            x[j + 1] = f2_hi(v);
          }
          if (R.out_f32) {
            if (jb == 1) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
            }
            if (whole) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<float4*>(stage + sw128_off(lane, 8 * j)) =
                    make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&p.map_out[R.mo], stage, 64 * half + 32 * jb, it.h, tok + 32 * quarter);
                bulk_commit_group();
              }
            } else if (row < n) {
              float* o = static_cast<float*>(R.out) + at + 32 * jb;
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4*>(o + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
            }
          } else {
            uint4 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              b[j] = make_uint4(pack_bf16x2(x[8 * j], x[8 * j + 1]), pack_bf16x2(x[8 * j + 2], x[8 * j + 3]),
                                pack_bf16x2(x[8 * j + 4], x[8 * j + 5]), pack_bf16x2(x[8 * j + 6], x[8 * j + 7]));
            if (whole) {
#pragma unroll
              for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(stage + sw128_off(lane, 32 * jb + 8 * j)) = b[j];
            } else if (row < n) {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(R.out) + at + 32 * jb;
#pragma unroll
              for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(o + 8 * j) = b[j];
            }
          }
        }
        if (whole && !R.out_f32) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&p.map_out[R.mo], stage, 64 * half, it.h, tok + 32 * quarter);
            bulk_commit_group();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  } else {
    set_regs<Sh::kRegsRest, Sh::kRegs>();
  }
  if (wid == Sh::kTmaWarp) {
    // ------------------------------------------------------------------ copies
    if (lane == 0) {
      // Items are drawn one ahead of the walk: the first by the block's number, then from a counter, so that a
      // CTA with short ones takes more.
      int i = blockIdx.x;
      for (; ok; ++items) {
        const uint32_t slot = items & 1, use = items >> 1;
        if (use > 0 && !(ok = la_wait(&sm.item_free[slot], (use - 1) & 1, sm))) break;
        *reinterpret_cast<volatile int*>(&sm.item[slot]) = i;
        mbar_arrive(&sm.item_full[slot]);
        if (i >= n_items) break;
        const int drawn = i;
        i = (int)gridDim.x + atomicAdd(&p.hd->ticket[kOut], 1);
        if (!la_item<kOut>(p, roles, drawn, it)) continue;
        const LaRole& R = *it.R;
        const int hq = it.h / R.div_q, hk = it.h / R.div_k, hv = it.h / R.div_v;
        for (int c = 0; c < it.nch; ++c, ++cc) {
          int n;
          const int tok = la_chunk_at(it, c, n);
#pragma unroll
          for (uint32_t x = 0; x < Sh::kPerChunk; ++x) {
            const LaTile<kOut> t = LaTile<kOut>::of(cc, x);
            if (t.use > 0 && !(ok = la_wait(&sm.free_[t.slot], (t.use - 1) & 1, sm))) break;
            const bool key = x == 0, val = x == Sh::kTileV;
            if (blockIdx.x != 0 || (int)loaded != p.withheld) {
              mbar_arrive_expect_tx(&sm.full[t.slot], kTile);
              load_tile(t.at(sm), &p.map[key ? R.mk : val ? R.mv : R.mq], key ? hk : val ? hv : hq, tok, &sm.full[t.slot]);
            }
            ++loaded;
          }
          if (!ok) break;
        }
      }
    }
  } else if (wid == Sh::kMmaWarp) {
    // ------------------------------------------------------------------ products
    // One elected lane issues: elect.sync keeps the branch and the descriptors uniform. With a test of
    // the lane number each product took 57 cycles to issue (its operands move to uniform registers
    // one by one), close to the 64 cycles it takes to run; elected it takes under 32. For the same reason
    // the trip counts and the outcomes of the waits are made uniform (shuffles and votes).
    // A chunk's order is Q K^T, Q S, the state's product, P V: the two in the middle run while the map is made.
    const uint32_t id_qk = idesc_bf16(128, 128, 0, 0), id_mn = idesc_bf16(128, 128, 0, 1);
    const uint64_t ds = mnmajor_desc(smem_u32(sm.s), kTile / 2, 0);
    // The ring's next tile and the descriptors of its first: kept as the walk goes, so that little is left to
    // compute between a chunk's last product and the next one's first.
    const uint64_t kmaj0 = kmajor_desc(smem_u32(sm.tiles), kTile / 2, 0), mnmaj0 = mnmajor_desc(smem_u32(sm.tiles), kTile / 2, 0);
    uint32_t next_slot = 0, next_use = 0;
    auto next_tile = [&]() {
      LaTile<kOut> t(next_slot, next_use);
      if (++next_slot == Sh::kSlots) {
        next_slot = 0;
        next_use ^= 1;
      }
      return t;
    };
    auto tile_at = [&](uint64_t first, const LaTile<kOut>& t) { return first + (uint64_t)(t.slot * (kTile >> 4)); };
    while (ok && next_item(it)) {
      const int nch = __shfl_sync(0xffffffffu, it.nch, 0);
      const int exact = __shfl_sync(0xffffffffu, it.exact, 0);
      const bool strong = kOut && __shfl_sync(0xffffffffu, (int)it.strong, 0);
      for (int c = 0; ok && c < nch; ++c, ++cc) {
        const uint32_t par = cc & 1, kvb = cc % Sh::kKv, kvu = cc / Sh::kKv, tkv = tm + kColKV + 128 * kvb;
        const LaTile<kOut> tk = next_tile(), tq = kOut ? next_tile() : tk, tv = next_tile();
        const uint64_t dv = tile_at(mnmaj0, tv);
        if constexpr (kOut) {
          const uint64_t dk = tile_at(kmaj0, tk), dq = tile_at(kmaj0, tq);
          if (!(ok = tk.wait_full(sm) && tq.wait_full(sm))) break;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_bf16(tm + kColQK, kmajor_step(dq, kTile / 2, ks), kmajor_step(dk, kTile / 2, ks), id_qk, ks > 0);
            umma_commit(&sm.qk_full);
          }
          __syncwarp();
          // this chunk's state is in place, and the outputs of the chunk before have been read
          if (!(ok = all_ok(la_wait(&sm.s_ready, par, sm) && (cc == 0 || la_wait(&sm.o_free, (cc - 1) & 1, sm))))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_bf16(tm + kColO, kmajor_step(dq, kTile / 2, ks), mnmajor_step(ds, ks), id_mn, ks > 0);
            umma_commit(&sm.qs_done);
            umma_commit(&sm.free_[tq.slot]);
          }
          __syncwarp();
        }
        const bool three = c >= exact;
        // (the accumulator is free: with outputs s_ready says so too)
        if (!(ok = all_ok(tv.wait_full(sm) && (kOut || kvu == 0 || la_wait(&sm.kv_free[kvb], (kvu - 1) & 1, sm))))) break;
        // Products go out in groups as large as their operands allow: the pipe drains while this warp waits.
        if (kOut && !three) {
          // (the last quarter's keys come after the others': one group of warps converts all four)
          if (!(ok = all_ok(la_wait(&sm.kt_ready[3], par, sm)))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t ka = tm + Sh::kColKt;
#pragma unroll
            for (int x = 0; x < 16; ++x) {  // two terms of eight steps of 16 tokens
              umma_bf16_ts(tkv, ka + la_kt_col<kOut>(x >> 2, false) + 16 * ((x >> 1) & 1) + 8 * (x & 1),
                           mnmajor_step(dv, 2 * (x >> 2) + (x & 1)), id_mn, x > 0);
              if ((x & 3) == 3) umma_commit(&sm.kt_free[x >> 2]);
            }
            umma_commit(&sm.kv_full[kvb]);
            umma_commit(&sm.free_[tk.slot]);
          }
          __syncwarp();
        } else if (kOut) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {  // 32 tokens at a time
            if (!(ok = all_ok(la_wait(&sm.kt_ready[q], par, sm)))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t ka = tm + Sh::kColKt + la_kt_col<kOut>(q, true);
              const uint64_t dvq = dv + (uint64_t)q * (4096u >> 4);
#pragma unroll
              for (int x = 0; x < 6; ++x)
                umma_bf16_ts(tkv, ka + 16 * (x >> 1) + 8 * (x & 1), mnmajor_step(dvq, x & 1), id_mn, x > 0 ? 1u : (uint32_t)q);
              umma_commit(&sm.kt_free[q]);
              if (q == 3) {
                umma_commit(&sm.kv_full[kvb]);
                umma_commit(&sm.free_[tk.slot]);
              }
            }
            __syncwarp();
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < 4; q += 2) {  // 64 tokens at a time, as the two groups of warps convert them
            if (!(ok = all_ok(la_wait(&sm.kt_ready[q], par, sm) && la_wait(&sm.kt_ready[q + 1], par, sm)))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t ka = tm + Sh::kColKt + la_kt_col<kOut>(q, true);
              const uint64_t dvq = dv + (uint64_t)q * (4096u >> 4);
#pragma unroll
              for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  umma_bf16_ts(tkv, ka + 48 * y + 16 * (x >> 1) + 8 * (x & 1), mnmajor_step(dvq, 2 * y + (x & 1)), id_mn,
                               x + y > 0 ? 1u : (uint32_t)q);
                if (three) {
                  umma_bf16_ts(tkv, ka + 48 * y + 32, mnmajor_step(dvq, 2 * y), id_mn, 1);
                  umma_bf16_ts(tkv, ka + 48 * y + 40, mnmajor_step(dvq, 2 * y + 1), id_mn, 1);
                }
                umma_commit(&sm.kt_free[q + y]);
              }
              if (q == 2) {
                umma_commit(&sm.kv_full[kvb]);
                umma_commit(&sm.free_[tk.slot]);
                umma_commit(&sm.free_[tv.slot]);
              }
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        if constexpr (kOut) {
#pragma unroll 1
          for (int j = 0; j < 2; ++j) {  // P V for 64 key tokens
            // a strong decay: both halves of O have their row factors before the first product is added to any
            if (!(ok = all_ok(la_wait(&sm.p_ready[j], par, sm) && (!strong || la_wait(&sm.p_ready[1], par, sm))))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dvj = dv + (uint64_t)j * (8192u >> 4);
#pragma unroll
              for (int x = 0; x < 8; ++x)  // two terms of four steps
                umma_bf16_ts(tm + kColO, tm + kColQK + 64 * j + 16 * (x & 3) + 8 * (x >> 2), mnmajor_step(dvj, x & 3), id_mn, 1);
              if (j == 1) {
                umma_commit(&sm.o_full);
                umma_commit(&sm.free_[tv.slot]);
              }
            }
            __syncwarp();
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (sm.abort) {
    // Copies still in flight land before the shared memory goes, whichever role has given up.
    if (wid == Sh::kTmaWarp && lane == 0)
      for (uint32_t x = loaded < Sh::kSlots ? 0 : loaded - Sh::kSlots; x < loaded; ++x)
        mbar_wait(&sm.full[x % Sh::kSlots], (x / Sh::kSlots) & 1, sm.budget);
    // Products still in flight: everything issued reads shared memory that no copy writes any more; a last
    // commit, waited for with a limit, orders them before the tensor memory goes.
    if (wid == Sh::kMmaWarp) {
      if (elect_one()) {
        umma_commit(&sm.drain);
        mbar_wait(&sm.drain, 0, kWaitBudget);
        la_status(p.hd, kErrTimeout);
      }
      __syncwarp();
    }
    __syncthreads();
  }
  if (wid == Sh::kMmaWarp) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------------------------------- scan

// Start states of the segments from their end states from zero, in place: one thread per head and
// four elements walks the documents in order (blockIdx.y = 1: the state gradients, from the end), every blockIdx.z-th
// one where no document can fork from another. The slots
// of a document do not depend on one another, so eight are read ahead of the recurrence. Each slot is read and
// written once: 19 segments of 8 heads, 20 MB through L2 in 8 us, most of it the recurrence's latency.
__global__ void __launch_bounds__(256) la_scan_kernel(const __grid_constant__ LaParams p) {
  griddep_wait();
  griddep_launch_dependents();
  if (!p.hd->scan) return;
  const int h = blockIdx.x / 16, e = ((blockIdx.x % 16) * 256 + threadIdx.x) * 4;
  const float g = la_decay(p, h);
  const bool rev = blockIdx.y != 0;
  const int seg_tok = p.hd->seg_chunks * kLaChunk;
  const size_t per = (size_t)p.Hv * kLaState;
  const size_t off = (size_t)h * kLaState + e;
  auto at = [&](float* base, int i) { return reinterpret_cast<float4*>(base + i * per + off); };
  auto cat = [&](const float* base, int i) { return *reinterpret_cast<const float4*>(base + i * per + off); };
  auto add = [](const float4& a, const float4& b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); };
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const float l_full = decay_pow(g, (float)seg_tok);
  float* slots = rev ? p.slot_r : p.slot_f;
  if (rev && p.init_idx)
    for (int d = 0; d < p.N; ++d)
      if (p.is_src[d]) *at(p.acc, d) = zero;
  for (int i = blockIdx.z; i < p.N; i += gridDim.z) {
    const int d = rev ? p.N - 1 - i : i;
    const int s0 = p.seg0[d], cnt = p.seg0[d + 1] - s0;
    const int idx = p.init_idx ? p.init_idx[d] : -1;
    const bool fork = idx >= 0 && idx >= p.n_init, src = p.init_idx && p.is_src[d] != 0;
    if (cnt == 1 && !fork && !src) continue;
    const int len = p.cu[d + 1] - p.cu[d];
    // an empty document hands its start state on, whatever the decay
    const float l_last = len > 0 ? decay_pow(g, (float)(len - (cnt - 1) * seg_tok)) : 1.f;
    float4 S;
    if (rev) {
      S = p.dfinal ? cat(p.dfinal, d) : zero;
      if (src) S = add(S, *at(p.acc, d));
    } else {
      S = fork ? *at(p.fin, idx - p.n_init) : idx >= 0 ? cat(p.start, idx) : zero;
    }
    for (int k0 = 0; k0 < cnt; k0 += 8) {
      float4 b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = k0 + j;  // in the walk's order; the last one's end state may not have been asked for
        const bool need = k < cnt && (k < cnt - 1 || (rev ? fork || (cnt > 1 && p.end_rev) : src || cnt > 1));
        b[j] = need ? *at(slots, rev ? s0 + cnt - 1 - k : s0 + k) : zero;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = k0 + j;
        if (k >= cnt) break;
        const int q = rev ? cnt - 1 - k : k;
        *at(slots, s0 + q) = S;
        const float l = q == cnt - 1 ? l_last : l_full;
        S = make_float4(fmaf(S.x, l, b[j].x), fmaf(S.y, l, b[j].y), fmaf(S.z, l, b[j].z), fmaf(S.w, l, b[j].w));
      }
    }
    if (rev) {
      if (fork) *at(p.acc, idx - p.n_init) = add(*at(p.acc, idx - p.n_init), S);
      if (p.end_rev) *at(p.end_rev, d) = S;
    } else {
      if (src) *at(p.fin, d) = S;
      if (p.end_fwd) *at(p.end_fwd, d) = S;
    }
  }
}

// ---------------------------------------------------------------------------------------- sums

// dq, dk of the shared key heads: the sum over each group's value heads, in their order. Bound by HBM traffic: four
// partial sums in, one bf16 out, 604 MB at 65536 tokens and 8 value heads in 87 us (6.9 TB/s).
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
  // entries along the grid's x, which has room for any pool; a state is 16 blocks
  const int x = blockIdx.x / (16 * p.Hv);
  const size_t e = ((size_t)(blockIdx.x % (16 * p.Hv)) * 256 + threadIdx.x) * 4, per = (size_t)p.Hv * kLaState;
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
         ((int64_t)N + T / kLaChunk) * H_v < ((int64_t)1 << 29) && H_v <= 4096;
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
    const int smem = sizeof(LaSmem);
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
  p->min_seg = L->min_seg;
  p->num_sms = *num_sms;
  p->bwd = c.bwd;
  const TestWithhold test = test_withhold();
  p->withheld = test.copy;
  p->budget = test.budget;
  return GDN_OK;
}

// 32 rows of one head, as a warp's outputs (or fp32 partial sums) are staged
bool la_part_map(CUtensorMap* m, void* out, int T, int Hv) {
  return make_tmap_f32_3d(m, out, kDim, Hv, T, kDim * 4, (uint64_t)Hv * kDim * 4, 32, 1, 32);
}
bool la_out_map(CUtensorMap* m, void* out, int T, int Hv) {
  return make_tmap_bf16_3d(m, out, kDim, Hv, T, kDim * 2, (uint64_t)Hv * kDim * 2, 64, 1, 32);
}

void la_launch_chunks(LaParams& p, const LaLayout& L, bool out, int roles, int sms, cudaStream_t s) {
  p.n_roles = roles;
  const int64_t items = L.smax * p.Hv * roles;
  const dim3 grid((unsigned)(items < sms ? items : sms));
  const size_t smem = sizeof(LaSmem);
  if (out)
    launch_early(la_chunk_kernel<true>, grid, LaShape<true>::kThreads, smem, s, p);
  else
    launch_early(la_chunk_kernel<false>, grid, LaShape<false>::kThreads, smem, s, p);
}

// Plan, and, where documents are cut or may fork, the segments' start states.
void la_launch_starts(const LaParams& p, const LaLayout& L, const LaRole& fwd, const LaRole* rev, int sms,
                      cudaStream_t s) {
  launch_early(la_plan_kernel, dim3(1), kLaPlanThreads, 0, s, p);
  if (!L.min_seg && !p.init_idx) return;
  LaParams a = p;
  a.role[0] = fwd;
  if (rev) a.role[1] = *rev;
  la_launch_chunks(a, L, false, rev ? 2 : 1, sms, s);
  // without forks the documents do not depend on one another
  const unsigned docs = p.init_idx ? 1 : (unsigned)(p.N < 8 ? p.N : 8);
  launch_early(la_scan_kernel, dim3(16 * p.Hv, rev ? 2 : 1, docs), 256, 0, s, a);
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
  const LaRole fwd{kMapQ, kMapK, kMapV, 0, G, G, 1, 0, 0, 1.f, scale, out, 0, final_state};
  if (T > 0 && !la_out_map(&p.map_out[0], out, T, H_v)) return GDN_ERR_CUDA;
  p.end_fwd = final_state;
  la_launch_starts(p, L, fwd, nullptr, sms, s);
  p.role[0] = fwd;
  la_launch_chunks(p, L, true, 1, sms, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_la_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                          const int32_t* cu_seqlens, int N, int T, int H_k, int H_v, int head_dim,
                          const int64_t* strides, const int32_t* init_idx, const float* initial_state, int n_init,
                          float scale, const void* dout, const float* dfinal_state, void* dq, void* dk, void* dv,
                          float* dinitial_state, void* workspace, size_t ws_bytes, gdn_stream_t stream) {
  using namespace gdn;
  if (T > 0 && (!dq || !dk || !dv)) return GDN_ERR_INVALID_ARG;
  if (n_init > 0 && (!dinitial_state || (int64_t)H_v * n_init > INT32_MAX / 16)) return GDN_ERR_INVALID_ARG;
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
  const LaRole fwd{kMapQ, kMapK, kMapV, 0, G, G, 1, 0, 0, 1.f, scale, nullptr, 0, nullptr};
  const LaRole rdq{kMapDo, kMapV, kMapK, 0, 1, 1, G, 0, 1, 1.f, scale, G > 1 ? (void*)part_q : dq, G > 1, nullptr};
  const LaRole rdv{kMapK, kMapQ, kMapDo, 1, G, G, 1, 1, 0, scale, 1.f, dv, 0, dstart};
  const LaRole rdk{kMapV, kMapDo, kMapQ, 2, 1, 1, G, 1, 1, scale, 1.f, G > 1 ? (void*)part_k : dk, G > 1, nullptr};
  if (T > 0 && (!la_out_map(&p.map_out[1], dv, T, H_v) ||
                (G == 1 && (!la_out_map(&p.map_out[0], dq, T, H_v) || !la_out_map(&p.map_out[2], dk, T, H_v))) ||
                (G > 1 && (!la_part_map(&p.map_out[0], part_q, T, H_v) || !la_part_map(&p.map_out[2], part_k, T, H_v)))))
    return GDN_ERR_CUDA;
  p.end_rev = dstart;
  la_launch_starts(p, L, fwd, &rdv, sms, s);
  p.role[0] = rdq;
  p.role[1] = rdv;
  p.role[2] = rdk;
  la_launch_chunks(p, L, true, 3, sms, s);
  if (G > 1 && T > 0) {
    const LaGroupParams gp{part_q, part_k, static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk),
                           (int64_t)T * H_k * 32, G};
    const int64_t blocks = (gp.n4 + 255) / 256;
    launch_early(la_group_sum_kernel, dim3((unsigned)(blocks < 16 * sms ? blocks : 16 * sms), 2), 256, 0, s, gp);
  }
  if (n_init > 0) {
    const LaInitParams ip{dstart, init_idx, p.hd, dinitial_state, N, H_v};
    launch_early(la_init_sum_kernel, dim3((unsigned)(16 * H_v * (int64_t)n_init)), 256, 0, s, ip);
  }
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
