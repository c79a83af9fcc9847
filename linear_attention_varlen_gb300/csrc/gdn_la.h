// Decayed linear attention over packed documents: parameters shared by the host entry points and
// the kernels (csrc/gdn_la.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gdn_common.cuh"

namespace gdn {

constexpr int kLaChunk = 128;  // tokens per chunk: one 128 x 128 tensor-core tile
constexpr int kLaState = kDim * kDim;

// A segment: consecutive chunks of one document that one CTA per head walks.
struct LaSeg {
  int32_t doc, tok0, ntok;
  int32_t k, nseg;       // place in the document
  int32_t src_fwd;       // state before the segment: -1 zero, >= 0 pool entry, -2 slot of this segment
  int32_t slot;          // its number, documents in order
  int32_t need;          // bit 0: the end state from zero is needed (slots), bit 1: the same in reverse time;
                         // bit 2: documents fork from this one, bit 3: it is a fork; bit 4: the state gradient
                         // after it is its slot (else the document's dfinal, or zero)
};

struct LaHeader {
  int32_t status;
  int32_t n_segs;
  int32_t scan;          // some document needs the scan over its segments (or a fork)
  int32_t seg_chunks;    // longest segment (0 = documents are not cut)
  int32_t ticket[2];     // items drawn by the states-only walk and by the output walk
  int32_t n_starts;      // segments of the states-only walk: all, or none where nothing needs the scan
  int32_t pad[57];
};
static_assert(sizeof(LaHeader) == 256, "header is 256 bytes");

// Workspace (byte offsets). Slots hold one state (64 KB) per segment and head: first the segment's
// end state from zero, then, after the scan, the state the segment starts from.
struct LaLayout {
  size_t header, segs, seg0, is_src, slot_f, slot_r, fin, acc, dstart, part_q, part_k, total;
  int64_t smax;
  int min_seg;  // shortest segment (chunks); 0 = documents are not cut
};

// Shortest segment (chunks) that the planner may cut documents into: a quarter of what gives one (segment,
// head) item to each SM, so that the slots stay a bounded part of memory; 0 where no document is long
// enough for a cut to pay (below eight chunks the two extra kernels cost more than they save).
inline int la_min_seg(int T, int Hv, int num_sms) {
  const int64_t chunks = (int64_t)T / kLaChunk + 1;
  if (chunks < 8) return 0;
  const int64_t L = (chunks * Hv + 4 * num_sms - 1) / (4 * num_sms);
  return (int)(L < 2 ? 2 : L);
}

inline LaLayout la_layout(int N, int T, int Hk, int Hv, bool has_init, bool bwd, int num_sms) {
  LaLayout L{};
  L.min_seg = la_min_seg(T, Hv, num_sms);
  L.smax = N + (L.min_seg ? (int64_t)T / ((int64_t)L.min_seg * kLaChunk) : 0);
  const size_t state = (size_t)Hv * kLaState * sizeof(float);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.header = take(sizeof(LaHeader));
  L.segs = take(sizeof(LaSeg) * L.smax);
  L.seg0 = take(sizeof(int32_t) * (N + 1));
  L.is_src = take(sizeof(int32_t) * N);
  const size_t slots = (L.min_seg || has_init) ? state * L.smax : 0;
  L.slot_f = take(slots);
  L.slot_r = take(bwd ? slots : 0);
  L.fin = take(has_init ? state * N : 0);               // final states of forked documents
  L.acc = take(has_init && bwd ? state * N : 0);        // gradients that forks send back
  L.dstart = take(has_init && bwd ? state * N : 0);     // start-state gradient of each document
  const size_t part = (bwd && Hv != Hk) ? (size_t)T * Hv * kDim * sizeof(float) : 0;
  L.part_q = take(part);
  L.part_k = take(part);
  L.total = o;
  return L;
}

}  // namespace gdn
