// Selective scan over packed documents: parameters shared by the host entry points and the kernels
// (csrc/gdn_ssm.cu).
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "gdn_common.cuh"

namespace gdn {

constexpr int kSsmSegStep = 16;  // segments are multiples of it, of one at least
// Tokens between two states that the backward keeps, and a tile of its walk in reverse. Eight states or fewer go with twice
// the channels to a warp, and half the tile lets two CTAs share an SM.
__host__ __device__ constexpr int ssm_tile(int Sp) { return Sp <= 8 ? 8 : 16; }
static_assert(kSsmSegStep % ssm_tile(8) == 0 && kSsmSegStep % ssm_tile(16) == 0, "segments are whole tiles");
// Warps of a walk that segments are cut for, sixteen to each SM (that is what an SM holds forward; a few more than fit
// cost nothing, and long segments of ragged documents leave SMs idle: at most as many as fit took 203 instead of 187 us
// for 9001 tokens of 12 documents).
constexpr int kSsmFill = 16 * 152;
constexpr int kSsmMaxState = 64;

// A segment: consecutive tokens of one document that one warp walks for its channels.
struct SsmSeg {
  int32_t doc, tok0, ntok;
  int32_t last;         // of its document
  int32_t src;          // state before it: -1 zero, >= 0 pool entry, -2 its slot
  int32_t need;         // the end state from zero is needed
  int32_t pad[2];
};

struct SsmHeader {
  int32_t status;
  int32_t n_segs;
  int32_t deep;      // some fork's source is a fork
  int32_t pad[61];
};
static_assert(sizeof(SsmHeader) == 256, "header is 256 bytes");

__host__ __device__ constexpr int ssm_padded(int S) { return S <= 8 ? 8 : S <= 16 ? 16 : S <= 32 ? 32 : 64; }
// channels to a warp of the walks forward in time, and of the backward's walk
__host__ __device__ constexpr int ssm_walk_channels(int Sp) { return Sp <= 16 ? 64 : Sp == 32 ? 32 : 16; }
__host__ __device__ constexpr int ssm_grad_channels(int Sp) { return 4 * 32 / (Sp / 4); }
constexpr int kSsmWarps = 4;  // warps to a CTA

// Workspace (byte offsets). State-sized arrays hold [Sp / 4][C][4] floats: four states of one channel together,
// channels beside one another.
struct SsmLayout {
  size_t header, segs, seg0, kind, link, maps, slot, sums, slot_r, ckpt, csum, dstart, fin, part_a, part_c, part_m, total;
  int64_t smax;  // segments at most
  int64_t room, tiles;  // segments and tiles that there is room for
  int seg_tokens;  // most tokens to a segment
  int parts;  // CTAs of the backward's walk to a group of channels
};

inline SsmLayout ssm_layout(int N, int T, int C, int S, int G, bool bwd) {
  SsmLayout L{};
  const int Sp = ssm_padded(S);
  const int ch = ssm_walk_channels(Sp);
  const int64_t blocks = (int64_t)G * ((C / G + ch - 1) / ch), each = ((int64_t)T * blocks + kSsmFill - 1) / kSsmFill;
  // With few channels segments could be shorter than they are worth: a walk takes about 0.3 us a token, the scan over a
  // document's segments 1 us for sixteen. Documents are taken to be up to four times as long as the mean.
  const int64_t doc = 4 * (int64_t)T / N < T ? 4 * (int64_t)T / N : T;
  int64_t worth = kSsmSegStep;
  while (5 * worth * worth < doc) worth += kSsmSegStep;
  const int64_t most = each > worth ? each : worth, len = ((most < T ? most : T) + kSsmSegStep - 1) / kSsmSegStep * kSsmSegStep;
  L.seg_tokens = (int)(len < kSsmSegStep ? kSsmSegStep : len);
  L.smax = N + (int64_t)T / L.seg_tokens;
  // Segments grow in steps, so fewer tokens can have more of them. The room is that of any call of no more documents and
  // tokens, which makes the size monotonic: one workspace serves the largest call and all below it. A segment that is not
  // its whole batch has at least kSsmSegStep tokens, T blocks / kSsmFill and sqrt(doc / 5), where doc is T up to four
  // documents and else 4 T / N rounded down, at least 2 T / N once it is two; so T over it is at most the least of these.
  const int64_t by_worth = (int64_t)std::sqrt(2.5 * T * (N > 2 ? N : 2)) + 1, by_fill = kSsmFill / blocks;
  const int64_t more = std::max<int64_t>(1, std::min(by_fill, by_worth));
  L.room = N + std::min<int64_t>(more, T / kSsmSegStep);
  L.tiles = L.room + T / ssm_tile(Sp) + 1;
  const int per = kSsmWarps * ssm_grad_channels(Sp);
  L.parts = (C / G + per - 1) / per;
  const size_t state = (size_t)C * Sp * sizeof(float);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.header = take(sizeof(SsmHeader));
  L.segs = take(sizeof(SsmSeg) * L.room);
  L.seg0 = take(sizeof(int32_t) * (N + 1));
  L.kind = take(sizeof(int32_t) * N);
  L.maps = take((size_t)T * G * 2 * Sp * sizeof(float));  // b and c in fp32, token by token
  L.slot = take(state * L.room);                          // end states from zero, then start states
  L.sums = take(sizeof(float) * C * L.room);              // time of each segment
  if (bwd) {
    L.link = take(sizeof(int2) * N);                      // documents of the same pool entry
    L.slot_r = take(state * L.room);                      // the same for the state's gradient, in reverse
    L.ckpt = take(state * L.tiles);                       // states from zero at each tile of a segment
    L.csum = take(sizeof(float) * C * L.tiles);           // time from the segment's start to each tile
    L.dstart = take(state * N);
    L.fin = take(state * N);                              // final states of documents that others start from
    L.part_a = take(state * L.room);                      // sums of each segment: da,
    L.part_c = take(sizeof(float) * 2 * C * L.room);      //   dskip and ddt_bias
    L.part_m = take((size_t)L.parts * T * G * 2 * Sp * sizeof(float));  // db and dc of each CTA's channels
  }
  L.total = o;
  return L;
}

}  // namespace gdn
