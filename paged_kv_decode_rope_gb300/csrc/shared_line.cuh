// shared_line.cuh -- what the two kernels of paged_gqa_decode_shared agree on: how the
// shared pages' work is cut, and where its pieces are.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// What a tile costs besides its steps, in steps. With 1, 2, 4 and 8: 256 sequences behind
// 2000 tokens 38.3, 37.8, 35.9 and 36.7 us, behind three documents 127.3, 127.0, 125.7 and
// 125.9, 64 prompts of 4 beams 37.6, 37.4, 36.7 and 37.2, 30 of 8 answers 53.6, 53.4, 53.7
// and 55.3.
constexpr int kUnitCost = 4;
constexpr int kStepKeys = 64, kStepPages = kStepKeys / kPage;

// A sequence's shared blocks and its place in its tile in one word.
constexpr int kPlaceShift = 24;
static_assert(kPlaceShift + 7 <= 31, "128 members of a tile");
__device__ __forceinline__ int shared_of(int word) { return word & ((1 << kPlaceShift) - 1); }
__device__ __forceinline__ int place_of(int word) { return word >> kPlaceShift; }

// Steps of a tile that lie before offset x of its cost.
__device__ __forceinline__ int steps_before(int x) { return max(x - kUnitCost, 0); }
// How much of the line, all kv heads', a CTA has (the last ones less).
__device__ __forceinline__ long long share_of(long long total, int ctas) { return (total + ctas - 1) / ctas; }

// The pieces of the shared pages' tiles, in the workspace.
struct SharedPieces {
  int4* tiles;   // [B + 1] of each sequence's tile: where it begins on a kv head's line, its cost, shared blocks, the
                 // sequence's place in it; last the line's length
  float2* ml;    // rows' {m, l}, base 2
  float* o;      // rows' O, not normalised
  int ctas;      // of the first kernel
};
// Row (member i of the tile of kv head h that begins at sequence b0, head g of the
// group) of CTA c's piece is row (h B + b0) G + i G + g + 128 c.

// The pieces of a sequence's tile (its entry of `tiles`) and kv head h: CTAs c0 ..
// c1's (none: c1 < c0).
struct PieceRange {
  long long x, share;  // where the tile is on the line, and a CTA's share of it
  int cost, c0, c1;
};
__device__ __forceinline__ PieceRange pieces_of(int4 tile, int length, int ctas, int hkv, int h) {
  PieceRange r = {static_cast<long long>(h) * length + tile.x, share_of(static_cast<long long>(length) * hkv, ctas), tile.y, 0, -1};
  if (r.cost > 0) {
    r.c0 = static_cast<int>(r.x / r.share);
    r.c1 = static_cast<int>((r.x + r.cost - 1) / r.share);
  }
  return r;
}

// Whether CTA c of the range has a piece (a share that begins or ends in what a tile
// costs besides its steps may have none).
__device__ __forceinline__ bool has_piece(const PieceRange& r, int c) {
  const int s0 = steps_before(static_cast<int>(max(r.share * c - r.x, 0ll)));
  const int s1 = steps_before(static_cast<int>(min(r.share * (c + 1) - r.x, static_cast<long long>(r.cost))));
  return s1 > s0;
}

}  // namespace pkv
