// How the tiles of a product are shared out over pairs of CTAs (internal): whole tiles in waves over the pairs; what is left over is
// split along s, the dimension that is summed. For host and device alike, without a GPU's state, so that a schedule can be replayed.
#pragma once

#include "common.cuh"

namespace gs {
namespace {

constexpr int kTile = 256;                 // of a pair, both ways; a CTA loads and holds 128 rows of each operand

// Division of 0 <= n < 2^31 by a divisor that the host knows: d = ceil(2^(32 + shift) / divisor) with 2^(shift - 1) < divisor <= 2^shift
// leaves the quotient exact (the excess of d, below the divisor, times n stays below 2^(32 + shift)).
struct Divisor {
  uint32_t by, shift;
  uint64_t d;
  __host__ __device__ __forceinline__ int of(int n) const {
    // d has 33 bits: its top bit adds n itself
    const uint32_t high = (uint32_t)((uint64_t)(uint32_t)n * (uint32_t)d >> 32);
    return (int)(((uint64_t)high + ((d >> 32) ? (uint32_t)n : 0u)) >> shift);
  }
};

inline Divisor divisor(int64_t by) {
  Divisor v;
  v.by = (uint32_t)by;
  v.shift = 0;
  while ((1ull << v.shift) < (uint64_t)by) ++v.shift;
  v.d = (uint64_t)((((unsigned __int128)1 << (32 + v.shift)) + by - 1) / by);
  return v;
}

// Tile t: bands of `band` tiles of the shorter way, along the longer, so that the tiles under way at a time share rows of both operands.
struct Order {
  int tiles, band, last_band, bands;       // the last band's width
  int wide;                                // the longer way is that of the columns
  Divisor per_band, in_band, in_last;
};

__host__ __device__ __forceinline__ void place_of(int t, const Order& o, int& m, int& n) {
  const int b = o.per_band.of(t), left = t - b * (int)o.per_band.by;
  const bool last = b == o.bands - 1;
  const int width = last ? o.last_band : o.band;
  const int y = last ? o.in_last.of(left) : o.in_band.of(left), x = b * o.band + left - y * width;
  m = o.wide ? x : y;
  n = o.wide ? y : x;
}

// A part has at least 4 blocks (88 tokens of 8383 x 103 bf16: 14 us, with parts of 2 and each row joined by one warp 28).
constexpr int64_t kPiece = 4;

struct Plan {
  Order order;
  int tiles, blocks, pairs, waves, piece, group, span;
};

// rows x cols of D, `blocks` of 128 bytes along s. `stacked`: every tile is a part (or several), since more rows than one are added up to a
// row of the result; there are no more tiles than pairs.
inline Plan plan_of(int64_t rows, int64_t cols, int64_t blocks, int band, int pairs, bool stacked = false) {
  Plan p;
  const int64_t m = rows > 0 ? cdiv(rows, kTile) : 1, n = cdiv(cols, kTile), across = m < n ? m : n, along = m < n ? n : m;
  Order& o = p.order;
  p.tiles = o.tiles = (int)(m * n);
  o.wide = m < n;
  o.band = (int)(across < band ? across : band);
  o.bands = (int)cdiv(across, o.band);
  o.last_band = (int)(across - (int64_t)(o.bands - 1) * o.band);
  o.per_band = divisor(along * o.band);
  o.in_band = divisor(o.band);
  o.in_last = divisor(o.last_band);
  p.blocks = (int)blocks;
  p.pairs = pairs;
  p.waves = stacked ? 0 : p.tiles / p.pairs;     // (as many stacked tiles as pairs are parts all the same, each with its own slot)
  const int64_t left = p.tiles - (int64_t)p.waves * p.pairs;
  // Where all tiles are split, pairs that take the tiles of a band side by side go through the same blocks at the same time, so that
  // the operand that they share is read from memory once.
  p.group = p.waves == 0 && o.bands == 1 && o.band < p.pairs / 2 ? o.band : 1;
  const int64_t even = cdiv(left / p.group * blocks, p.pairs / p.group), piece = even < kPiece ? kPiece : even;
  // Splitting costs a part's way out and back, and a launch: worth it where it saves 36 blocks (2300 x 2900 x 8192 integers, where it
  // saves 31 of 64: 56 us split, 49 whole; 42 x 117 x 6965, 51 of 55: 11 split, 23 whole). Stacked planes are added up in any case.
  p.piece = stacked ? (int)(piece < blocks ? piece : blocks) : left && blocks - piece >= 36 ? (int)piece : 0;
  // Where a whole number of parts a tile keeps four fifths of the pairs busy, the tiles are cut at the same places, and all pairs go
  // through the same blocks at the same time: both operands are read from memory once (gradient by the input of 4000 x 85000 x 512: 296 us
  // with 64 of 74 pairs, 333 with all and ranges that begin anywhere).
  p.span = p.blocks;
  const int64_t cuts = p.waves == 0 ? p.pairs / p.tiles : 0;
  if (p.piece && cuts > 1 && cuts * p.tiles * 5 >= 4 * p.pairs && cdiv(blocks, cuts) >= kPiece) {
    p.piece = (int)cdiv(blocks, cuts);
    p.span = (int)(cuts * p.piece);
  }
  return p;
}

// The i-th part of a pair's work: blocks [from, to) of a tile, and whether they are all of it (else its place among the parts).
struct Part {
  int m, n, from, to, slot;
  bool whole;
};

// `A` has order, blocks, pairs, waves, piece, group and span of a Plan, and stacked.
template <class A>
__host__ __device__ __forceinline__ bool part_of(const A& a, int pair, int i, Part& p) {
  int tile;
  p.slot = 0;
  if (i < a.waves || a.piece == 0) {
    tile = pair + i * a.pairs;
    if (tile >= a.order.tiles) return false;
    p.from = 0;
    p.to = a.blocks;
  } else {
    const int k = i - a.waves;                                  // a pair's range of blocks meets at most two tiles
    const int set = pair / a.group, member = pair - set * a.group;
    const int64_t all = (int64_t)((a.order.tiles - a.waves * a.pairs) / a.group) * a.span;
    const int64_t first = (int64_t)set * a.piece, last = all < first + a.piece ? all : first + a.piece;
    if (first >= last) return false;
    const int64_t t = first / a.span + k, begin = t * a.span, end = begin + a.blocks;
    const int64_t from = first > begin ? first : begin, to = last < end ? last : end;
    if (from >= to) return false;
    tile = a.waves * a.pairs + (int)t * a.group + member;
    p.from = (int)(from - begin);
    p.to = (int)(to - begin);
    p.slot = pair * 2 + k;
  }
  p.whole = p.to - p.from == a.blocks && !a.stacked;
  place_of(tile, a.order, p.m, p.n);
  return true;
}

// Where the parts of the t-th split tile lie: `count` of them, along s, the k-th in slot(k).
struct Parts {
  int64_t from;
  int first, count, piece, group, member;
  __host__ __device__ __forceinline__ int64_t slot(int k) const {
    const int64_t part = first + k;                             // a range that begins before this tile has it as its second
    return (part * group + member) * 2 + (part * piece < from ? 1 : 0);
  }
};

__host__ __device__ __forceinline__ Parts parts_of(int t, int blocks, int piece, int group, int span) {
  Parts p;
  const int set = t / group;
  p.member = t - set * group;
  p.from = (int64_t)set * span;
  p.first = (int)(p.from / piece);
  p.count = (int)((p.from + blocks - 1) / piece) - p.first + 1;
  p.piece = piece;
  p.group = group;
  return p;
}

}  // namespace
}  // namespace gs
