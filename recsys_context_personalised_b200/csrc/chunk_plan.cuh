// How the attention of new tokens over a paged cache is cut into work, shared by
// the kernels and by a host program that checks it on the CPU (no CUDA types).
//
// An item is (sample b, kv head, row tile): `rt` consecutive new tokens with all the query
// heads that read the kv head.  It covers the key blocks (`1 << bn_shift` positions each,
// aligned) that its rows see.  All items' blocks, in the order (b, head, tile, block), form
// one line that is cut into equal parts, one per worker: every worker gets the
// same number of blocks whatever the lengths are.  An item cut by a part's
// border is finished by joining its pieces.
#pragma once

#include <stdint.h>

#include "paged.cuh"

namespace gdpa {

// sum of floor((a i + b) / m) over 0 <= i < n, for a, b >= 0, m > 0: the lattice points under a line, by the known
// descent of Euclid's algorithm.  Whole multiples of m in a and b are sums in closed form; what is left lies under a line
// of slope below 1, whose points are counted along the other axis, where a and m have changed places.
GDPA_HD int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t ans = 0;
  while (n > 0) {
    if (a >= m) {
      ans += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      ans += n * (b / m);
      b %= m;
    }
    const int64_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return ans;
}

// One sample: n new tokens at positions ctx .. ctx + n - 1 (ctx may be negative).
struct ChunkSample {
  int32_t n, ctx, window, rt, bn_shift;

  GDPA_HD int32_t tiles() const { return (n + rt - 1) / rt; }
  GDPA_HD int32_t tokens(int32_t tile) const {
    const int32_t left = n - tile * rt;
    return left < rt ? left : rt;
  }
  // positions that some row of the tile sees: [lo, hi); hi <= lo when there is none
  GDPA_HD int32_t lo(int32_t tile) const {
    const int64_t p = (int64_t)ctx + (int64_t)tile * rt - window + 1;
    return p > 0 ? (int32_t)p : 0;
  }
  GDPA_HD int32_t hi(int32_t tile) const { return ctx + tile * rt + tokens(tile); }
  GDPA_HD int32_t first_block(int32_t tile) const { return lo(tile) >> bn_shift; }
  // key blocks of the tile; a tile that sees nothing counts as one block, so
  // that a worker visits it and writes its empty rows
  GDPA_HD int32_t blocks(int32_t tile) const {
    const int32_t h = hi(tile);
    return h <= 0 ? 1 : ((h - 1) >> bn_shift) - first_block(tile) + 1;
  }
  // sum of blocks(u) over u < tile
  GDPA_HD int64_t blocks_before(int32_t tile) const {
    if (tile <= 4) {
      int64_t s = 0;
      for (int32_t u = 0; u < tile; ++u) s += blocks(u);
      return s;
    }
    const int32_t whole = n / rt;                        // tiles with all rt tokens
    const int32_t f = tile < whole ? tile : whole;
    int32_t neg = 0;                                     // tiles that lie before position 0
    if (ctx < 0) {
      neg = -ctx / rt;
      if (neg > f) neg = f;
    }
    int64_t s = neg;
    // last blocks: floor((ctx + (u + 1) rt - 1) / bn)
    const int64_t bn = (int64_t)1 << bn_shift;
    s += floor_sum(f - neg, bn, rt, (int64_t)ctx + (int64_t)(neg + 1) * rt - 1) + (f - neg);
    // first blocks: floor(max(0, ctx + u rt - window + 1) / bn)
    const int64_t v = (int64_t)window - 1 - ctx;
    int64_t u0 = v <= 0 ? 0 : (v + rt - 1) / rt;
    if (u0 < neg) u0 = neg;
    if (u0 < f) s -= floor_sum(f - u0, bn, rt, (int64_t)ctx + u0 * rt - window + 1);
    return tile > f ? s + blocks(f) : s;
  }
};

// First block of worker w's part of a line of `total` blocks.  The longer parts come
// first, so that of a line shorter than the workers the empty parts are the last ones and an
// item's pieces lie in neighbouring workers.
GDPA_HD int64_t part_start(int64_t total, int32_t workers, int32_t w) {
  const int64_t rest = total % workers;
  return total / workers * w + (w < rest ? w : rest);
}

// Place of block x (0 <= x < heads * per_head) of a sample's line.
struct ChunkPlace {
  int32_t head, tile, block;
};
GDPA_HD ChunkPlace place_of(const ChunkSample& s, int64_t x) {
  const int32_t tiles = s.tiles();
  const int64_t per = s.blocks_before(tiles);
  ChunkPlace p;
  p.head = (int32_t)(x / per);
  x -= p.head * per;
  int32_t lo = 0, hi = tiles - 1;                         // largest tile with blocks_before <= x
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (s.blocks_before(mid) <= x) lo = mid; else hi = mid - 1;
  }
  p.tile = lo;
  p.block = (int32_t)(x - s.blocks_before(lo));
  return p;
}

}  // namespace gdpa
