// Shared by the kernels for attention of new tokens over a paged cache
// (chunk.cu: few rows per sample and the joining of pieces; chunk_sm100.cu: many rows).
#pragma once

#include <cudaTypedefs.h>

#include "chunk_plan.cuh"
#include "layer_launch.cuh"
#include "sm100.cuh"

namespace gdpa {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

constexpr uint64_t kChunkTimeoutNs = 2000000000ull;   // 2 s per wait; a healthy wait is microseconds

// log2 of the positions of a block of the kernel for few rows: 64 at dh = 128, 256 at dh = 32 (16 KB of K)
constexpr int chunk_rows_shift(int dh) { return dh == 128 ? 6 : dh == 64 ? 7 : 8; }

// A piece of an item whose blocks are shared with other workers (or none:
// tokens = 0).  Its rows' (max in log2 units, sum) and unnormalised O are at the
// same index of the workspace's ml and po arrays.
struct __align__(16) ChunkPiece {
  // row r of a tile: token r / group of the tile, head head0 + r % group
  int32_t token0, tokens, head0;
  int32_t ends;                           // this piece holds the item's last block
};

struct ChunkArgs {
  const int32_t* offsets;
  const int32_t* kv_len;
  const int32_t* table;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                // [hq, T] or NULL
  int32_t* status;           // [workers]
  ChunkPiece* piece;         // [2 * workers]: a part's first (0) and last (1) unfinished item
  float2* ml;                // [2 * workers, rows]
  float* po;                 // [2 * workers, dh / 4, rows, 4]
  int64_t T;
  int32_t B, hq, hk, group;  // group = hq / hk
  int32_t max_n, window, bn_shift;
  int32_t rt, rt1, rows, tile_rows;           // an item: rt tokens in tiles of rt1 tokens, rows in tiles of tile_rows
  int32_t num_pages, max_pages, page_shift;
  int32_t workers;
  float scale_log2;          // scale * log2(e)
};

__device__ __forceinline__ ChunkSample load_sample(const ChunkArgs& a, int b, int32_t& token0,
                                                   int& bad) {
  const int32_t lo = __ldg(a.offsets + b), hi = __ldg(a.offsets + b + 1);
  int32_t kv = __ldg(a.kv_len + b);
  ChunkSample s;
  s.window = a.window;
  s.rt = a.rt;
  s.bn_shift = a.bn_shift;
  token0 = lo;
  if (lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_n) {
    bad = 1;
    s.n = 0;
    s.ctx = 0;
    return s;
  }
  const int64_t room = (int64_t)a.max_pages << a.page_shift;
  if (kv > room) {
    bad = 1;
    kv = (int32_t)room;
  }
  if (kv < 0) {
    bad = 1;
    kv = 0;
  }
  s.n = hi - lo;
  s.ctx = kv - s.n;
  return s;
}

// Where a worker's part of the line begins, found by the whole block (blockDim.x a multiple
// of 32, at most 1024): every thread sums the blocks of a run of samples, one
// scan over the threads places the run that holds the part's first block, and
// that run's thread walks its samples.
struct ChunkStart {
  int64_t count;             // blocks of this worker
  int32_t b;                 // its first block's sample, and the place within it
  ChunkPlace at;
  int32_t bad;
};
__device__ __forceinline__ void find_start(const ChunkArgs& a, int worker, ChunkStart* out,
                                           int64_t* scan /* 33 shared words */) {
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int run = (a.B + nt - 1) / nt;
  const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
  int64_t mine = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    int32_t t0;
    const ChunkSample s = load_sample(a, b, t0, bad);
    if (s.n > 0) mine += s.blocks_before(s.tiles()) * a.hk;
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (tid == 0) {
    out->bad = 0;
    out->count = 0;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  if (bad) out->bad = 1;
  int64_t before = 0, total = 0;
  for (int w = 0; w < nt >> 5; ++w) {
    const int64_t v = scan[w];
    if (w < warp) before += v;
    total += v;
  }
  const int64_t x0 = part_start(total, a.workers, worker), x1 = part_start(total, a.workers, worker + 1);
  int64_t lo = before + upto - mine;
  if (x1 > x0 && x0 >= lo && x0 < lo + mine) {
    for (int b = b0; b < b1; ++b) {
      int32_t t0;
      const ChunkSample s = load_sample(a, b, t0, bad);
      if (s.n == 0) continue;
      const int64_t w = s.blocks_before(s.tiles()) * a.hk;
      if (x0 < lo + w) {
        out->count = x1 - x0;
        out->b = b;
        out->at = place_of(s, x0 - lo);
        break;
      }
      lo += w;
    }
  }
  __syncthreads();
}

// The tensor maps of a call: Q as boxes of rt1 tokens x group heads, K and V
// as boxes of the rows of a page that lie in one block of `bn` positions; `ch` elements wide.
bool chunk_maps(const ChunkArgs& a, const gdpa_cache_t& c, int dh, int ch, int bn,
                CUtensorMapSwizzle sw, CUtensorMap* q, CUtensorMap* k, CUtensorMap* v);

// Many rows per sample (chunk_sm100.cu), one worker per SM.
cudaError_t launch_chunk_tiles(const ChunkArgs& a, const gdpa_cache_t& c, cudaStream_t st);

// Joins the pieces of the items that a part's border cuts, and the workers'
// status words into the workspace's.
cudaError_t launch_chunk_join(const ChunkArgs& a, int dh, WsHeader* ws, cudaStream_t st);

}  // namespace gdpa
