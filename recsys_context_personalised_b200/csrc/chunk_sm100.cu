// Attention of many new tokens per sample over a paged key/value cache: the tcgen05 kernel.
//
//   O_i = sum_p softmax_p(scale q_i . k_p) v_p,   p in (pos_i - window, pos_i]
//
// Bound: the tensor core and the exp2 unit.  Per 128 x 128 block of logits a tile needs
// 4 * 128 * 128 * dh tensor FLOPs (1,024 cycles at dh = 128) and 128 * 128 exp2 (1,024
// cycles of the MUFU unit), so a CTA keeps two tiles in flight: while one tile's softmax
// runs, the tensor core works for the other.
//
// An item is a pair of consecutive row tiles A and B of one (sample, kv head): up to
// 128 rows each, rt1 tokens with all the query heads of the kv head, so that one load
// of a key block serves every row that sees it.  The items' 128-position blocks form
// one line, cut into equal parts, one per CTA (chunk_plan.cuh); an item cut by a
// part's border leaves unnormalised pieces that launch_chunk_join joins.
//
// CTA = 12 warps, one per SM:
//   warp 0      TMA producer: Q of a visit (a run of one item's blocks), K and V page by page
//   warp 1      MMA issuer: per block PV_A(j), S_A(j+1), PV_B(j), S_B(j+1)
//   warp 2      TMEM allocator; zeroes the V rows of an item's first and last block
//               that no row of the item sees (0 * NaN would reach O through the product)
//   warps 4-7   softmax of tile A, warps 8-11 of tile B (thread = row = TMEM lane)
//
// TMEM columns: S_A [0,128), S_B [128,256), O_A [256, 256+dh), O_B [256+dh, 256+2dh).  P_X (packed
// bf16) aliases the first 64 columns of S_X, so S_X(j+1) is issued behind PV_X(j).  P goes out in two
// halves of 64 keys; the product of the first runs while the second is computed.
//
// Softmax: online, the running offset kept while a block's maximum stays within 2^8 of it (a published device of
// attention kernels: softmax does not depend on the offset, and 2^8 is far from overflow).  P is rounded to
// bf16, the precision of the MMA's operand; its sum l is taken before that.
//
// The code is kept short and its rare parts out of line: a launch fetches it cold, and the warps
// waited for instructions most of the time with separate masked and unmasked paths
// (48 sessions of up to 700 events in a 256-event window 0.28 ms, in this form 0.14 ms, and 0.12 ms with the masks
// by bit tests).
#include <limits.h>
#include <math.h>

#include "chunk_internal.cuh"

namespace gdpa {
namespace {

using namespace sm100;

constexpr int kThreadsT = 384;
constexpr int kBNT = 128, kBNTShift = 7;

// A run of one item's blocks, [u0, u1) of the context's 128-position blocks.
struct __align__(16) Visit {
  int32_t u0, u1;
  int32_t b0[2], b1[2];      // blocks of it that tile A / B sees
  int32_t pos0, token0;      // position and global index of the first token
  int32_t tok[2];            // tokens of tile A / B
  int32_t kvh, flags;
};
enum { kBegins = 1, kEnds = 2 };   // the item's first / last block is among them

template <int DH>
struct CfgT {
  static constexpr int CH = DH < 64 ? DH : 64;          // elements per swizzled row
  static constexpr int NCH = DH / CH;
  static constexpr uint32_t ROWB = CH * 2;
  static constexpr uint32_t CHUNKB = 128 * ROWB;        // one [128 x CH] chunk
  static constexpr uint32_t TILEB = NCH * CHUNKB;
  static constexpr uint32_t SW = DH < 64 ? kSw64 : kSw128;
  static constexpr uint32_t ATOM = 8 * ROWB;
  static constexpr int QST = DH == 128 ? 1 : 2;         // Q stages (a stage = tiles A and B)
  static constexpr int NS = DH == 32 ? 16 : DH == 64 ? 10 : 5;   // K/V ring slots
  static constexpr int NV = 8;                          // barriers of V blocks that pass warp 2
  static_assert((NS + 1) / 2 <= NV, "as many as V blocks in flight");
  static constexpr uint32_t COL_S = 0, COL_O = 256;
  static constexpr int B_QFULL = 0, B_QEMPTY = 2, B_SFULL = 4, B_PFULL = 6, B_OFULL = 10, B_OEMPTY = 12,
                       B_DRAIN = 14, B_VRAW = 15, B_KVFULL = B_VRAW + NV, B_KVEMPTY = B_KVFULL + NS,
                       NBAR = B_KVEMPTY + NS;
  static constexpr uint32_t OFF_Q = 0, OFF_KV = QST * 2 * TILEB, OFF_CTL = OFF_KV + NS * TILEB;
  static constexpr uint32_t CTL_TMEM = 8 * NBAR, CTL_ABORT = CTL_TMEM + 4,
                            CTL_VISIT = (CTL_ABORT + 4 + 15) / 16 * 16,
                            CTL_BYTES = CTL_VISIT + QST * sizeof(Visit);
  static constexpr uint32_t USED = 1024 + OFF_CTL + CTL_BYTES;
  // at least 120 KB so that two CTAs never share an SM (each allocates all 512 TMEM columns)
  static constexpr uint32_t SMEM = USED > 120u * 1024u ? USED : 120u * 1024u;
  static_assert(SMEM + 512 <= 232448u, "shared memory of a CTA, the static part with it");
};

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// The products and commits of a converged warp, issued by the elected lane under a predicate (not on
// a branch of its own, so that the operands stay in uniform registers).
__device__ __forceinline__ void mma_ss_if(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 l, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n\t}" ::"r"(on), "r"(d), "l"(a),
      "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, l;\n\tsetp.ne.b32 l, %0, 0;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "@l tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n\t}" ::"r"(on), "r"(d), "r"(a),
      "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred l;\n\tsetp.ne.b32 l, %0, 0;\n\t"
      "@l tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(on),
      "r"(bar)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int DH>
__global__ void __launch_bounds__(kThreadsT, 1)
chunk_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const ChunkArgs a) {
  using C = CfgT<DH>;
  constexpr uint32_t IDESC_S = idesc_bf16(128, 128, 0, 0);
  constexpr uint32_t IDESC_O = idesc_bf16(128, DH, 0, 1);
  extern __shared__ uint8_t smem_raw[];
  __shared__ ChunkStart start;
  __shared__ int64_t scan[33];
  __shared__ int bad_page;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + C::OFF_Q, sKV = base + C::OFF_KV;
  uint8_t* ctl = gbase + C::OFF_CTL;
  const uint32_t bar0 = smem_u32(ctl);
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctl + C::CTL_TMEM);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctl + C::CTL_ABORT);
  Visit* visits = reinterpret_cast<Visit*>(ctl + C::CTL_VISIT);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::B_QFULL + i), 1);
      mbar_init(bar(C::B_QEMPTY + i), 10);     // the MMA issuer, warp 2 and the 8 softmax warps
      mbar_init(bar(C::B_SFULL + i), 1);
      mbar_init(bar(C::B_PFULL + i), 4);
      mbar_init(bar(C::B_PFULL + 2 + i), 4);
      mbar_init(bar(C::B_OFULL + i), 1);
      mbar_init(bar(C::B_OEMPTY + i), 4);
    }
    mbar_init(bar(C::B_DRAIN), 1);
    for (int i = 0; i < C::NV; ++i) mbar_init(bar(C::B_VRAW + i), 1);
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(bar(C::B_KVFULL + i), 1);
      mbar_init(bar(C::B_KVEMPTY + i), 1);
    }
    *abort_flag = 0;
    bad_page = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 2) a.piece[2 * worker + threadIdx.x].tokens = 0;
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  find_start(a, worker, &start, scan);            // (synchronises the block)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const int64_t count = start.count;              // blocks of this worker

  // The visit in stage vn % QST, in registers.
  auto open_visit = [&](uint32_t vn, Visit& v) -> bool {
    const uint32_t qs = vn % C::QST;
    if (!mbar_wait(bar(C::B_QFULL + qs), (vn / C::QST) & 1u, abort_flag, kChunkTimeoutNs)) return false;
    v = visits[qs];
    return true;
  };
  // Does the item see only a part of block j (V rows outside are zeroed)?
  const int window = a.window;
  auto pair_lo = [&](const Visit& v) -> int {
    const int64_t p = (int64_t)v.pos0 - window + 1;
    return p > 0 ? (int)p : 0;
  };
  auto pair_hi = [&](const Visit& v) -> int { return v.pos0 + v.tok[0] + v.tok[1]; };

  if (warp < 4) {
    setmaxnreg_dec<80>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      const int pr = min(kBNT, 1 << a.page_shift);            // rows of a page piece
      const int pieces = kBNT / pr;
      int b = start.b;
      ChunkPlace at = start.at;
      int32_t token0 = 0;
      int bad = 0;
      ChunkSample s = {};
      int64_t left = count;
      if (left > 0) s = load_sample(a, b, token0, bad);
      uint32_t slot = 0, phase = 0, vn = 0, edges = 0;
      bool ok = true;
      while (ok && left > 0) {
        // a visit: the rest of this item, or of this worker's part
        const int nb = s.blocks(at.tile), first = s.first_block(at.tile);
        const int take = (int)min((int64_t)(nb - at.block), left);
        const int lo = s.lo(at.tile), hi = s.hi(at.tile), i0 = at.tile * s.rt;
        const int kvh = at.head;
        const int u0 = first + at.block, u1 = u0 + take;
        const uint32_t qs = vn % C::QST;
        ok = mbar_wait(bar(C::B_QEMPTY + qs), ((vn / C::QST) & 1u) ^ 1u, abort_flag, kChunkTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          Visit v;
          v.u0 = u0;
          v.u1 = u1;
          v.pos0 = s.ctx + i0;
          v.token0 = token0 + i0;
          v.tok[0] = min(a.rt1, s.n - i0);
          v.tok[1] = min(a.rt1, s.n - i0 - v.tok[0]);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int p = v.pos0 + x * a.rt1;                 // the tile's first position
            const int64_t l = (int64_t)p - window + 1;
            const int h = p + v.tok[x];
            const bool some = v.tok[x] > 0 && h > 0;
            v.b0[x] = max(u0, l > 0 ? (int)(l >> kBNTShift) : 0);
            v.b1[x] = some ? min(u1, ((h - 1) >> kBNTShift) + 1) : 0;
            if (v.b1[x] <= v.b0[x]) v.b0[x] = v.b1[x] = 0;
          }
          v.kvh = kvh;
          v.flags = (at.block == 0 ? kBegins : 0) | (at.block + take == nb ? kEnds : 0);
          visits[qs] = v;
          const bool two = v.tok[1] > 0;
          const uint32_t qb = (uint32_t)(a.rt1 * a.group) * DH * 2;
          const uint32_t qaddr = sQ + qs * 2 * C::TILEB;
          mbar_expect_tx(bar(C::B_QFULL + qs), two ? 2 * qb : qb);
#pragma unroll
          for (int c = 0; c < C::NCH; ++c) {
            tma_load_3d(qaddr + c * C::CHUNKB, &tmQ, bar(C::B_QFULL + qs), c * C::CH,
                        kvh * a.group, token0 + i0);
            if (two)
              tma_load_3d(qaddr + C::TILEB + c * C::CHUNKB, &tmQ, bar(C::B_QFULL + qs), c * C::CH,
                          kvh * a.group, token0 + i0 + a.rt1);
          }
        }
        __syncwarp();
        ++vn;
        for (int j = u0; ok && j < u1; ++j) {
          const int key0 = j << kBNTShift;
          int32_t page = -1;
          bool load = false;
          if (lane < pieces) {
            const int64_t p0 = (int64_t)key0 + lane * pr;
            load = p0 < hi && p0 + pr > lo;
            if (load) {
              page = page_of(a.table + (int64_t)b * a.max_pages, a.max_pages, a.num_pages,
                             a.page_shift, p0);
              if (page < 0) {
                load = false;
                bad_page = 1;
              }
            }
          }
          const uint32_t mask = __ballot_sync(0xffffffffu, load);
          const uint32_t bytes = (uint32_t)__popc(mask) * pr * DH * 2;
          const int pc = lane / C::NCH, c = lane - pc * C::NCH;   // one lane per (piece, chunk of dh)
          const int32_t id = __shfl_sync(0xffffffffu, page, pc < pieces ? pc : 0);
          const bool edge = key0 < lo || hi - key0 < kBNT;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = ok && mbar_wait(bar(C::B_KVEMPTY + slot), phase ^ 1u, abort_flag, kChunkTimeoutNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // V blocks with rows to zero land on warp 2's barrier, which passes them on
            const uint32_t full = kv && edge ? bar(C::B_VRAW + edges % C::NV) : bar(C::B_KVFULL + slot);
            if (lane == 0) mbar_expect_tx(full, bytes);
            __syncwarp();
            if (pc < pieces && (mask >> pc & 1u))
              tma_load_4d(sKV + slot * C::TILEB + c * C::CHUNKB + pc * pr * C::ROWB,
                          kv ? &tmV : &tmK, full, c * C::CH,
                          (key0 + pc * pr) & ((1 << a.page_shift) - 1), kvh, id);
            if (kv && edge) ++edges;
            if (++slot == (uint32_t)C::NS) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
        left -= take;
        at.block += take;
        if (at.block == nb) {
          at.block = 0;
          if (++at.tile == s.tiles()) {
            at.tile = 0;
            if (++at.head == a.hk) {
              at.head = 0;
              if (left > 0) {
                do {
                  ++b;
                  s = load_sample(a, b, token0, bad);
                } while (s.n == 0);
              }
            }
          }
        }
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      // Both tiles in one in-order stream, PV_A(j), S_A(j+1), PV_B(j), S_B(j+1).  The whole warp walks the blocks and
      // one elected lane issues under a predicate: values that are the same in the warp (as a
      // broadcast tells the compiler) stay in uniform registers, where the descriptors have to be.
      auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
      const uint32_t tm = (uint32_t)uni((int)tmem);
      const uint32_t leader = elect_one();
      // a negative scale: the products of -Q, and its absolute value in the softmax
      const uint32_t idesc_s = IDESC_S | (a.scale_log2 < 0.f ? 1u << 13 : 0u);
      uint32_t slot = 0, phase = 0, vn = 0, qs = 0, pbit = 0, obit = 0;
      auto wait = [&](int b, uint32_t parity) -> bool {
        const bool w = __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, kChunkTimeoutNs));
        tc_fence_after();
        return w;
      };
      auto take = [&]() -> int {
        if (!wait(C::B_KVFULL + slot, phase)) return -1;
        const int r = (int)slot;
        if (++slot == (uint32_t)C::NS) {
          slot = 0;
          phase ^= 1u;
        }
        return r;
      };
      const int64_t steps = ((int64_t)uni((int)(count >> 32)) << 32) | (uint32_t)uni((int)count);
      // block j of the products with P, block nj (of a visit that may be the next one) of S
      int j = -1, nj = -1, u1 = 0, cb0[2] = {0, 0}, cb1[2] = {0, 0}, nb0[2] = {0, 0}, nb1[2] = {0, 0};
      bool ok = true;
      for (int64_t it = 0; ok && it <= steps && steps > 0; ++it) {
        int v = -1, k = -1;
        if (it > 0) ok = (v = take()) >= 0;
        if (ok && it < steps) {
          if (++nj >= u1) {                                   // the next visit
            qs = vn % C::QST;
            ok = wait(C::B_QFULL + qs, (vn / C::QST) & 1u);
            ++vn;
            const Visit& r = visits[qs];
            nj = uni(r.u0);
            u1 = uni(r.u1);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              nb0[x] = uni(r.b0[x]);
              nb1[x] = uni(r.b1[x]);
            }
          }
          ok = ok && (k = take()) >= 0;
        }
        if (!ok) break;
#pragma unroll 1
        for (int x = 0; ok && x < 2; ++x) {
          const int c0 = x ? cb0[1] : cb0[0], c1 = x ? cb1[1] : cb1[0];
          const int n0 = x ? nb0[1] : nb0[0], n1 = x ? nb1[1] : nb1[0];
          if (v >= 0 && j >= c0 && j < c1) {                  // O_X += P_X(j) V(j)
            const bool first = j == c0, last = j == c1 - 1;
            const uint64_t v0 = smem_desc(sKV + v * C::TILEB, C::CHUNKB, C::ATOM, C::SW);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = wait(C::B_PFULL + 2 * x + h, (pbit >> x) & 1u);
              if (ok && h == 0 && first) ok = wait(C::B_OEMPTY + x, ((obit >> x) & 1u) ^ 1u);
              if (!ok) break;
#pragma unroll
              for (int q = 4 * h; q < 4 * h + 4; ++q)
                mma_ts_if(leader, tm + C::COL_O + DH * x, tm + C::COL_S + 128 * x + q * 8,
                          desc_advance(v0, q * 2 * C::ATOM), IDESC_O, q > 0 || !first ? 1u : 0u);
            }
            if (!ok) break;
            pbit ^= 1u << x;
            if (last) {
              commit_if(leader, bar(C::B_OFULL + x));
              obit ^= 1u << x;
            }
          }
          if (k >= 0 && nj >= n0 && nj < n1) {                // S_X(nj)
            const uint64_t a0 = smem_desc(sQ + (qs * 2 + x) * C::TILEB, 16, C::ATOM, C::SW);
            const uint64_t b0 = smem_desc(sKV + k * C::TILEB, 16, C::ATOM, C::SW);
#pragma unroll
            for (int q = 0; q < DH / 16; ++q) {
              const uint32_t off = (q / (C::CH / 16)) * C::CHUNKB + (q % (C::CH / 16)) * 32;
              mma_ss_if(leader, tm + C::COL_S + 128 * x, desc_advance(a0, off), desc_advance(b0, off),
                        idesc_s, q > 0 ? 1u : 0u);
            }
            commit_if(leader, bar(C::B_SFULL + x));
          }
        }
        if (!ok) break;
        if (v >= 0) commit_if(leader, bar(C::B_KVEMPTY + v));
        if (k >= 0) commit_if(leader, bar(C::B_KVEMPTY + k));
        if (k >= 0 && nj == u1 - 1) commit_if(leader, bar(C::B_QEMPTY + qs));
        __syncwarp();
        j = nj;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          cb0[x] = nb0[x];
          cb1[x] = nb1[x];
        }
      }
    } else if (warp == 2) {
      // ------------------------------------- rows of V that the item does not see
      uint32_t pos = 0, edges = 0;                            // pos: blocks so far
      Visit v;
      bool ok = true;
      int64_t left = count;
      for (uint32_t vn = 0; ok && left > 0; ++vn) {
        ok = __all_sync(0xffffffffu, open_visit(vn, v));
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_QEMPTY + vn % C::QST));
        const int lo = pair_lo(v), hi = pair_hi(v);
        for (int j = v.u0; j < v.u1; ++j, ++pos) {
          const int key0 = j << kBNTShift;
          if (!(key0 < lo || hi - key0 < kBNT)) continue;
          const uint32_t slot = (2 * pos + 1) % C::NS;
          ok = mbar_wait(bar(C::B_VRAW + edges % C::NV), (edges / C::NV) & 1u, abort_flag, kChunkTimeoutNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++edges;
          constexpr int UPR = C::ROWB / 16;                   // 16-byte units of a row of a chunk
          for (int e = lane; e < kBNT * UPR; e += 32) {
            const int key = key0 + e / UPR;
            if (key >= lo && key < hi) continue;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               sKV + slot * C::TILEB + c * C::CHUNKB + e * 16),
                           "r"(0)
                           : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_KVFULL + slot));
        }
        left -= v.u1 - v.u0;
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    setmaxnreg_inc<208>();
    const int x = (warp - 4) >> 2;                // tile: 0 = A, 1 = B
    const int quad = warp & 3;                    // TMEM lane quadrant
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t my_s = tmem + lane_off + C::COL_S + 128 * x;
    const uint32_t my_o = tmem + lane_off + C::COL_O + DH * x;
    const int tk = row / a.group, hd = row - tk * a.group;
    // |scale| (S holds the products of -Q for a negative one); of a zero scale so little is kept that
    // every logit is 0 and a masked one still -inf
    const float c2 = fmaxf(fabsf(a.scale_log2), 1e-30f);
    const float2 c2v = make_float2(c2, c2);
    uint32_t sc = 0, oc = 0;
    int64_t left = count;
    bool ok = true;
    Visit v;
    for (uint32_t vn = 0; ok && left > 0; ++vn) {
      ok = __all_sync(0xffffffffu, open_visit(vn, v));
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::B_QEMPTY + vn % C::QST));
      left -= v.u1 - v.u0;
      const int tokens = x ? v.tok[1] : v.tok[0];
      if (tokens <= 0) continue;
      const int j0 = x ? v.b0[1] : v.b0[0], j1 = x ? v.b1[1] : v.b1[0];
      const int head0 = v.kvh * a.group;
      const bool store = tk < tokens;
      const bool dead = quad * 32 >= tokens * a.group;       // no row of this warp is stored
      // the row sees the positions [low, pos]; the whole warp sees [wlow, wpos]
      const int pos = v.pos0 + x * a.rt1 + tk;
      const int low = (int)max((int64_t)pos - window + 1, (int64_t)0);
      const int wpos = __reduce_min_sync(0xffffffffu, store ? pos : INT_MAX);
      const int wlow = __reduce_max_sync(0xffffffffu, store ? low : 0);
      float m_run = 0.f, l_run = 0.f;
      for (int j = j0; j < j1; ++j, ++sc) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_SFULL + x), sc & 1u, abort_flag, kChunkTimeoutNs));
        if (!ok) break;
        tc_fence_after();
        // (PV_x(j-1), which reads P_x and writes O_x, is done: S_x(j) came behind it)
        if (dead) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(C::B_PFULL + 2 * x));
            mbar_arrive(bar(C::B_PFULL + 2 * x + 1));
          }
          continue;
        }
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld_x32(my_s + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
        tmem_wait_ld();
        const int key0 = j << kBNTShift;
        if (__builtin_expect(key0 < wlow || wpos - key0 < kBNT - 1, 0)) {   // positions outside [low, pos]
          const int clo = low - key0, chi = pos - key0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            // bits lo .. hi of a word (tests of constant bits cost half of two comparisons each)
            const int lo = clo - 32 * w, hi = chi - 32 * w;
            uint32_t m = lo <= 0 ? 0xffffffffu : lo > 31 ? 0u : 0xffffffffu << lo;
            m &= hi >= 31 ? 0xffffffffu : hi < 0 ? 0u : 0xffffffffu >> (31 - hi);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              s[32 * w + i] = (m >> i) & 1u ? s[32 * w + i] : __float_as_uint(-INFINITY);
          }
        }
        float e4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) e4[u] = __uint_as_float(s[u]);
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            e4[u] = max3(e4[u], __uint_as_float(s[i + 2 * u]), __uint_as_float(s[i + 2 * u + 1]));
#pragma unroll
        for (int u = 0; u < 4; ++u) e4[u] = fmaxf(e4[u], __uint_as_float(s[124 + u]));
        const float top = max3(fmaxf(e4[0], e4[1]), e4[2], e4[3]) * c2;
        // a first visible key (l = 0) sets the offset, a maximum beyond 2^8 of it moves it
        const bool move = l_run == 0.f ? top != -INFINITY : top > m_run + 8.f;
        if (__builtin_expect(__any_sync(0xffffffffu, move), 0)) {
          const float alpha = move ? ex2_approx(m_run - top) : 1.f;
          if (move) m_run = top;
          if (__any_sync(0xffffffffu, move && l_run != 0.f)) {
            const float f = l_run != 0.f ? alpha : 0.f;
            l_run *= f;
#pragma unroll 1
            for (int c = 0; c < DH; c += 16) {
              uint32_t ov[16];
              tmem_ld_x16(my_o + c, ov);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f);
              tmem_st_x16(my_o + c, ov);
            }
          }
        }
        const float2 negm = make_float2(-m_run, -m_run);
        float2 acc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[u] = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[64 * h + 2 * i]),
                                                    __uint_as_float(s[64 * h + 2 * i + 1])), c2v, negm);
            const float2 e = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            acc[i & 3] = __fadd2_rn(acc[i & 3], e);
            pk[i] = pack_bf16x2(e.x, e.y);
          }
          tmem_st_x32(my_s + 32 * h, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_PFULL + 2 * x + h));
        }
        const float2 r = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        l_run += r.x + r.y;
        if (!ok) break;
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      const bool has_o = j1 > j0;
      if (has_o) {
        const bool w = mbar_wait(bar(C::B_OFULL + x), oc & 1u, abort_flag, kChunkTimeoutNs);
        ok = __all_sync(0xffffffffu, w);
        if (!ok) break;
        ++oc;
        tc_fence_after();
      }
      const bool whole = (v.flags & kBegins) && (v.flags & kEnds);
      const int64_t at = 2 * worker + ((v.flags & kBegins) ? 1 : 0);
      if (!whole && x == 0 && threadIdx.x == 128) {
        ChunkPiece pc = {};
        pc.token0 = v.token0;
        pc.tokens = v.tok[0] + v.tok[1];
        pc.head0 = head0;
        pc.ends = (v.flags & kEnds) ? 1 : 0;
        a.piece[at] = pc;
      }
      auto free_o = [&]() {                      // the O accumulator is read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_OEMPTY + x));
      };
      if (dead) {
        if (has_o) free_o();
        continue;
      }
      // a whole row of O is normalised and stored by its thread, 32 bytes (one sector) at a time;
      // a row of a piece goes to the workspace as it is
      const int pr = x * 128 + row;
      const int64_t t = v.token0 + x * a.rt1 + tk;
      const float inv = l_run > 0.f || l_run != l_run ? 1.f / l_run : 0.f;
      if (store && whole && a.lse)
        a.lse[(int64_t)(head0 + hd) * a.T + t] =
            l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
      if (store && !whole) a.ml[at * a.rows + pr] = make_float2(m_run, l_run);
      __nv_bfloat16* o = a.o + (t * a.hq + head0 + hd) * DH;
      float* po = a.po + at * a.rows * DH + pr * 4;
#pragma unroll 1
      for (int c = 0; c < DH; c += 16) {
        uint32_t ov[16];
        if (has_o) {
          tmem_ld_x16(my_o + c, ov);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) ov[i] = 0u;
        }
        if (store && whole) {
          uint32_t p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            p[i] = pack_bf16x2(__uint_as_float(ov[2 * i]) * inv, __uint_as_float(ov[2 * i + 1]) * inv);
          reinterpret_cast<uint4*>(o + c)[0] = make_uint4(p[0], p[1], p[2], p[3]);
          reinterpret_cast<uint4*>(o + c)[1] = make_uint4(p[4], p[5], p[6], p[7]);
        } else if (store) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(po + (int64_t)(c / 4 + i) * a.rows * 4) =
                make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
        }
        __syncwarp();
      }
      if (has_o) free_o();
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  __syncthreads();
  if (*abort_flag) {
    volatile int never = 0;
    if (warp == 1 && elect_one()) {
      mma_commit(bar(C::B_DRAIN));                       // all MMAs issued so far
      mbar_wait(bar(C::B_DRAIN), 0, &never, kChunkTimeoutNs);
    }
    if (warp == 0 && lane == 0) {                         // let copies in flight land
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 200000ull) {
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0)
    a.status[worker] = *abort_flag ? GDPA_ERR_TIMEOUT
                                   : start.bad || bad_page ? GDPA_ERR_INVALID_ARG : GDPA_OK;
}

template <int DH>
cudaError_t launch_tiles(const ChunkArgs& a, const gdpa_cache_t& c, cudaStream_t st) {
  using C = CfgT<DH>;
  CUtensorMap mq, mk, mv;
  const CUtensorMapSwizzle sw = DH < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!chunk_maps(a, c, DH, C::CH, kBNT, sw, &mq, &mk, &mv)) return cudaErrorInvalidValue;
  auto kern = chunk_tiles_kernel<DH>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, (int)C::SMEM, done);
  if (e != cudaSuccess) return e;
  KernelScope ks_("gdpa_chunk_tiles", st);
  kern<<<a.workers, kThreadsT, C::SMEM, st>>>(mq, mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_tiles(const ChunkArgs& a, const gdpa_cache_t& c, cudaStream_t st) {
  return c.dh == 32 ? launch_tiles<32>(a, c, st)
                    : c.dh == 64 ? launch_tiles<64>(a, c, st) : launch_tiles<128>(a, c, st);
}

}  // namespace gdpa
