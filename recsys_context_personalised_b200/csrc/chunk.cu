// Attention of a few new tokens per sample over a paged key/value cache (the
// serving form of the sliding-window attention), the join of its pieces, and
// the entry points.
//
//   O_i = sum_p softmax_p(scale q_i . k_p) v_p,   p in (pos_i - window, pos_i]
//
// Bound: memory, the visible cache rows once.  One row of queries per sample and
// head makes 2 products per loaded element, so the query heads that share a kv
// head (and the sample's new tokens) form the 16 (or 32) rows of one tile and
// every loaded key serves them all.  The work is cut into equal runs of
// blocks (chunk_plan.cuh), two workers per SM.
//
// A worker is a CTA of 5 warps: warp 4 loads (Q, and K and V blocks of 16 KB through a
// ring of TMA slots, one copy per page piece), warps 0-3 each take 16 of every
// 64 positions: S = Q K^T (mma.sync m16n8k16, which at these row counts is
// far from bounding), an online softmax with running max and sum in fp32, and
// O += P V with P rounded to bf16 (the precision of the output).
// The warps' (max, sum, O) meet in shared memory at the end of the item, where each thread joins and
// stores a part of the rows.
#include <math.h>
#include <stdio.h>

#include "chunk_internal.cuh"

namespace gdpa {
namespace {

using namespace sm100;

constexpr int kWarps = 4, kSub = 16 * kWarps;      // consumer warps, and the positions that they take at a time
constexpr int kThreadsC = (kWarps + 1) * 32;

// What the loader tells the consumers about one block.
struct BlockMeta {
  int32_t key0;              // position of the block's first row
  int32_t lo, hi;            // positions that some row of the tile sees
  int32_t pos0, tokens;      // first token's position, tokens of the tile
  int32_t token0;            // global index of the first token
  int32_t kvh;               // kv head
  int32_t flags;             // kFirst | kLast of this worker's visit of the item; kBegins | kEnds of the item
};
enum { kFirst = 1, kLast = 2, kBegins = 4, kEnds = 8 };

template <int DH, int MT>
struct Cfg {
  static constexpr int R = 16 * MT;                       // rows of a tile
  static constexpr int kBN = 8192 / DH, kBNShift = chunk_rows_shift(DH);   // positions of a block (16 KB of K)
  static_assert(1 << kBNShift == kBN, "positions of a block");
  static constexpr int CH = DH < 64 ? DH : 64;            // elements per swizzled row
  static constexpr int NCH = DH / CH;
  static constexpr uint32_t ROWB = CH * 2;
  static constexpr uint32_t SLOTB = kBN * DH * 2;         // one K or V block
  static constexpr uint32_t CHUNKB = kBN * ROWB;
  static constexpr uint32_t QB = R * DH * 2, QCHUNKB = R * ROWB;
  static constexpr int QST = 2;                           // Q stages
  static constexpr int NS = DH == 128 ? 4 : DH == 64 ? (MT == 1 ? 5 : 4) : MT == 1 ? 6 : 5;   // K/V ring slots
  static constexpr int NM = 32;                           // meta ring (blocks in flight < NM)
  // merge: every warp's O (fp32) and (max, sum)
  static constexpr uint32_t OFF_Q = 0, OFF_KV = (QST * QB + 1023) / 1024 * 1024,
                            OFF_MRG = OFF_KV + NS * SLOTB, MRGB = kWarps * R * (DH + 4) * 4,
                            OFF_ML = OFF_MRG + MRGB, OFF_META = OFF_ML + kWarps * R * 8,
                            OFF_CTL = OFF_META + NM * sizeof(BlockMeta);
  static constexpr int B_KVFULL = 0, B_KVEMPTY = NS, B_QFULL = 2 * NS, B_QEMPTY = 2 * NS + QST,
                       B_JOIN = 2 * NS + 2 * QST, B_FREE = B_JOIN + 1, NBAR = B_JOIN + 2;
  static constexpr uint32_t SMEM = 1024 + OFF_CTL + 8 * NBAR + 16;
  static_assert(SMEM <= 113 * 1024, "two workers share an SM");
  static_assert(NS / 2 + 2 < NM, "meta ring");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16-byte unit `u` of row r of a swizzled [rows x CH] chunk
template <int CH>
__device__ __forceinline__ uint32_t unit_addr(uint32_t base, int r, int u) {
  if constexpr (CH == 64) return base + r * 128 + ((u ^ (r & 7)) << 4);
  return base + r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
}

template <int DH, int MT>
__global__ void __launch_bounds__(kThreadsC, 2)
chunk_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const ChunkArgs a) {
  using C = Cfg<DH, MT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ChunkStart start;
  __shared__ int64_t scan[33];
  __shared__ int bad_page;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  BlockMeta* meta = reinterpret_cast<BlockMeta*>(gbase + C::OFF_META);
  const uint32_t bar0 = base + C::OFF_CTL;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::OFF_CTL + 8 * C::NBAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(bar(C::B_KVFULL + i), 1);
      mbar_init(bar(C::B_KVEMPTY + i), kWarps);
    }
    for (int i = 0; i < C::QST; ++i) {
      mbar_init(bar(C::B_QFULL + i), 1);
      mbar_init(bar(C::B_QEMPTY + i), kWarps);
    }
    mbar_init(bar(C::B_JOIN), kWarps);
    mbar_init(bar(C::B_FREE), kWarps);
    *abort_flag = 0;
    bad_page = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 2) a.piece[2 * worker + threadIdx.x].tokens = 0;
  find_start(a, worker, &start, scan);            // (synchronises the block)
  pdl_trigger();
  const int64_t count = start.count;

  if (warp == kWarps) {
    // -------------------------------------------------------------- loader
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    const int pr = min(C::kBN, 1 << a.page_shift);          // rows of a page piece
    const int pieces = C::kBN / pr;
    int b = start.b;
    ChunkPlace at = start.at;
    int32_t token0 = 0;
    int bad = 0;
    ChunkSample s = {};
    int64_t left = count;
    if (left > 0) s = load_sample(a, b, token0, bad);
    uint32_t slot = 0, phase = 0, mslot = 0, qn = 0;
    bool ok = true, fresh = true, begins = false;   // this worker visits the item's first block
    while (ok && left > 0) {
      const int nb = s.blocks(at.tile);
      const int lo = s.lo(at.tile), hi = s.hi(at.tile), kb0 = s.first_block(at.tile);
      const int tokens = s.tokens(at.tile), i0 = at.tile * s.rt;
      if (fresh) {
        begins = at.block == 0;
        // Q of the item: the kv head's `group` heads of `rt` tokens (rows past the item are never stored)
        const uint32_t qs = qn % C::QST, qph = (qn / C::QST) & 1u;
        ok = mbar_wait(bar(C::B_QEMPTY + qs), qph ^ 1u, abort_flag, kChunkTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(bar(C::B_QFULL + qs), (uint32_t)(a.rt * a.group) * DH * 2);
#pragma unroll
          for (int c = 0; c < C::NCH; ++c)
            tma_load_3d(base + C::OFF_Q + qs * C::QB + c * C::QCHUNKB, &tmQ, bar(C::B_QFULL + qs),
                        c * C::CH, at.head * a.group, token0 + i0);
        }
        ++qn;
      }
      const int key0 = (kb0 + at.block) << C::kBNShift;
      // page pieces of this block that hold a visible position: lanes 0 .. pieces - 1
      int32_t page = -1;
      bool load = false;
      if (lane < pieces) {
        const int p0 = key0 + lane * pr;
        load = p0 < hi && p0 + pr > lo;
        if (load) {
          page = page_of(a.table + (int64_t)b * a.max_pages, a.max_pages, a.num_pages, a.page_shift, p0);
          if (page < 0) {
            load = false;
            bad_page = 1;
          }
        }
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, load);
      const uint32_t bytes = (uint32_t)__popc(mask) * pr * DH * 2;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        ok = ok && mbar_wait(bar(C::B_KVEMPTY + slot), phase ^ 1u, abort_flag, kChunkTimeoutNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          if (kv == 0) {
            BlockMeta m;
            m.key0 = key0;
            m.lo = lo;
            m.hi = hi;
            m.pos0 = s.ctx + i0;
            m.tokens = tokens;
            m.token0 = token0 + i0;
            m.kvh = at.head;
            m.flags = (fresh ? kFirst : 0) | (begins ? kBegins : 0) |
                      (at.block == nb - 1 ? kEnds : 0) |
                      (at.block == nb - 1 || left == 1 ? kLast : 0);
            meta[mslot] = m;
          }
          mbar_expect_tx(bar(C::B_KVFULL + slot), bytes);
        }
        __syncwarp();
        // one lane per (piece, chunk of dh)
        const int pc = lane / C::NCH, c = lane - pc * C::NCH;
        const int32_t id = __shfl_sync(0xffffffffu, page, pc < pieces ? pc : 0);
        if (pc < pieces && (mask >> pc & 1u))
          tma_load_4d(base + C::OFF_KV + slot * C::SLOTB + c * C::CHUNKB + pc * pr * C::ROWB,
                      kv ? &tmV : &tmK, bar(C::B_KVFULL + slot), c * C::CH,
                      (key0 + pc * pr) & ((1 << a.page_shift) - 1), at.head, id);
        if (++slot == (uint32_t)C::NS) {
          slot = 0;
          phase ^= 1u;
        }
      }
      if (++mslot == (uint32_t)C::NM) mslot = 0;
      --left;
      fresh = false;
      if (++at.block == nb) {
        at.block = 0;
        fresh = true;
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
  } else {
    // ----------------------------------------------------------- consumers
    const int g8 = lane >> 2, t4 = lane & 3;
    const int mat = lane >> 3, r8 = lane & 7;
    float o[MT][DH / 8][4];
    float mx[MT][2], sum[MT][2];
    int pos[MT][2];
    uint32_t slot = 0, phase = 0, mslot = 0, qn = 0, merges = 0;
    uint32_t sq = 0;
    float* mrg = reinterpret_cast<float*>(gbase + C::OFF_MRG);
    float2* mls = reinterpret_cast<float2*>(gbase + C::OFF_ML);
    bool ok = true;
    auto wait = [&](int b, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, kChunkTimeoutNs));
    };
    auto arrive = [&](int b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    for (int64_t i = 0; i < count; ++i) {
      if (!wait(C::B_KVFULL + slot, phase)) break;
      const BlockMeta m = meta[mslot];
      if (++mslot == (uint32_t)C::NM) mslot = 0;
      if (m.flags & kFirst) {
        const uint32_t qs = qn % C::QST, qph = (qn / C::QST) & 1u;
        if (!wait(C::B_QFULL + qs, qph)) break;
        sq = base + C::OFF_Q + qs * C::QB;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mx[mt][x] = -INFINITY;
            sum[mt][x] = 0.f;
            pos[mt][x] = m.pos0 + (mt * 16 + x * 8 + g8) / a.group;
          }
#pragma unroll
          for (int n = 0; n < DH / 8; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[mt][n][x] = 0.f;
        }
      }
      const uint32_t kslot = slot;
      if (++slot == (uint32_t)C::NS) {
        slot = 0;
        phase ^= 1u;
      }
      const uint32_t sk = base + C::OFF_KV + kslot * C::SLOTB, sv = base + C::OFF_KV + slot * C::SLOTB;
      bool have_v = false;
#pragma unroll 1
      for (int kw = warp * 16; kw < C::kBN; kw += kSub) {   // this warp's next 16 positions
        if (m.key0 + kw >= m.hi || m.key0 + kw + 16 <= m.lo) continue;   // (no row of the tile sees one)
        // S = Q K^T
        float s[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[mt][0][x] = s[mt][1][x] = 0.f;
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          constexpr int PER = C::CH / 16;                   // 16-element steps per chunk
          uint32_t kb[4];
          ldsm4(unit_addr<C::CH>(sk + (k / PER) * C::CHUNKB, kw + (mat >> 1) * 8 + r8,
                                 (k % PER) * 2 + (mat & 1)), kb);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t qa[4];
            ldsm4(unit_addr<C::CH>(sq + (k / PER) * C::QCHUNKB, mt * 16 + (mat & 1) * 8 + r8,
                                   (k % PER) * 2 + (mat >> 1)), qa);
            mma16816(s[mt][0], qa, kb[0], kb[1]);
            mma16816(s[mt][1], qa, kb[2], kb[3]);
          }
        }
        // online softmax; positions outside (pos - window, pos] are masked by selection
        const int kp = m.key0 + kw + t4 * 2;                // + 8 n + j
        uint32_t p[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float big[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int row = x >> 1, key = kp + 8 * n + (x & 1);
              const bool see = key <= pos[mt][row] && (int64_t)key > (int64_t)pos[mt][row] - a.window &&
                               key >= 0;
              s[mt][n][x] = see ? s[mt][n][x] * a.scale_log2 : -INFINITY;
              big[row] = fmaxf(big[row], s[mt][n][x]);
            }
#pragma unroll
          for (int row = 0; row < 2; ++row) {
            big[row] = fmaxf(big[row], __shfl_xor_sync(0xffffffffu, big[row], 1));
            big[row] = fmaxf(big[row], __shfl_xor_sync(0xffffffffu, big[row], 2));
          }
          // a row's offset moves only when its maximum grew by more than 2^8 (a published device of attention kernels:
          // softmax does not depend on the offset, and 2^8 is far from overflow).  Each row decides for itself, and one that stays
          // is scaled by exactly 1: the tile's rows behind the item hold what was there before (or other
          // samples' queries) and must not change a bit of the others
          bool move[2];
#pragma unroll
          for (int row = 0; row < 2; ++row) move[row] = big[row] > mx[mt][row] + 8.f;
          if (__any_sync(0xffffffffu, move[0] || move[1])) {
            float f[2];
#pragma unroll
            for (int row = 0; row < 2; ++row) {
              f[row] = move[row] ? ex2_approx(mx[mt][row] - big[row]) : 1.f;
              if (move[row]) mx[mt][row] = big[row];
              sum[mt][row] *= f[row];
            }
#pragma unroll
            for (int n = 0; n < DH / 8; ++n) {
              o[mt][n][0] *= f[0];
              o[mt][n][1] *= f[0];
              o[mt][n][2] *= f[1];
              o[mt][n][3] *= f[1];
            }
          }
          float e[2][4];
#pragma unroll
          for (int row = 0; row < 2; ++row) {
            const float off = mx[mt][row] == -INFINITY ? 0.f : mx[mt][row];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                e[n][row * 2 + j] = ex2_approx(s[mt][n][row * 2 + j] - off);
                sum[mt][row] += e[n][row * 2 + j];
              }
          }
          p[mt][0] = pack_bf16x2(e[0][0], e[0][1]);
          p[mt][1] = pack_bf16x2(e[0][2], e[0][3]);
          p[mt][2] = pack_bf16x2(e[1][0], e[1][1]);
          p[mt][3] = pack_bf16x2(e[1][2], e[1][3]);
        }
        // O += P V
        if (!have_v) {
          ok = wait(C::B_KVFULL + slot, phase);
          if (!ok) break;
          have_v = true;
        }
        // V rows that no row of the tile sees may hold anything (NaN): they enter as zeros
        const bool edge = m.key0 + kw < m.lo || m.key0 + kw + 16 > m.hi;
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (edge)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k0 = kp + 8 * h;
            keep[h] = (k0 >= m.lo && k0 < m.hi ? 0x0000ffffu : 0u) |
                      (k0 + 1 >= m.lo && k0 + 1 < m.hi ? 0xffff0000u : 0u);
          }
#pragma unroll
        for (int n = 0; n < DH / 16; ++n) {
          constexpr int PER = C::CH / 16;
          uint32_t vb[4];
          ldsm4t(unit_addr<C::CH>(sv + (n / PER) * C::CHUNKB, kw + (mat & 1) * 8 + r8,
                                  (n % PER) * 2 + (mat >> 1)), vb);
          if (edge) {
            vb[0] &= keep[0];
            vb[1] &= keep[1];
            vb[2] &= keep[0];
            vb[3] &= keep[1];
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816(o[mt][2 * n], p[mt], vb[0], vb[1]);
            mma16816(o[mt][2 * n + 1], p[mt], vb[2], vb[3]);
          }
        }
      }
      // (a slot is given back only once its copy has landed, read or not)
      if (ok && !have_v) ok = wait(C::B_KVFULL + slot, phase);
      if (!ok) break;
      arrive(C::B_KVEMPTY + kslot);
      arrive(C::B_KVEMPTY + slot);
      if (++slot == (uint32_t)C::NS) {
        slot = 0;
        phase ^= 1u;
      }
      if (!(m.flags & kLast)) continue;
      arrive(C::B_QEMPTY + qn % C::QST);
      ++qn;

      // ------------------------------------------- the item (or piece) is done
      if (merges > 0 && !wait(C::B_FREE, (merges - 1) & 1u)) break;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int row = 0; row < 2; ++row) {
          sum[mt][row] += __shfl_xor_sync(0xffffffffu, sum[mt][row], 1);
          sum[mt][row] += __shfl_xor_sync(0xffffffffu, sum[mt][row], 2);
          const int r = warp * C::R + mt * 16 + row * 8 + g8;
          if (t4 == 0) mls[r] = make_float2(mx[mt][row], sum[mt][row]);
#pragma unroll
          for (int n = 0; n < DH / 8; ++n)
            *reinterpret_cast<float2*>(mrg + r * (DH + 4) + n * 8 + t4 * 2) =
                make_float2(o[mt][n][2 * row], o[mt][n][2 * row + 1]);
        }
      arrive(C::B_JOIN);
      if (!wait(C::B_JOIN, merges & 1u)) break;
      const int head0 = m.kvh * a.group;
      const bool whole = (m.flags & kBegins) && (m.flags & kEnds);
      // a piece that holds the item's first block is the part's last, else its first
      const int64_t at = 2 * worker + ((m.flags & kBegins) ? 1 : 0);
      if (!whole && threadIdx.x == 0) {
        ChunkPiece pc = {};
        pc.token0 = m.token0;
        pc.tokens = m.tokens;
        pc.head0 = head0;
        pc.ends = (m.flags & kEnds) ? 1 : 0;
        a.piece[at] = pc;
      }
      // four columns of a row to a thread: along the rows of O, or along the workspace's row groups
#pragma unroll 1
      for (int e = threadIdx.x; e < C::R * DH / 4; e += kWarps * 32) {
        const int r = whole ? e / (DH / 4) : e % C::R, c4 = whole ? e % (DH / 4) : e / C::R;
        const int tk = r / a.group, h = r - tk * a.group;
        if (tk >= m.tokens) continue;
        float2 ml[kWarps];
        float top = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          ml[w] = mls[w * C::R + r];
          top = fmaxf(top, ml[w].x);
        }
        const float off = top == -INFINITY ? 0.f : top;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2_approx(ml[w].x - off);
          const float4 x = *reinterpret_cast<const float4*>(mrg + (w * C::R + r) * (DH + 4) + c4 * 4);
          l = fmaf(ml[w].y, f, l);
          v.x = fmaf(x.x, f, v.x);
          v.y = fmaf(x.y, f, v.y);
          v.z = fmaf(x.z, f, v.z);
          v.w = fmaf(x.w, f, v.w);
        }
        if (whole) {
          const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
          const int64_t t = m.token0 + tk;
          *reinterpret_cast<uint2*>(a.o + (t * a.hq + head0 + h) * DH + c4 * 4) =
              make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
          if (a.lse && c4 == 0)
            a.lse[(int64_t)(head0 + h) * a.T + t] =
                l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(a.po + at * a.rows * DH + ((int64_t)c4 * a.rows + r) * 4) = v;
          if (c4 == 0) a.ml[at * a.rows + r] = make_float2(top, l);
        }
      }
      arrive(C::B_FREE);
      ++merges;
    }
  }
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {                    // let copies in flight land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  __syncthreads();
  if (threadIdx.x == 0)
    a.status[worker] = *abort_flag ? GDPA_ERR_TIMEOUT
                                   : start.bad || bad_page ? GDPA_ERR_INVALID_ARG : GDPA_OK;
}

struct Partial {                                              // of one row and 4 columns
  float m, l;
  float4 o;
};
__device__ __forceinline__ void merge(Partial& a, const float2 ml, const float4 v) {
  if (ml.y == 0.f) return;                                    // a piece that this row sees nothing of
  const float top = fmaxf(a.m, ml.x);
  const float f = sm100::ex2_approx(a.m - top), g = sm100::ex2_approx(ml.x - top);
  a.m = top;
  a.l = a.l * f + ml.y * g;
  a.o.x = a.o.x * f + v.x * g;
  a.o.y = a.o.y * f + v.y * g;
  a.o.z = a.o.z * f + v.z * g;
  a.o.w = a.o.w * f + v.w * g;
}

// Joins the pieces of the item that begins in worker blockIdx.x's part and ends
// in a later one, 8 rows (blockIdx.y) to a block: a warp to 16 columns of every SPLIT-th
// piece, merged in the workers' order, then the splits in theirs.
template <int DH, int SPLIT>
__global__ void __launch_bounds__(DH / 16 * SPLIT * 32)
chunk_join_kernel(const ChunkArgs a, WsHeader* ws) {
  constexpr int GROUPS = DH / 16;
  __shared__ float4 sacc[SPLIT][GROUPS][32];
  __shared__ float2 sml[SPLIT][GROUPS][8];
  __shared__ int worst;
  const int w = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (w == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) worst = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.workers; i += blockDim.x)
      if (a.status[i]) atomicMax(&worst, a.status[i]);
    __syncthreads();
    if (threadIdx.x == 0) ws->status = worst;
  }
  const ChunkPiece first = a.piece[2 * w + 1];
  const int cg = warp % GROUPS, sp = warp / GROUPS, r8 = lane & 7, c4 = lane >> 3;
  const int r = blockIdx.y * 8 + r8, x = r / a.tile_rows, rr = r - x * a.tile_rows;
  const int tk = rr / a.group, h = rr - tk * a.group;
  const bool live = tk < a.rt1 && x * a.rt1 + tk < first.tokens;
  if (!__any_sync(0xffffffffu, live)) return;                 // (the same in every warp of the block)
  // worker of the item's last piece: the next one that holds the item's end
  int last = w + 1;
  for (; last < a.workers; last += 32) {
    const int i = last + lane;
    const bool stop = i >= a.workers - 1 || a.piece[2 * i].ends || a.piece[2 * i].tokens == 0;
    const uint32_t m = __ballot_sync(0xffffffffu, stop);
    if (m) {
      last += __ffs(m) - 1;
      break;
    }
  }
  last = min(last, a.workers - 1);
  Partial p = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  const int64_t col = ((int64_t)(cg * 4 + c4) * a.rows + r) * 4;
  if (live) {
    constexpr int U = 4;
    for (int i = w + sp; i <= last; i += U * SPLIT) {
      float2 ml[U];
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u * SPLIT;
        const int64_t at = k == w ? 2 * w + 1 : 2 * k;
        ml[u] = make_float2(0.f, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k <= last) {
          ml[u] = a.ml[at * a.rows + r];
          v[u] = *reinterpret_cast<const float4*>(a.po + at * a.rows * DH + col);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) merge(p, ml[u], v[u]);
    }
  }
  if constexpr (SPLIT > 1) {
    sacc[sp][cg][lane] = p.o;
    if (c4 == 0) sml[sp][cg][r8] = make_float2(p.m, p.l);
    __syncthreads();
    if (sp > 0) return;
#pragma unroll
    for (int i = 1; i < SPLIT; ++i) merge(p, sml[i][cg][r8], sacc[i][cg][lane]);
  }
  if (!live) return;
  const float inv = p.l > 0.f || p.l != p.l ? 1.f / p.l : 0.f;
  const int64_t t = first.token0 + x * a.rt1 + tk;
  *reinterpret_cast<uint2*>(a.o + (t * a.hq + first.head0 + h) * DH + (cg * 4 + c4) * 4) =
      make_uint2(sm100::pack_bf16x2(p.o.x * inv, p.o.y * inv),
                 sm100::pack_bf16x2(p.o.z * inv, p.o.w * inv));
  if (a.lse && cg == 0 && c4 == 0)
    a.lse[(int64_t)(first.head0 + h) * a.T + t] =
        p.l == 0.f ? -INFINITY : (p.m + log2f(p.l)) * 0.69314718055994531f;
}

template <int DH, int MT>
cudaError_t launch_rows(const ChunkArgs& a, const gdpa_cache_t& c, cudaStream_t st) {
  using C = Cfg<DH, MT>;
  CUtensorMap mq, mk, mv;
  const CUtensorMapSwizzle sw = DH < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!chunk_maps(a, c, DH, C::CH, C::kBN, sw, &mq, &mk, &mv)) return cudaErrorInvalidValue;
  auto kern = chunk_rows_kernel<DH, MT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kern, (int)C::SMEM, done);
  if (e != cudaSuccess) return e;
  KernelScope ks_("gdpa_chunk_rows", st);
  kern<<<a.workers, kThreadsC, C::SMEM, st>>>(mq, mk, mv, a);
  return cudaGetLastError();
}

// How a call is cut.  `tiles`: the tcgen05 kernel of chunk_sm100.cu.
struct ChunkLayout {
  bool tiles;
  int mt, rows, tile_rows, rt1, rt, workers;
  size_t status_off, piece_off, ml_off, po_off, total;
};
ChunkLayout chunk_layout(const gdpa_cache_t& c, int hq, int max_n) {
  ChunkLayout L;
  const int group = hq / c.hk;
  // one row tile of 16, or of 32, where it holds all of a sample's rows; pairs of 128-row
  // tiles on the tensor core's tcgen05 path beyond that.  At dh = 128 a thread has no registers for 32 rows of O
  // beside the rest: 32 rows over 8 x 15 k positions, 8 kv heads, took 199 us in one tile of 32 and 100 us on the
  // tcgen05 path (dh = 64: 75 and 83 us).
  const int64_t need = (int64_t)group * (max_n > 1 ? max_n : 1);   // (0: a batch of padding alone)
  L.tiles = need > (c.dh == 128 ? 16 : 32);
  L.mt = need <= 16 ? 1 : 2;
  L.tile_rows = L.tiles ? 128 : 16 * L.mt;
  L.rows = L.tiles ? 256 : L.tile_rows;
  L.rt1 = L.tile_rows / group;
  L.rt = L.tiles ? 2 * L.rt1 : L.rt1;
  L.workers = (L.tiles ? 1 : 2) * device_sm_count();
  L.status_off = sizeof(WsHeader);
  L.piece_off = align_up(L.status_off + 4 * (size_t)L.workers, 256);
  L.ml_off = align_up(L.piece_off + 2 * sizeof(ChunkPiece) * (size_t)L.workers, 256);
  L.po_off = align_up(L.ml_off + 2 * sizeof(float2) * (size_t)L.workers * L.rows, 256);
  L.total = align_up(L.po_off + 2 * sizeof(float) * (size_t)L.workers * L.rows * c.dh, 256);
  return L;
}

gdpa_status_t check_chunk(const gdpa_cache_t* c, int32_t B, int32_t hq, int64_t T, int32_t max_n) {
  const gdpa_status_t s = check_cache(c, B);
  if (s != GDPA_OK) return s;
  if (hq < 1 || hq % c->hk || T < 0 || T >= (int64_t)1 << 31 || max_n < 0) return GDPA_ERR_INVALID_ARG;
  if (hq / c->hk > 128 || (int64_t)hq * c->dh > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  return GDPA_OK;
}

gdpa_status_t finish(cudaError_t e) {
  if (e == cudaSuccess) return GDPA_OK;
  fprintf(stderr, "gdpa: CUDA error %d (%s)\n", (int)e, cudaGetErrorString(e));
  return GDPA_ERR_CUDA;
}

}  // namespace

bool chunk_maps(const ChunkArgs& a, const gdpa_cache_t& c, int dh, int ch, int bn,
                CUtensorMapSwizzle sw, CUtensorMap* q, CUtensorMap* k, CUtensorMap* v) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  auto make = [&](CUtensorMap* m, int dims, const void* p, const cuuint64_t* size,
                  const cuuint64_t* stride, const cuuint32_t* box) {
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, const_cast<void*>(p), size, stride, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t row = (cuuint64_t)dh * 2;
  const cuuint64_t qsize[3] = {(cuuint64_t)dh, (cuuint64_t)a.hq, (cuuint64_t)a.T};
  const cuuint64_t qstride[2] = {row, a.hq * row};
  const cuuint32_t qbox[3] = {(cuuint32_t)ch, (cuuint32_t)a.group, (cuuint32_t)a.rt1};
  const cuuint64_t size[4] = {(cuuint64_t)dh, (cuuint64_t)c.page, (cuuint64_t)c.hk,
                              (cuuint64_t)c.num_pages};
  const cuuint64_t stride[3] = {row, c.page * row, (cuuint64_t)c.hk * c.page * row};
  const cuuint32_t box[4] = {(cuuint32_t)ch, (cuuint32_t)(c.page < bn ? c.page : bn), 1, 1};
  return make(q, 3, a.q, qsize, qstride, qbox) && make(k, 4, c.k, size, stride, box) &&
         make(v, 4, c.v, size, stride, box);
}

template <int DH, int SPLIT>
cudaError_t launch_join(const ChunkArgs& a, WsHeader* ws, cudaStream_t st) {
  KernelScope ks_("gdpa_chunk_join", st);
  return launch_dependent(chunk_join_kernel<DH, SPLIT>, dim3(a.workers, a.rows / 8),
                          dim3(DH / 16 * SPLIT * 32), st, a, ws);
}
cudaError_t launch_chunk_join(const ChunkArgs& a, int dh, WsHeader* ws, cudaStream_t st) {
  // few items leave many pieces to each (about workers / items): 512 threads share them.  (Rows behind the last
  // sample are none of the at most B * max_n tokens.)
  const int64_t most = (int64_t)a.B * a.max_n, tokens = a.T < most ? a.T : most;
  const int64_t tiles = tokens / a.rt > a.B ? tokens / a.rt : a.B;
  const bool many = tiles * a.hk * 8 < a.workers;
  if (dh == 32) return many ? launch_join<32, 8>(a, ws, st) : launch_join<32, 1>(a, ws, st);
  if (dh == 64) return many ? launch_join<64, 4>(a, ws, st) : launch_join<64, 1>(a, ws, st);
  return many ? launch_join<128, 2>(a, ws, st) : launch_join<128, 1>(a, ws, st);
}

}  // namespace gdpa

using namespace gdpa;

extern "C" gdpa_status_t gdpa_chunk_workspace_size(const gdpa_cache_t* cache, int32_t B, int32_t hq,
                                                   int64_t T, int32_t max_n, size_t* bytes) {
  const gdpa_status_t s = check_chunk(cache, B, hq, T, max_n);
  if (s != GDPA_OK) return s;
  if (!bytes || (int64_t)max_n * B < T) return GDPA_ERR_INVALID_ARG;   // (the samples' tokens)
  *bytes = chunk_layout(*cache, hq, max_n).total;
  return GDPA_OK;
}

extern "C" gdpa_status_t gdpa_chunk_fwd(const gdpa_cache_t* cache, int32_t B, int32_t hq, int64_t T,
                                        int32_t max_n, int32_t window, float scale, const void* q,
                                        const int32_t* offsets, const int32_t* kv_len, void* o,
                                        float* lse, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  reset_launch_count();
  const gdpa_status_t s = check_chunk(cache, B, hq, T, max_n);
  if (s != GDPA_OK) return s;
  if (window < 1 || !(scale - scale == 0.f)) return GDPA_ERR_INVALID_ARG;
  if (!offsets || !kv_len || (T > 0 && (!q || !o))) return GDPA_ERR_INVALID_ARG;
  if (((uintptr_t)q & 15u) || ((uintptr_t)o & 15u) || ((uintptr_t)offsets & 3u) ||
      ((uintptr_t)kv_len & 3u) || ((uintptr_t)lse & 3u))
    return GDPA_ERR_INVALID_ARG;
  const ChunkLayout L = chunk_layout(*cache, hq, max_n);
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < L.total)
    return GDPA_ERR_WORKSPACE;
  const cudaStream_t st = (cudaStream_t)stream;
  if (T == 0) return finish(cudaMemsetAsync(workspace, 0, sizeof(WsHeader), st));
  ChunkArgs a = {};
  a.offsets = offsets;
  a.kv_len = kv_len;
  a.table = cache->page_table;
  a.q = (const __nv_bfloat16*)q;
  a.o = (__nv_bfloat16*)o;
  a.lse = lse;
  char* ws = (char*)workspace;
  a.status = (int32_t*)(ws + L.status_off);
  a.piece = (ChunkPiece*)(ws + L.piece_off);
  a.ml = (float2*)(ws + L.ml_off);
  a.po = (float*)(ws + L.po_off);
  a.T = T;
  a.B = B;
  a.hq = hq;
  a.hk = cache->hk;
  a.group = hq / cache->hk;
  a.max_n = max_n;
  a.window = window;
  a.rt = L.rt;
  a.rt1 = L.rt1;
  a.rows = L.rows;
  a.tile_rows = L.tile_rows;
  a.bn_shift = L.tiles ? 7 : chunk_rows_shift(cache->dh);
  a.num_pages = cache->num_pages;
  a.max_pages = cache->max_pages;
  a.page_shift = log2_int(cache->page);
  a.workers = L.workers;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaError_t e;
#define GDPA_ROWS(DH) \
  (L.mt == 1 ? launch_rows<DH, 1>(a, *cache, st) : launch_rows<DH, 2>(a, *cache, st))
  e = L.tiles            ? launch_chunk_tiles(a, *cache, st)
      : cache->dh == 32 ? GDPA_ROWS(32)
      : cache->dh == 64 ? GDPA_ROWS(64)
                        : launch_rows<128, 1>(a, *cache, st);
#undef GDPA_ROWS
  if (e == cudaSuccess) e = launch_chunk_join(a, cache->dh, (WsHeader*)workspace, st);
  return finish(e);
}
