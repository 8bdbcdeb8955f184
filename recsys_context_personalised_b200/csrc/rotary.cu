// Rotary positions and the append to a paged key/value cache.
//
// Rotary: within the first `rot` elements of a head, pair i (elements (2i, 2i+1)
// interleaved, or (i, i + rot/2)) turns by the angle pos * w_i and is scaled by
// mscale; w_i = base^(-2i/rot), slowed for long contexts (rotary_frequencies).
// The gradient is the same map with the angle's sign reversed.
//
// Angles: pos * w_i / (2 pi) turns is taken modulo 1 exactly, by one 64-bit
// integer product with w_i / (2 pi) held as a 0.64 fixed-point fraction, so a
// position of 2^31 is as accurate (2^-33 turns) as position 1; the remaining
// turn in [-1/2, 1/2) goes to sincospif as an fp32 value.
//
// Bound: memory (each element is read and written once).  A block takes a few
// tokens with all their heads: it first writes the (cos, sin) of its tokens to
// shared memory, once for all heads; then a thread takes the (cos, sin) of one piece of a token's heads into
// registers and walks the heads with it in 16-byte vectors.  Measured (copy: 6.5 TB/s): 144 k tokens of 32
// bf16 heads of 64 199 us, 5.9 TB/s; the append of 49 k tokens, 32 + 8 + 8 heads of 128, 206 us, 5.8 TB/s.
#include <math.h>
#include <stdio.h>

#include "layer_launch.cuh"
#include "paged.cuh"

namespace gdpa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kMaxTok = 8;       // tokens of a block (16: append 227 instead of 214 us)

struct RotArgs {
  uint64_t turn[64];             // w_i / (2 pi) in units of 2^-64 turns
  float mscale;
  int rot, dh, B, interleaved, inverse;
  int tok;                       // tokens per block
  int64_t T;
  const int32_t* offsets;        // [B + 1], or NULL with `positions`
  const int32_t* kv_len;         // [B]: the last token's position + 1; NULL: n_b
  const int32_t* positions;      // [T], or NULL
  // plain rotation: x -> y, h heads; append: q -> q_out (hq heads, may be absent)
  const void* x;
  void* y;
  int64_t x_stride, y_stride;
  int h;
  // append
  const void *k, *v;
  int64_t k_stride, v_stride;
  void *cache_k, *cache_v;
  const int32_t* table;
  int hk, page_shift, num_pages, max_pages;
  WsHeader* status;
};

template <typename E> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

enum RotPath { kInterleaved, kHalves, kPairs };

// Piece `u` of a head row, the same in every head of a token:
//   kInterleaved  one vector of pairs (4 or 2 to a vector)
//   kHalves       the halves are whole vectors: u < half / N: the two vectors of N pairs; then the vectors past rot
//   kPairs        otherwise: u < half: pair u; then the single elements past rot (an in-place row has one
//                 owner per pair)
template <typename E, int PATH>
struct Piece {
  using V = Vec16<E>;
  static constexpr int N = V::N, C = PATH == kInterleaved ? N / 2 : PATH == kHalves ? N : 1;
  struct Data {
    uint4 a, b;
  };
  float2 cs[C];
  int at;                       // of its first element in the row
  bool turn;

  // `tab`: the token's (cos, sin); pairs past rot turn by nothing
  __device__ __forceinline__ Piece(const float2* tab, int half, int u) {
    const int p = PATH == kPairs ? u : u * C;
    turn = p < half;
    at = PATH == kInterleaved ? u * N : turn ? p : half + p;
#pragma unroll
    for (int i = 0; i < C; ++i) cs[i] = p + i < half ? tab[p + i] : make_float2(1.f, 0.f);
  }
  __device__ __forceinline__ Data load(const E* row, int half) const {
    Data d;
    if constexpr (PATH == kPairs) {
      d.a.x = raw(row[at]);
      if (turn) d.b.x = raw(row[at + half]);
    } else {
      d.a = *reinterpret_cast<const uint4*>(row + at);
      if (PATH == kHalves && turn) d.b = *reinterpret_cast<const uint4*>(row + at + half);
    }
    return d;
  }
  __device__ __forceinline__ void store(E* row, int half, const Data& d) const {
    if constexpr (PATH == kInterleaved) {
      if (!turn) {
        *reinterpret_cast<uint4*>(row + at) = d.a;
        return;
      }
      float f[N];
      V::unpack(d.a, f);
#pragma unroll
      for (int i = 0; i < C; ++i) rotate(f[2 * i], f[2 * i + 1], cs[i], u_exact(i));
      *reinterpret_cast<uint4*>(row + at) = V::pack(f);
    } else if constexpr (PATH == kHalves) {
      if (!turn) {
        *reinterpret_cast<uint4*>(row + at) = d.a;
        return;
      }
      float f[N], g[N];
      V::unpack(d.a, f);
      V::unpack(d.b, g);
#pragma unroll
      for (int i = 0; i < C; ++i) rotate(f[i], g[i], cs[i], true);
      *reinterpret_cast<uint4*>(row + at) = V::pack(f);
      *reinterpret_cast<uint4*>(row + at + half) = V::pack(g);
    } else {
      float x = Elem<E>::to_f(elem(d.a.x));
      if (!turn) {
        row[at] = elem(d.a.x);
        return;
      }
      float y = Elem<E>::to_f(elem(d.b.x));
      rotate(x, y, cs[0], true);
      row[at] = Elem<E>::from_f(x);
      row[at + half] = Elem<E>::from_f(y);
    }
  }

 private:
  // (a vector that rot ends in: its pairs past rot are only copied, whatever they hold)
  __device__ __forceinline__ bool u_exact(int i) const { return cs[i].x != 1.f || cs[i].y != 0.f; }
  static __device__ __forceinline__ void rotate(float& x, float& y, float2 c, bool on) {
    const float p = x * c.x - y * c.y, q = x * c.y + y * c.x;
    x = on ? p : x;
    y = on ? q : y;
  }
  static __device__ __forceinline__ uint32_t raw(E v) {
    if constexpr (sizeof(E) == 2) return *reinterpret_cast<const uint16_t*>(&v);
    else return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ E elem(uint32_t v) {
    if constexpr (sizeof(E) == 2) {
      const uint16_t h = (uint16_t)v;
      return *reinterpret_cast<const E*>(&h);
    } else {
      return *reinterpret_cast<const E*>(&v);
    }
  }
};

// The piece in heads s, s + slots, ... of a token: src_step, dst_step elements from head to head.  Two
// heads' loads go out before their stores (which might alias the next loads, for all the compiler knows).
template <typename P, typename E>
__device__ __forceinline__ void walk_heads(const P& piece, const E* src, int src_step, E* dst, int64_t dst_step,
                                           int heads, int s, int slots, int half) {
  for (int j = s; j < heads; j += 2 * slots) {
    const int k = j + slots;
    const typename P::Data d0 = piece.load(src + (int64_t)j * src_step, half);
    typename P::Data d1;
    if (k < heads) d1 = piece.load(src + (int64_t)k * src_step, half);
    piece.store(dst + j * dst_step, half, d0);
    if (k < heads) piece.store(dst + k * dst_step, half, d1);
  }
}

// Sample of token t: the largest b with offsets[b] <= t, by one warp, 32
// entries a round (two dependent loads for up to 1023 samples).  Stays inside
// [0, B] whatever the offsets hold; B when t lies behind the last sample, -1
// when it lies before the first.
__device__ __forceinline__ int warp_sample(const int32_t* offsets, int B, int64_t t, int lane) {
  int lo = 0, n = B + 1;
  for (;;) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    const bool below = i < n && (int64_t)__ldg(offsets + lo + i) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, below));
    if (c == 0) return lo == 0 ? -1 : lo;
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
    if (step == 1) return lo;
  }
}

// (Halves hold twice the vectors and (cos, sin): 64 registers, the other paths run in 40.)
template <typename E, int PATH, bool APPEND>
__global__ void __launch_bounds__(kRotThreads, PATH == kHalves ? 4 : 6)
rotary_kernel(const __grid_constant__ RotArgs a) {
  __shared__ float2 cs[kMaxTok * 64];
  __shared__ int64_t dst_row[kMaxTok];     // append: element offset of the cache row (head 0), or -1
  __shared__ int64_t pos_of[kMaxTok];
  __shared__ int live[kMaxTok];
  constexpr int N = Vec16<E>::N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * a.tok;
  const int nt = (int)min((int64_t)a.tok, a.T - t0);
  const int half = a.rot >> 1;

  for (int i = warp; i < nt; i += kRotThreads / 32) {
    const int64_t t = t0 + i;
    int b = 0;
    bool ok = true;
    int64_t pos = 0, row = -1;
    if (a.offsets) {
      b = warp_sample(a.offsets, a.B, t, lane);
      ok = b >= 0 && b < a.B;
    }
    if (ok) {
      if (a.positions) {
        pos = a.positions[t];
      } else {
        const int32_t lo = a.offsets[b], hi = a.offsets[b + 1];
        pos = (a.kv_len ? (int64_t)a.kv_len[b] - (hi - (int64_t)lo) : 0) + (t - lo);
      }
      if constexpr (APPEND) {
        if (pos >= 0) {
          const int32_t id = page_of(a.table + (int64_t)b * a.max_pages, a.max_pages, a.num_pages,
                                     a.page_shift, pos);
          if (id >= 0)
            row = cache_row(id, 0, a.hk, a.page_shift, (int)(pos & ((1 << a.page_shift) - 1)), a.dh);
          else if (lane == 0 && a.status)
            report(a.status, GDPA_ERR_INVALID_ARG);
        }
      }
    }
    if (lane == 0) {
      live[i] = ok;
      pos_of[i] = pos;
      dst_row[i] = row;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nt * half; e += kRotThreads) {
    const int i = e / half, p = e - i * half;
    // frac(pos * turn) as a signed 64-bit fraction: |angle| <= half a turn
    const int64_t frac = (int64_t)((uint64_t)pos_of[i] * a.turn[p]);
    float s, c;
    sincospif((float)(frac >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    cs[i * half + p] = make_float2(c * a.mscale, (a.inverse ? -s : s) * a.mscale);
  }
  __syncthreads();

  // threads: (token, slot, piece), pieces fastest; `slots` threads share the heads of a token's piece
  const int units = PATH == kInterleaved ? a.dh / N : PATH == kHalves ? (a.dh - half) / N : a.dh - half;
  const int ph = 1 << a.page_shift;
  {
    const int slots = max(1, kRotThreads / (nt * units)), per = slots * units;
    for (int e = threadIdx.x; e < nt * per; e += kRotThreads) {
      const int i = e / per, r = e - i * per, slot = r / units, u = r - slot * units;
      if (!live[i]) continue;
      const int64_t t = t0 + i;
      const Piece<E, PATH> piece(cs + i * half, half, u);
      walk_heads(piece, reinterpret_cast<const E*>(a.x) + t * a.x_stride, a.dh,
                 reinterpret_cast<E*>(a.y) + t * a.y_stride, (int64_t)a.dh, a.h, slot, slots, half);
      if constexpr (APPEND)
        if (dst_row[i] >= 0)
          walk_heads(piece, reinterpret_cast<const E*>(a.k) + t * a.k_stride, a.dh,
                     reinterpret_cast<E*>(a.cache_k) + dst_row[i], (int64_t)ph * a.dh, a.hk, slot, slots,
                     half);
    }
  }
  if constexpr (APPEND) {                    // the values: vectors as they are
    const int slots = max(1, kRotThreads / (nt * (a.dh / N))), per = slots * (a.dh / N);
    for (int e = threadIdx.x; e < nt * per; e += kRotThreads) {
      const int i = e / per, r = e - i * per, slot = r / (a.dh / N), u = r - slot * (a.dh / N);
      if (dst_row[i] < 0) continue;
      const Piece<E, kInterleaved> copy(cs, 0, u);
      walk_heads(copy, reinterpret_cast<const E*>(a.v) + (t0 + i) * a.v_stride, a.dh,
                 reinterpret_cast<E*>(a.cache_v) + dst_row[i], (int64_t)ph * a.dh, a.hk, slot, slots, 0);
    }
  }
}

bool finite(double x) { return x == x && x - x == 0.0; }

gdpa_status_t check_spec(const gdpa_rotary_t* r, int32_t dh) {
  if (!r) return GDPA_ERR_INVALID_ARG;
  if (r->rot < 2 || (r->rot & 1) || r->rot > dh) return GDPA_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return GDPA_ERR_INVALID_ARG;
  if (!finite(r->base) || r->base < 1.0 || !finite(r->factor) || r->factor < 1.0 ||
      r->trained_len < 0 || !finite(r->mscale))
    return GDPA_ERR_INVALID_ARG;
  if (r->trained_len > 0 && (!finite(r->low) || !finite(r->high) || !(r->high > r->low)))
    return GDPA_ERR_INVALID_ARG;
  return GDPA_OK;
}

// w_i / (2 pi) as 0.64 fixed point (w_i <= 1, so below 0.16 turns).
// A frequency that makes more than `high` turns within the trained length stays,
// one that makes fewer than `low` is divided by `factor`, linearly in between.
void rotary_frequencies(const gdpa_rotary_t& r, uint64_t (&turn)[64]) {
  const long double two_pi = 6.283185307179586476925286766559L;
  // (by repeated multiplication: 63 roundings of 2^-64, nothing beside the 2^-64 turns of the result, where
  // a power for every pair would take longer than the kernel on a few tokens)
  const long double step = powl((long double)r.base, -2.0L / r.rot);
  long double power = 1.0L;
  for (int i = 0; i < r.rot / 2; ++i, power *= step) {
    long double w = power, keep = 0.0L;
    if (r.trained_len > 0) {
      keep = (r.trained_len * w / two_pi - r.low) / ((long double)r.high - r.low);
      keep = keep < 0.0L ? 0.0L : keep > 1.0L ? 1.0L : keep;
    }
    w *= keep + (1.0L - keep) / r.factor;
    turn[i] = (uint64_t)(w / two_pi * 18446744073709551616.0L);
  }
}

template <typename E, bool APPEND>
cudaError_t launch_rotary(RotArgs& a, const char* name, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  // a few tokens per block: at most kMaxTok, fewer when the call has too few
  // tokens to give every SM four blocks
  int64_t tok = a.T / (4 * (int64_t)device_sm_count());
  a.tok = (int)(tok < 1 ? 1 : tok > kMaxTok ? kMaxTok : tok);
  const int64_t blocks = (a.T + a.tok - 1) / a.tok;
  const int half = a.rot / 2;
  KernelScope ks_(name, st);
  if (a.interleaved)
    rotary_kernel<E, kInterleaved, APPEND><<<(unsigned)blocks, kRotThreads, 0, st>>>(a);
  else if (half % Vec16<E>::N == 0)
    rotary_kernel<E, kHalves, APPEND><<<(unsigned)blocks, kRotThreads, 0, st>>>(a);
  else
    rotary_kernel<E, kPairs, APPEND><<<(unsigned)blocks, kRotThreads, 0, st>>>(a);
  return cudaGetLastError();
}

gdpa_status_t finish(cudaError_t e) {
  if (e == cudaSuccess) return GDPA_OK;
  fprintf(stderr, "gdpa: CUDA error %d (%s)\n", (int)e, cudaGetErrorString(e));
  return GDPA_ERR_CUDA;
}

bool off16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
bool off4(const void* p) { return ((uintptr_t)p & 3u) != 0; }

}  // namespace
}  // namespace gdpa

using namespace gdpa;

extern "C" gdpa_status_t gdpa_rotary(const gdpa_rotary_t* r, int32_t dtype, int32_t B, int32_t h,
                                     int32_t dh, int64_t T, const int32_t* offsets,
                                     const int32_t* kv_len, const int32_t* positions,
                                     const void* x, int64_t x_stride, void* y, int64_t y_stride,
                                     int32_t inverse, void* stream) {
  reset_launch_count();
  if (dtype != GDPA_DTYPE_F32 && dtype != GDPA_DTYPE_BF16) return GDPA_ERR_INVALID_ARG;
  if (h < 1 || T < 0 || T >= (int64_t)1 << 31 || B < 0) return GDPA_ERR_INVALID_ARG;
  if (dh != 32 && dh != 64 && dh != 128) return GDPA_ERR_UNSUPPORTED;
  const gdpa_status_t s = check_spec(r, dh);
  if (s != GDPA_OK) return s;
  if ((!offsets && !positions) || (offsets && B < 1) || (kv_len && !offsets) ||
      (kv_len && positions))
    return GDPA_ERR_INVALID_ARG;
  const int vec = dtype == GDPA_DTYPE_BF16 ? 8 : 4;
  if ((int64_t)h * dh > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  if (x_stride < (int64_t)h * dh || y_stride < (int64_t)h * dh || x_stride % vec || y_stride % vec)
    return GDPA_ERR_INVALID_ARG;
  if (T > 0 && (!x || !y)) return GDPA_ERR_INVALID_ARG;
  if (x == y && x_stride != y_stride) return GDPA_ERR_INVALID_ARG;
  if (off16(x) || off16(y) || off4(offsets) || off4(kv_len) || off4(positions))
    return GDPA_ERR_INVALID_ARG;
  RotArgs a = {};
  rotary_frequencies(*r, a.turn);
  a.mscale = (float)r->mscale;
  a.rot = r->rot;
  a.interleaved = r->interleaved;
  a.inverse = inverse != 0;
  a.dh = dh;
  a.B = B;
  a.T = T;
  a.offsets = offsets;
  a.kv_len = kv_len;
  a.positions = positions;
  a.x = x;
  a.y = y;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.h = h;
  const cudaStream_t st = (cudaStream_t)stream;
  return finish(dtype == GDPA_DTYPE_BF16
                    ? launch_rotary<__nv_bfloat16, false>(a, "gdpa_rotary", st)
                    : launch_rotary<float, false>(a, "gdpa_rotary", st));
}

extern "C" gdpa_status_t gdpa_cache_append(const gdpa_rotary_t* r, const gdpa_cache_t* c,
                                           int32_t B, int32_t hq, int64_t T,
                                           const int32_t* offsets, const int32_t* kv_len,
                                           const void* q, int64_t q_stride, void* q_out,
                                           const void* k, int64_t k_stride, const void* v,
                                           int64_t v_stride, void* status_ws, void* stream) {
  reset_launch_count();
  gdpa_status_t s = check_cache(c, B);
  if (s != GDPA_OK) return s;
  if (T < 0 || T >= (int64_t)1 << 31 || hq < 0) return GDPA_ERR_INVALID_ARG;
  if (r) {
    s = check_spec(r, c->dh);
    if (s != GDPA_OK) return s;
  }
  if (!offsets || !kv_len || (T > 0 && (!k || !v))) return GDPA_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr) || (q && hq < 1)) return GDPA_ERR_INVALID_ARG;
  const int64_t kw = (int64_t)c->hk * c->dh, qw = (int64_t)hq * c->dh;
  if (kw > (1 << 20) || qw > (1 << 20)) return GDPA_ERR_UNSUPPORTED;
  if (k_stride < kw || v_stride < kw || k_stride % 8 || v_stride % 8 ||
      (q && (q_stride < qw || q_stride % 8)) || (q && q == q_out && q_stride != qw))
    return GDPA_ERR_INVALID_ARG;
  if (off16(q) || off16(q_out) || off16(k) || off16(v) || off4(offsets) || off4(kv_len))
    return GDPA_ERR_INVALID_ARG;
  if (status_ws && ((uintptr_t)status_ws & 255u)) return GDPA_ERR_WORKSPACE;
  const cudaStream_t st = (cudaStream_t)stream;
  RotArgs a = {};
  if (r) {
    rotary_frequencies(*r, a.turn);
    a.mscale = (float)r->mscale;
    a.rot = r->rot;
    a.interleaved = r->interleaved;
  } else {
    a.rot = 0;               // nothing turns: the interleaved path copies every vector
    a.interleaved = 1;
  }
  a.dh = c->dh;
  a.B = B;
  a.T = T;
  a.offsets = offsets;
  a.kv_len = kv_len;
  a.x = q;
  a.y = q_out;
  a.x_stride = q_stride;
  a.y_stride = qw;
  a.h = q ? hq : 0;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cache_k = c->k;
  a.cache_v = c->v;
  a.table = c->page_table;
  a.hk = c->hk;
  a.page_shift = log2_int(c->page);
  a.num_pages = c->num_pages;
  a.max_pages = c->max_pages;
  a.status = (WsHeader*)status_ws;
  if (status_ws) {
    const cudaError_t e = cudaMemsetAsync(status_ws, 0, sizeof(int32_t), st);
    if (e != cudaSuccess) return finish(e);
  }
  return finish(launch_rotary<__nv_bfloat16, true>(a, "gdpa_cache_append", st));
}
