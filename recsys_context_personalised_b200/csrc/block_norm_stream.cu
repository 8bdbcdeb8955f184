// The block norm on rows streamed through shared memory (formulas: block_norm.cu).
//
// Bound: memory, every row once.  A row belongs to one warp (or to a few where it is
// wide), a group of warps walks a contiguous range of rows, and every warp keeps the next rows of its
// columns in flight by bulk copies into a ring of its own: the copies need no registers, so the
// bytes in flight (about 100 KB an SM) do not depend on what the arithmetic holds, and a row's
// reductions are shuffles within a warp, or a barrier of a row's few warps, that no other row waits for.
// Measured (copy: 6.5 TB/s): 132 k rows of 2048 bf16 with a gate per element forward 483 us, 5.6 TB/s; backward 66 k
// rows of 1024 with a gate per element 197 us, 5.4 TB/s, 126 k rows with shared gates 303 us, 5.1 TB/s.
//
// The weights' gradients (and a shared gate's) accumulate in fp32 registers over the range, in the
// rows' order, and go to the workspace once.
#include <math.h>

#include "block_norm.cuh"
#include "sm100.cuh"

namespace gdpa {
namespace {

using namespace sm100;

// Warps of a block (one block to an SM) and 16-byte vectors of a row that a thread holds: forward y in
// fp32 (4 vectors: 467 us at 2048 wide instead of 447, 8 in 8 warps: 635); backward y, dn, f, G, the gate and up
// to three sums, for which 16 warps have too few registers and 8 hide too little (1024 wide, shared
// gates: 496 and 458 us where 12 warps took 360).
constexpr int kWarpsFwd = 16, kWarpsBwd = 12, kWarpsWide = 16, kMaxFwd = 2, kMaxBwd = 2;
// Rows in flight of a warp, the current one among them.  Two are enough, and what a longer ring takes is missing
// in L1, which holds the weights: backward, 1024 wide, 4 rows 360 us, 2 rows 326 us.
constexpr int kStages = 2;
constexpr uint32_t kRingBytes = 192 * 1024;          // of a block, at most; up to 32 KB of sums come behind it
static_assert(kStages * 5 * kWarpsWide * (kMaxBwd * 512 + 32) <= kRingBytes && kMaxFwd <= kMaxBwd &&
                  kWarpsFwd <= kWarpsWide && kWarpsBwd <= kWarpsWide,
              "a ring for five tensors of the widest plan");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Which columns of a warp's segment a thread holds, and how they are read and written.  AL (rows of whole
// 16-byte units): vector i of a thread is VEC neighbouring columns.  Otherwise rows start at any element: the
// VEC columns lie 32 apart, so that a warp's access is contiguous, and each is tested against the segment's
// end; a column past it reads as 0.  Values come in pairs, for the packed arithmetic.
template <typename E, bool AL>
struct Cols {
  static constexpr int VEC = 16 / sizeof(E), P = VEC / 2;

  // does vector i hold any column (of this thread, AL; of the warp) below n
  static __device__ __forceinline__ bool any(int i, int lane, int n) {
    return AL ? (i * 32 + lane) * VEC < n : i * 32 * VEC < n;
  }
  static __device__ __forceinline__ int col(int i, int lane, int k) {
    return AL ? (i * 32 + lane) * VEC + k : (i * VEC + k) * 32 + lane;
  }
  template <typename F>
  static __device__ __forceinline__ void each(int i, int lane, int n, float2 (&f)[P], F read) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int c = col(i, lane, 2 * k), d = col(i, lane, 2 * k + 1);
      f[k] = make_float2(c < n ? read(c) : 0.f, d < n ? read(d) : 0.f);
    }
  }
  // from shared memory: `addr` of the segment's first element
  static __device__ __forceinline__ void shared(uint32_t addr, int i, int lane, int n, float2 (&f)[P]) {
    if constexpr (AL) {
      uint32_t w[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(addr + (i * 32 + lane) * 16));
      if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          f[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          f[k] = make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
      }
    } else {
      each(i, lane, n, f, [&](int c) -> float {
        if constexpr (sizeof(E) == 2) {
          uint16_t v;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr + c * 2));
          return __uint_as_float((uint32_t)v << 16);
        } else {
          float v;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr + c * 4));
          return v;
        }
      });
    }
  }
  // fp32 weights of the segment
  static __device__ __forceinline__ void weights(const float* w, int i, int lane, int n, float2 (&f)[P]) {
    if constexpr (AL) {
#pragma unroll
      for (int k = 0; k < P; k += 2) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(w + (i * 32 + lane) * VEC + 2 * k));
        f[k] = make_float2(v.x, v.y);
        f[k + 1] = make_float2(v.z, v.w);
      }
    } else {
      each(i, lane, n, f, [&](int c) { return __ldg(w + c); });
    }
  }
  static __device__ __forceinline__ void global(const E* p, int i, int lane, int n, float2 (&f)[P]) {
    if constexpr (AL) {
      Raw<E, VEC> r;
      r.load(p, (i * 32 + lane) * VEC);
      r.get(reinterpret_cast<float*>(f));
    } else {
      each(i, lane, n, f, [&](int c) { return Elem<E>::to_f(__ldg(p + c)); });
    }
  }
  static __device__ __forceinline__ void put(E* p, int i, int lane, int n, const float2 (&f)[P]) {
    if constexpr (AL) {
      Raw<E, VEC>::store(p, (i * 32 + lane) * VEC, reinterpret_cast<const float*>(f));
    } else {
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int c = col(i, lane, 2 * k), d = col(i, lane, 2 * k + 1);
        if (c < n) p[c] = Elem<E>::from_f(f[k].x);
        if (d < n) p[d] = Elem<E>::from_f(f[k].y);
      }
    }
  }
  static __device__ __forceinline__ void each_at(const float* p, int i, int lane, int n, float2 (&f)[P]) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int c = col(i, lane, 2 * k), d = col(i, lane, 2 * k + 1);
      f[k] = make_float2(AL || c < n ? p[c] : 0.f, AL || d < n ? p[d] : 0.f);
    }
  }
  // fp32 sums, in shared or global memory: v <- op(v, f)
  template <typename F>
  static __device__ __forceinline__ void sums(float* p, int i, int lane, int n, const float2 (&f)[P], F op) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const int c = col(i, lane, 2 * k), d = col(i, lane, 2 * k + 1);
      if (AL || c < n) p[c] = op(p[c], f[k].x);
      if (AL || d < n) p[d] = op(p[d], f[k].y);
    }
  }
};
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
// act of the gate, by selection
template <int P>
__device__ __forceinline__ void act(float2 (&z)[P], int sigmoid) {
#pragma unroll
  for (int k = 0; k < P; ++k)
    z[k] = make_float2(sigmoid ? logistic(z[k].x) : z[k].x, sigmoid ? logistic(z[k].y) : z[k].y);
}
// act in place, and its slope
template <int P>
__device__ __forceinline__ void act(float2 (&z)[P], int sigmoid, float2 (&slope)[P]) {
#pragma unroll
  for (int k = 0; k < P; ++k) {
    gate_slope(z[k].x, sigmoid, z[k].x, slope[k].x);
    gate_slope(z[k].y, sigmoid, z[k].y, slope[k].y);
  }
}

// The rows of one warp: its columns [col0, col0 + n) of the group's rows [t0, t1), NT tensors, in a
// ring of kStages rows.  A copy takes whole 16-byte units: of rows that start anywhere (not AL) the units around
// them, of the tensors' last bytes those that make a whole unit, and the rest by plain loads.
// Waits have a limit.  A warp whose wait ran out lets the copies in flight land and copies no more, but walks through
// its rows all the same, since the row's other warps meet it at barriers: `poison` makes its sums NaN from that row on,
// and with them what all of the row's warps make of them.  (Each of its later waits ends at the block's
// flag, within some 5 us.)  132 k rows of 2048 forward: 477 us without any of this, 483 in this form, 500 to 510 with a
// branch on the wait's result in the rows' path.
template <typename E, int NV, int NT, bool AL>
struct Stream {
  static constexpr int VEC = 16 / sizeof(E), SEG = NV * 32 * VEC;
  static constexpr uint32_t SEGB = SEG * sizeof(E) + (AL ? 0 : 32), ROWB = NT * SEGB;
  const E* src[NT];             // the tensors
  uint32_t ring, bar;
  int64_t t0, t1, whole;        // whole: bytes of a tensor in whole units
  int d, col0, n, stage;
  uint32_t phase;
  int limit;                    // this thread copies the rows below it (lane 0; others 0); -1: its wait ran out
  float poison;                 // 1, or NaN
  volatile int* abort_flag;

  __device__ __forceinline__ int64_t first(int64_t t) const { return (t * d + col0) * (int64_t)sizeof(E); }
  __device__ __forceinline__ void issue(int64_t t, int slot, bool copy = true) {
    if (t < limit) {
      const int64_t b0 = first(t), b1 = b0 + n * (int)sizeof(E);
      const int64_t a0 = AL ? b0 : b0 & ~(int64_t)15;
      const int64_t a1 = AL ? b1 : min((b1 + 15) & ~(int64_t)15, whole);
      const uint32_t bytes = n > 0 && a1 > a0 ? (uint32_t)(a1 - a0) : 0u;
      mbar_expect_tx(bar + 8 * slot, bytes * NT);
      if (bytes > 0 && copy)
#pragma unroll
        for (int k = 0; k < NT; ++k)
          bulk_load(ring + slot * ROWB + k * SEGB, reinterpret_cast<const char*>(src[k]) + a0, bytes,
                    bar + 8 * slot);
    }
  }
  // (lost: the self-test of the waits; the group's first row does not come)
  __device__ __forceinline__ void start(int lane, bool lost) {
    stage = 0;
    phase = 0;
    limit = lane == 0 ? (int)t1 : 0;
    for (int s = 0; s < kStages; ++s) issue(t0 + s, s, !(lost && s == 0));
  }
  // Waits for row t, the current one.
  __device__ __forceinline__ void wait(const NormArgs& a, int64_t t, int lane) {
    const bool ok = mbar_wait(bar + 8 * stage, phase, abort_flag, a.wait_ns);
    if (!ok) {                  // (in some of the threads, or all)
      if (t < limit) {
        volatile int never = 0;
        for (int i = 0; i < kStages && t + i < t1; ++i)
          mbar_wait(bar + 8 * ((stage + i) % kStages), phase ^ (uint32_t)((stage + i) / kStages), &never, a.wait_ns);
      }
      limit = -1;
    }
    if (!AL) {
      base = (uint32_t)(first(t) & 15);
      const int64_t b0 = first(t), b1 = b0 + n * (int)sizeof(E);
      if (b1 > whole) {                            // (the last row's last few elements)
        const int c = (int)((max(whole, b0) - b0) / (int)sizeof(E)) + lane;
        if (c < n)
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            const E v = src[k][t * d + col0 + c];
            const uint32_t to = at(k) + c * sizeof(E);
            if constexpr (sizeof(E) == 2)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(*reinterpret_cast<const uint16_t*>(&v)) : "memory");
            else
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"((float)v) : "memory");
          }
        __syncwarp();
      }
    }
    poison = __all_sync(0xffffffffu, limit >= 0) ? 1.f : NAN;
  }
  uint32_t base = 0;            // of the row's first element in the copied units
  __device__ __forceinline__ uint32_t at(int k) const { return ring + stage * ROWB + k * SEGB + base; }
  // The current row (t) has been read: its place takes a later one.
  __device__ __forceinline__ void next(int64_t t) {
    __syncwarp();
    issue(t + kStages, stage);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

// Sums of K values over a row's warps (every thread gets them): shuffles, then for a row of several
// warps a pass through shared memory between them (two halves in turn, so one barrier is enough).
template <int K>
__device__ __forceinline__ void row_sum_w(float (&v)[K], int W, int wi, int gi, float* buf, int& flip) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (W == 1) return;
  float* b = buf + flip * (kWarpsFwd * 6) + gi * W * K;
  flip ^= 1;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[wi * K + k] = v[k];
  named_bar_sync(1 + gi, W * 32);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int i = 0; i < W; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += b[i * K + k];
}

// What a call has is fixed at compile time (GATE: a gdpa_gate_t): branches on it inside the row would
// make the compiler move the row's registers around.
template <typename E, int NV, bool AL, bool BLOCK, bool POST, int GATE>
__global__ void __launch_bounds__(kWarpsFwd * 32, 1)
norm_stream_fwd_kernel(const NormArgs a, int W) {
  using St = Stream<E, NV, BLOCK ? (GATE == GDPA_GATE_TOKEN ? 3 : 2) : 1, AL>;
  using Co = Cols<E, AL>;
  constexpr int P = Co::P;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarpsFwd * kStages];
  __shared__ float buf[2 * 6 * kWarpsFwd];
  __shared__ int abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gi = warp / W, wi = warp - gi * W, g = blockIdx.x * (blockDim.x / 32 / W) + gi;
  if (threadIdx.x < kWarpsFwd * kStages) mbar_init(smem_u32(&bars[threadIdx.x]), 1);
  if (threadIdx.x == 0) abort_s = 0;
  fence_mbar_init();
  __syncthreads();
  St st;
  const int col0 = wi * St::SEG, n = max(0, min(St::SEG, a.d - col0));
  st.col0 = col0;
  st.n = n;
  st.d = a.d;
  st.whole = a.T * a.d * (int64_t)sizeof(E) & ~(int64_t)15;
  st.src[0] = reinterpret_cast<const E*>(a.x);
  if constexpr (BLOCK) st.src[1] = reinterpret_cast<const E*>(a.f);
  if constexpr (GATE == GDPA_GATE_TOKEN) st.src[2] = reinterpret_cast<const E*>(a.gate);
  st.ring = smem_u32(smem) + warp * (kStages * St::ROWB);
  st.bar = smem_u32(&bars[warp * kStages]);
  st.abort_flag = &abort_s;
  st.t0 = g < a.groups ? group_row(a.T, a.groups, g) : 0;
  st.t1 = g < a.groups ? group_row(a.T, a.groups, g + 1) : 0;
  st.start(lane, wi == 0 && st.t0 <= a.lost_row && a.lost_row < st.t1);
  int flip = 0;
  SampleWalk walk;
  walk.next = -1;
  walk.b = 0;
  for (int64_t t = st.t0; t < st.t1; ++t) {
    st.wait(a, t, lane);
    float2 y[NV][P];
    bool live = true;
    if constexpr (BLOCK) {
      float scale = a.alpha * st.poison;
      if constexpr (POST) {
        float2 q[2] = {two(0.f), two(0.f)};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (Co::any(i, lane, n)) {
            float2 f[P];
            Co::shared(st.at(1), i, lane, n, f);
#pragma unroll
            for (int k = 0; k < P; ++k) q[k & 1] = __ffma2_rn(f[k], f[k], q[k & 1]);
          }
        }
        float v[1] = {((q[0].x + q[1].x) + (q[0].y + q[1].y)) * st.poison};
        row_sum_w(v, W, wi, gi, buf, flip);
        scale *= rsqrtf(fmaf(v[0], a.inv_d, a.eps));
      }
      if constexpr (GATE == GDPA_GATE_SAMPLE) {
        walk.at(a, t);
        live = walk.live(a);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (Co::any(i, lane, n)) {
          float2 f[P], w[P];
          Co::shared(st.at(0), i, lane, n, y[i]);
          Co::shared(st.at(1), i, lane, n, f);
#pragma unroll
          for (int k = 0; k < P; ++k) f[k] = __fmul2_rn(f[k], two(scale));
          if constexpr (POST) {
            Co::weights(a.w_post + col0, i, lane, n, w);
#pragma unroll
            for (int k = 0; k < P; ++k) f[k] = __fmul2_rn(f[k], w[k]);
          }
          if constexpr (GATE != GDPA_GATE_NONE) {
            if constexpr (GATE == GDPA_GATE_TOKEN)
              Co::shared(st.at(2), i, lane, n, w);
            else
              Co::global(reinterpret_cast<const E*>(a.gate) + (int64_t)(live ? walk.b : 0) * a.d + col0, i, lane, n, w);
            act(w, a.sigmoid);
          }
#pragma unroll
          for (int k = 0; k < P; ++k)
            y[i][k] = GATE != GDPA_GATE_NONE ? __ffma2_rn(w[k], f[k], y[i][k]) : __fadd2_rn(f[k], y[i][k]);
          if (live) Co::put(reinterpret_cast<E*>(a.y) + t * a.d + col0, i, lane, n, y[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (Co::any(i, lane, n)) {
          Co::shared(st.at(0), i, lane, n, y[i]);
#pragma unroll
          for (int k = 0; k < P; ++k) y[i][k] = __fmul2_rn(y[i][k], two(st.poison));
        }
      }
    }
    st.next(t);
    if (a.w_pre) {
      float2 q[2] = {two(0.f), two(0.f)};
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (Co::any(i, lane, n))
#pragma unroll
          for (int k = 0; k < P; ++k) q[k & 1] = __ffma2_rn(y[i][k], y[i][k], q[k & 1]);
      float v[1] = {(q[0].x + q[1].x) + (q[0].y + q[1].y)};
      row_sum_w(v, W, wi, gi, buf, flip);
      const float scale = rsqrtf(fmaf(v[0], a.inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (Co::any(i, lane, n) && live) {
          float2 w[P];
          Co::weights(a.w_pre + col0, i, lane, n, w);
#pragma unroll
          for (int k = 0; k < P; ++k) y[i][k] = __fmul2_rn(y[i][k], __fmul2_rn(w[k], two(scale)));
          Co::put(reinterpret_cast<E*>(a.n) + t * a.d + col0, i, lane, n, y[i]);
        }
      }
    }
  }
}

// (A gate of GDPA_GATE_SAMPLE is one row per sample, whose gradient accumulates over the sample's rows.)
// WARPS: kWarpsBwd, or kWarpsWide for rows that more warps have to share: 128 registers spill some of the row,
// still far from the registers' form (14 k bf16 rows of 8192 624 us, there 1187).
template <typename E, int NV, int WARPS, bool AL, bool BLOCK, bool PRE, bool POST, int GATE>
__global__ void __launch_bounds__(WARPS * 32, 1)
norm_stream_bwd_kernel(const NormArgs a, int W) {
  pdl_trigger();
  constexpr bool SHARED = GATE == GDPA_GATE_SAMPLE;
  // the tensors, in the order dy, y, dn, f, token gate
  constexpr int KY = 1, KN = 2, KF = PRE ? 3 : 1, KZ = KF + 1;
  using St = Stream<E, NV, KF + (BLOCK ? 1 : 0) + (GATE == GDPA_GATE_TOKEN ? 1 : 0), AL>;
  using Co = Cols<E, AL>;
  constexpr int P = Co::P;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarpsFwd * kStages];
  __shared__ float buf[2 * 6 * kWarpsFwd];
  __shared__ int abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gi = warp / W, wi = warp - gi * W, g = blockIdx.x * (blockDim.x / 32 / W) + gi;
  if (threadIdx.x < kWarpsFwd * kStages) mbar_init(smem_u32(&bars[threadIdx.x]), 1);
  if (threadIdx.x == 0) abort_s = 0;
  fence_mbar_init();
  __syncthreads();
  St st;
  const int col0 = wi * St::SEG, n = max(0, min(St::SEG, a.d - col0));
  st.col0 = col0;
  st.n = n;
  st.d = a.d;
  st.whole = a.T * a.d * (int64_t)sizeof(E) & ~(int64_t)15;
  st.src[0] = reinterpret_cast<const E*>(a.dy ? a.dy : a.dn);     // (no dy: unused)
  if constexpr (PRE) {
    st.src[KY] = reinterpret_cast<const E*>(a.x);
    st.src[KN] = reinterpret_cast<const E*>(a.dn);
  }
  if constexpr (BLOCK) st.src[KF] = reinterpret_cast<const E*>(a.f);
  if constexpr (GATE == GDPA_GATE_TOKEN) st.src[KZ] = reinterpret_cast<const E*>(a.gate);
  st.ring = smem_u32(smem) + warp * (kStages * St::ROWB);
  st.bar = smem_u32(&bars[warp * kStages]);
  st.abort_flag = &abort_s;
  st.t0 = g < a.groups ? group_row(a.T, a.groups, g) : 0;
  st.t1 = g < a.groups ? group_row(a.T, a.groups, g + 1) : 0;
  st.start(lane, wi == 0 && st.t0 <= a.lost_row && a.lost_row < st.t1);
  int flip = 0;
  float2 apost[SHARED ? 1 : NV][P], apre[NV][P], agate[SHARED ? NV : 1][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) {
      apre[i][k] = two(0.f);
      if constexpr (SHARED) agate[i][k] = two(0.f);
      if constexpr (!SHARED) apost[i][k] = two(0.f);
    }
  // A shared gate: agate holds the sum over the sample's rows of alpha G fh, of which both the gate's
  // gradient (times w_post act') and w_post's (times act) are made when the sample ends; the latter's sum
  // stays in shared memory between samples.
  float* const spost = reinterpret_cast<float*>(smem + (size_t)(blockDim.x / 32) * kStages * St::ROWB) +
                       warp * St::SEG;
  if constexpr (SHARED && POST)
    for (int c = lane; c < St::SEG; c += 32) spost[c] = 0.f;
  SampleWalk walk;
  walk.next = -1;
  walk.b = 0;
  // the gate of this thread's columns: a sample's act(gate) (times w_post), or a row's gate as it is (act
  // is taken twice rather than kept with its slope: registers)
  float2 z[GATE != GDPA_GATE_NONE ? NV : 1][P];
  // the rows of sample walk.b that this group holds are done: their gate gradient goes out whole, or as
  // a piece (slot 1 when it holds the sample's first row)
  auto flush = [&]() {
    if constexpr (SHARED) {
      if (!walk.live(a)) return;
      const int64_t lo = max((int64_t)__ldg(a.offsets + walk.b), (int64_t)0);
      const int64_t hi = min(walk.next, a.T);
      float* out = lo >= st.t0 && hi <= st.t1
                       ? a.dgate_sample + (int64_t)walk.b * a.d
                       : a.part_gate + ((int64_t)g * 2 + (lo >= st.t0 ? 1 : 0)) * a.d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (Co::any(i, lane, n)) {
          float2 s[P], w[P];
          Co::global(reinterpret_cast<const E*>(a.gate) + (int64_t)walk.b * a.d + col0, i, lane, n, s);
          float2 ds[P];
          act(s, a.sigmoid, ds);
          if constexpr (POST) Co::weights(a.w_post + col0, i, lane, n, w);
          float2 v[P];
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const float2 sum = agate[i][k];
            agate[i][k] = two(0.f);
            v[k] = __fmul2_rn(POST ? __fmul2_rn(sum, w[k]) : sum, ds[k]);
            if constexpr (POST) s[k] = __fmul2_rn(sum, s[k]);
          }
          Co::sums(out + col0, i, lane, n, v, [](float, float y) { return y; });
          if constexpr (POST) Co::sums(spost, i, lane, n, s, [](float x, float y) { return x + y; });
        }
      }
    }
  };
  // (columns past the row hold zeros throughout and are never stored)
  float2 y[PRE ? NV : 1][P], dn[PRE ? NV : 1][P], f[BLOCK ? NV : 1][P], G[NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) {
      G[i][k] = two(0.f);
      if constexpr (PRE) y[i][k] = dn[i][k] = two(0.f);
      if constexpr (BLOCK) f[i][k] = two(0.f);
      if constexpr (GATE != GDPA_GATE_NONE) z[i][k] = two(0.f);
    }
  for (int64_t t = st.t0; t < st.t1; ++t) {
    st.wait(a, t, lane);
    bool live = true;
    if constexpr (SHARED) {
      if (t >= walk.next) {
        if (t > st.t0) flush();
        walk.seek(a, t);
        if (walk.live(a))
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (Co::any(i, lane, n)) {
              Co::global(reinterpret_cast<const E*>(a.gate) + (int64_t)walk.b * a.d + col0, i, lane, n, z[i]);
              act(z[i], a.sigmoid);
              if constexpr (POST) {
                float2 w[P];
                Co::weights(a.w_post + col0, i, lane, n, w);
#pragma unroll
                for (int k = 0; k < P; ++k) z[i][k] = __fmul2_rn(z[i][k], w[k]);
              }
            }
          }
      }
      live = walk.live(a);
    }
    if (!live) {                       // (the same for all of the row's warps) adds nothing anywhere
      st.next(t);
      continue;
    }
    // The row into registers, with all the sums of its two norms at once: of y^2, w_pre dn y and f^2, and, with
    // s = act w_post f, of s dy, s w_pre dn and s y, of which mean(w_post du fh) is made (G is linear in them),
    // so that nothing of the row waits for a second sum.
    float2 q[6];
#pragma unroll
    for (int k = 0; k < 6; ++k) q[k] = two(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (Co::any(i, lane, n)) {
        float2 wn[P], s[P];
        Co::shared(st.at(0), i, lane, n, G[i]);
        if (!a.dy)
#pragma unroll
          for (int k = 0; k < P; ++k) G[i][k] = two(0.f);
        if constexpr (PRE) {
          Co::shared(st.at(KY), i, lane, n, y[i]);
          Co::shared(st.at(KN), i, lane, n, dn[i]);
          Co::weights(a.w_pre + col0, i, lane, n, wn);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            wn[k] = __fmul2_rn(wn[k], dn[i][k]);
            q[0] = __ffma2_rn(y[i][k], y[i][k], q[0]);
            q[1] = __ffma2_rn(wn[k], y[i][k], q[1]);
          }
        }
        if constexpr (BLOCK) Co::shared(st.at(KF), i, lane, n, f[i]);
        if constexpr (GATE == GDPA_GATE_TOKEN) {
          Co::shared(st.at(KZ), i, lane, n, z[i]);
        }
        if constexpr (POST) {
          float2 az[P];
          if constexpr (GATE == GDPA_GATE_TOKEN) {
#pragma unroll
            for (int k = 0; k < P; ++k) az[k] = z[i][k];
            act(az, a.sigmoid);
          }
          if constexpr (!SHARED) Co::weights(a.w_post + col0, i, lane, n, s);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            if constexpr (SHARED) s[k] = z[i][k];             // (act w_post)
            if constexpr (GATE == GDPA_GATE_TOKEN) s[k] = __fmul2_rn(s[k], az[k]);
            s[k] = __fmul2_rn(s[k], f[i][k]);
            q[2] = __ffma2_rn(f[i][k], f[i][k], q[2]);
            q[3] = __ffma2_rn(s[k], G[i][k], q[3]);
            if constexpr (PRE) {
              q[4] = __ffma2_rn(s[k], wn[k], q[4]);
              q[5] = __ffma2_rn(s[k], y[i][k], q[5]);
            }
          }
        }
      }
    }
    st.next(t);
    constexpr int K = POST ? PRE ? 6 : 4 : 2;
    float v[6];
#pragma unroll
    for (int k = 0; k < 6; ++k) v[k] = q[k].x + q[k].y;
    if constexpr (PRE) v[0] *= st.poison;
    if constexpr (POST) v[2] *= st.poison;
    if constexpr (PRE || POST) row_sum_w(*reinterpret_cast<float(*)[K]>(v), W, wi, gi, buf, flip);
    const float sy = rsqrtf(fmaf(v[0], a.inv_d, a.eps));
    const float my = v[1] * sy * a.inv_d;                  // mean(w_pre dn yh)
    const float sf = POST ? rsqrtf(fmaf(v[2], a.inv_d, a.eps)) : 1.f;
    // mean(w_post du fh)
    const float mf = a.alpha * sf * a.inv_d * (PRE ? fmaf(sy, fmaf(-my * sy, v[5], v[4]), v[3]) : v[3]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (Co::any(i, lane, n)) {
        if constexpr (PRE) {
          float2 w[P];
          Co::weights(a.w_pre + col0, i, lane, n, w);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const float2 yh = __fmul2_rn(y[i][k], two(sy));
            G[i][k] = __ffma2_rn(two(sy), __ffma2_rn(yh, two(-my), __fmul2_rn(dn[i][k], w[k])), G[i][k]);
            apre[i][k] = __ffma2_rn(dn[i][k], yh, apre[i][k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < P; ++k) G[i][k] = __fmul2_rn(G[i][k], two(st.poison));
        }
        Co::put(reinterpret_cast<E*>(a.dx) + t * a.d + col0, i, lane, n, G[i]);
        if constexpr (BLOCK) {         // G: alpha G, alpha act w_post G (without act for a token gate's slope), df
          float2 w[P], dz[P];
          float2 slope[P];
          if constexpr (GATE == GDPA_GATE_TOKEN) act(z[i], a.sigmoid, slope);
          if constexpr (POST && !SHARED) Co::weights(a.w_post + col0, i, lane, n, w);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            G[i][k] = __fmul2_rn(G[i][k], two(a.alpha));
            if constexpr (POST) f[i][k] = __fmul2_rn(f[i][k], two(sf));
            float2 e = __fmul2_rn(G[i][k], f[i][k]);                    // alpha G fh
            if constexpr (SHARED) agate[i][k] = __fadd2_rn(agate[i][k], e);
            if constexpr (GATE != GDPA_GATE_NONE) G[i][k] = __fmul2_rn(G[i][k], z[i][k]);
            if constexpr (POST && !SHARED) {
              G[i][k] = __fmul2_rn(G[i][k], w[k]);
              apost[i][k] = GATE == GDPA_GATE_TOKEN ? __ffma2_rn(e, z[i][k], apost[i][k])
                                                    : __fadd2_rn(apost[i][k], e);
            }
            if constexpr (GATE == GDPA_GATE_TOKEN) {                    // alpha G u act'
              if constexpr (POST) e = __fmul2_rn(e, w[k]);
              dz[k] = __fmul2_rn(e, slope[k]);
            }
            if constexpr (POST) G[i][k] = __fmul2_rn(two(sf), __ffma2_rn(f[i][k], two(-mf), G[i][k]));
          }
          Co::put(reinterpret_cast<E*>(a.df) + t * a.d + col0, i, lane, n, G[i]);
          if constexpr (GATE == GDPA_GATE_TOKEN) Co::put(reinterpret_cast<E*>(a.dgate) + t * a.d + col0, i, lane, n, dz);
        }
      }
    }
  }
  if (SHARED && st.t1 > st.t0) flush();
  // the block's weight gradients: its groups in order, through shared memory (every copy has landed)
  __syncthreads();
  if (threadIdx.x == 0) a.status[blockIdx.x] = abort_s ? GDPA_ERR_TIMEOUT : GDPA_OK;
  float* sums = reinterpret_cast<float*>(smem);
  for (int which = 0; which < 2; ++which) {
    float* out = which ? a.part_pre : a.part_post;
    if (!out) continue;
    for (int r = 0; r < (int)blockDim.x / 32 / W; ++r) {
      if (gi == r)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (Co::any(i, lane, n)) {
            float2 v[P];
            if (SHARED && !which) {
              Co::each_at(spost, i, lane, n, v);
            } else {
#pragma unroll
              for (int k = 0; k < P; ++k) v[k] = which ? apre[i][k] : apost[SHARED ? 0 : i][k];
            }
            Co::sums(sums + col0, i, lane, n, v, [&](float x, float y) { return r == 0 ? y : x + y; });
          }
        }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) out[(int64_t)blockIdx.x * a.d + c] = sums[c];
    __syncthreads();
  }
}

struct Kernel {
  void (*fn)(const NormArgs, int);
  std::atomic<uint64_t>* allowed;     // devices that have its shared memory allowed
};
template <void (*FN)(const NormArgs, int)>
Kernel entry() {
  static std::atomic<uint64_t> allowed{0};
  return {FN, &allowed};
}

// WARPS = 0: forward
template <typename E, int NV, int WARPS, bool AL, bool PRE, bool POST, int GATE>
Kernel kernel_of() {
  if constexpr (WARPS > 0)
    return entry<norm_stream_bwd_kernel<E, NV, WARPS, AL, true, PRE, POST, GATE>>();
  else
    return entry<norm_stream_fwd_kernel<E, NV, AL, true, POST, GATE>>();
}
template <typename E, int NV, int WARPS, bool AL, bool PRE, bool POST>
Kernel kernel_of(const NormArgs& a) {
  if (a.gate_kind == GDPA_GATE_TOKEN) return kernel_of<E, NV, WARPS, AL, PRE, POST, GDPA_GATE_TOKEN>();
  if (a.gate_kind == GDPA_GATE_SAMPLE) return kernel_of<E, NV, WARPS, AL, PRE, POST, GDPA_GATE_SAMPLE>();
  return kernel_of<E, NV, WARPS, AL, PRE, POST, GDPA_GATE_NONE>();
}
template <typename E, int NV, int WARPS, bool AL>
Kernel kernel_of(const NormArgs& a) {
  if (!a.f) {
    if constexpr (WARPS > 0)
      return entry<norm_stream_bwd_kernel<E, NV, WARPS, AL, false, true, false, GDPA_GATE_NONE>>();
    else
      return entry<norm_stream_fwd_kernel<E, NV, AL, false, false, GDPA_GATE_NONE>>();
  }
  if constexpr (WARPS > 0)            // (forward, n is a test beside the row's sum)
    if (!a.w_pre)
      return a.w_post ? kernel_of<E, NV, WARPS, AL, false, true>(a)
                      : kernel_of<E, NV, WARPS, AL, false, false>(a);
  return a.w_post ? kernel_of<E, NV, WARPS, AL, true, true>(a) : kernel_of<E, NV, WARPS, AL, true, false>(a);
}

template <typename E, bool AL>
Kernel dispatch(const NormArgs& a, const StreamPlan& p, bool backward) {
  if (!backward)
    return p.nv == kMaxFwd ? kernel_of<E, kMaxFwd, 0, AL>(a) : kernel_of<E, kMaxFwd / 2, 0, AL>(a);
  if (p.warps > kWarpsBwd) return kernel_of<E, kMaxBwd, kWarpsWide, AL>(a);
  return p.nv == kMaxBwd ? kernel_of<E, kMaxBwd, kWarpsBwd, AL>(a) : kernel_of<E, kMaxBwd / 2, kWarpsBwd, AL>(a);
}

}  // namespace

StreamPlan stream_plan(int64_t T, int d, int dtype, bool backward, int gate_kind) {
  StreamPlan p = {};
  const int tensors = (backward ? 4 : 2) + (gate_kind == GDPA_GATE_TOKEN ? 1 : 0);   // at most
  const int es = dtype == GDPA_DTYPE_BF16 ? 2 : 4, vec = 16 / es;
  const bool aligned = d % vec == 0;
  // Narrow rows fill few lanes of a warp: many of them are quicker in the registers' form, which puts several
  // into a warp (14 k bf16 rows of 64 forward 4.3 us and streamed 8.6, of 130 already 21 and 11).  Backward, registers
  // and streamed, token gate, bf16: rows of 64 14.7 and 8.1 us at 500 rows, 16.9 and 14.9 at 8 k, 19.6 and 21.1 at
  // 16 k, 30.2 and 58.1 at 64 k; rows of 100 are quicker streamed at every length (32.8 and 25.7 at 16 k).  Wider
  // rows are too (64 rows of 1024 4.0 and 3.9 us, 14 k 37 and 29).
  if (d < 128 && (!backward || T > 8192)) return p;
  const int most = backward ? kMaxBwd : kMaxFwd;
  int nv = most / 2;
  while (nv < most && nv * 32 * vec < d) nv *= 2;
  const int w = (d + nv * 32 * vec - 1) / (nv * 32 * vec);
  const int most_warps = !backward ? kWarpsFwd : w <= kWarpsBwd ? kWarpsBwd : kWarpsWide;
  const int warps = most_warps / w * w;
  if (warps == 0) return p;
  int64_t groups = (int64_t)device_sm_count() * (warps / w);
  if (groups > T) groups = T;
  const uint32_t row = (uint32_t)(nv * 32 * vec * es + (aligned ? 0 : 32)) * tensors * warps;   // of every warp
  p.nv = nv;
  p.warps_row = w;
  p.warps = warps;
  p.groups = (int)groups;
  p.blocks = (int)((groups + warps / w - 1) / (warps / w));
  p.smem = (size_t)kStages * row;
  if (backward && p.smem < (size_t)d * 4) p.smem = (size_t)d * 4;
  if (backward && gate_kind == GDPA_GATE_SAMPLE) p.smem += (size_t)warps * nv * 32 * vec * 4;   // w_post's sums
  return p;
}

cudaError_t launch_norm_stream(const NormArgs& a, const StreamPlan& p, int dtype, bool backward,
                               cudaStream_t st) {
  const bool bf16 = dtype == GDPA_DTYPE_BF16, aligned = a.d % (bf16 ? 8 : 4) == 0;
  const Kernel kern = bf16 ? aligned ? dispatch<__nv_bfloat16, true>(a, p, backward)
                               : dispatch<__nv_bfloat16, false>(a, p, backward)
                     : aligned ? dispatch<float, true>(a, p, backward)
                               : dispatch<float, false>(a, p, backward);
  const cudaError_t e = allow_smem(kern.fn, (int)kRingBytes + 32 * 1024, *kern.allowed);
  if (e != cudaSuccess) return e;
  KernelScope ks_(backward ? "gdpa_block_norm_bwd" : "gdpa_block_norm_fwd", st);
  kern.fn<<<p.blocks, p.warps * 32, p.smem, st>>>(a, p.warps_row);
  return cudaGetLastError();
}

}  // namespace gdpa
