// Shared by the block norm's kernels (block_norm.cu: any width, rows in registers;
// block_norm_stream.cu: rows streamed through shared memory).
#pragma once

#include "layer_launch.cuh"

namespace gdpa {

struct NormArgs {
  const void *x, *f, *gate;      // backward: x is the forward's y
  const float *w_post, *w_pre;
  const int32_t* offsets;        // sample gates: [B + 1]
  void *y, *n;                   // forward outputs
  const void *dy, *dn;           // backward inputs
  void *dx, *df, *dgate;         // backward outputs (dgate: token gates)
  float* dgate_sample;           // [B, d] (sample gates)
  float *part_post, *part_pre;   // [blocks, d] partial weight gradients
  float* part_gate;              // [groups, 2, d] partial sample-gate gradients
  int32_t* status;               // [blocks] (streamed backward): GDPA_OK or GDPA_ERR_TIMEOUT
  int64_t T;
  int64_t lost_row;              // -1; the self-test of the waits: a row of the group whose first row does not arrive
  uint64_t wait_ns;              // limit of a wait
  int d, B, groups;
  float alpha, eps, inv_d;
  int gate_kind, sigmoid;
};

// 1 / (1 + exp(-z)): the product's rounding moves the exponential by 2^-24 |z log2 e| relatively, ex2 and
// the reciprocal are off by 2^-22 and 2^-23; no denormals (a value below 2^-126 is 0)
__device__ __forceinline__ float logistic(float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// act(z) and act'(z).  From t = exp(-|z|), so that the slope keeps its relative precision where act is close
// to 1 (act (1 - act) of a rounded act loses it).
__device__ __forceinline__ void gate_slope(float z, int sigmoid, float& act, float& slope) {
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fabsf(z) * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
  const float s = t * r;                     // 1 / (1 + exp(|z|))
  act = sigmoid ? (z >= 0.f ? r : s) : z;
  slope = sigmoid ? s * r : 1.f;
}

// VEC consecutive elements of a row as floats (VEC * sizeof(E) = 16, or one element)
template <typename E, int VEC> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    r = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + i));
  }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p) + i) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Raw<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    r = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i));
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = r.x;
    f[1] = r.y;
    f[2] = r.z;
    f[3] = r.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* f) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i) =
        make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <typename E> struct Raw<E, 1> {
  E r;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    r = __ldg(reinterpret_cast<const E*>(p) + i);
  }
  __device__ __forceinline__ void get(float* f) const { f[0] = Elem<E>::to_f(r); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* f) {
    reinterpret_cast<E*>(p)[i] = Elem<E>::from_f(f[0]);
  }
};

// VEC fp32 weights from column `col` on (1 without weights); they stay in L1 between rows.
template <int VEC>
__device__ __forceinline__ void weights(const float* w, int col, float (&f)[VEC]) {
  if (!w) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = 1.f;
  } else if constexpr (VEC == 1) {
    f[0] = __ldg(w + col);
  } else {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + col + k));
      f[k] = v.x;
      f[k + 1] = v.y;
      f[k + 2] = v.z;
      f[k + 3] = v.w;
    }
  }
}

// First row of group g of a call with `groups` groups over T rows.
__host__ __device__ __forceinline__ int64_t group_row(int64_t T, int groups, int g) {
  return T * g / groups;
}
// The group that holds row t.
__device__ __forceinline__ int row_group(int64_t T, int groups, int64_t t) {
  int g = (int)(((t + 1) * groups - 1) / T);
  while (g > 0 && group_row(T, groups, g) > t) --g;
  while (g + 1 < groups && group_row(T, groups, g + 1) <= t) ++g;
  return g;
}

// Sample of row t: the largest b with offsets[b] <= t (B when behind the last, -1 before the first).
__device__ __forceinline__ int sample_of(const int32_t* offsets, int B, int64_t t) {
  int lo = -1, hi = B;          // offsets[lo] <= t < offsets[hi + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)__ldg(offsets + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Walks a group's rows keeping the sample of the current row.
struct SampleWalk {
  int b;
  int64_t next;                  // first row of the next sample
  __device__ __forceinline__ void seek(const NormArgs& a, int64_t t) {
    b = sample_of(a.offsets, a.B, t);
    next = b >= a.B ? (int64_t)1 << 62 : (int64_t)__ldg(a.offsets + b + 1);
  }
  // returns true when the sample changed
  __device__ __forceinline__ bool at(const NormArgs& a, int64_t t) {
    if (t < next) return false;
    seek(a, t);
    return true;
  }
  __device__ __forceinline__ bool live(const NormArgs& a) const { return b >= 0 && b < a.B; }
};

// How a call of the streaming kernels is cut (nv = 0: they do not take it).
struct StreamPlan {
  int nv, warps_row, warps, groups, blocks;
  size_t smem;
};
StreamPlan stream_plan(int64_t T, int d, int dtype, bool backward, int gate_kind);
cudaError_t launch_norm_stream(const NormArgs& a, const StreamPlan& p, int dtype, bool backward,
                               cudaStream_t st);

}  // namespace gdpa
