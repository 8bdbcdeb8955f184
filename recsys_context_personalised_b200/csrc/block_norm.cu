// Norms before and after a block, fused with its gate and residual scale.
//
// Forward, per row (token) of width d:
//   u = w_post f / rms(f)  (or f),  y = x + alpha act(gate) u,  n = w_pre y / rms(y)
// with rms(v) = sqrt(mean(v^2) + eps) and act the identity or the logistic.
// Backward, for dy and dn:
//   G = dy + r_y (w_pre dn - yh mean(w_pre dn yh)),  yh = y r_y,  r = 1 / rms
//   dx = G,  du = alpha act(gate) G,  dgate = alpha act'(gate) G u
//   df = r_f (w_post du - fh mean(w_post du fh)),    fh = f r_f
//   dw_pre = sum_t dn yh,  dw_post = sum_t du fh
//
// This file has the entry points and the form that keeps rows in registers, for many narrow rows and very
// wide fp32 ones; block_norm_stream.cu has the form for all others.
//
// Bound: memory, every row once.  A row is spread over TPR threads that keep
// it in registers (NV vectors of VEC elements each) between its two
// reductions.  A group of TPR threads walks a contiguous range of rows, with the
// next row's loads issued before the current row's reductions; the weights'
// and a sample-shared gate's gradients accumulate in fp32 registers over the
// range and go to the workspace once, where a second kernel adds them up in a
// fixed order (no atomics: the same inputs give the same bits).
//
// n is taken from the unrounded y; all sums and statistics are fp32.
#include <math.h>
#include <stdio.h>

#include "block_norm.cuh"

namespace gdpa {
namespace {

// Sums of K values over the TPR threads of a row (every thread gets them).
// Rows that span warps pass through shared memory; `buf` alternates between
// two halves so that one __syncthreads per reduction is enough.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int tpr, float* buf, int& flip) {
#pragma unroll
  for (int k = 0; k < K; ++k)
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (tpr <= 32) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* b = buf + flip * 64;
  flip ^= 1;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) b[warp * K + k] = v[k];
  __syncthreads();
  const int w0 = (threadIdx.x / tpr) * (tpr >> 5), nw = tpr >> 5;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int i = 0; i < nw; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += b[(w0 + i) * K + k];
}

template <typename E, int VEC, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_fwd_kernel(const NormArgs a, int tpr) {
  __shared__ float buf[128];
  int flip = 0;
  using R = Raw<E, VEC>;
  const int rpb = blockDim.x / tpr, gi = threadIdx.x / tpr, tid = threadIdx.x - gi * tpr;
  const int g = blockIdx.x * rpb + gi;
  const bool mine = g < a.groups;
  int64_t t = mine ? group_row(a.T, a.groups, g) : 0;
  const int64_t t1 = mine ? group_row(a.T, a.groups, g + 1) : 0;
  // every group of a block takes the same number of steps (the reductions synchronise the block)
  const int64_t steps = (a.T + a.groups - 1) / a.groups;
  int col[NV];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * tpr + tid) * VEC;
    in[i] = col[i] < a.d;
  }
  float gs[NV][VEC];             // act(gate): of this row, or of this sample
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) gs[i][k] = 1.f;
  R rx[NV] = {}, rf[NV] = {}, rg[NV] = {};
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i] && row < t1) {
        rx[i].load(a.x, row * a.d + col[i]);
        if (a.f) rf[i].load(a.f, row * a.d + col[i]);
        if (a.gate_kind == GDPA_GATE_TOKEN) rg[i].load(a.gate, row * a.d + col[i]);
      }
  };
  SampleWalk walk;
  walk.next = -1;
  walk.b = 0;
  fetch(t);
  for (int64_t s = 0; s < steps; ++s, ++t) {
    float x[NV][VEC], f[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i].get(x[i]);
      rf[i].get(f[i]);
      if (a.gate_kind == GDPA_GATE_TOKEN) {
        rg[i].get(gs[i]);
        if (a.sigmoid)
#pragma unroll
          for (int k = 0; k < VEC; ++k) gs[i][k] = logistic(gs[i][k]);
      }
    }
    bool live = t < t1;
    fetch(t + 1);
    if (a.f) {
      float scale = 1.f;
      if (a.w_post) {
        float v[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < VEC; ++k)
            if (in[i]) v[0] = fmaf(f[i][k], f[i][k], v[0]);
        row_sum(v, tpr, buf, flip);
        scale = 1.f / sqrtf(fmaf(v[0], a.inv_d, a.eps));
      }
      if (a.gate_kind == GDPA_GATE_SAMPLE && live) {
        if (walk.at(a, t) && walk.live(a)) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (in[i]) {
              R r;
              r.load(a.gate, (int64_t)walk.b * a.d + col[i]);
              r.get(gs[i]);
              if (a.sigmoid)
#pragma unroll
                for (int k = 0; k < VEC; ++k) gs[i][k] = logistic(gs[i][k]);
            }
        }
        live = walk.live(a);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i]) {
          float w[VEC];
          weights<VEC>(a.w_post, col[i], w);
#pragma unroll
          for (int k = 0; k < VEC; ++k)
            x[i][k] = fmaf(a.alpha * gs[i][k], f[i][k] * scale * w[k], x[i][k]);
        }
      if (live)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (in[i]) R::store(a.y, t * a.d + col[i], x[i]);
    }
    if (a.w_pre) {
      float v[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if (in[i]) v[0] = fmaf(x[i][k], x[i][k], v[0]);
      row_sum(v, tpr, buf, flip);
      const float scale = 1.f / sqrtf(fmaf(v[0], a.inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i] && live) {
          float w[VEC];
          weights<VEC>(a.w_pre, col[i], w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) x[i][k] *= scale * w[k];
          R::store(a.n, t * a.d + col[i], x[i]);
        }
    }
  }
}

template <typename E, int VEC, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_kernel(const NormArgs a, int tpr) {
  pdl_trigger();
  __shared__ float buf[128];
  int flip = 0;
  using R = Raw<E, VEC>;
  const int rpb = blockDim.x / tpr, gi = threadIdx.x / tpr, tid = threadIdx.x - gi * tpr;
  const int g = blockIdx.x * rpb + gi;
  const bool mine = g < a.groups;
  const int64_t t0 = mine ? group_row(a.T, a.groups, g) : 0;
  const int64_t t1 = mine ? group_row(a.T, a.groups, g + 1) : 0;
  const int64_t steps = (a.T + a.groups - 1) / a.groups;
  int col[NV];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * tpr + tid) * VEC;
    in[i] = col[i] < a.d;
  }
  float apost[NV][VEC], apre[NV][VEC], agate[NV][VEC], gs[NV][VEC], slope[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      apost[i][k] = apre[i][k] = agate[i][k] = 0.f;
      gs[i][k] = slope[i][k] = 1.f;
    }
  R ry[NV] = {}, rf[NV] = {}, rz[NV] = {}, rdy[NV] = {}, rdn[NV] = {};
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i] && row < t1) {
        const int64_t at = row * a.d + col[i];
        if (a.w_pre) {
          ry[i].load(a.x, at);
          rdn[i].load(a.dn, at);
        }
        if (a.dy) rdy[i].load(a.dy, at);
        if (a.f) rf[i].load(a.f, at);
        if (a.gate_kind == GDPA_GATE_TOKEN) rz[i].load(a.gate, at);
      }
  };
  SampleWalk walk;
  walk.next = -1;
  walk.b = 0;
  // the rows of sample walk.b that this group holds are done: their gate gradient
  // goes out whole, or as a piece (slot 1 when it holds the sample's first row)
  auto flush = [&]() {
    if (!walk.live(a)) return;
    const int64_t lo = max((int64_t)__ldg(a.offsets + walk.b), (int64_t)0);
    const int64_t hi = min(walk.next, a.T);
    float* out;
    if (lo >= t0 && hi <= t1)
      out = a.dgate_sample + (int64_t)walk.b * a.d;
    else
      out = a.part_gate + ((int64_t)g * 2 + (lo >= t0 ? 1 : 0)) * a.d;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i])
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          out[col[i] + k] = agate[i][k] * slope[i][k] * a.alpha;
          agate[i][k] = 0.f;
        }
  };
  fetch(t0);
  int64_t t = t0;
  for (int64_t s = 0; s < steps; ++s, ++t) {
    float y[NV][VEC], f[NV][VEC], G[NV][VEC], dn[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ry[i].get(y[i]);
      rf[i].get(f[i]);
      rdy[i].get(G[i]);
      rdn[i].get(dn[i]);
      if (a.gate_kind == GDPA_GATE_TOKEN) {
        rz[i].get(gs[i]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) gate_slope(gs[i][k], a.sigmoid, gs[i][k], slope[i][k]);
      }
    }
    bool live = t < t1;
    fetch(t + 1);
    if (a.gate_kind == GDPA_GATE_SAMPLE && live) {
      if (t >= walk.next) {
        if (s > 0) flush();
        walk.seek(a, t);
        if (walk.live(a))
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (in[i]) {
              R r;
              r.load(a.gate, (int64_t)walk.b * a.d + col[i]);
              r.get(gs[i]);
#pragma unroll
              for (int k = 0; k < VEC; ++k) gate_slope(gs[i][k], a.sigmoid, gs[i][k], slope[i][k]);
            }
      }
      live = walk.live(a);
    }
    // sums of y^2, w_pre dn y and f^2 (a row that is not live adds nothing anywhere)
    float v[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) {
        float w[VEC];
        weights<VEC>(a.w_pre, col[i], w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          v[0] = fmaf(y[i][k], y[i][k], v[0]);
          v[1] = fmaf(dn[i][k] * w[k], y[i][k], v[1]);
          v[2] = fmaf(f[i][k], f[i][k], v[2]);
        }
      }
    row_sum(v, tpr, buf, flip);
    const float sy = 1.f / sqrtf(fmaf(v[0], a.inv_d, a.eps));
    const float my = v[1] * sy * a.inv_d;                  // mean(w_pre dn yh)
    const float sf = a.w_post ? 1.f / sqrtf(fmaf(v[2], a.inv_d, a.eps)) : 1.f;
    float m2[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      if (a.w_pre) {
        float w[VEC];
        weights<VEC>(a.w_pre, col[i], w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float yh = y[i][k] * sy;
          G[i][k] = fmaf(sy, fmaf(-yh, my, dn[i][k] * w[k]), G[i][k]);
          if (live) apre[i][k] = fmaf(dn[i][k], yh, apre[i][k]);
        }
      }
      if (a.w_post) {
        float w[VEC];
        weights<VEC>(a.w_post, col[i], w);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          f[i][k] *= sf;                                   // fh
          const float du = a.alpha * gs[i][k] * G[i][k];
          if (live) apost[i][k] = fmaf(du, f[i][k], apost[i][k]);
          m2[0] = fmaf(du * w[k], f[i][k], m2[0]);
        }
      }
    }
    if (a.w_post) row_sum(m2, tpr, buf, flip);
    const float mf = m2[0] * a.inv_d;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!in[i]) continue;
      const int64_t at = t * a.d + col[i];
      R::store(a.dx, at, G[i]);
      if (!a.f) continue;
      float dz[VEC], w[VEC];
      weights<VEC>(a.w_post, col[i], w);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float gu = G[i][k] * f[i][k] * w[k];          // G u
        dz[k] = a.alpha * gu * slope[i][k];
        if (a.gate_kind == GDPA_GATE_SAMPLE) agate[i][k] += gu;
        const float wd = w[k] * (a.alpha * gs[i][k] * G[i][k]);
        f[i][k] = a.w_post ? sf * fmaf(-f[i][k], mf, wd) : wd;
      }
      R::store(a.df, at, f[i]);
      if (a.gate_kind == GDPA_GATE_TOKEN) R::store(a.dgate, at, dz);
    }
  }
  if (a.gate_kind == GDPA_GATE_SAMPLE && t1 > t0) {
    // the last sample of the range (its rows end here, or go on in the next group)
    flush();
  }
  // the block's weight gradients: its groups in order, through shared memory
  extern __shared__ float sums[];
  for (int which = 0; which < 2; ++which) {
    float* out = which ? a.part_pre : a.part_post;
    if (!out) continue;
    for (int r = 0; r < rpb; ++r) {
      if (gi == r)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (in[i])
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
              const float v = which ? apre[i][k] : apost[i][k];
              if (r == 0) sums[col[i] + k] = v; else sums[col[i] + k] += v;
            }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.d; c += blockDim.x)
      out[(int64_t)blockIdx.x * a.d + c] = sums[c];
    __syncthreads();
  }
}

// Adds up the partial weight gradients (blockIdx.y = 0: post, 1: pre), 32 columns to a block of
// 32 x 32 threads, and (blockIdx.y = 2) joins the pieces of the sample gates' gradients.  The first block also
// takes the streamed blocks' status words together into the workspace's.
__global__ void __launch_bounds__(1024)
norm_join_kernel(const NormArgs a, float* dw_post, float* dw_pre, int blocks, WsHeader* ws) {
  __shared__ float s[32][33];
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int worst = GDPA_OK;
    if (a.status)
      for (int i = threadIdx.x; i < blocks; i += blockDim.x) worst |= a.status[i];
    worst = __syncthreads_or(worst);
    if (threadIdx.x == 0) ws->status = worst ? GDPA_ERR_TIMEOUT : GDPA_OK;
  }
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  if (blockIdx.y < 2) {
    const float* part = blockIdx.y ? a.part_pre : a.part_post;
    float* out = blockIdx.y ? dw_pre : dw_post;
    if (!part) return;
    for (int c0 = blockIdx.x * 32; c0 < a.d; c0 += gridDim.x * 32) {
      const int c = c0 + tx;
      float v = 0.f;
      if (c < a.d)
        for (int r = ty; r < blocks; r += 32) v += part[(int64_t)r * a.d + c];
      s[ty][tx] = v;
      __syncthreads();
      if (ty == 0 && c < a.d) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) sum += s[r][tx];
        out[c] = sum;
      }
      __syncthreads();
    }
    return;
  }
  if (a.gate_kind != GDPA_GATE_SAMPLE) return;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int64_t lo = max((int64_t)__ldg(a.offsets + b), (int64_t)0);
    const int64_t hi = min((int64_t)__ldg(a.offsets + b + 1), a.T);
    if (hi <= lo) {
      for (int c = threadIdx.x; c < a.d; c += blockDim.x)
        a.dgate_sample[(int64_t)b * a.d + c] = 0.f;
      continue;
    }
    const int g0 = row_group(a.T, a.groups, lo), g1 = row_group(a.T, a.groups, hi - 1);
    if (g0 == g1) continue;                                 // written whole
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
      float v = a.part_gate[((int64_t)g0 * 2 + 1) * a.d + c];
      for (int g = g0 + 1; g <= g1; ++g) v += a.part_gate[(int64_t)g * 2 * a.d + c];
      a.dgate_sample[(int64_t)b * a.d + c] = v;
    }
  }
}

constexpr int kMaxWidth = 8192;

// How a call is cut: TPR threads to a row, rpb rows to a block, `groups` row ranges.
struct Plan {
  int vec, nv, tpr, threads, rpb, groups, blocks;
  StreamPlan stream;
};
Plan plan(int64_t T, int d, int dtype, bool backward, int gate_kind) {
  Plan p = {};
  p.stream = stream_plan(T, d, dtype, backward, gate_kind);
  if (p.stream.nv) {
    p.groups = p.stream.groups;
    p.blocks = p.stream.blocks;
    return p;
  }
  const int v16 = dtype == GDPA_DTYPE_BF16 ? 8 : 4;
  p.vec = d % v16 == 0 ? v16 : 1;
  const int nvec = d / p.vec;
  // one vector to a thread while 512 threads hold the row, and four elements to
  // a thread where they are loaded one by one
  p.nv = p.vec == 1 ? 4 : 1;
  while (p.nv * 512 < nvec) p.nv *= 2;
  p.tpr = 8;
  while (p.tpr * p.nv < nvec) p.tpr *= 2;
  p.threads = p.tpr > 256 ? p.tpr : 256;
  p.rpb = p.threads / p.tpr;
  const int64_t most = (int64_t)device_sm_count() * (backward ? 512 / p.threads : 1024 / p.threads);
  int64_t blocks = (T + p.rpb - 1) / p.rpb;
  if (blocks > most) blocks = most;
  if (blocks < 1) blocks = 1;
  p.groups = (int)(blocks * p.rpb < T ? blocks * p.rpb : T);
  p.blocks = (p.groups + p.rpb - 1) / p.rpb;
  return p;
}

// Workspace of the backward: the header, the blocks' status words and partial sums, the pieces of sample gates.
struct NormSpace {
  size_t status, post, pre, gate, total;
};
NormSpace norm_space(const Plan& p, int d, int gate_kind) {
  const size_t part = align_up((size_t)p.blocks * d * 4, 256);
  NormSpace w;
  w.status = sizeof(WsHeader);
  w.post = w.status + align_up((size_t)p.blocks * 4, 256);
  w.pre = w.post + part;
  w.gate = w.pre + part;
  w.total = w.gate + (gate_kind == GDPA_GATE_SAMPLE ? align_up((size_t)p.groups * 2 * d * 4, 256) : 0);
  return w;
}

constexpr uint64_t kNormTimeoutNs = 2000000000ull;   // 2 s per wait; a healthy wait is microseconds
// What gdpa_selftest_norm_wait has left for this thread's next call.
thread_local int64_t next_lost_row = -1;
thread_local uint64_t next_wait_ns = kNormTimeoutNs;

template <typename E, int VEC, int NV>
cudaError_t launch_fwd(const NormArgs& a, const Plan& p, cudaStream_t st) {
  KernelScope ks_("gdpa_block_norm_fwd", st);
  norm_fwd_kernel<E, VEC, NV, 512, (VEC * NV <= 8 ? 2 : 1)><<<p.blocks, p.threads, 0, st>>>(a, p.tpr);
  return cudaGetLastError();
}
template <typename E, int VEC, int NV>
cudaError_t launch_bwd(const NormArgs& a, const Plan& p, cudaStream_t st) {
  KernelScope ks_("gdpa_block_norm_bwd", st);
  norm_bwd_kernel<E, VEC, NV, 512, 1><<<p.blocks, p.threads, (size_t)a.d * 4, st>>>(a, p.tpr);
  return cudaGetLastError();
}

template <typename E, int V16>
cudaError_t dispatch(const NormArgs& a, const Plan& p, bool backward, cudaStream_t st) {
#define GDPA_NORM(VEC, NV) \
  return backward ? launch_bwd<E, VEC, NV>(a, p, st) : launch_fwd<E, VEC, NV>(a, p, st)
  // (what stream_plan leaves: rows narrower than 128, and fp32 rows beyond 4,096)
  if (p.vec == 1 && p.nv == 4) GDPA_NORM(1, 4);
  if (p.vec > 1 && p.nv == 1) GDPA_NORM(V16, 1);
  if constexpr (V16 == 4) {
    if (p.vec == 1) GDPA_NORM(1, 16);
    GDPA_NORM(4, 4);
  }
  return cudaErrorInvalidValue;
#undef GDPA_NORM
}

gdpa_status_t check_norm(const gdpa_block_norm_t* p) {
  if (!p) return GDPA_ERR_INVALID_ARG;
  if (p->dtype != GDPA_DTYPE_F32 && p->dtype != GDPA_DTYPE_BF16) return GDPA_ERR_INVALID_ARG;
  if (p->T < 0 || p->T >= (int64_t)1 << 31 || p->d < 1) return GDPA_ERR_INVALID_ARG;
  if (p->gate < GDPA_GATE_NONE || p->gate > GDPA_GATE_SAMPLE) return GDPA_ERR_INVALID_ARG;
  if (p->gate == GDPA_GATE_SAMPLE && p->B < 1) return GDPA_ERR_INVALID_ARG;
  if (!(p->alpha - p->alpha == 0.f) || !(p->eps >= 0.f) || !(p->eps - p->eps == 0.f))
    return GDPA_ERR_INVALID_ARG;
  if (p->d > kMaxWidth) return GDPA_ERR_UNSUPPORTED;
  return GDPA_OK;
}

bool off16(const void* p) { return ((uintptr_t)p & 15u) != 0; }
bool off4(const void* p) { return ((uintptr_t)p & 3u) != 0; }

gdpa_status_t finish(cudaError_t e) {
  if (e == cudaSuccess) return GDPA_OK;
  fprintf(stderr, "gdpa: CUDA error %d (%s)\n", (int)e, cudaGetErrorString(e));
  return GDPA_ERR_CUDA;
}

NormArgs base_args(const gdpa_block_norm_t* p) {
  NormArgs a = {};
  a.T = p->T;
  a.d = p->d;
  a.B = p->B;
  a.alpha = p->alpha;
  a.eps = p->eps;
  a.inv_d = 1.f / (float)p->d;
  a.gate_kind = p->gate;
  a.sigmoid = p->sigmoid != 0;
  a.lost_row = next_lost_row;
  a.wait_ns = next_wait_ns;
  next_lost_row = -1;
  next_wait_ns = kNormTimeoutNs;
  return a;
}

}  // namespace
}  // namespace gdpa

using namespace gdpa;

extern "C" gdpa_status_t gdpa_block_norm_fwd(const gdpa_block_norm_t* p, const int32_t* offsets,
                                             const void* x, const void* f, const void* gate,
                                             const float* w_post, const float* w_pre, void* y,
                                             void* n, void* stream) {
  reset_launch_count();
  gdpa_status_t s = check_norm(p);
  if (s != GDPA_OK) return s;
  const bool empty = p->T == 0;
  // (tensors without rows have no address)
  if (!empty && !f && (p->gate != GDPA_GATE_NONE || w_post || y)) return GDPA_ERR_INVALID_ARG;
  if (!empty && !f && !w_pre) return GDPA_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != (n != nullptr) && !empty) return GDPA_ERR_INVALID_ARG;
  if (!empty && (!x || (f && !y))) return GDPA_ERR_INVALID_ARG;
  if ((p->gate != GDPA_GATE_NONE) != (gate != nullptr) && !empty) return GDPA_ERR_INVALID_ARG;
  if (p->gate == GDPA_GATE_SAMPLE && !offsets) return GDPA_ERR_INVALID_ARG;
  if (off16(x) || off16(f) || off16(gate) || off16(y) || off16(n) || off16(w_post) || off16(w_pre) ||
      off4(offsets))
    return GDPA_ERR_INVALID_ARG;
  if (empty) return GDPA_OK;
  NormArgs a = base_args(p);
  a.x = x;
  a.f = f;
  a.gate = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.offsets = offsets;
  a.y = y;
  a.n = n;
  const Plan pl = plan(p->T, p->d, p->dtype, false, p->gate);
  a.groups = pl.groups;
  const cudaStream_t st = (cudaStream_t)stream;
  if (pl.stream.nv) return finish(launch_norm_stream(a, pl.stream, p->dtype, false, st));
  return finish(p->dtype == GDPA_DTYPE_BF16 ? dispatch<__nv_bfloat16, 8>(a, pl, false, st)
                                            : dispatch<float, 4>(a, pl, false, st));
}

extern "C" gdpa_status_t gdpa_block_norm_bwd_workspace_size(const gdpa_block_norm_t* p,
                                                            size_t* bytes) {
  const gdpa_status_t s = check_norm(p);
  if (s != GDPA_OK) return s;
  if (!bytes) return GDPA_ERR_INVALID_ARG;
  *bytes = norm_space(plan(p->T, p->d, p->dtype, true, p->gate), p->d, p->gate).total;
  return GDPA_OK;
}

extern "C" gdpa_status_t gdpa_block_norm_bwd(const gdpa_block_norm_t* p, const int32_t* offsets,
                                             const void* y, const void* f, const void* gate,
                                             const float* w_post, const float* w_pre,
                                             const void* dy, const void* dn, void* dx, void* df,
                                             void* dgate, float* dw_post, float* dw_pre,
                                             void* workspace, size_t workspace_bytes,
                                             void* stream) {
  reset_launch_count();
  gdpa_status_t s = check_norm(p);
  if (s != GDPA_OK) return s;
  const bool empty = p->T == 0;
  if (!empty && !f && (p->gate != GDPA_GATE_NONE || w_post || df)) return GDPA_ERR_INVALID_ARG;
  if (!empty && !f && !w_pre) return GDPA_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != (dw_pre != nullptr) || (w_post != nullptr) != (dw_post != nullptr))
    return GDPA_ERR_INVALID_ARG;
  if (!empty) {
    if (!dx || (f && !df) || (w_pre && (!y || !dn)) || (!w_pre && !dy)) return GDPA_ERR_INVALID_ARG;
    if ((p->gate != GDPA_GATE_NONE) != (gate != nullptr)) return GDPA_ERR_INVALID_ARG;
    if (p->gate == GDPA_GATE_TOKEN && !dgate) return GDPA_ERR_INVALID_ARG;
  }
  if (p->gate == GDPA_GATE_SAMPLE && (!offsets || !dgate)) return GDPA_ERR_INVALID_ARG;
  if (off16(y) || off16(f) || off16(gate) || off16(dy) || off16(dn) || off16(dx) || off16(df) ||
      off16(dgate) || off16(w_post) || off16(w_pre) || off4(dw_post) || off4(dw_pre) || off4(offsets))
    return GDPA_ERR_INVALID_ARG;
  const Plan pl = plan(p->T, p->d, p->dtype, true, p->gate);
  const NormSpace space = norm_space(pl, p->d, p->gate);
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < space.total) return GDPA_ERR_WORKSPACE;
  const cudaStream_t st = (cudaStream_t)stream;
  if (empty) {
    cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(WsHeader), st);
    if (e == cudaSuccess && dw_post) e = cudaMemsetAsync(dw_post, 0, (size_t)p->d * 4, st);
    if (e == cudaSuccess && dw_pre) e = cudaMemsetAsync(dw_pre, 0, (size_t)p->d * 4, st);
    if (e == cudaSuccess && p->gate == GDPA_GATE_SAMPLE)
      e = cudaMemsetAsync(dgate, 0, (size_t)p->B * p->d * 4, st);
    return finish(e);
  }
  NormArgs a = base_args(p);
  a.x = y;
  a.f = f;
  a.gate = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.offsets = offsets;
  a.dy = dy;
  a.dn = dn;
  a.dx = dx;
  a.df = df;
  if (p->gate == GDPA_GATE_SAMPLE)
    a.dgate_sample = (float*)dgate;
  else
    a.dgate = dgate;
  a.groups = pl.groups;
  char* const ws = (char*)workspace;
  a.status = pl.stream.nv ? (int32_t*)(ws + space.status) : nullptr;
  a.part_post = w_post ? (float*)(ws + space.post) : nullptr;
  a.part_pre = w_pre ? (float*)(ws + space.pre) : nullptr;
  a.part_gate = (float*)(ws + space.gate);
  cudaError_t e = pl.stream.nv ? launch_norm_stream(a, pl.stream, p->dtype, true, st)
                  : p->dtype == GDPA_DTYPE_BF16 ? dispatch<__nv_bfloat16, 8>(a, pl, true, st)
                                                : dispatch<float, 4>(a, pl, true, st);
  if (e == cudaSuccess) {
    KernelScope ks_("gdpa_block_norm_join", st);
    const int cols = w_post || w_pre ? (p->d + 31) / 32 : 1;
    const int rows = p->gate == GDPA_GATE_SAMPLE ? (p->B < 1024 ? p->B : 1024) : 0;
    e = launch_dependent(norm_join_kernel,
                         dim3(cols > rows ? cols : rows, p->gate == GDPA_GATE_SAMPLE ? 3 : 2), dim3(1024),
                         st, a, dw_post, dw_pre, pl.blocks, (WsHeader*)workspace);
  }
  return finish(e);
}

extern "C" gdpa_status_t gdpa_selftest_norm_wait(int64_t row, uint32_t timeout_us) {
  if (row < 0 || timeout_us == 0 || timeout_us > 5000000u) return GDPA_ERR_INVALID_ARG;
  next_lost_row = row;
  next_wait_ns = 1000ull * timeout_us;
  return GDPA_OK;
}
