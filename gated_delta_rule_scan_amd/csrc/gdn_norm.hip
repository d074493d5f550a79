// The seam between two blocks: norm of the block's output, gate, residual, norm
// for the next block; and its gradients.
//
// Per row, with r(z) = 1 / sqrt(mean z^2 + eps), y^ = y r(y), h^ = h r(h):
//
//   u = wp y^ (or y),  h = alpha x + g u,  n = w h^
//
//   dH  = dh + r(h) (w dn - h^ mean(w dn h^))         the gradient of h
//   dx  = alpha dH,  dg = sum dH u,  dw = sum dn h^
//   dy  = r(y) (b - y^ mean(b y^)), b = wp g dH (or dy = g dH),  dwp = sum g dH y^
//
// Memory-bound: four rows a token forward, six backward.  A row stays in
// registers between its reductions, 8 or 16 channels a lane over one, four or
// sixteen waves; parameters and the sums over rows stay in registers over all
// of a workgroup's rows.  Those sums go to the workspace, one partial each per
// workgroup, and a second kernel adds them in a fixed order.
#include "gdn_layer.h"

namespace gdn {
namespace {

// Sum over a wave, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// WAVES waves per row, E channels per lane in vectors of VEC.
template <typename MT, int WAVES, int E, int VEC>
struct Lanes {
  static constexpr int kRows = WAVES < 4 ? 4 / WAVES : 1;  // rows of a workgroup at a time
  static constexpr int kThreads = WAVES * kRows * 64;
  static constexpr int kWidth = WAVES * 64 * E;
  int64_t D;
  int col0;  // the lane's first channel
  float* red;
  int phase = 0;

  __device__ __forceinline__ int col(int v) const { return v * WAVES * 64 * VEC + col0; }

  template <typename T>
  __device__ __forceinline__ void load(const T* p, float (&x)[E]) const {
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
      T t[VEC];
      if (col(v) < D) {
        __builtin_memcpy(t, __builtin_assume_aligned(p + col(v), VEC * sizeof(T) < 16 ? VEC * sizeof(T) : 16), sizeof(t));
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[v * VEC + e] = (float)t[e];
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[v * VEC + e] = 0.0f;
      }
    }
  }
  // parameters: fp32, aligned to their type only
  __device__ __forceinline__ void param(const float* p, float (&x)[E], float none) const {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = col(i / VEC) + i % VEC;
      x[i] = p && c < D ? p[c] : none;
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&x)[E]) const {
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
      if (col(v) >= D) continue;
      T t[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) t[e] = (T)x[v * VEC + e];
      __builtin_memcpy(__builtin_assume_aligned(p + col(v), VEC * sizeof(T) < 16 ? VEC * sizeof(T) : 16), t, sizeof(t));
    }
  }
  // K sums over the row, in all its lanes.  Several waves join theirs in LDS;
  // two buffers in turn, so that one barrier a call is enough.
  template <int K>
  __device__ __forceinline__ void sum(float (&s)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = wave_sum(s[k]);
    if constexpr (WAVES > 1) {
      float* buf = red + phase * (2 * WAVES);
      phase ^= 1;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[k * WAVES + (threadIdx.x >> 6)] = s[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        s[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s[k] += buf[k * WAVES + w];
      }
    }
  }
};

// The rows of a workgroup: a run of one sequence's, or rows of no sequence.
struct Run {
  SeqItem s;
  int64_t t0, t1;   // rows of the run
  int64_t limit;    // ... with those behind the last sequence
};

__device__ __forceinline__ Run run_of(const NormArgs& a) {
  Run r;
  if (a.off) {
    r.s = find_packed(a.off, a.B, a.T, a.chunk, blockIdx.x);
  } else {
    r.s.b = blockIdx.x / a.chunks;
    r.s.chunk = blockIdx.x % a.chunks;
    r.s.row0 = 0;
    r.s.len = a.T;
  }
  const int64_t all = a.off && a.zero_unused && r.s.b == a.B - 1 ? a.T - r.s.row0 : r.s.len;
  r.t0 = r.s.chunk * a.chunk;
  r.t1 = r.t0 + a.chunk < r.s.len ? r.t0 + a.chunk : r.s.len;
  r.limit = r.t0 + a.chunk < all ? r.t0 + a.chunk : all;
  return r;
}

template <typename MT, int WAVES, int E, int VEC>
__global__ __launch_bounds__((Lanes<MT, WAVES, E, VEC>::kThreads)) void norm_kernel(NormArgs a) {
  typedef Lanes<MT, WAVES, E, VEC> L;
  __shared__ float red[4 * WAVES];
  const int sub = L::kRows > 1 ? threadIdx.x / (64 * WAVES) : 0;
  L lanes{a.D, (int)(threadIdx.x % (64 * WAVES)) * VEC, red};
  const Run r = run_of(a);
  if (r.t0 >= r.limit) return;
  const float inv_d = 1.0f / (float)a.D;
  float g[E], pw[E], w[E];
  lanes.param(a.gate ? a.gate + r.s.b * a.gate_sb : nullptr, g, 1.0f);
  lanes.param(a.post, pw, 1.0f);
  lanes.param(a.weight, w, 1.0f);
  for (int64_t t = r.t0 + sub; t < r.limit; t += L::kRows) {
    const int64_t row = r.s.row0 + t, b = a.off ? 0 : r.s.b;
    float x[E], y[E];
    MT* h = static_cast<MT*>(a.h) + b * a.h_sb + row * a.h_st;
    MT* n = static_cast<MT*>(a.n) + b * a.n_sb + row * a.n_st;
    if (t >= r.t1) {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = 0.0f;
      if (a.h) lanes.store(h, x);
      if (a.n) lanes.store(n, x);
      continue;
    }
    lanes.load(static_cast<const MT*>(a.x) + b * a.x_sb + row * a.x_st, x);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] *= a.alpha;
    if (a.y) {
      lanes.load(static_cast<const MT*>(a.y) + b * a.y_sb + row * a.y_st, y);
      if (a.post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] = fmaf(y[i], y[i], s[0]);
        lanes.sum(s);
        const float ry = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] *= ry * pw[i];
      }
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = fmaf(g[i], y[i], x[i]);
    }
    if (a.h) lanes.store(h, x);
    if (a.n) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] = fmaf(x[i], x[i], s[0]);
      lanes.sum(s);
      const float rh = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] *= rh * w[i];
      lanes.store(n, x);
    }
  }
}

template <typename MT, int WAVES, int E, int VEC>
__global__ __launch_bounds__((Lanes<MT, WAVES, E, VEC>::kThreads)) void norm_back_kernel(NormArgs a) {
  typedef Lanes<MT, WAVES, E, VEC> L;
  __shared__ float red[4 * WAVES];
  const int sub = L::kRows > 1 ? threadIdx.x / (64 * WAVES) : 0;
  L lanes{a.D, (int)(threadIdx.x % (64 * WAVES)) * VEC, red};
  const Run r = run_of(a);
  const float inv_d = 1.0f / (float)a.D;
  float g[E], pw[E], w[E], dg[E], dpw[E], dw[E];
  lanes.param(a.gate ? a.gate + r.s.b * a.gate_sb : nullptr, g, 1.0f);
  lanes.param(a.post, pw, 1.0f);
  lanes.param(a.weight, w, 1.0f);
#pragma unroll
  for (int i = 0; i < E; ++i) dg[i] = dpw[i] = dw[i] = 0.0f;
  for (int64_t t = r.t0 + sub; t < r.limit; t += L::kRows) {
    const int64_t row = r.s.row0 + t, b = a.off ? 0 : r.s.b;
    MT* dx = static_cast<MT*>(a.dx) + b * a.dx_sb + row * a.dx_st;
    MT* dy = static_cast<MT*>(a.dy) + b * a.dy_sb + row * a.dy_st;
    float h[E], y[E], u[E], d[E], dn[E];
    if (t >= r.t1) {
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = 0.0f;
      if (a.dx) lanes.store(dx, d);
      if (a.dy) lanes.store(dy, d);
      continue;
    }
    lanes.load(static_cast<const MT*>(a.x) + b * a.x_sb + row * a.x_st, h);
    if (a.y) {
      lanes.load(static_cast<const MT*>(a.y) + b * a.y_sb + row * a.y_st, y);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = 0.0f;
    }
    if (a.h) {
      lanes.load(static_cast<const MT*>(a.h) + b * a.h_sb + row * a.h_st, d);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = 0.0f;
    }
    float ry = 1.0f;
    if (a.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) s[0] = fmaf(y[i], y[i], s[0]);
      lanes.sum(s);
      ry = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      y[i] *= ry;            // y^ (without a norm: y)
      u[i] = y[i] * pw[i];
      h[i] = fmaf(g[i], u[i], a.alpha * h[i]);
    }
    if (a.n) {
      lanes.load(static_cast<const MT*>(a.n) + b * a.n_sb + row * a.n_st, dn);
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        s[0] = fmaf(h[i], h[i], s[0]);
        s[1] = fmaf(w[i] * dn[i], h[i], s[1]);
      }
      lanes.sum(s);
      const float rh = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
      const float c = s[1] * rh * inv_d;  // mean(w dn h^)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float hh = h[i] * rh;
        dw[i] = fmaf(dn[i], hh, dw[i]);
        d[i] = fmaf(rh, fmaf(-hh, c, w[i] * dn[i]), d[i]);
      }
    }
    if (a.dx) {
#pragma unroll
      for (int i = 0; i < E; ++i) h[i] = a.alpha * d[i];
      lanes.store(dx, h);
    }
    if (!a.y) continue;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      dg[i] = fmaf(d[i], u[i], dg[i]);
      d[i] *= g[i];
    }
    if (a.post) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        dpw[i] = fmaf(d[i], y[i], dpw[i]);
        d[i] *= pw[i];
        s[0] = fmaf(d[i], y[i], s[0]);
      }
      lanes.sum(s);
      const float c = s[0] * inv_d;
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = ry * fmaf(-y[i], c, d[i]);
    }
    if (a.dy) lanes.store(dy, d);
  }
  // the sums over these rows: zero where the run is empty
  float* part = a.parts + (blockIdx.x * (int64_t)L::kRows + sub) * a.sums * a.D;
  auto put = [&](const float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = lanes.col(i / VEC) + i % VEC;
      if (c < a.D) part[c] = x[i];
    }
    part += a.D;
  };
  if (a.dgate) put(dg);
  if (a.dpost) put(dpw);
  if (a.dweight) put(dw);
}

// Partial sums [parts][sums][D] to gradients: a workgroup takes 64 channels of
// one gradient (of one sequence's, where the gate is per sequence), its waves
// every sixteenth partial, joined in order.
__global__ __launch_bounds__(1024) void norm_sums_kernel(NormArgs a) {
  __shared__ float red[16][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t tiles = (a.D + 63) / 64;
  const int64_t c = (blockIdx.x % tiles) * 64 + lane;
  int64_t which = blockIdx.x / tiles;  // gates, then the others
  const int64_t gates = a.dgate ? (a.gate_sb ? a.B : 1) : 0;
  int64_t first = 0, last = a.items;
  int kind = 0;
  float* to;
  if (which < gates) {
    to = a.dgate + which * a.D;
    if (a.gate_sb) {
      if (a.off) {
        const int64_t lo = clamp64(a.off[which], 0, a.T), hi = clamp64(a.off[which + 1], lo, a.T);
        first = lo / a.chunk + which;
        last = first + (hi - lo + a.chunk - 1) / a.chunk;
      } else {
        first = which * a.chunks;
        last = first + a.chunks;
      }
    }
  } else {
    which -= gates;
    kind = (a.dgate ? 1 : 0) + (int)which;
    to = which == 0 && a.dpost ? a.dpost : a.dweight;
  }
  first *= a.rows;
  last *= a.rows;
  float s = 0.0f;
  if (c < a.D)
    for (int64_t p = first + wave; p < last; p += 16) s += a.parts[(p * a.sums + kind) * a.D + c];
  red[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= a.D) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += red[i][lane];
  to[c] = s;
}

// rows of a workgroup at a time, by the channels
int rows_at_once(int64_t D) { return D <= 1024 ? 4 : 1; }

template <typename MT, int WAVES, int E, int VEC>
hipError_t norm_launch(const NormArgs& a, bool backward, hipStream_t stream) {
  typedef Lanes<MT, WAVES, E, VEC> L;
  if (!grid_fits(a.items, L::kThreads)) return hipErrorNotSupported;
  if (backward)
    hipLaunchKernelGGL((norm_back_kernel<MT, WAVES, E, VEC>), dim3((unsigned)a.items), dim3(L::kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_kernel<MT, WAVES, E, VEC>), dim3((unsigned)a.items), dim3(L::kThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename MT, int VEC>
hipError_t norm_by_width(const NormArgs& a, bool backward, hipStream_t stream) {
  if (a.D <= 512) return norm_launch<MT, 1, 8, VEC>(a, backward, stream);
  if (a.D <= 1024) return norm_launch<MT, 1, 16, VEC>(a, backward, stream);
  if (a.D <= 2048) return norm_launch<MT, 4, 8, VEC>(a, backward, stream);
  if (a.D <= 4096) return norm_launch<MT, 4, 16, VEC>(a, backward, stream);
  if (a.D <= 8192) return norm_launch<MT, 16, 8, VEC>(a, backward, stream);
  return norm_launch<MT, 16, 16, VEC>(a, backward, stream);
}

template <typename MT>
hipError_t norm_for(const NormArgs& a, bool aligned, bool backward, hipStream_t stream) {
  return aligned ? norm_by_width<MT, 16 / sizeof(MT)>(a, backward, stream) : norm_by_width<MT, 1>(a, backward, stream);
}

}  // namespace

NormPlan norm_plan(int64_t B, int64_t T, int64_t D, bool packed, bool backward) {
  NormPlan p;
  // rows a workgroup: many enough that its parameters and partial sums cost
  // little beside them, with workgroups enough for every compute unit
  const int64_t at_once = p.rows = rows_at_once(D), workgroups = backward ? 1024 : 2048;
  const int64_t rows = packed ? T : B * T;
  p.chunk = (rows + workgroups - 1) / workgroups;
  p.chunk = (p.chunk + at_once - 1) / at_once * at_once;
  if (p.chunk < at_once) p.chunk = at_once;
  p.chunks = (T + p.chunk - 1) / p.chunk;
  p.items = packed ? T / p.chunk + B : B * p.chunks;
  return p;
}

template <typename MT>
hipError_t launch_norm(const NormArgs& a, bool aligned, hipStream_t stream) {
  return a.items ? norm_for<MT>(a, aligned, false, stream) : hipSuccess;
}

template <typename MT>
hipError_t launch_norm_back(const NormArgs& a, bool aligned, hipStream_t stream) {
  if (a.items) {
    const hipError_t e = norm_for<MT>(a, aligned, true, stream);
    if (e != hipSuccess) return e;
  }
  const int64_t outs = (a.dgate ? (a.gate_sb ? a.B : 1) : 0) + (a.dpost ? 1 : 0) + (a.dweight ? 1 : 0);
  if (!outs) return hipSuccess;
  const int64_t blocks = outs * ((a.D + 63) / 64);
  if (!grid_fits(blocks, 1024)) return hipErrorNotSupported;
  hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)blocks), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

template hipError_t launch_norm<float>(const NormArgs&, bool, hipStream_t);
template hipError_t launch_norm<bf16>(const NormArgs&, bool, hipStream_t);
template hipError_t launch_norm_back<float>(const NormArgs&, bool, hipStream_t);
template hipError_t launch_norm_back<bf16>(const NormArgs&, bool, hipStream_t);

}  // namespace gdn
