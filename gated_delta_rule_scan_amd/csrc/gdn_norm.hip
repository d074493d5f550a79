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
// registers between its reductions, 4 to 16 channels a lane over a quarter of a
// wave to sixteen waves, and so do, over all of a workgroup's rows, the parameters
// (forward) and the sums over rows.  Those sums go to the workspace, one partial each
// per workgroup, and a second kernel adds them in a fixed order.  bf16: forward 65520
// x 2048 in 193 us (5.6 TB/s), backward 32760 x 2048 in 151 (5.3 TB/s) and 6 for
// the sums; above 8192 channels the backward kernel spills (4096 x 16384: 516 us,
// 1.6 TB/s).
#include "gdn_layer.h"

namespace gdn {
namespace {

// Sum over LANES lanes of a wave (16, 32 or 64), in each of them: quads, eights
// and sixteens by row permutations, then pairs of rows and the halves swapped.
template <int LANES>
__device__ __forceinline__ float wave_sum(float x) {
  auto add = [](float v, int moved) { return v + __builtin_bit_cast(float, moved); };
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0xB1, 0xF, 0xF, true));   // quad: 1 0 3 2
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x4E, 0xF, 0xF, true));   // quad: 2 3 0 1
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x141, 0xF, 0xF, true));  // half row mirrored
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x140, 0xF, 0xF, true));  // row mirrored
  if constexpr (LANES == 16) return x;
  if constexpr (LANES == 64) return over_groups(x, [](float a, float b) { return a + b; });
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned a = r[0], b = r[1];
  return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

// Waves of a compute unit at a time, by registers and LDS.  A call has
// workgroups for so many, so that all of them run from its start to its end.
constexpr int waves_at_once(int waves, int E, size_t size, bool backward) {
  if (waves == 16) return 16;
  if (backward) return E == 16 ? 8 : 16;
  return E == 16 ? (size == 4 ? 12 : 16) : 20;
}

// Threads of a workgroup: rows of up to a wave come by four waves.
constexpr int threads_of(int lanes) { return lanes <= 64 ? 256 : lanes; }

// LANES lanes per row, E channels per lane in vectors of 16 bytes.
// Rows that are not WHOLE (off 16 bytes, or not of whole vectors) are moved in
// vectors too, which the memory takes at any address; the last one of a row ends
// with the row, so that its first channels are the neighbour's as well.  Those are
// left out of sums, and written twice they are the same; in a call in place the
// waves wait for each other's loads, since a neighbour could have written them
// before they are read.  bf16 in microseconds, so against channel by channel:
// forward 8000 x 4003 51 and 88, 20000 x 1001 29 and 49; backward 101 and 124, 55
// and 67.
template <typename MT, int LANES, int E, bool WHOLE>
struct Lanes {
  static constexpr int VEC = 16 / sizeof(MT) < E ? 16 / sizeof(MT) : E;
  static constexpr int WAVES = LANES <= 64 ? 1 : LANES / 64;
  static_assert(WAVES == 1 || WAVES >= 4, "waves that share a row have the workgroup's barriers to themselves");
  static constexpr int kRows = WAVES == 1 ? 256 / LANES : 1;  // rows of a workgroup at a time
  static constexpr int kThreads = threads_of(LANES);
  static constexpr int kAlign = WHOLE ? VEC * sizeof(MT) : sizeof(MT);
  // a lane's channels of a row as they lie in memory: what is in flight for the next row
  struct Raw {
    MT v[E];
  };
  // whether a row's loads are under way while the one before is worked on
  static constexpr bool kAhead = LANES * E <= 8192;
  int64_t D;
  int col0;  // the lane's first channel
  float* red;
  int phase = 0;
  mutable int sums_taken = 0;
  bool some_twice = false;  // the wave has a vector that was moved

  // a vector's first channel, were it not moved back; whether the lane has it at all; how far it is moved
  __device__ __forceinline__ int place(int v) const { return v * LANES * VEC + col0; }
  __device__ __forceinline__ bool live(int v) const { return place(v) < D; }
  __device__ __forceinline__ int col(int v) const {
    if constexpr (WHOLE) return place(v);
    return live(v) && place(v) + VEC > D && !narrow() ? (int)D - VEC : place(v);
  }
  // the row has not one whole vector (wider kernels than the narrowest have no such rows)
  __device__ __forceinline__ bool narrow() const { return !WHOLE && LANES == 16 && D < VEC; }
  __device__ __forceinline__ int twice(int v) const { return place(v) - col(v); }
  // sum over the lane's own channels of a b
  __device__ __forceinline__ float dot(const float (&a)[E], const float (&b)[E]) const {
    float s = 0.0f;
    if (!WHOLE && some_twice) {
#pragma unroll
      for (int i = 0; i < E; ++i) s = i % VEC >= twice(i / VEC) ? fmaf(a[i], b[i], s) : s;
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) s = fmaf(a[i], b[i], s);
    }
    return s;
  }
  // before a row is written, in a call in place: every wave of it has its loads, of this row and the next
  __device__ __forceinline__ void loaded(bool in_place) const {
    if (WHOLE || WAVES == 1 || !in_place) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }
  // (by the whole wave, before anything else)
  __device__ __forceinline__ void begin() {
    bool any = false;
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) any = any || twice(v) != 0;
    some_twice = !WHOLE && __any(any);
  }

  __device__ __forceinline__ void load(const MT* p, Raw& x) const {
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
      // (rows are read once: with the hint for that the backward call of 32760 x 2048 took 160 us, without 175)
      typedef MT vec __attribute__((ext_vector_type(VEC), aligned(kAlign)));
      vec q = (vec)(MT)0.0f;
      if (narrow()) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (col(v) + e < D) q[e] = p[col(v) + e];
      } else if (live(v)) {
        q = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p + col(v)));
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) x.v[v * VEC + e] = q[e];
    }
  }
  static __device__ __forceinline__ void open(const Raw& r, float (&x)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = (float)r.v[i];
  }
  // The parameters g, wp and w, ones where they are not given.  Up to 8192
  // channels they are loaded once: the forward kernel keeps them in registers,
  // the backward one, which has sums there, in LDS (in LDS the forward call of
  // 65520 x 2048 took 215 us, in registers 194).
  static constexpr bool kOnce = LANES * E <= 8192;
  __device__ __forceinline__ void param(const float* p, float (&x)[E]) const {
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
      if (p && live(v) && !narrow()) {
        __builtin_memcpy(x + v * VEC, p + col(v), VEC * 4);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[v * VEC + e] = narrow() && p && col(v) + e < D ? p[col(v) + e] : 1.0f;
      }
    }
  }
  // In LDS a vector's pieces of 16 bytes lie LANES pieces apart, so that a
  // wave's lanes read side by side: [v][piece][lane].
  static constexpr int kStage = kOnce ? LANES * E : 4;
  static constexpr int kPiece = VEC < 4 ? VEC : 4;
  __device__ __forceinline__ void stage(const float* p, float* to) const {
    if constexpr (kOnce)
      for (int i = threadIdx.x; i < kStage; i += kThreads) {
        const int at = i / (LANES * VEC) * (LANES * VEC) + i / kPiece % LANES * VEC;  // its vector's place
        int c = at + i / (LANES * kPiece) % (VEC / kPiece) * kPiece + i % kPiece;
        if (!WHOLE && at < D && at + VEC > D && !narrow()) c -= at + VEC - (int)D;
        to[i] = p && c < D ? p[c] : 1.0f;
      }
  }
  __device__ __forceinline__ void param(const float* p, const float* staged, float (&x)[E]) const {
    if constexpr (!kOnce) return param(p, x);
#pragma unroll
    for (int i = 0; i < E; i += kPiece)
      __builtin_memcpy(x + i, __builtin_assume_aligned(staged + i * LANES + col0 / VEC * kPiece, kPiece * 4), kPiece * 4);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* p, const float (&x)[E]) const {
    // (partial sums, fp32, lie at rows of D words)
    typedef T vec __attribute__((ext_vector_type(VEC), aligned(sizeof(T) == sizeof(MT) ? kAlign : 4)));
#pragma unroll
    for (int v = 0; v < E / VEC; ++v) {
      if (narrow()) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (col(v) + e < D) p[col(v) + e] = (T)x[v * VEC + e];
      } else if (live(v)) {
        vec q;
#pragma unroll
        for (int e = 0; e < VEC; ++e) q[e] = (T)x[v * VEC + e];
        *reinterpret_cast<vec*>(p + col(v)) = q;
      }
    }
  }
  // K sums over the row, in all its lanes.  Several waves join theirs in LDS;
  // two buffers in turn, so that one barrier a call is enough.
  template <int K>
  __device__ __forceinline__ void sum(float (&s)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = wave_sum<(LANES < 64 ? LANES : 64)>(s[k]);
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

// A lane's sums over rows: in registers, or (the widest rows) in LDS, where
// each lane has places of its own.
template <typename L, int E, bool REGISTERS>
struct Sum {
  float x[E];
  __device__ __forceinline__ explicit Sum(const L&) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = 0.0f;
  }
  __device__ __forceinline__ void add(const float (&y)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] += y[i];
  }
  __device__ __forceinline__ void get(float (&y)[E]) const {
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = x[i];
  }
};
template <typename L, int E>
struct Sum<L, E, false> {
  f32x4* at;
  __device__ __forceinline__ explicit Sum(const L& lanes) {
    __shared__ f32x4 places[2 * (E / 4) * L::kThreads];  // (of dgate and dpost)
    at = places + lanes.sums_taken * (E / 4 * L::kThreads) + threadIdx.x;
    ++lanes.sums_taken;
#pragma unroll
    for (int v = 0; v < E / 4; ++v) at[v * L::kThreads] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void add(const float (&y)[E]) {
#pragma unroll
    for (int v = 0; v < E / 4; ++v) at[v * L::kThreads] += f32x4{y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]};
  }
  __device__ __forceinline__ void get(float (&y)[E]) const {
#pragma unroll
    for (int v = 0; v < E / 4; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[4 * v + e] = at[v * L::kThreads][e];
  }
};

// The rows of a workgroup: of a sequence that is cut into n runs, run i takes
// rows i, i + n, i + 2n, ... (R neighbouring ones in a row's place, where R are
// taken at a time), so that the workgroups of a call read side by side; runs of
// neighbouring rows start at distances that may all fall on the same memory
// channels (32 rows of 4096 bytes a run, forward: 255 us against 248).  Rows of no
// sequence lie behind the last one's, `chunk` of them a run.
struct Run {
  int64_t b, row0, len;   // the sequence, its first row and rows
  int64_t t, step;        // the first row of this lane's, and the distance of the others
  int64_t u0, u1;         // rows of no sequence
};

template <int R>
__device__ __forceinline__ Run run_of(const NormArgs& a, int sub) {
  const int64_t item = a.first + blockIdx.x;
  SeqItem s;
  if (a.off) {
    s = find_packed(a.off, a.B, a.T, a.chunk, item);
  } else {
    s.b = item / a.chunks;
    s.chunk = item % a.chunks;
    s.row0 = 0;
    s.len = a.T;
  }
  Run r;
  r.b = s.b;
  r.row0 = s.row0;
  r.len = s.len;
  const int64_t runs = (s.len + a.chunk - 1) / a.chunk;
  r.t = s.chunk >= 0 && s.chunk < runs ? s.chunk * R + sub : s.len;  // (below zero: in front of the first sequence)
  r.step = runs * R;
  const int64_t all = a.off && a.zero_unused && s.b == a.B - 1 ? a.T - s.row0 : s.len;
  r.u0 = s.chunk * a.chunk > s.len ? s.chunk * a.chunk : s.len;
  r.u1 = (s.chunk + 1) * a.chunk < all ? (s.chunk + 1) * a.chunk : all;
  return r;
}

template <typename MT, int LANES, int E, bool WHOLE>
__global__ __launch_bounds__(threads_of(LANES), (waves_at_once(LANES / 64, E, sizeof(MT), false) / 4)) void norm_kernel(NormArgs a) {
  typedef Lanes<MT, LANES, E, WHOLE> L;
  __shared__ float red[4 * L::WAVES];
  const int sub = L::kRows > 1 ? threadIdx.x / LANES : 0;
  L lanes{a.D, (int)(threadIdx.x % LANES) * L::VEC, red};
  const Run r = run_of<L::kRows>(a, sub);
  const int64_t b = a.off ? 0 : r.b;
  const MT* x_rows = static_cast<const MT*>(a.x) + b * a.x_sb;
  const MT* y_rows = static_cast<const MT*>(a.y) + b * a.y_sb;
  MT* h_rows = static_cast<MT*>(a.h) + b * a.h_sb;
  MT* n_rows = static_cast<MT*>(a.n) + b * a.n_sb;
  // the next row's loads are under way while this one's sums are taken
  typename L::Raw rx, ry;
  int64_t t = r.t;
  if (t < r.len) {
    lanes.load(x_rows + (r.row0 + t) * a.x_st, rx);
    if (a.y) lanes.load(y_rows + (r.row0 + t) * a.y_st, ry);
  }
  const float inv_d = 1.0f / (float)a.D;
  lanes.begin();
  const float* gate = a.gate ? a.gate + r.b * a.gate_sb : nullptr;
  float x[E], y[E], g[E], pw[E], w[E];
  if (L::kOnce) {
    lanes.param(gate, g);
    lanes.param(a.post, pw);
    lanes.param(a.weight, w);
  }
  for (; t < r.len; t += r.step) {
    const int64_t row = r.row0 + t;
    L::open(rx, x);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] *= a.alpha;
    if (a.y) L::open(ry, y);
    if (t + r.step < r.len) {
      lanes.load(x_rows + (row + r.step) * a.x_st, rx);
      if (a.y) lanes.load(y_rows + (row + r.step) * a.y_st, ry);
    }
    asm volatile("" ::: "memory");  // (the loads are issued here, not where they are used)
    lanes.loaded(a.h == a.x);
    if (a.y) {
      if (a.post) {
        float s[1] = {lanes.dot(y, y)};
        lanes.sum(s);
        const float inv = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
        if (!L::kOnce) lanes.param(a.post, pw);
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] *= inv * pw[i];
      }
      if (!L::kOnce) lanes.param(gate, g);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = fmaf(g[i], y[i], x[i]);
    }
    if (a.h) lanes.store(h_rows + row * a.h_st, x);
    if (a.n) {
      float s[1] = {lanes.dot(x, x)};
      lanes.sum(s);
      const float inv = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
      if (!L::kOnce) lanes.param(a.weight, w);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] *= inv * w[i];
      lanes.store(n_rows + row * a.n_st, x);
    }
  }
  // rows of no sequence
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = 0.0f;
  for (t = r.u0 + sub; t < r.u1; t += L::kRows) {
    if (a.h) lanes.store(h_rows + (r.row0 + t) * a.h_st, x);
    if (a.n) lanes.store(n_rows + (r.row0 + t) * a.n_st, x);
  }
}

template <typename MT, int LANES, int E, bool WHOLE>
__global__ __launch_bounds__(threads_of(LANES), (waves_at_once(LANES / 64, E, sizeof(MT), true) / 4)) void norm_back_kernel(NormArgs a) {
  typedef Lanes<MT, LANES, E, WHOLE> L;
  __shared__ float red[4 * L::WAVES];
  const int sub = L::kRows > 1 ? threadIdx.x / LANES : 0;
  L lanes{a.D, (int)(threadIdx.x % LANES) * L::VEC, red};
  const Run r = run_of<L::kRows>(a, sub);
  const int64_t b = a.off ? 0 : r.b;
  const MT* x_rows = static_cast<const MT*>(a.x) + b * a.x_sb;
  const MT* y_rows = static_cast<const MT*>(a.y) + b * a.y_sb;
  const MT* dh_rows = static_cast<const MT*>(a.h) + b * a.h_sb;
  const MT* dn_rows = static_cast<const MT*>(a.n) + b * a.n_sb;
  MT* dx_rows = static_cast<MT*>(a.dx) + b * a.dx_sb;
  MT* dy_rows = static_cast<MT*>(a.dy) + b * a.dy_sb;
  typename L::Raw rx, ry, rdh, rdn;
  auto load = [&](int64_t row) {
    lanes.load(x_rows + row * a.x_st, rx);
    if (a.y) lanes.load(y_rows + row * a.y_st, ry);
    if (a.h) lanes.load(dh_rows + row * a.h_st, rdh);
    if (a.n) lanes.load(dn_rows + row * a.n_st, rdn);
  };
  int64_t t = r.t;
  if (t < r.len) load(r.row0 + t);
  const float inv_d = 1.0f / (float)a.D;
  lanes.begin();
  const float* gate = a.gate ? a.gate + r.b * a.gate_sb : nullptr;
  __shared__ __align__(16) float params[3][L::kStage];
  lanes.stage(gate, params[0]);
  lanes.stage(a.post, params[1]);
  lanes.stage(a.weight, params[2]);
  __syncthreads();
  float g[E], pw[E], dw[E];
  Sum<L, E, L::kOnce> dg(lanes), dpw(lanes);
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = 0.0f;
  for (; t < r.len; t += r.step) {
    const int64_t row = r.row0 + t;
    asm volatile("" ::: "memory");  // (parameters are not kept in registers over the rows)
    float h[E], y[E], d[E], dn[E];
    if (!L::kAhead && t != r.t) load(row);
    L::open(rx, h);
#pragma unroll
    for (int i = 0; i < E; ++i) y[i] = d[i] = dn[i] = 0.0f;
    if (a.y) L::open(ry, y);
    if (a.h) L::open(rdh, d);
    if (a.n) L::open(rdn, dn);
    if (L::kAhead && t + r.step < r.len) load(row + r.step);
    lanes.loaded(a.dx == a.h);
    float ry_ = 1.0f;
    if (a.post) {
      float s[1] = {lanes.dot(y, y)};
      lanes.sum(s);
      ry_ = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
    }
    lanes.param(gate, params[0], g);
    lanes.param(a.post, params[1], pw);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      y[i] *= ry_;  // y^ (without a norm: y)
      h[i] = fmaf(g[i], y[i] * pw[i], a.alpha * h[i]);
    }
    if (a.n) {
      float w[E];  // weight, then weight dn
      lanes.param(a.weight, params[2], w);
#pragma unroll
      for (int i = 0; i < E; ++i) w[i] *= dn[i];
      float s[2] = {lanes.dot(h, h), lanes.dot(w, h)};
      lanes.sum(s);
      const float rh = 1.0f / sqrtf(fmaf(s[0], inv_d, a.eps));
      const float c = s[1] * rh * inv_d;  // mean(w dn h^)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float hh = h[i] * rh;
        dw[i] = fmaf(dn[i], hh, dw[i]);
        d[i] = fmaf(rh, fmaf(-hh, c, w[i]), d[i]);
      }
    }
    if (a.dx) {
#pragma unroll
      for (int i = 0; i < E; ++i) h[i] = a.alpha * d[i];
      lanes.store(dx_rows + row * a.dx_st, h);
    }
    if (!a.y) continue;
    asm volatile("" ::: "memory");  // (nor over the sums before)
    lanes.param(gate, params[0], g);
    lanes.param(a.post, params[1], pw);
    float u[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      u[i] = d[i] * (y[i] * pw[i]);
      d[i] *= g[i];
    }
    if (a.dgate) dg.add(u);
    if (a.post) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        u[i] = d[i] * y[i];
        d[i] *= pw[i];
      }
      if (a.dpost) dpw.add(u);
      float s[1] = {lanes.dot(d, y)};
      lanes.sum(s);
      const float c = s[0] * inv_d;
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = ry_ * fmaf(-y[i], c, d[i]);
    }
    if (a.dy) lanes.store(dy_rows + row * a.dy_st, d);
  }
  float u[E];
  // rows of no sequence
  float zero[E];
#pragma unroll
  for (int i = 0; i < E; ++i) zero[i] = 0.0f;
  for (t = r.u0 + sub; t < r.u1; t += L::kRows) {
    if (a.dx) lanes.store(dx_rows + (r.row0 + t) * a.dx_st, zero);
    if (a.dy) lanes.store(dy_rows + (r.row0 + t) * a.dy_st, zero);
  }
  // the sums over these rows: zero where the run is empty.  Rows that were
  // taken side by side are added first.
  float* part = a.parts + (a.first + blockIdx.x) * a.sums * a.D;
  auto put = [&](float (&x)[E]) {
    if constexpr (L::kRows > 1) {
      __shared__ float side[L::kRows - 1][E * LANES];
      __syncthreads();
      if (sub > 0)
#pragma unroll
        for (int i = 0; i < E; ++i) side[sub - 1][i * LANES + threadIdx.x % LANES] = x[i];
      __syncthreads();
      if (sub == 0)
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
          for (int k = 0; k < L::kRows - 1; ++k) x[i] += side[k][i * LANES + threadIdx.x];
    }
    if (sub == 0) lanes.store(part, x);
    part += a.D;
  };
  if (a.dgate) {
    dg.get(u);
    put(u);
  }
  if (a.dpost) {
    dpw.get(u);
    put(u);
  }
  if (a.dweight) put(dw);
}

// Partial sums [parts][sums][D] to gradients: a workgroup takes 32 channels of
// one gradient (of one sequence's, where the gate is per sequence), its half
// waves every 16th partial, joined in order.  (41 sequences' gates, a few partials
// each: with sixteen waves a workgroup the whole call took 99 us, with eight 95.)
__global__ __launch_bounds__(512) void norm_sums_kernel(NormArgs a) {
  __shared__ float red[16][32];
  const int half = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tiles = (a.D + 31) / 32;
  const int64_t c = (blockIdx.x % tiles) * 32 + lane;
  int64_t which = a.first + blockIdx.x / tiles;  // gates, then the others
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
  // (sixteen loads under way at a time, the last ones too: the sum is a chain of their latencies)
  float s = 0.0f;
  if (c < a.D) {
    const float* from = a.parts + kind * a.D + c;
    const int64_t step = a.sums * a.D;
    for (int64_t p = first + half; p < last; p += 16 * 16) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = from[(p + 16 * i < last ? p + 16 * i : p) * step];
#pragma unroll
      for (int i = 0; i < 16; ++i) s = p + 16 * i < last ? s + v[i] : s;
    }
  }
  red[half][lane] = s;
  __syncthreads();
  if (half != 0 || c >= a.D) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += red[i][lane];
  to[c] = s;
}

// A row's lanes and a lane's channels, by the row's width.  Rows up to 256
// channels share a wave: a row alone has too few bytes under way (with a wave
// per row 93750 x 64 took 30 us in bf16 and 29 in fp32, so 12 and 18).
struct Width {
  int64_t D;
  int lanes, E;
};
template <bool HALF, bool BACKWARD>
constexpr Width kWidths[] = {{64, 16, 4},
                             {128, 32, 4},
                             {256, HALF ? 32 : 64, HALF ? 8 : 4},
                             {512, 64, 8},
                             {1024, 64, 16},
                             {2048, 256, 8},
                             {4096, BACKWARD ? 512 : 256, BACKWARD ? 8 : 16},
                             {8192, BACKWARD ? 1024 : 512, BACKWARD ? 8 : 16},
                             {16384, 1024, 16}};

template <typename MT, bool WHOLE, bool BACKWARD, int I = 0>
hipError_t norm_by_width(const NormArgs& a, hipStream_t stream) {
  constexpr Width w = kWidths<sizeof(MT) == 2, BACKWARD>[I];
  if constexpr (w.D < 16384)
    if (a.D > w.D) return norm_by_width<MT, WHOLE, BACKWARD, I + 1>(a, stream);
  constexpr int kThreads = threads_of(w.lanes);
  NormArgs part = a;
  return in_launches(a.items, 1, kThreads, [&](int64_t first, dim3 blocks) {
    part.first = first;
    if constexpr (BACKWARD)
      hipLaunchKernelGGL((norm_back_kernel<MT, w.lanes, w.E, WHOLE>), blocks, dim3(kThreads), 0, stream, part);
    else
      hipLaunchKernelGGL((norm_kernel<MT, w.lanes, w.E, WHOLE>), blocks, dim3(kThreads), 0, stream, part);
  });
}

template <typename MT, bool BACKWARD>
hipError_t norm_for(const NormArgs& a, bool aligned, hipStream_t stream) {
  return aligned ? norm_by_width<MT, true, BACKWARD>(a, stream) : norm_by_width<MT, false, BACKWARD>(a, stream);
}

}  // namespace

NormPlan norm_plan(int64_t B, int64_t T, int64_t D, bool half, bool packed, bool backward) {
  NormPlan p;
  const Width* widths = half ? (backward ? kWidths<true, true> : kWidths<true, false>) : backward ? kWidths<false, true> : kWidths<false, false>;
  while (D > widths->D && widths->D < 16384) ++widths;
  const Width& w = *widths;
  const int64_t at_once = w.lanes <= 64 ? 256 / w.lanes : 1;
  int64_t workgroups = 256 * (waves_at_once(w.lanes / 64, w.E, half ? 2 : 4, backward) * 64 / threads_of(w.lanes));
  if (workgroups < 256) workgroups = 256;
  const int64_t rows = packed ? T : B * T;
  // (a packed batch has up to a workgroup a sequence more)
  if (packed) workgroups = B < workgroups / 2 ? workgroups - B : workgroups / 2;
  p.chunk = (rows + workgroups - 1) / workgroups;
  p.chunk = (p.chunk + at_once - 1) / at_once * at_once;
  if (p.chunk < at_once) p.chunk = at_once;
  p.chunks = (T + p.chunk - 1) / p.chunk;
  p.items = packed ? T / p.chunk + B : B * p.chunks;
  return p;
}

template <typename MT>
hipError_t launch_norm(const NormArgs& a, bool aligned, hipStream_t stream) {
  return norm_for<MT, false>(a, aligned, stream);
}

template <typename MT>
hipError_t launch_norm_back(const NormArgs& a, bool aligned, hipStream_t stream) {
  const hipError_t e = norm_for<MT, true>(a, aligned, stream);
  if (e != hipSuccess) return e;
  const int64_t outs = (a.dgate ? (a.gate_sb ? a.B : 1) : 0) + (a.dpost ? 1 : 0) + (a.dweight ? 1 : 0);
  NormArgs part = a;
  return in_launches(outs, (a.D + 31) / 32, 512, [&](int64_t first, dim3 blocks) {
    part.first = first;
    hipLaunchKernelGGL(norm_sums_kernel, blocks, dim3(512), 0, stream, part);
  });
}

template hipError_t launch_norm<float>(const NormArgs&, bool, hipStream_t);
template hipError_t launch_norm<bf16>(const NormArgs&, bool, hipStream_t);
template hipError_t launch_norm_back<float>(const NormArgs&, bool, hipStream_t);
template hipError_t launch_norm_back<bf16>(const NormArgs&, bool, hipStream_t);

}  // namespace gdn
