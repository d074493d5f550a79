// Selective state space scan, for prompts and for single tokens: per channel
// d an fp32 state h of N entries,
//
//   dt' = softplus(dt + bias),  h_n = exp(dt' A_n) h_n + dt' x B_n,
//   y = sum_n h_n C_n + skip x,  out = y silu(z)
#include "gdn_layer.h"

namespace gdn {
namespace {

__device__ __forceinline__ float step_size(const SsmArgs& a, float dt, float bias) {
  const float v = dt + bias;
  return a.softplus ? softplus(v) : v;
}

// ---- prompts ----
// The decay depends on channel and state entry, so nothing here is a product
// of matrices: per token, channel and entry a pass takes one exponential (two
// issue slots), the products dt A and dt x B, the update and the readout --
// bound by the vector units, not by memory.
//
// A lane owns a channel and NN state entries in registers and walks the tokens
// in order, so rows of x, dt, z and out move in whole cache lines; the B and C
// of kStage tokens wait in LDS as fp32 and reach every lane by broadcast
// reads.  CT waves of a workgroup take neighbouring channel tiles of the same
// tokens; more than NN entries are split over waves, whose partial readouts
// meet in LDS.
//
// Too few channels to fill the GPU: sequences are cut into chunks and three
// kernels run.  The first (STATES) finds each chunk's end state from a zero
// start, and the sum of its step sizes: a chunk's whole decay is exp(A sum
// dt).  The second (carry) turns those into the state that enters each chunk;
// the third is the scan itself from there.  The first costs the exponentials
// once more, about 0.7 of the scan; a sequence's last chunk, and with it a
// sequence of one chunk, is spared it.

constexpr int kStage = 16;  // tokens whose B and C are staged at a time
constexpr int kAhead = 4;   // tokens of x, dt and z in flight per lane

struct Chunk {
  int64_t b;            // sequence
  int64_t item;         // its place in the workspace
  int64_t t0, t1, len;  // tokens of the sequence
  int64_t row0;         // first row of a packed sequence
  bool work;
};

__device__ __forceinline__ Chunk chunk_of(const SsmArgs& a, int64_t item) {
  Chunk c;
  c.item = item;
  int64_t k;
  if (a.off) {
    const SeqItem s = find_packed(a.off, a.B, a.T, a.chunk, item);
    c.b = s.b;
    c.len = s.len;
    c.row0 = s.row0;
    k = s.chunk;
  } else {
    c.b = item / a.chunks;
    k = item - c.b * a.chunks;
    c.len = a.T;
    c.row0 = 0;
  }
  c.t0 = k * a.chunk;
  c.t1 = c.t0 + a.chunk < c.len ? c.t0 + a.chunk : c.len;
  c.work = k >= 0 && (c.t0 < c.len || k == 0);
  return c;
}

template <typename MT, int NN, int CT, bool STATES>
__global__ __launch_bounds__(1024) void ssm_kernel(SsmArgs a, int NG, int tiles_per_group) {
  extern __shared__ __align__(16) float lds[];  // [kStage][B, C][NG * NN], then partial readouts
  const int NP = NG * NN, N = (int)a.N;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ng = wave / CT, ct = wave % CT;     // this wave's entries and channel tile
  const unsigned tiles = (unsigned)tiles_per_group * (unsigned)a.G;
  const Chunk c = chunk_of(a, blockIdx.x / tiles);
  if (!c.work) return;
  if (STATES && c.t1 >= c.len) return;  // nothing follows the last chunk
  const unsigned tile = blockIdx.x % tiles, g = tile / (unsigned)tiles_per_group;
  // the wave's first channel (uniform) and the lane's behind it; lanes without
  // a channel repeat the group's last one and store nothing
  const int64_t per = a.D / a.G, end = (g + 1) * per;
  const int64_t want = g * per + ((int64_t)(tile % (unsigned)tiles_per_group) * CT + ct) * 64;
  const int64_t d0 = want < end ? want : end - 1;
  const bool live = want + lane < end;
  const unsigned dl = live ? lane : (unsigned)(end - 1 - d0);
  const int64_t d = d0 + dl;
  const int64_t slot = slot_of(a.index, c.b, a.slots);

  auto base = [&](int64_t sb, int64_t st) { return a.off ? c.row0 * st : c.b * sb; };
  const MT* x = static_cast<const MT*>(a.x) + base(a.x_sb, a.x_st) + d0;
  const MT* dt = static_cast<const MT*>(a.dt) + base(a.dt_sb, a.dt_st) + d0;
  const MT* z = a.z ? static_cast<const MT*>(a.z) + base(a.z_sb, a.z_st) + d0 : nullptr;
  MT* out = static_cast<MT*>(a.out) + base(a.o_sb, a.o_st) + d0;
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.skip ? a.skip[d] : 0.0f;

  float A[NN], h[NN];
#pragma unroll
  for (int i = 0; i < NN; ++i) {
    const int n = ng * NN + i;
    const bool in = n < N;
    A[i] = in ? a.A[d * N + n] * kLog2e : 0.0f;
    h[i] = 0.0f;
    if (!STATES && in) {
      if (a.ends) h[i] = a.ends[(c.item * N + n) * a.D + d];
      else if (a.state_in && slot >= 0) h[i] = a.state_in[(slot * a.D + d) * N + n];
    }
  }

  // B and C of kStage tokens: one element a thread and round; a round covers
  // whole tokens, so a thread keeps its column
  constexpr int STEP = CT * 64 / (2 * NN), ROUNDS = kStage / STEP;
  static_assert(kStage % STEP == 0 && STEP > 0, "rounds cover the stage");
  const int col = tid % (2 * NP), first = tid / (2 * NP);
  const bool isC = col >= NP;
  const int n_col = isC ? col - NP : col;
  const bool stages = n_col < N && !(STATES && isC);
  const int64_t bc_st = isC ? a.c_st : a.b_st;
  const MT* bc = static_cast<const MT*>(isC ? a.Cm : a.Bm) + (isC ? base(a.c_sb, a.c_st) : base(a.b_sb, a.b_st)) +
                 g * a.N + (n_col < N ? n_col : 0);
  MT sv[ROUNDS];
  auto load_bc = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int64_t u = t + first + i * STEP;
      sv[i] = stages && u < c.t1 ? bc[u * bc_st] : (MT)0.0f;
    }
  };
  // x, dt and z of kAhead tokens; past the end the last token repeats
  MT xv[kAhead], dv[kAhead], zv[kAhead];
  auto load_rows = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t u = t + i < c.t1 ? t + i : c.t1 - 1;
      xv[i] = (x + u * a.x_st)[dl];
      dv[i] = (dt + u * a.dt_st)[dl];
      if (!STATES && NG == 1) zv[i] = z ? (z + u * a.z_st)[dl] : (MT)0.0f;
    }
  };

  float total = 0.0f;
  if (c.t0 < c.t1) {
    load_bc(c.t0);
    load_rows(c.t0);
  }
  for (int64_t tb = c.t0; tb < c.t1; tb += kStage) {
    __syncthreads();  // the stage before is read
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) lds[(first + i * STEP) * 2 * NP + col] = to_float(sv[i]);
    __syncthreads();
    if (tb + kStage < c.t1) load_bc(tb + kStage);
#pragma unroll 1
    for (int part = 0; part < kStage && tb + part < c.t1; part += kAhead) {
      const int64_t t = tb + part;
      MT xc[kAhead], dc[kAhead], zc[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        xc[i] = xv[i];
        dc[i] = dv[i];
        zc[i] = zv[i];
      }
      if (t + kAhead < c.t1) load_rows(t + kAhead);
      float* partial = lds + kStage * 2 * NP + wave * kAhead * 64 + lane;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float xi = to_float(xc[i]);
        const float s = t + i < c.t1 ? step_size(a, to_float(dc[i]), bias) : 0.0f;  // past the end: decay 1, no input
        const float u = s * xi;
        if (STATES) total += s;
        const float* bcl = lds + (part + i) * 2 * NP + ng * NN;
        float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int j = 0; j < NN / 4; ++j) {
          const f32x4 B = *reinterpret_cast<const f32x4*>(bcl + 4 * j);
          f32x4 C = {0.f, 0.f, 0.f, 0.f};
          if (!STATES) C = *reinterpret_cast<const f32x4*>(bcl + NP + 4 * j);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int n = 4 * j + m;
            h[n] = fmaf(hw_exp2(s * A[n]), h[n], u * B[m]);
            if (!STATES) {
              if (m & 1) y1 = fmaf(h[n], C[m], y1);
              else y0 = fmaf(h[n], C[m], y0);
            }
          }
        }
        if (!STATES) {
          if (NG == 1) {
            float y = fmaf(skip, xi, y0 + y1);
            if (z) y *= silu(to_float(zc[i]));
            if (live && t + i < c.t1) (out + (t + i) * a.o_st)[dl] = (MT)y;
          } else {
            partial[i * 64] = y0 + y1;
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // one token's operands in registers at a time
      }
      if (!STATES && NG > 1) {
        // the waves of a channel tile share out the tokens' sums
        __syncthreads();
        for (int i = ng; i < kAhead; i += NG) {
          const int64_t u = t + i;
          if (u >= c.t1) break;
          const float* p = lds + kStage * 2 * NP + (ct * kAhead + i) * 64 + lane;
          float y = skip * to_float((x + u * a.x_st)[dl]);
          for (int k = 0; k < NG; ++k) y += p[k * CT * kAhead * 64];
          if (z) y *= silu(to_float((z + u * a.z_st)[dl]));
          if (live) (out + u * a.o_st)[dl] = (MT)y;
        }
        __syncthreads();
      }
    }
  }
  if (STATES) {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NN; ++i)
      if (ng * NN + i < N) a.ends[(c.item * N + ng * NN + i) * a.D + d] = h[i];
    if (ng == 0) a.steps[c.item * a.D + d] = total;
  } else if (a.state_out && slot >= 0 && live && c.t1 >= c.len) {
#pragma unroll
    for (int i = 0; i < NN; ++i)
      if (ng * NN + i < N) a.state_out[(slot * a.D + d) * N + ng * NN + i] = h[i];
  }
}

// Chunk end states become entering states, in place: a thread per channel and
// state entry of a sequence walks its chunks.
constexpr int kCarry = 8;  // chunks in flight

__global__ __launch_bounds__(256) void ssm_carry_kernel(SsmArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, DN = a.D * a.N;
  if (i >= a.B * DN) return;
  const int64_t b = i / DN, r = i - b * DN, n = r / a.D, d = r - n * a.D;
  int64_t item0 = b * a.chunks, len = a.T;
  if (a.off) {
    const int64_t row0 = clamp64(a.off[b], 0, a.T);
    item0 = row0 / a.chunk + b;
    len = clamp64(a.off[b + 1], row0, a.T) - row0;
  }
  const int64_t chunks = len > a.chunk ? (len + a.chunk - 1) / a.chunk : 1;
  const int64_t slot = slot_of(a.index, b, a.slots);
  const float A = a.A[d * a.N + n] * kLog2e;
  float h = a.state_in && slot >= 0 ? a.state_in[(slot * a.D + d) * a.N + n] : 0.0f;
  float* ends = a.ends + (item0 * a.N + n) * a.D + d;
  const float* steps = a.steps + item0 * a.D + d;
  for (int64_t c = 0; c < chunks; c += kCarry) {
    float e[kCarry], s[kCarry];
#pragma unroll
    for (int k = 0; k < kCarry; ++k) {
      const bool in = c + k < chunks - 1;  // the last chunk has no end state here
      e[k] = in ? ends[(c + k) * DN] : 0.0f;
      s[k] = in ? steps[(c + k) * a.D] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kCarry; ++k) {
      if (c + k < chunks) ends[(c + k) * DN] = h;
      h = fmaf(hw_exp2(s[k] * A), h, e[k]);
    }
  }
}

// One token per sequence: 1 << lanes_log2 lanes share a channel, each taking V
// neighbouring state entries at a time, so a wave's state accesses are
// contiguous.  Memory-bound on the state, read and written once.
template <typename MT, int V>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a, int lanes_log2, int channel_tiles) {
  const int L = 1 << lanes_log2;
  const int64_t b = blockIdx.x / channel_tiles;
  const int64_t d = (int64_t)(blockIdx.x % channel_tiles) * (256 >> lanes_log2) + (threadIdx.x >> lanes_log2);
  const int l = threadIdx.x & (L - 1);
  const int64_t slot = slot_of(a.index, b, a.slots);
  if (slot < 0 || d >= a.D) return;
  const int64_t g = d / (a.D / a.G);
  const float x = to_float(static_cast<const MT*>(a.x)[b * a.x_sb + d]);
  const float dt =
      step_size(a, to_float(static_cast<const MT*>(a.dt)[b * a.dt_sb + d]), a.dt_bias ? a.dt_bias[d] : 0.0f);
  const MT* Bm = static_cast<const MT*>(a.Bm) + b * a.b_sb + g * a.N;
  const MT* Cm = static_cast<const MT*>(a.Cm) + b * a.c_sb + g * a.N;
  float* st = a.state_out + (slot * a.D + d) * a.N;
  float y = 0.0f;
  for (int n = l * V; n < a.N; n += L * V) {
    float h[V], A[V];
    __builtin_memcpy(h, __builtin_assume_aligned(st + n, V * 4), V * 4);
    __builtin_memcpy(A, __builtin_assume_aligned(a.A + d * a.N + n, V * 4), V * 4);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      h[e] = fmaf(hw_exp2(dt * A[e] * kLog2e), h[e], dt * x * to_float(Bm[n + e]));
      y = fmaf(h[e], to_float(Cm[n + e]), y);
    }
    __builtin_memcpy(__builtin_assume_aligned(st + n, V * 4), h, V * 4);
  }
  for (int m = L >> 1; m >= 1; m >>= 1) y += __shfl_xor(y, m, 64);
  if (l == 0) {
    if (a.skip) y = fmaf(a.skip[d], x, y);
    if (a.z) y *= silu(to_float(static_cast<const MT*>(a.z)[b * a.z_sb + d]));
    static_cast<MT*>(a.out)[b * a.o_sb + d] = (MT)y;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename MT, int NN, int CT>
hipError_t ssm_launch(const SsmArgs& a, hipStream_t stream) {
  const int64_t per = a.D / a.G, tiles = (per + 64 * CT - 1) / (64 * CT);
  const int NG = (int)((a.N + NN - 1) / NN), threads = NG * CT * 64;
  const int64_t items = a.off ? a.T / a.chunk + a.B : a.B * a.chunks, blocks = items * a.G * tiles;
  const int64_t carries = (a.B * a.D * a.N + 255) / 256;
  if (!grid_fits(blocks, threads) || !grid_fits(carries, 256) || tiles > 0x7FFFFFFF) return hipErrorNotSupported;
  const size_t stage = (size_t)kStage * 2 * NG * NN * sizeof(float);
  const size_t partials = NG > 1 ? (size_t)NG * CT * kAhead * 64 * sizeof(float) : 0;
  if (a.ends) {
    hipLaunchKernelGGL((ssm_kernel<MT, NN, CT, true>), dim3((unsigned)blocks), dim3(threads), (unsigned)stage, stream, a,
                       NG, (int)tiles);
    hipLaunchKernelGGL(ssm_carry_kernel, dim3((unsigned)carries), dim3(256), 0, stream, a);
  }
  hipLaunchKernelGGL((ssm_kernel<MT, NN, CT, false>), dim3((unsigned)blocks), dim3(threads), (unsigned)(stage + partials),
                     stream, a, NG, (int)tiles);
  return hipGetLastError();
}

}  // namespace

SsmPlan ssm_plan(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, bool packed) {
  SsmPlan p;
  const int64_t waves = G * ((D / G + 63) / 64) * ((N + 15) / 16);  // of one sequence
  const int64_t rows = packed ? T : B * T;
  p.split = packed || B * waves < 768;
  int64_t chunk = (rows * waves / 4096 + kStage - 1) / kStage * kStage;
  if (chunk < 64) chunk = 64;
  if (chunk < T / 128) chunk = (T / 128 + kStage) / kStage * kStage;
  if (!p.split || chunk >= T) {
    p.split = false;
    chunk = T < 1 ? 1 : T;
  }
  p.chunk = chunk;
  p.chunks = T < 1 ? 1 : (T + chunk - 1) / chunk;
  p.ends_bytes = p.total_bytes = 0;
  if (p.split) {
    const int64_t items = packed ? T / chunk + B : B * p.chunks;
    // (no overflow: a split leaves D N below 2^23)
    const size_t entries = (size_t)(items * D);
    p.ends_bytes = align_up(entries * N * 4, 256);
    p.total_bytes = p.ends_bytes + align_up(entries * 4, 256);
  }
  return p;
}

template <typename MT>
hipError_t launch_ssm(const SsmArgs& a, hipStream_t stream) {
  // channel tiles per workgroup: four waves' worth, fewer where the entries
  // already split over waves or the group has fewer channels
  const int64_t tiles = (a.D / a.G + 63) / 64;
  if (a.N <= 8) return ssm_launch<MT, 8, 4>(a, stream);
  if (a.N <= 16 && tiles > 2) return ssm_launch<MT, 16, 4>(a, stream);
  if (a.N <= 32 && tiles > 1) return ssm_launch<MT, 16, 2>(a, stream);
  return ssm_launch<MT, 16, 1>(a, stream);
}

template <typename MT>
hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t stream) {
  const bool v4 = a.N % 4 == 0 && aligned16(a.state_out) && aligned16(a.A);
  const int64_t lanes = v4 ? a.N / 4 : a.N;
  int l = 0;
  while (l < 6 && ((int64_t)1 << l) < lanes) ++l;
  const int64_t ctiles = (a.D + (256 >> l) - 1) / (256 >> l);
  if (!grid_fits(a.B * ctiles, 256)) return hipErrorNotSupported;
  if (v4)
    hipLaunchKernelGGL((ssm_step_kernel<MT, 4>), dim3((unsigned)(a.B * ctiles)), dim3(256), 0, stream, a, l, (int)ctiles);
  else
    hipLaunchKernelGGL((ssm_step_kernel<MT, 1>), dim3((unsigned)(a.B * ctiles)), dim3(256), 0, stream, a, l, (int)ctiles);
  return hipGetLastError();
}

template hipError_t launch_ssm<float>(const SsmArgs&, hipStream_t);
template hipError_t launch_ssm<bf16>(const SsmArgs&, hipStream_t);
template hipError_t launch_ssm_step<float>(const SsmArgs&, hipStream_t);
template hipError_t launch_ssm_step<bf16>(const SsmArgs&, hipStream_t);

}  // namespace gdn
