// Arguments and device helpers of the layer operators: short causal
// convolution, selective scan, rotary positions, single-token steps.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_common.h"

namespace gdn {

// ---- arguments ----

struct ConvArgs {
  const void* x;
  const float* weight;
  const float* bias;
  const void* state_in;
  void* state_out;
  void* out;
  const int32_t* off;    // packed batch: sequence offsets, else null
  const int32_t* index;  // state slots, or null
  int64_t B, T, D, slots;
  int64_t x_sb, x_st, o_sb, o_st;
  int silu;
  int zero_unused;       // rows of no sequence become zero
  int batches;           // runs of kConvRows tokens per thread
};

struct SsmArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* Bm;
  const void* Cm;
  const void* z;
  const float* dt_bias;
  const float* skip;
  const float* state_in;
  float* state_out;
  void* out;
  const int32_t* off;
  const int32_t* index;
  int64_t B, T, D, N, G, slots;
  int64_t x_sb, x_st, dt_sb, dt_st, z_sb, z_st, b_sb, b_st, c_sb, c_st, o_sb, o_st;
  int softplus;
  int zero_unused;
  int vec4;  // entries of A and of the states come in whole, aligned 16-byte pieces
  // prompts: tokens per chunk, chunks of an unpacked sequence, and where
  // sequences are split (else null) the workspace: chunk end states, then
  // entering states [item][D][N], and sums of step sizes [item][D]
  int64_t chunk, chunks;
  float* ends;
  float* steps;
};

// How a selective scan over prompts is split, and the workspace that takes.
struct SsmPlan {
  bool split;
  int64_t chunk, chunks;
  size_t ends_bytes, total_bytes;
};
SsmPlan ssm_plan(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, bool packed);

struct RotaryArgs {
  const void* q;
  const void* k;
  void* qo;
  void* ko;
  const double* freq;
  const void* pos;
  int64_t B, T, tokens, position0;
  int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh;
  int64_t qo_sb, qo_st, qo_sh, ko_sb, ko_st, ko_sh;
  int Hq, Hk, d, rot;
  int bits, axes;
  int edge[4];           // first pair behind each axis
  int interleaved, inverse, in_place_q, in_place_k;
  int token_tile;        // tokens per workgroup
  int head_split;        // workgroups that share one tile's heads
  float scale;
};

struct StepArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* log_alpha;
  const float* beta;
  float* state;
  float* out;
  const int32_t* index;
  const void* gate;
  const float* norm_weight;
  float norm_eps;
  int64_t B, H, slots;
  int dv;
  int erase, exclusive, zero_unused;
};

// ---- launchers (host) ----
template <typename MT>
hipError_t launch_conv(const ConvArgs& a, int width, bool aligned, hipStream_t stream);
template <typename MT>
hipError_t launch_conv_step(const ConvArgs& a, int width, bool aligned, hipStream_t stream);
template <typename MT>
hipError_t launch_ssm(const SsmArgs& a, hipStream_t stream);
template <typename MT>
hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t stream);
template <typename MT>
hipError_t launch_rotary(const RotaryArgs& a, bool aligned, hipStream_t stream);
template <typename MT>
hipError_t launch_step(const StepArgs& a, int dk, hipStream_t stream);

// Blocks of `threads` that one launch may have (the launch's work items are
// counted in 32 bits).
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= (((int64_t)1 << 32) - 1) / threads && blocks <= 0x7FFFFFFF; }

// ---- small device helpers ----

template <typename MT>
__device__ __forceinline__ float to_float(MT x) { return (float)x; }

// 2^x, log2 x and 1/x by the hardware instructions (1 ulp)
__device__ __forceinline__ float hw_exp2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float hw_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

constexpr float kLog2e = 1.4426950408889634f;

// x * sigmoid(x) = x / (1 + 2^(-x log2 e)); -inf gives NaN like the formula
__device__ __forceinline__ float silu(float x) { return x * hw_rcp(1.0f + hw_exp2(-kLog2e * x)); }

// log(1 + e^x) = max(x, 0) + log1p(t), t = e^-|x| in (0, 1].  log1p(t) =
// 2 atanh(s), s = t / (2 + t) <= 1/3: no cancellation, so small steps keep
// their relative precision.  2 atanh(s) / s as a polynomial of degree four in
// s^2, the one of least relative error on [0, 1/9] (8e-9, found by exchange).
__device__ __forceinline__ float softplus(float x) {
  const float t = hw_exp2(-kLog2e * fabsf(x));
  const float s = t * hw_rcp(2.0f + t);
  const float w = s * s;
  float p = 0.28178334f;
  p = fmaf(p, w, 0.27960601f);
  p = fmaf(p, w, 0.40024909f);
  p = fmaf(p, w, 0.66666317f);
  p = fmaf(p, w, 2.0f);
  return fmaf(s, p, fmaxf(x, 0.0f));
}

// Slot of sequence b, or -1 (no state): an index outside 0..slots-1 is no slot.
__device__ __forceinline__ int64_t slot_of(const int32_t* index, int64_t b, int64_t slots) {
  if (!index) return b;
  const int64_t s = index[b];
  return s >= 0 && s < slots ? s : -1;
}

// ---- packed batches ----
// Sequence s of a packed batch owns the items floor(off[s] / C) + s onwards,
// one per chunk of C tokens: off[s + 1] >= off[s] + len makes the next
// sequence's first item lie at least ceil(len / C) (and at least 1) further,
// so items never collide, an empty sequence still has one item, and
// floor(T / C) + B items hold them all.  An item past its sequence's chunks
// has nothing to do; those behind the last sequence's hold the rows behind it,
// all of them: its items go on up to floor(T / C) + B - 1, chunks enough for
// T - off[B - 1] tokens.
struct SeqItem {
  int64_t b;      // sequence
  int64_t row0;   // its first row in a packed buffer (0 for equal sequences)
  int64_t len;    // its tokens
  int64_t chunk;  // this item's chunk
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// The sequence of packed item `i`: a search by whole waves, 64 candidates a
// round (one round up to 64 sequences).  Every lane gets the same answer; the
// result is in range whatever the offsets hold.
__device__ __forceinline__ SeqItem find_packed(const int32_t* off, int64_t B, int64_t T, int64_t C, int64_t i) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, hi = B;  // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) / 64;
    const int64_t s = lo + lane * step;
    bool in = false;
    if (s < hi) in = clamp64(off[s], 0, T) / C + s <= i;
    const unsigned long long m = __ballot(in);
    const int n = m == 0 ? 0 : 63 - __builtin_clzll(m);
    lo += n * step;
    hi = lo + step < hi ? lo + step : hi;
  }
  SeqItem r;
  r.b = lo;
  r.row0 = clamp64(off[lo], 0, T);
  r.len = clamp64(off[lo + 1], r.row0, T) - r.row0;
  r.chunk = i - (r.row0 / C + lo);
  return r;
}

}  // namespace gdn
