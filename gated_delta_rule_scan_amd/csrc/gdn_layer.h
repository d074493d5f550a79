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

// rows into the cache (k, v read) or out of it (k, v written)
struct KvArgs {
  void* k;
  void* v;
  void* k_cache;
  void* v_cache;
  uint8_t* k_scales;
  uint8_t* v_scales;
  const int32_t* off;
  const int32_t* table;
  const int32_t* start;
  int64_t B, T, width, pages;
  int64_t k_sb, k_st, k_sh, v_sb, v_st, v_sh;
  int Hk, d;
  int page_bits;         // log2 of the tokens of a page
  int zero_unused;
  int chunk_bits;        // log2 of the tokens per workgroup
  int heads;             // heads per workgroup
  int64_t chunks;        // runs of tokens per sequence (not packed)
  int64_t first;         // of the launch's runs
};

struct AttendArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* lengths;
  int64_t B, width, pages;
  int64_t q_sb, q_sh, o_sb, o_sh;
  int64_t window, sinks;
  int64_t tiles;         // that a sequence may have (about)
  int Hq, Hk, d, page_bits;
  int q_aligned;         // every row of q starts on 16 bytes
  int once;              // pools are read past the caches
  float scale;
  int64_t first;         // of the launch's items (sequences, in the join)
  int64_t items;         // runs of tiles; the workspace, or null where no sequence can be split:
  int32_t* plan;         // [B][2] first item and items of a sequence
  float* parts;          // [items][Hq][d] sums of weighted values
  float* stats;          // [items][Hq][2] maximum, sum of weights
};

// How a call's sequences are cut, and the workspace that takes.
struct AttendPlan {
  int64_t items;
  size_t plan_bytes, parts_bytes, total_bytes;
};
AttendPlan attend_plan(int64_t B, int64_t Hq, int64_t Hk, int64_t d, bool half, int64_t reach, int64_t window, int64_t sinks);

struct NormArgs {
  const void* x;
  const void* y;
  void* h;               // backward: dh, read
  void* n;               // backward: dn, read
  void* dx;
  void* dy;
  const float* gate;
  const float* post;
  const float* weight;
  const int32_t* off;
  int64_t B, T, D;
  int64_t x_sb, x_st, y_sb, y_st, h_sb, h_st, n_sb, n_st, dx_sb, dx_st, dy_sb, dy_st;
  int64_t gate_sb;
  float alpha, eps;
  int zero_unused;
  int64_t chunk;         // rows per workgroup
  int64_t chunks;        // workgroups per sequence (not packed)
  int64_t items;         // workgroups
  int64_t first;         // of the launch's (of the gradients, in their sums)
  // backward: the sums over a workgroup's rows [item][sums][D], and where
  // the gradients' sums go (null: not wanted)
  float* parts;
  int sums;
  float* dgate;
  float* dpost;
  float* dweight;
};

// How the rows of a seam are divided among workgroups.
struct NormPlan {
  int64_t chunk, chunks, items;
};
NormPlan norm_plan(int64_t B, int64_t T, int64_t D, bool half, bool packed, bool backward);

// ---- launchers (host) ----
template <typename MT>
hipError_t launch_kv(const KvArgs& a, int format, bool write, bool aligned, hipStream_t stream);
template <typename MT>
hipError_t launch_attend(const AttendArgs& a, int format, hipStream_t stream);
template <typename MT>
hipError_t launch_norm(const NormArgs& a, bool aligned, hipStream_t stream);
template <typename MT>
hipError_t launch_norm_back(const NormArgs& a, bool aligned, hipStream_t stream);
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

// Work of `count` parts, each of `blocks` blocks, in as many launches as that
// takes: launch(first part, its blocks).
template <typename Launch>
hipError_t in_launches(int64_t count, int64_t blocks, int threads, Launch launch) {
  const int64_t most = (((int64_t)1 << 32) - 1) / threads / blocks;
  for (int64_t at = 0; at < count; at += most) {
    launch(at, dim3((unsigned)((count - at < most ? count - at : most) * blocks)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

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

// Joins x over the four lane groups of sixteen, for every place in a group:
// rows of 16 lanes are swapped by pairs, then the wave's halves.  (The swapped
// words are copied before they are taken as floats: a bit cast of a vector's
// element takes the first one.)
template <typename Join>
__device__ __forceinline__ float over_groups(float x, Join join) {
  unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned a = r[0], b = r[1];
  u = __builtin_bit_cast(unsigned, join(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned c = s[0], d = s[1];
  return join(__builtin_bit_cast(float, c), __builtin_bit_cast(float, d));
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
