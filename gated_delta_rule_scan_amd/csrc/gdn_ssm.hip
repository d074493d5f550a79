// Selective state space scan, for prompts and for single tokens: per channel
// d an fp32 state h of N entries,
//
//   dt' = softplus(dt + bias),  h_n = exp(dt' A_n) h_n + dt' x B_n,
//   y = sum_n h_n C_n + skip x,  out = y silu(z)
#include <type_traits>

#include "gdn_layer.h"

namespace gdn {
namespace {

__device__ __forceinline__ float step_size(const SsmArgs& a, float dt, float bias) {
  const float v = dt + bias, p = softplus(v);
  return a.softplus ? p : v;
}

// A for base-2 exponents.  Minus infinity becomes the lowest number: its
// product with a step size of zero is zero, not NaN.
constexpr float kLargest = 3.402823466e38f;
__device__ __forceinline__ float rate(float A) {
  const float r = A * kLog2e;
  return r < -kLargest ? -kLargest : r;
}

// ---- prompts ----
// Per token, channel and state entry a pass takes one exponential (the issue
// time of three multiply-adds), the products dt A and dt x B, the update and
// the readout; the decay depends on channel and entry, so nothing here is a
// product of matrices, and the vector units bound it, not memory.  (The input
// and readout products as 4 x 4 x 1 matrix instructions were right but 10%
// slower: such an instruction issues as long as three multiply-adds too, and
// nothing overlaps it.)
//
// A lane owns a channel and NN state entries in registers and walks the tokens
// in order, so rows of x, dt, z and out move in whole cache lines.  The B and C
// of the next kStage tokens wait in the wave's own part of LDS as fp32 and
// reach all lanes by 16-byte broadcast reads; waves do not wait for each other.
// More than 32 entries are split over waves that do, to add up their partial
// readouts in LDS.
//
// Too few channels to fill the GPU: sequences are cut into chunks and three
// kernels run.  The first (STATES) finds each chunk's end state from a zero
// start, and the sum of its step sizes: a chunk's whole decay is exp(A sum
// dt).  The second (carry) turns those into the state that enters each chunk;
// the third is the scan itself from there.  The first costs the exponentials
// once more; a sequence's last chunk, and with it a sequence of one chunk, is
// spared it.
//
// 32768 tokens x 2048 channels x 16 entries, bf16, gated: 411-420 us (under a
// profiler, which slows them, first pass 200, carry 11, scan 255-263).  The scan
// issues 115 vector instructions per token and wave, 80 of them the formula's,
// 20 of them exponentials and reciprocals; at their measured issue times (3.1
// and 9 cycles, four waves a SIMD) 200 us.  Its memory traffic alone would take
// 107 us.

// Tokens computed while the next ones' inputs are in flight (4: 435 us against
// 427 with 8 at the size above).
constexpr int kStage = 8;

struct Chunk {
  int64_t b;            // sequence
  int64_t item;         // its place in the workspace
  int64_t t0, t1, len;  // tokens of the sequence
  int64_t row0;         // first row of a packed sequence
  int64_t clear;        // rows of no sequence from this item's tokens on, up to this one (0: none)
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
  // the last sequence's items also hold the rows behind it
  c.clear = 0;
  if (a.zero_unused && a.off && c.b == a.B - 1 && k >= 0) {
    c.clear = a.T - c.row0 < c.t0 + a.chunk ? a.T - c.row0 : c.t0 + a.chunk;
    if (c.clear <= c.t1 || c.clear <= c.t0) c.clear = 0;
  }
  return c;
}

// One element through a buffer resource: uniform base, the lane's offset, a
// uniform offset (bytes).
// A loaded value as its bits in a register of its own, converted where it is
// used: bf16 values held as such get packed in pairs right behind their loads,
// which waits for the loads there.
template <typename MT>
__device__ __forceinline__ unsigned buffer_load(rsrc_t r, unsigned lane_off, unsigned off) {
  if constexpr (sizeof(MT) == 2) return (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, (int)lane_off, (int)off, 0);
  else return __builtin_amdgcn_raw_buffer_load_b32(r, (int)lane_off, (int)off, 0);
}
template <typename MT>
__device__ __forceinline__ float from_bits(unsigned bits) {
  return __builtin_bit_cast(float, sizeof(MT) == 2 ? bits << 16 : bits);
}
template <typename MT>
__device__ __forceinline__ void buffer_store(MT v, rsrc_t r, unsigned lane_off, unsigned off) {
  if constexpr (sizeof(MT) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, v), r, (int)lane_off, (int)off, 0);
  else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v), r, (int)lane_off, (int)off, 0);
}
// Resources reach kReach bytes; a lane offset of kNowhere lies outside of any,
// so its loads give zero and its stores are dropped.
constexpr unsigned kReach = 0x7FFFFFFFu, kNowhere = 0x80000000u;

// A lane's state entries, `wide` of NN (the rest zero); vec4: rows of whole,
// aligned 16-byte pieces.
template <int NN>
__device__ __forceinline__ void load_entries(const float* p, int wide, int vec4, float (&v)[NN]) {
  if (vec4) {
#pragma unroll
    for (int i = 0; i < NN; i += 4) {
      const f32x4 q = i < wide ? *reinterpret_cast<const f32x4*>(p + i) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i + e] = q[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NN; ++i) v[i] = i < wide ? p[i] : 0.0f;
  }
}
template <int NN>
__device__ __forceinline__ void store_entries(float* p, int wide, int vec4, const float (&v)[NN]) {
  if (vec4) {
#pragma unroll
    for (int i = 0; i < NN; i += 4)
      if (i < wide) *reinterpret_cast<f32x4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < NN; ++i)
      if (i < wide) p[i] = v[i];
  }
}

// PADDED, for the readout: some wave has fewer than NN entries.  The rest stay
// zero by their zero B, but for an infinite input, whose product with it is NaN:
// such a token's are cleared, and its readout taken again.  (One test a token,
// below 1%; a mask an entry took 4% with up to 32 entries and 13% with more.)
template <typename MT, int NN, bool STATES, bool MULTI, bool GATE, bool PADDED>
__global__ __launch_bounds__(512, NN == 32 ? 2 : 4) void ssm_kernel(SsmArgs a, int waves_n, int CT, int tiles_per_group) {
  constexpr int ES = sizeof(MT), STEP = 64 / NN;       // tokens of B (or C) that a wave loads at a time
  constexpr int ROUNDS = kStage / STEP;
  static_assert(kStage % STEP == 0, "whole rounds");
  extern __shared__ __align__(16) float lds[];         // per wave [B, C][kStage][NN]; with MULTI then [wave][kStage][64]
  const int NG = MULTI ? waves_n : 1;                  // waves that share a channel tile's entries
  const int N = (int)a.N;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ng = wave / CT, ct = wave % CT;            // this wave's entries and channel tile
  const unsigned tiles = (unsigned)tiles_per_group * (unsigned)a.G;
  const Chunk c = chunk_of(a, blockIdx.x / tiles);
  if (STATES ? !c.work || c.t1 >= c.len : !c.work && !c.clear) return;  // (nothing follows a sequence's last chunk)
  const unsigned tile = blockIdx.x % tiles, g = tile / (unsigned)tiles_per_group;
  // the wave's first channel (uniform) and the lane's behind it; lanes without
  // a channel repeat the group's last one and store nothing
  const int64_t per = a.D / a.G, end = (g + 1) * per;
  const int64_t want = g * per + ((int64_t)(tile % (unsigned)tiles_per_group) * CT + ct) * 64;
  if ((STATES || !MULTI) && want >= end) return;  // the whole wave, and nobody waits for it
  const int64_t d0 = want < end ? want : end - 1;
  const bool live = want + lane < end;
  const unsigned dl = live ? lane : (unsigned)(end - 1 - d0);
  const int64_t d = d0 + dl;
  if (!STATES && c.clear) {
    if (live && ng == 0)
      for (int64_t t = c.t0 > c.t1 ? c.t0 : c.t1; t < c.clear; ++t) static_cast<MT*>(a.out)[(c.row0 + t) * a.o_st + d] = (MT)0.0f;
    if (!c.work) return;  // the whole workgroup
  }
  const int64_t slot = slot_of(a.index, c.b, a.slots);
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.skip ? a.skip[d] : 0.0f;

  const int wide = N - ng * NN < NN ? N - ng * NN : NN;  // entries of this wave
  const int64_t row = d * N + ng * NN;                   // of the channel's entries in A and in one state
  float A[NN], h[NN];
  load_entries(a.A + row, wide, a.vec4, A);
#pragma unroll
  for (int i = 0; i < NN; ++i) {
    A[i] = rate(A[i]);
    h[i] = 0.0f;
  }
  if (!STATES) {
    if (a.ends) load_entries(a.ends + c.item * a.D * N + row, wide, a.vec4, h);
    else if (a.state_in && slot >= 0) load_entries(a.state_in + slot * a.D * N + row, wide, a.vec4, h);
  }

  // Uniform pointers at the first token not yet loaded (out: stored); bytes
  // from token to token fit 32 bits.
  auto start = [&](const void* p, int64_t sb, int64_t st, int64_t col) {
    return static_cast<const char*>(p) + ((a.off ? c.row0 * st : c.b * sb) + c.t0 * st + col) * ES;
  };
  const char* px = start(a.x, a.x_sb, a.x_st, d0);
  const char* pd = start(a.dt, a.dt_sb, a.dt_st, d0);
  const char* pz = a.z ? start(a.z, a.z_sb, a.z_st, d0) : nullptr;
  const char* po = start(a.out, a.o_sb, a.o_st, d0);
  const char* pb = start(a.Bm, a.b_sb, a.b_st, g * a.N + ng * NN);
  const char* pc = start(a.Cm, a.c_sb, a.c_st, g * a.N + ng * NN);
  const unsigned sx = (unsigned)(a.x_st * ES), sd = (unsigned)(a.dt_st * ES), sz = (unsigned)(a.z_st * ES);
  const unsigned so = (unsigned)(a.o_st * ES), sb = (unsigned)(a.b_st * ES), sc = (unsigned)(a.c_st * ES);
  const unsigned lane_in = dl * ES, lane_out = live ? lane * ES : kNowhere;

  // B and C: a lane loads one entry of one of STEP tokens.  The resource ends
  // with the chunk's last token: behind it, and behind entry N, B and C are
  // zero.
  float* stage = lds + wave * 2 * kStage * NN;
  const int bt = lane / NN, bn = lane % NN;
  const unsigned lane_b = bn < wide ? bt * sb + bn * ES : kNowhere, lane_c = bn < wide ? bt * sc + bn * ES : kNowhere;
  unsigned bv[ROUNDS], cv[ROUNDS];
  auto load_bc = [&](int left) {  // left: tokens from pb, pc on
    auto records = [&](unsigned st) {
      const uint64_t n = (uint64_t)(left - 1) * st + wide * ES;
      return n < kReach ? (unsigned)n : kReach;
    };
    const rsrc_t rb = make_rsrc(pb, records(sb)), rc = make_rsrc(pc, records(sc));
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      bv[i] = buffer_load<MT>(rb, lane_b + i * STEP * sb, 0);
      if (!STATES) cv[i] = buffer_load<MT>(rc, lane_c + i * STEP * sc, 0);
    }
    pb += (uint64_t)kStage * sb;
    pc += (uint64_t)kStage * sc;
  };
  // x, dt and z of kStage tokens; past the end the last token repeats
  unsigned xv[kStage], dv[kStage], zv[kStage];
  auto load_rows = [&](int left) {  // left: tokens from px, pd, pz on
    const rsrc_t rx = make_rsrc(px, kReach), rd = make_rsrc(pd, kReach), rz = make_rsrc(pz, kReach);
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      const unsigned k = i < left ? i : left - 1;
      xv[i] = buffer_load<MT>(rx, lane_in, k * sx);
      dv[i] = buffer_load<MT>(rd, lane_in, k * sd);
      if (GATE) zv[i] = buffer_load<MT>(rz, lane_in, k * sz);
    }
    if (GATE) pz += (uint64_t)kStage * sz;
    px += (uint64_t)kStage * sx;
    pd += (uint64_t)kStage * sd;
  };

  constexpr int kWhole = MULTI || NN == 8 ? 1 : NN / 2 + 1;         // entries that every wave has
  unsigned there = wide < 32 ? (1u << wide) - 1 : 0xFFFFFFFFu;  // bit n: entry n is there
  double total = 0.0;  // of the step sizes: a chunk may have very many
  float* partial = lds + NG * CT * 2 * kStage * NN + wave * kStage * 64 + lane;
  int left = (int)(c.t1 - c.t0);  // tokens not yet computed
  if (left > 0) {
    load_bc(left);
    load_rows(left);
  }
  while (left > 0) {
    // (a wave's LDS accesses keep their order: no barrier)
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      stage[i * 64 + lane] = from_bits<MT>(bv[i]);
      if (!STATES) stage[kStage * NN + i * 64 + lane] = from_bits<MT>(cv[i]);
    }
    __builtin_amdgcn_wave_barrier();
    float xc[kStage], dc[kStage], zc[kStage];
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      xc[i] = from_bits<MT>(xv[i]);
      dc[i] = from_bits<MT>(dv[i]);
      if (GATE) zc[i] = from_bits<MT>(zv[i]);
    }
    if (left > kStage) {
      load_bc(left - kStage);
      load_rows(left - kStage);
    }
    const rsrc_t ro = make_rsrc(po, kReach);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kStage; ++i) {
      // past the end: decay 1, no input (infinite x or dt too), no store; a
      // branch instead keeps tokens from overlapping (412 -> 436 us at the size
      // above), a second copy of the loop spills
      const bool in = i < left;
      const float step = step_size(a, dc[i], bias);
      const float s = in ? step : 0.0f, u = in ? step * xc[i] : 0.0f;
      if (STATES) sum += s;
      float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
      for (int j = 0; j < NN / 4; ++j) {
        const f32x4 B = *reinterpret_cast<const f32x4*>(stage + i * NN + 4 * j);
        f32x4 C = {0.f, 0.f, 0.f, 0.f};
        if (!STATES) C = *reinterpret_cast<const f32x4*>(stage + kStage * NN + i * NN + 4 * j);
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
      if (PADDED && __builtin_expect(__any(!(fabsf(u) <= kLargest)), 0)) {
        asm volatile("" : "+s"(there));  // masks made here: kept ready for all tokens they spill
        y0 = y1 = 0.0f;
#pragma unroll
        for (int n = 0; n < NN; ++n) {
          if (n >= kWhole && !(there >> n & 1)) h[n] = 0.0f;
          (n & 1 ? y1 : y0) = fmaf(h[n], stage[kStage * NN + i * NN + n], n & 1 ? y1 : y0);
        }
      }
      if (!STATES && !MULTI) {
        float y = fmaf(skip, a.skip ? xc[i] : 0.0f, y0 + y1);  // (no skip: nothing of x, infinite perhaps)
        if (GATE) y *= silu(zc[i]);
        buffer_store<MT>((MT)y, ro, in ? lane_out : kNowhere, i * so);
      }
      if (!STATES && MULTI) partial[i * 64] = y0 + y1;
      __builtin_amdgcn_sched_barrier(0);  // one token's B and C in registers at a time
    }
    if (STATES) total += (double)sum;
    if (!STATES && MULTI) {
      // the waves of a channel tile take turns at the tokens' sums
      __syncthreads();
      int turn = ng;
#pragma unroll
      for (int i = 0; i < kStage; ++i) {
        if (turn == 0 && i < left) {
          const float* p = lds + NG * CT * 2 * kStage * NN + (ct * kStage + i) * 64 + lane;
          float y = a.skip ? skip * xc[i] : 0.0f;
          for (int k = 0; k < NG; ++k) y += p[k * CT * kStage * 64];
          if (GATE) y *= silu(zc[i]);
          buffer_store<MT>((MT)y, ro, lane_out, i * so);
        }
        turn = (turn ? turn : NG) - 1;
      }
      __syncthreads();
    }
    po += (uint64_t)kStage * so;
    left -= kStage;
  }
  if (!live) return;
  if (STATES) {
    store_entries(a.ends + c.item * a.D * N + row, wide, a.vec4, h);
    if (ng == 0) a.steps[c.item * a.D + d] = (float)total;
  } else if (a.state_out && slot >= 0 && c.t1 >= c.len) {
    store_entries(a.state_out + slot * a.D * N + row, wide, a.vec4, h);
  }
}

// The base-2 exponent of a chunk's decay, of its sum of step sizes; and the state
// behind a chunk, of the one that enters it and the one from zero.  A decay that
// rounds to zero is a product of many above zero, which keep an infinite state,
// or zero by an infinite step or rate, where that state has no value (0 * inf is
// NaN).  EXACT tells the two apart; without it both give NaN, and nothing that
// follows from NaN is a number: so chunks are walked without, and once more
// with it if the result is NaN (with it at once: 72 -> 73 us at 2048 tokens of
// 4096 channels).
__device__ __forceinline__ float decay_exponent(float steps, float rate) {
  return rate == -kLargest && steps > 0.0f ? -INFINITY : steps * rate;
}
template <bool EXACT>
__device__ __forceinline__ float behind(float h, float exponent, float end) {
  const float decay = hw_exp2(exponent), next = fmaf(decay, h, end);
  return EXACT && decay == 0.0f && exponent > -INFINITY && fabsf(h) == INFINITY ? h + end : next;
}

// Chunk end states become entering states, in place: a thread per channel and
// state entry of a sequence walks its chunks, kCarry of them in flight.  More
// chunks than that: PARTS threads take kCarry each at a time, join their parts'
// decays and end states in LDS, and go on from the state that enters theirs.
constexpr int kCarry = 16, kParts = 4;

template <int PARTS>
__global__ __launch_bounds__(256) void ssm_carry_kernel(SsmArgs a) {
  constexpr int ENTRIES = 256 / PARTS;
  __shared__ float2 joined[PARTS][ENTRIES];  // per part: its decay's exponent, and end state from zero
  const int64_t DN = a.D * a.N, tiles = (DN + ENTRIES - 1) / ENTRIES;
  const int i = threadIdx.x % ENTRIES, part = threadIdx.x / ENTRIES;
  const int64_t b = blockIdx.x / tiles, want = (blockIdx.x - b * tiles) * ENTRIES + i;
  const bool live = want < DN;
  const int64_t r = live ? want : DN - 1;
  const int64_t d = (uint64_t)r / (unsigned)a.N;
  int64_t item0 = b * a.chunks, len = a.T;
  if (a.off) {
    const int64_t row0 = clamp64(a.off[b], 0, a.T);
    item0 = row0 / a.chunk + b;
    len = clamp64(a.off[b + 1], row0, a.T) - row0;
  }
  const int64_t chunks = len > a.chunk ? (len + a.chunk - 1) / a.chunk : 1;
  const int64_t slot = slot_of(a.index, b, a.slots);
  const float A = rate(a.A[r]);
  float h = a.state_in && slot >= 0 ? a.state_in[slot * DN + r] : 0.0f;
  float* ends = a.ends + item0 * DN + r;
  const float* steps = a.steps + item0 * a.D + d;
  for (int64_t c0 = 0; c0 < chunks; c0 += PARTS * kCarry) {
    const int64_t c = c0 + part * kCarry;
    float e[kCarry], s[kCarry];
#pragma unroll
    for (int k = 0; k < kCarry; ++k) {
      const bool in = c + k < chunks - 1;  // the last chunk has no end state here
      e[k] = in ? ends[(c + k) * DN] : 0.0f;
      s[k] = in ? steps[(c + k) * a.D] : 0.0f;
    }
    // this part's chunks behind state g; STORE: the states that enter them
    auto walk = [&](float g, auto store) {
#pragma unroll
      for (int k = 0; k < kCarry; ++k) {
        if (store && live && c + k < chunks) ends[(c + k) * DN] = g;
        g = behind<false>(g, s[k] * A, e[k]);
      }
      return g;
    };
    // the same, EXACT, from memory: rare, and without registers of its own
    auto walk_exact = [&](float g, auto store) {
#pragma unroll 1
      for (int64_t k = c; k < c + kCarry && k < chunks; ++k) {
        const bool in = k < chunks - 1;
        const float end = in ? ends[k * DN] : 0.0f, step = in ? steps[k * a.D] : 0.0f;
        if (store && live) ends[k * DN] = g;
        g = behind<true>(g, decay_exponent(step, A), end);
      }
      return g;
    };
    constexpr std::true_type yes;
    constexpr std::false_type no;
    float sum = 0.0f, end = walk(PARTS > 1 ? 0.0f : h, no), next = end;
    bool exact = __any(isnan(end));
    if (PARTS > 1) {
      if (exact) end = walk_exact(0.0f, no);
#pragma unroll
      for (int k = 0; k < kCarry; ++k) sum += s[k];
      __syncthreads();  // the round before has been read
      joined[part][i] = make_float2(decay_exponent(sum, A), end);
      __syncthreads();
      const float start = h;
      auto join = [&](auto exactly) {
        h = next = start;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          const float2 j = joined[q][i];
          if (q < part) h = behind<decltype(exactly)::value>(h, j.x, j.y);
          next = behind<decltype(exactly)::value>(next, j.x, j.y);
        }
      };
      join(no);
      if (__any(isnan(next))) {
        exact = true;
        join(yes);
      }
    }
    // (without NaN so far there is none in this walk: its zero decays make zero products)
    const float g = exact ? walk_exact(h, yes) : walk(h, yes);
    h = PARTS > 1 ? next : g;
  }
}

// One token per sequence: 1 << lanes_log2 lanes share a channel, each taking V
// neighbouring state entries (with V = 1 up to four of them, 64 apart), so a
// wave's state accesses are contiguous; a thread takes kChannels channels.
// Memory-bound on the state, read and written once, and on the latency of
// what comes before: only the state's address waits for the slot index, and
// everything else is on its way by then.  128 sequences x 4096 channels x 16
// entries: 14.0 us for 72 MB (5.1 TB/s); with 1, 2, 4 channels a thread 18,
// 14.3, 15.6 us.
constexpr int kChannels = 2;

template <typename MT, int V>
struct __attribute__((aligned(V * sizeof(MT)))) Entries {
  MT e[V];
};

template <typename MT, int V>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a, int lanes_log2, int tiles_per_group, int bc_vec) {
  constexpr int PARTS = V == 4 ? 1 : 4;  // V = 4: 64 lanes hold the 256 entries there can be
  const int L = 1 << lanes_log2, rows = 256 >> lanes_log2, N = (int)a.N;
  const unsigned tiles = (unsigned)tiles_per_group * (unsigned)a.G;
  const int64_t b = blockIdx.x / tiles;
  const unsigned tile = blockIdx.x % tiles, g = tile / (unsigned)tiles_per_group;
  const int64_t per = a.D / a.G, end = (g + 1) * per;
  // the workgroup's first channel (uniform), and this thread's behind it;
  // channels behind the group's last repeat it and store nothing
  const int64_t base = g * per + (int64_t)(tile % (unsigned)tiles_per_group) * rows * kChannels;
  const int l = threadIdx.x & (L - 1), left = end - base < 0x10000 ? (int)(end - base) : 0x10000;
  const int64_t slot = slot_of(a.index, b, a.slots);
  unsigned c[kChannels];
  bool live[kChannels];
  float x[kChannels], dt[kChannels];
  Entries<float, V> A[PARTS][kChannels], h[PARTS][kChannels];
  Entries<MT, V> B[PARTS], C[PARTS];
  const MT* px = static_cast<const MT*>(a.x) + b * a.x_sb + base;
  const MT* pd = static_cast<const MT*>(a.dt) + b * a.dt_sb + base;
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    const int ch = (threadIdx.x >> lanes_log2) + i * rows;
    live[i] = ch < left;
    c[i] = live[i] ? ch : left - 1;
    x[i] = to_float(px[c[i]]);
    dt[i] = to_float(pd[c[i]]) + (a.dt_bias ? (a.dt_bias + base)[c[i]] : 0.0f);
  }
  // this thread finishes one of its channels (or all, with fewer lanes than channels)
  const int mine = L >= kChannels ? l % kChannels : 0;
  unsigned cf = c[0];
#pragma unroll
  for (int i = 1; i < kChannels; ++i) cf = mine == i ? c[i] : cf;
  const float zf = a.z ? to_float((static_cast<const MT*>(a.z) + b * a.z_sb + base)[cf]) : 0.0f;
  const float skipf = a.skip ? (a.skip + base)[cf] : 0.0f;
  const MT* Bm = static_cast<const MT*>(a.Bm) + b * a.b_sb + (int64_t)g * N;
  const MT* Cm = static_cast<const MT*>(a.Cm) + b * a.c_sb + (int64_t)g * N;
  const float* Ab = a.A + base * N;
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    const int n = (q * L + l) * V;
    const bool in = n < N;
#pragma unroll
    for (int e = 0; e < V; ++e) B[q].e[e] = C[q].e[e] = (MT)0.0f;
    if (in) {
      if (bc_vec) {
        B[q] = *reinterpret_cast<const Entries<MT, V>*>(Bm + n);
        C[q] = *reinterpret_cast<const Entries<MT, V>*>(Cm + n);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          B[q].e[e] = Bm[n + e];
          C[q].e[e] = Cm[n + e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kChannels; ++i) A[q][i] = *reinterpret_cast<const Entries<float, V>*>(Ab + c[i] * (unsigned)N + (in ? n : 0));
  }
  if (slot < 0) {  // the whole workgroup
    if (a.zero_unused) {
#pragma unroll
      for (int i = 0; i < kChannels; ++i)
        if (live[i] && l == 0) (static_cast<MT*>(a.out) + b * a.o_sb + base)[c[i]] = (MT)0.0f;
    }
    return;
  }
  float* S = a.state_out + (slot * a.D + base) * N;
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    const int n = (q * L + l) * V;
#pragma unroll
    for (int i = 0; i < kChannels; ++i)
      h[q][i] = *reinterpret_cast<const Entries<float, V>*>(S + c[i] * (unsigned)N + (n < N ? n : 0));
  }
  float y[kChannels];
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    const float s = step_size(a, dt[i], 0.0f), u = s * x[i];
    y[i] = 0.0f;
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      const int n = (q * L + l) * V;
      if (V == 1 && n >= N) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        h[q][i].e[e] = fmaf(hw_exp2(s * rate(A[q][i].e[e])), h[q][i].e[e], u * to_float(B[q].e[e]));
        y[i] = fmaf(h[q][i].e[e], to_float(C[q].e[e]), y[i]);
      }
      if (live[i] && n < N) *reinterpret_cast<Entries<float, V>*>(S + c[i] * (unsigned)N + n) = h[q][i];
    }
    if (V > 1 && l * V >= N) y[i] = 0.0f;  // a lane behind entry N ran entry 0's state, infinite perhaps
  }
  for (int m = L >> 1; m >= 1; m >>= 1) {
#pragma unroll
    for (int i = 0; i < kChannels; ++i) y[i] += __shfl_xor(y[i], m, 64);
  }
  MT* po = static_cast<MT*>(a.out) + b * a.o_sb + base;
#pragma unroll
  for (int i = 0; i < kChannels; ++i) {
    if (!live[i] || l != (L >= kChannels ? i : 0)) continue;
    const bool own = L >= kChannels || i == 0;  // whose gate and skip this thread holds
    const float sk = own ? skipf : a.skip ? (a.skip + base)[c[i]] : 0.0f;
    const float zi = own ? zf : a.z ? to_float((static_cast<const MT*>(a.z) + b * a.z_sb + base)[c[i]]) : 0.0f;
    const float v = a.skip ? fmaf(sk, x[i], y[i]) : y[i];
    po[c[i]] = (MT)(a.z ? v * silu(zi) : v);
  }
}

template <typename MT, int NN, bool PADDED>
auto scan_kernel(bool multi, bool gate) {
  constexpr bool kMulti = NN == 32;
  return multi ? (gate ? ssm_kernel<MT, NN, false, kMulti, true, PADDED> : ssm_kernel<MT, NN, false, kMulti, false, PADDED>)
               : (gate ? ssm_kernel<MT, NN, false, false, true, PADDED> : ssm_kernel<MT, NN, false, false, false, PADDED>);
}

template <typename MT, int NN>
hipError_t ssm_launch(const SsmArgs& a, hipStream_t stream) {
  // four waves a workgroup: channel tiles, fewer where the entries already
  // take several waves
  const int NG = (int)((a.N + NN - 1) / NN), CT = NG >= 4 ? 1 : 4 / NG, threads = NG * CT * 64;
  const int64_t per = a.D / a.G, tiles = (per + 64 * CT - 1) / (64 * CT);
  const int64_t items = a.off ? a.T / a.chunk + a.B : a.B * a.chunks, blocks = items * a.G * tiles;
  // parts where a sequence (a packed one of average length) fills half of them
  // (32 chunks: 38 -> 33 us at 512 tokens of 4096 channels; 9 of each packed
  // sequence: 147 -> 171 us at the sizes below)
  const int64_t chunks = a.off ? (a.T / a.B + a.chunk - 1) / a.chunk : a.chunks;
  const int parts = chunks >= kParts * kCarry / 2 ? kParts : 1;
  const int64_t carries = a.B * ((a.D * a.N * parts + 255) / 256);
  if (!grid_fits(blocks, threads) || (a.ends && !grid_fits(carries, 256))) return hipErrorNotSupported;
  constexpr bool kMulti = NN == 32;
  const bool multi = kMulti && NG > 1, padded = a.N % NN != 0;
  const unsigned stage = (unsigned)(NG * CT * kStage * 2 * NN * sizeof(float));
  const unsigned partials = multi ? (unsigned)(NG * CT * kStage * 64 * sizeof(float)) : 0;
  if (a.ends) {
    const auto states = multi ? ssm_kernel<MT, NN, true, kMulti, false, false> : ssm_kernel<MT, NN, true, false, false, false>;
    hipLaunchKernelGGL(states, dim3((unsigned)blocks), dim3(threads), stage, stream, a, NG, CT, (int)tiles);
    hipLaunchKernelGGL(parts > 1 ? ssm_carry_kernel<kParts> : ssm_carry_kernel<1>, dim3((unsigned)carries), dim3(256), 0, stream, a);
  }
  const auto scan = padded ? scan_kernel<MT, NN, true>(multi, a.z) : scan_kernel<MT, NN, false>(multi, a.z);
  hipLaunchKernelGGL(scan, dim3((unsigned)blocks), dim3(threads), stage + partials, stream, a, NG, CT, (int)tiles);
  return hipGetLastError();
}

}  // namespace

SsmPlan ssm_plan(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, bool packed) {
  SsmPlan p;
  const int64_t waves = G * ((D / G + 63) / 64) * ((N + 31) / 32);  // of one sequence
  const int64_t all = B < ((int64_t)1 << 40) / waves ? B * waves : (int64_t)1 << 40;
  // Waves that run at once (registers: four a SIMD up to 16 entries, else
  // two); chunks as short as that takes, but not so short that the carry over
  // them costs more than their tokens (4096 channels: 128 tokens in chunks of
  // 8, 16, 32: 20, 22, 30 us; 256: 29, 24, 31; 512: 35, 33, 34; 1024: 47, 47,
  // 45).
  // Packed sequences, whose lengths differ, are cut finer (twice the waves), so
  // that no long one is left alone at the end: 160 -> 147 us at 24 sequences,
  // 9001 tokens and 2048 channels.
  const int64_t room = N <= 16 ? 4096 : 2048;
  int64_t pieces;  // chunks of a sequence; of the whole packed batch (where every sequence may leave a rest)
  if (packed) pieces = 2 * room / waves - B > room / (4 * waves) ? 2 * room / waves - B : room / (4 * waves);
  else pieces = room / all;
  if (pieces < 1) pieces = 1;
  int64_t chunk = ((T + pieces - 1) / pieces + kStage - 1) / kStage * kStage;
  const int64_t least = T <= 128 ? kStage : T <= 512 ? 2 * kStage : 4 * kStage;
  if (chunk < least) chunk = least;
  // One kernel where most SIMDs have a wave anyway (512 tokens of 4096
  // channels: 8 sequences 189 us against 123 us split, 12: 189 and 186, 16: 191
  // and 223), or few tokens (0.35 us each at a wave a SIMD: 32 tokens 15.3 us
  // against 16.2, 40 tokens 18.0 against 16.6).
  p.split = T > 36 && chunk < T && (packed || all < 768);
  if (!p.split) chunk = T < 1 ? 1 : T;
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
  if (a.N <= 8) return ssm_launch<MT, 8>(a, stream);
  if (a.N <= 16) return ssm_launch<MT, 16>(a, stream);
  return ssm_launch<MT, 32>(a, stream);
}

template <typename MT>
hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t stream) {
  const int64_t lanes = a.vec4 ? a.N / 4 : a.N;
  int l = 0;
  while (l < 6 && ((int64_t)1 << l) < lanes) ++l;
  const int64_t rows = (256 >> l) * kChannels, ctiles = (a.D / a.G + rows - 1) / rows;
  if (!grid_fits(a.B * a.G * ctiles, 256)) return hipErrorNotSupported;
  auto quads = [&](const void* p, int64_t sb) {
    return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(MT)) == 0 && (a.B == 1 || sb % 4 == 0);
  };
  const int bc_vec = a.vec4 && quads(a.Bm, a.b_sb) && quads(a.Cm, a.c_sb);
  if (a.vec4)
    hipLaunchKernelGGL((ssm_step_kernel<MT, 4>), dim3((unsigned)(a.B * a.G * ctiles)), dim3(256), 0, stream, a, l, (int)ctiles,
                       bc_vec);
  else
    hipLaunchKernelGGL((ssm_step_kernel<MT, 1>), dim3((unsigned)(a.B * a.G * ctiles)), dim3(256), 0, stream, a, l, (int)ctiles,
                       1);
  return hipGetLastError();
}

template hipError_t launch_ssm<float>(const SsmArgs&, hipStream_t);
template hipError_t launch_ssm<bf16>(const SsmArgs&, hipStream_t);
template hipError_t launch_ssm_step<float>(const SsmArgs&, hipStream_t);
template hipError_t launch_ssm_step<bf16>(const SsmArgs&, hipStream_t);

}  // namespace gdn
