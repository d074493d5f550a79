// Rotary positions on q and k:
//
//   (u, v) -> scale (u cos - v sin, v cos + u sin),  angle = position inv_freq[i]
//
// Memory-bound: every element is read and written once.  The angles cost far
// more arithmetic than the turn itself but are shared by all heads of a token,
// so a workgroup takes a few tokens, puts scale cos and scale sin of their
// pairs into LDS once, and then streams all heads of those tokens through
// (few tokens: several workgroups share a token's heads, so that the GPU still
// fills).  2 x 32760 x (16 + 16) heads x 128 bf16: 191-194 us for 1.08 GB, 5.5
// TB/s, a large copy's rate; 4096 x (32 + 8): 16.0 us for 84 MB.
//
// The angle is reduced in 64 bits: the number of quarter turns position *
// inv_freq * 2 / pi, minus the nearest whole number, leaves f in [-1/2, 1/2]
// with an error of 2^-52 of the whole count (below fp32's own at any position
// under 2^26).  What is left is within an eighth of a turn, |f pi / 2| <=
// pi / 4, where the Taylor series of sine (to x^11) and cosine (to x^12) end
// below 1e-9.
#include "gdn_layer.h"

namespace gdn {
namespace {

__device__ __forceinline__ float2 cos_sin(double quarter_turns) {
  const double n = rint(quarter_turns);
  const float x = (float)(quarter_turns - n) * 1.57079632679489662f;
  const int quadrant = (int)(n - 4.0 * floor(n * 0.25));
  const float w = x * x;
  float s = fmaf(w, -2.50521084e-8f, 2.75573192e-6f);  // -1/11!, 1/9!
  s = fmaf(w, s, -1.98412698e-4f);                     // -1/7!
  s = fmaf(w, s, 8.33333333e-3f);                      // 1/5!
  s = fmaf(w, s, -1.66666667e-1f);                     // -1/3!
  s = fmaf(x * w, s, x);
  float c = fmaf(w, 2.08767570e-9f, -2.75573192e-7f);  // 1/12!, -1/10!
  c = fmaf(w, c, 2.48015873e-5f);                      // 1/8!
  c = fmaf(w, c, -1.38888889e-3f);                     // -1/6!
  c = fmaf(w, c, 4.16666667e-2f);                      // 1/4!
  c = fmaf(w, c, -0.5f);
  c = fmaf(w, c, 1.0f);
  const float cq = (quadrant & 1) ? s : c, sq = (quadrant & 1) ? c : s;
  // quadrants: (c, s), (-s, c), (-c, -s), (s, -c)
  return make_float2(quadrant == 1 || quadrant == 2 ? -cq : cq, quadrant >= 2 ? -sq : sq);
}

constexpr int kThreads = 256;

// V elements per access: 16 bytes of aligned rows, else one.  An item of a
// head row is, in the half layout, V pairs (two accesses), interleaved V / 2
// pairs (one access; a single pair with V = 1), or V channels behind the
// rotated ones.
template <typename MT, int V, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a, int items, int rows_per_pass) {
  extern __shared__ float2 cs[];  // [token_tile][pairs]
  const int pairs = a.rot / 2, heads = a.Hq + a.Hk;
  const int64_t tile = blockIdx.x / a.head_split, tok0 = tile * a.token_tile;
  const int part = (int)(blockIdx.x % a.head_split);
  const int ntok = (int)(a.tokens - tok0 < a.token_tile ? a.tokens - tok0 : a.token_tile);
  for (int i = threadIdx.x; i < ntok * pairs; i += kThreads) {
    const int p = i % pairs;
    const int64_t tok = tok0 + i / pairs;
    int axis = 0;
    while (axis < a.axes - 1 && p >= a.edge[axis]) ++axis;
    double pos;
    if (a.bits == 64) pos = (double)static_cast<const int64_t*>(a.pos)[axis * a.tokens + tok];
    else if (a.bits == 32) pos = (double)static_cast<const int32_t*>(a.pos)[axis * a.tokens + tok];
    else pos = (double)(a.position0 + tok % a.T);
    float2 r = cos_sin(pos * (a.freq[p] * 0.63661977236758134308));
    r.x *= a.scale;
    r.y *= a.inverse ? -a.scale : a.scale;
    cs[i] = r;
  }
  __syncthreads();
  const int lane_row = (int)threadIdx.x / items, j = (int)threadIdx.x % items;
  if (lane_row >= rows_per_pass) return;
  // heads part, part + head_split, ... of every token of the tile
  const int my_heads = (heads - part + a.head_split - 1) / a.head_split;
  if (my_heads <= 0) return;
  const int rot_items = INTERLEAVED ? (V == 1 ? pairs : a.rot / V) : pairs / V;
  int tl = lane_row / my_heads, hh = lane_row % my_heads;
  const int step_t = rows_per_pass / my_heads, step_h = rows_per_pass % my_heads;
  const int64_t b0 = tok0 / a.T, t0 = tok0 - b0 * a.T;
  while (tl < ntok) {
    const int h = part + hh * a.head_split;
    int64_t b = b0, t = t0 + tl;
    while (t >= a.T) {
      t -= a.T;
      ++b;
    }
    const bool isq = h < a.Hq;
    const MT* src = isq ? static_cast<const MT*>(a.q) + b * a.q_sb + t * a.q_st + h * a.q_sh
                        : static_cast<const MT*>(a.k) + b * a.k_sb + t * a.k_st + (h - a.Hq) * a.k_sh;
    MT* dst = isq ? static_cast<MT*>(a.qo) + b * a.qo_sb + t * a.qo_st + h * a.qo_sh
                  : static_cast<MT*>(a.ko) + b * a.ko_sb + t * a.ko_st + (h - a.Hq) * a.ko_sh;
    const float2* row = cs + tl * pairs;
    if (j < rot_items) {
      if constexpr (INTERLEAVED) {
        constexpr int E = V == 1 ? 2 : V;
        MT e[E];
        if constexpr (V == 1) {
          e[0] = src[2 * j];
          e[1] = src[2 * j + 1];
        } else {
          const f32x4 raw = *reinterpret_cast<const f32x4*>(src + j * V);
          __builtin_memcpy(e, &raw, 16);
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const float2 r = row[j * (E / 2) + i];
          const float u = to_float(e[2 * i]), v = to_float(e[2 * i + 1]);
          e[2 * i] = (MT)(u * r.x - v * r.y);
          e[2 * i + 1] = (MT)(v * r.x + u * r.y);
        }
        if constexpr (V == 1) {
          dst[2 * j] = e[0];
          dst[2 * j + 1] = e[1];
        } else {
          f32x4 raw;
          __builtin_memcpy(&raw, e, 16);
          *reinterpret_cast<f32x4*>(dst + j * V) = raw;
        }
      } else {
        MT eu[V], ev[V];
        if constexpr (V == 1) {
          eu[0] = src[j];
          ev[0] = src[pairs + j];
        } else {
          const f32x4 ru = *reinterpret_cast<const f32x4*>(src + j * V);
          const f32x4 rv = *reinterpret_cast<const f32x4*>(src + pairs + j * V);
          __builtin_memcpy(eu, &ru, 16);
          __builtin_memcpy(ev, &rv, 16);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 r = row[j * V + i];
          const float u = to_float(eu[i]), v = to_float(ev[i]);
          eu[i] = (MT)(u * r.x - v * r.y);
          ev[i] = (MT)(v * r.x + u * r.y);
        }
        if constexpr (V == 1) {
          dst[j] = eu[0];
          dst[pairs + j] = ev[0];
        } else {
          f32x4 ru, rv;
          __builtin_memcpy(&ru, eu, 16);
          __builtin_memcpy(&rv, ev, 16);
          *reinterpret_cast<f32x4*>(dst + j * V) = ru;
          *reinterpret_cast<f32x4*>(dst + pairs + j * V) = rv;
        }
      }
    } else if (!(isq ? a.in_place_q : a.in_place_k)) {
      const int c = a.rot + (j - rot_items) * V;  // channels that pass through
      if constexpr (V == 1) dst[c] = src[c];
      else *reinterpret_cast<f32x4*>(dst + c) = *reinterpret_cast<const f32x4*>(src + c);
    }
    tl += step_t;
    hh += step_h;
    if (hh >= my_heads) {
      hh -= my_heads;
      ++tl;
    }
  }
}

template <typename MT, int V, bool INTERLEAVED>
hipError_t rotary_launch(RotaryArgs a, hipStream_t stream) {
  const int pairs = a.rot / 2, heads = a.Hq + a.Hk;
  const int rot_items = INTERLEAVED ? (V == 1 ? pairs : a.rot / V) : pairs / V;
  const int items = rot_items + (a.d - a.rot) / V;
  if (items > kThreads) return hipErrorNotSupported;
  const int rows_per_pass = kThreads / items;
  // tokens per workgroup: about four passes over its rows (4096 x 40 heads of
  // 128: 2, 4, 8 passes 16.3, 16.9, 17.8 us; 65520 x 32: 197, 193, 200), within
  // 32 KB of angles; where that leaves fewer than eight workgroups per compute
  // unit, fewer, and with one token each its heads are shared among workgroups
  // (eight against two: 6.9 and 8.5 us at 1024 x 40 heads, 9.5 and 11.2 at 2048)
  int64_t tile = (4 * rows_per_pass + heads - 1) / heads;
  if (tile * pairs > 4096) tile = 4096 / pairs;
  if (tile < 1) tile = 1;
  a.head_split = 1;
  while (tile > 1 && (a.tokens + tile - 1) / tile < 2048) tile = (tile + 1) / 2;
  if (tile == 1) {
    const int most = (heads + rows_per_pass - 1) / rows_per_pass;
    while (a.head_split < most && a.tokens * a.head_split < 2048) ++a.head_split;
  }
  a.token_tile = (int)tile;
  const int64_t blocks = (a.tokens + tile - 1) / tile * a.head_split;
  if (!grid_fits(blocks, kThreads)) return hipErrorNotSupported;
  hipLaunchKernelGGL((rotary_kernel<MT, V, INTERLEAVED>), dim3((unsigned)blocks), dim3(kThreads),
                     (unsigned)(tile * pairs * sizeof(float2)), stream, a, items, rows_per_pass);
  return hipGetLastError();
}

}  // namespace

template <typename MT>
hipError_t launch_rotary(const RotaryArgs& a, bool aligned, hipStream_t stream) {
  constexpr int V = 16 / sizeof(MT);
  if (a.interleaved) return aligned ? rotary_launch<MT, V, true>(a, stream) : rotary_launch<MT, 1, true>(a, stream);
  return aligned ? rotary_launch<MT, V, false>(a, stream) : rotary_launch<MT, 1, false>(a, stream);
}

template hipError_t launch_rotary<float>(const RotaryArgs&, bool, hipStream_t);
template hipError_t launch_rotary<bf16>(const RotaryArgs&, bool, hipStream_t);

}  // namespace gdn
