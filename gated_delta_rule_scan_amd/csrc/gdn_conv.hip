// Short causal depthwise convolution over time, for prompts and for single
// tokens:
//
//   y[t, d] = act(bias[d] + sum_{j < W} w[d, j] x[t - (W - 1) + j, d])
//
// with the rows before a sequence's first taken from its state (the last
// W - 1 input rows).  Memory-bound: 2 W flops per element against one read
// and one write of it.
//
// Prompt split: a thread owns V neighbouring channels (16 bytes of a row) and a
// run of tokens, which it walks in batches of kConvRows.  A batch's rows are
// all in flight at once, the last W - 1 rows of the batch before stay in
// registers, and the next batch's loads are issued before the current one is
// computed; a run re-reads only its W - 1 rows of history.  A wave covers up to
// 64 V channels of a row, so rows are read and written in whole cache lines.
// 2 x 32760 x 2048 bf16, four taps: 105-109 us for 537 MB, 5.0 TB/s, the rate
// of a large copy.  A step of 64 x 2048: 3.6 us, its launch.
#include "gdn_layer.h"

namespace gdn {
namespace {

constexpr int kConvRows = 8;   // tokens in flight per thread

// V neighbouring channels as stored.  WHOLE: 16 bytes, and rows lie on 16 bytes
// and hold whole packs; else a pack may start at any element (unaligned
// accesses) and a row's last one may hold only `m` channels.
template <typename MT, int V>
struct Pack {
  MT e[V];
};
template <typename MT, int V, bool WHOLE>
__device__ __forceinline__ Pack<MT, V> load_pack(const MT* p, int m) {
  Pack<MT, V> r;
  if constexpr (WHOLE) {
    __builtin_memcpy(&r, __builtin_assume_aligned(p, 16), 16);
  } else if (m >= V) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r.e[e] = e < m ? p[e] : (MT)0.0f;
  }
  return r;
}
template <typename MT, int V>
__device__ __forceinline__ Pack<MT, V> zeros() {
  Pack<MT, V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.e[e] = (MT)0.0f;
  return r;
}
template <typename MT, int V, bool WHOLE>
__device__ __forceinline__ void store_pack(MT* p, const Pack<MT, V>& v, int m) {
  if constexpr (WHOLE) {
    __builtin_memcpy(__builtin_assume_aligned(p, 16), &v, 16);
  } else if (m >= V) {
    __builtin_memcpy(p, &v, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < m) p[e] = v.e[e];
  }
}

// row `pos` of a sequence: its own rows from `x`, the W - 1 before them from
// the state (zeros without one; spelled out here, since with zeros() the
// compiler splits and joins the pairs of every loaded row: 110 us at the size above)
template <typename MT, int W, int V, bool WHOLE>
__device__ __forceinline__ Pack<MT, V> load_row(const MT* x, int64_t st, const MT* state, int64_t D, int64_t pos, int m) {
  if (pos >= 0) return load_pack<MT, V, WHOLE>(x + pos * st, m);
  if (state) return load_pack<MT, V, WHOLE>(state + (W - 1 + pos) * D, m);
  Pack<MT, V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.e[e] = (MT)0.0f;
  return r;
}

template <typename MT, int W, int V, bool WHOLE>
__global__ __launch_bounds__(256) void conv_kernel(ConvArgs a, int tx_log2, int channel_tiles, int64_t chunks) {
  const int TX = 1 << tx_log2, TY = 256 >> tx_log2;
  const int tx = threadIdx.x & (TX - 1), ty = threadIdx.x >> tx_log2;
  const int64_t item = blockIdx.x / channel_tiles;
  const int64_t d = ((int64_t)(blockIdx.x % channel_tiles) * TX + tx) * V;
  const int64_t run = (int64_t)a.batches * kConvRows, C = run * TY;
  SeqItem s;
  int64_t x0, o0;
  if (a.off) {
    s = find_packed(a.off, a.B, a.T, C, item);
    x0 = s.row0 * a.x_st;
    o0 = s.row0 * a.o_st;
    // the last sequence's items also hold the rows behind it
    if (a.zero_unused && s.b == a.B - 1 && d < a.D && s.chunk >= 0) {
      int64_t t = s.chunk * C + ty * run;
      const int64_t rows = a.T - s.row0, t1 = t + run < rows ? t + run : rows;
      for (t = t > s.len ? t : s.len; t < t1; ++t)
        store_pack<MT, V, WHOLE>(static_cast<MT*>(a.out) + o0 + t * a.o_st + d, zeros<MT, V>(), a.D - d < V ? (int)(a.D - d) : V);
    }
  } else {
    s.b = item / chunks;
    s.chunk = item % chunks;
    s.len = a.T;
    x0 = s.b * a.x_sb;
    o0 = s.b * a.o_sb;
  }
  if (d >= a.D || s.chunk < 0) return;
  const int m = a.D - d < V ? (int)(a.D - d) : V;  // channels of this pack
  const int64_t t0 = s.chunk * C + ty * run;
  const bool writes_state = s.chunk == 0 && ty == 0 && a.state_out;
  if (t0 >= s.len && !writes_state) return;
  const MT* x = static_cast<const MT*>(a.x) + x0 + d;
  MT* out = static_cast<MT*>(a.out) + o0 + d;
  const int64_t slot = slot_of(a.index, s.b, a.slots);
  const MT* state = a.state_in && slot >= 0 ? static_cast<const MT*>(a.state_in) + slot * (W - 1) * a.D + d : nullptr;

  if (t0 < s.len) {
    float w[V][W], bias[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int64_t c = d + (e < m ? e : m - 1);
      bias[e] = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) w[e][j] = a.weight[c * W + j];
    }
    Pack<MT, V> r[kConvRows + W - 1], nx[kConvRows];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j] = load_row<MT, W, V, WHOLE>(x, a.x_st, state, a.D, t0 - (W - 1) + j, m);
    // tokens of the run, counted down; pointers at the rows to be loaded and
    // stored next
    int left = (int)(s.len - t0 < run ? s.len - t0 : run);
    const MT* px = x + t0 * a.x_st;
    MT* po = out + t0 * a.o_st;
    auto load = [&](int n) {  // the next kConvRows rows, of which n are there; the last one repeats
      if (n >= kConvRows) {
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) nx[i] = load_pack<MT, V, WHOLE>(px + i * a.x_st, m);
      } else {
#pragma unroll
        for (int i = 0; i < kConvRows; ++i) nx[i] = load_pack<MT, V, WHOLE>(px + (i < n ? i : n - 1) * a.x_st, m);
      }
      px += kConvRows * a.x_st;
    };
    load(left);
    while (left > 0) {
#pragma unroll
      for (int i = 0; i < kConvRows; ++i) r[W - 1 + i] = nx[i];
      if (left > kConvRows) load(left - kConvRows);
#pragma unroll
      for (int i = 0; i < kConvRows; ++i) {
        Pack<MT, V> y;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float acc = bias[e];
#pragma unroll
          for (int j = 0; j < W; ++j) acc = fmaf(w[e][j], to_float(r[i + j].e[e]), acc);
          y.e[e] = (MT)(a.silu ? silu(acc) : acc);
        }
        if (i < left) store_pack<MT, V, WHOLE>(po + i * a.o_st, y, m);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) r[j] = r[kConvRows + j];
      po += kConvRows * a.o_st;
      left -= kConvRows;
    }
  }
  // The final state: written by the thread that alone reads this sequence's
  // initial state for these channels, after that read, so the two may be one
  // buffer.
  if (writes_state && slot >= 0) {
    Pack<MT, V> keep[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) keep[j] = load_row<MT, W, V, WHOLE>(x, a.x_st, state, a.D, s.len - (W - 1) + j, m);
    MT* so = static_cast<MT*>(a.state_out) + slot * (W - 1) * a.D + d;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_pack<MT, V, WHOLE>(so + j * a.D, keep[j], m);
  }
}

// One token per sequence: a thread takes V channels of one sequence.
template <typename MT, int W, int V, bool WHOLE>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, int tx_log2, int channel_tiles) {
  const int TX = 1 << tx_log2, TY = 256 >> tx_log2;
  const int64_t b = (int64_t)(blockIdx.x / channel_tiles) * TY + (threadIdx.x >> tx_log2);
  const int64_t d = ((int64_t)(blockIdx.x % channel_tiles) * TX + (threadIdx.x & (TX - 1))) * V;
  if (b >= a.B || d >= a.D) return;
  const int m = a.D - d < V ? (int)(a.D - d) : V;  // channels of this pack
  // everything but the state is on its way before the slot is known
  const int64_t slot = slot_of(a.index, b, a.slots);
  Pack<MT, V> r[W], y;
  r[W - 1] = load_pack<MT, V, WHOLE>(static_cast<const MT*>(a.x) + b * a.x_sb + d, m);
  float w[V][W], bias[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int64_t c = d + (e < m ? e : m - 1);
    bias[e] = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[e][j] = a.weight[c * W + j];
  }
  MT* out = static_cast<MT*>(a.out) + b * a.o_sb + d;
  if (slot < 0) {
    if (a.zero_unused) store_pack<MT, V, WHOLE>(out, zeros<MT, V>(), m);
    return;
  }
  MT* state = static_cast<MT*>(a.state_out) + slot * (W - 1) * a.D + d;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) r[j] = load_pack<MT, V, WHOLE>(state + j * a.D, m);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float acc = bias[e];
#pragma unroll
    for (int j = 0; j < W; ++j) acc = fmaf(w[e][j], to_float(r[j].e[e]), acc);
    y.e[e] = (MT)(a.silu ? silu(acc) : acc);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_pack<MT, V, WHOLE>(state + j * a.D, r[j + 1], m);
  store_pack<MT, V, WHOLE>(out, y, m);
}

// lanes across channels: enough for the row, at most a wave
int lanes_log2(int64_t lanes) {
  int l = 3;
  while (l < 6 && ((int64_t)1 << l) < lanes) ++l;
  return l;
}

template <typename MT, int W, int V, bool WHOLE>
hipError_t conv_launch(ConvArgs a, hipStream_t stream) {
  const int64_t lanes = (a.D + V - 1) / V;
  const int txl = lanes_log2(lanes), TY = 256 >> txl;
  const int64_t ctiles = (lanes + ((int64_t)1 << txl) - 1) >> txl;
  // four batches a run where that still gives every compute unit eight waves
  // (2048 in all): 108 us against 130 with one and 117 with two at 2 x 32760 x
  // 2048 bf16.  Less work takes one, for more threads: 6.6 us against 12.5 at
  // 1024 x 2048, 11.8 against 14.3 at 4096.  So do packs off 16 bytes: 36 us
  // against 38 at 20011 x 1001 fp32.
  const int64_t rows = a.off ? a.T : a.B * a.T;
  a.batches = ((rows * ctiles) << txl) >= (int64_t)2048 * 64 * 4 * kConvRows ? (WHOLE ? 4 : 1) : 1;
  const int64_t C = (int64_t)a.batches * kConvRows * TY;
  const int64_t chunks = (a.T + C - 1) / C > 0 ? (a.T + C - 1) / C : 1;
  const int64_t items = a.off ? a.T / C + a.B : a.B * chunks;
  if (!grid_fits(items * ctiles, 256)) return hipErrorNotSupported;
  hipLaunchKernelGGL((conv_kernel<MT, W, V, WHOLE>), dim3((unsigned)(items * ctiles)), dim3(256), 0, stream, a, txl, (int)ctiles,
                     chunks);
  return hipGetLastError();
}

template <typename MT, int W, int V, bool WHOLE>
hipError_t conv_step_launch(const ConvArgs& a, hipStream_t stream) {
  const int64_t lanes = (a.D + V - 1) / V;
  const int txl = lanes_log2(lanes), TY = 256 >> txl;
  const int64_t ctiles = (lanes + ((int64_t)1 << txl) - 1) >> txl, items = (a.B + TY - 1) / TY;
  if (!grid_fits(items * ctiles, 256)) return hipErrorNotSupported;
  hipLaunchKernelGGL((conv_step_kernel<MT, W, V, WHOLE>), dim3((unsigned)(items * ctiles)), dim3(256), 0, stream, a, txl,
                     (int)ctiles);
  return hipGetLastError();
}

}  // namespace

// Rows off 16 bytes: two fp32 channels or one bf16 channel a thread.  Of 20011 x
// 1001: fp32 with 1, 2, 4 channels 42, 39, 48 us, bf16 with 1, 2 26, 29 us.
template <typename MT>
hipError_t launch_conv(const ConvArgs& a, int width, bool aligned, hipStream_t stream) {
  constexpr int V = 16 / sizeof(MT), U = sizeof(MT) == 4 ? 2 : 1;
  if (width == 2) return aligned ? conv_launch<MT, 2, V, true>(a, stream) : conv_launch<MT, 2, U, false>(a, stream);
  if (width == 3) return aligned ? conv_launch<MT, 3, V, true>(a, stream) : conv_launch<MT, 3, U, false>(a, stream);
  return aligned ? conv_launch<MT, 4, V, true>(a, stream) : conv_launch<MT, 4, U, false>(a, stream);
}

template <typename MT>
hipError_t launch_conv_step(const ConvArgs& a, int width, bool aligned, hipStream_t stream) {
  constexpr int V = 16 / sizeof(MT), U = sizeof(MT) == 4 ? 2 : 1;
  if (width == 2) return aligned ? conv_step_launch<MT, 2, V, true>(a, stream) : conv_step_launch<MT, 2, U, false>(a, stream);
  if (width == 3) return aligned ? conv_step_launch<MT, 3, V, true>(a, stream) : conv_step_launch<MT, 3, U, false>(a, stream);
  return aligned ? conv_step_launch<MT, 4, V, true>(a, stream) : conv_step_launch<MT, 4, U, false>(a, stream);
}

template hipError_t launch_conv<float>(const ConvArgs&, int, bool, hipStream_t);
template hipError_t launch_conv<bf16>(const ConvArgs&, int, bool, hipStream_t);
template hipError_t launch_conv_step<float>(const ConvArgs&, int, bool, hipStream_t);
template hipError_t launch_conv_step<bf16>(const ConvArgs&, int, bool, hipStream_t);

}  // namespace gdn
