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

// A wave walks one channel of one sequence token by token; lane l holds the
// state entries l, l + 64, ...
constexpr int kMaxN = 256;

template <typename MT>
__global__ __launch_bounds__(256) void ssm_kernel(SsmArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wave >= a.B * a.D) return;
  const int64_t b = wave / a.D, d = wave % a.D;
  int64_t r0 = 0, len = a.T;
  int64_t xb = b * a.x_sb, db = b * a.dt_sb, zb = b * a.z_sb, bb = b * a.b_sb, cb = b * a.c_sb, ob = b * a.o_sb;
  if (a.off) {
    r0 = clamp64(a.off[b], 0, a.T);
    len = clamp64(a.off[b + 1], r0, a.T) - r0;
    xb = db = zb = bb = cb = ob = 0;
  }
  const int64_t slot = slot_of(a.index, b, a.slots), g = d / (a.D / a.G);
  float h[kMaxN / 64], A[kMaxN / 64];
#pragma unroll
  for (int i = 0; i < kMaxN / 64; ++i) {
    const int n = lane + 64 * i;
    A[i] = n < a.N ? a.A[d * a.N + n] * kLog2e : 0.0f;
    h[i] = n < a.N && a.state_in && slot >= 0 ? a.state_in[(slot * a.D + d) * a.N + n] : 0.0f;
  }
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.skip ? a.skip[d] : 0.0f;
  for (int64_t t = r0; t < r0 + len; ++t) {
    const float x = to_float(static_cast<const MT*>(a.x)[xb + t * a.x_st + d]);
    const float dt = step_size(a, to_float(static_cast<const MT*>(a.dt)[db + t * a.dt_st + d]), bias);
    float y = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxN / 64; ++i) {
      const int n = lane + 64 * i;
      if (n >= a.N) break;
      const float B = to_float(static_cast<const MT*>(a.Bm)[bb + t * a.b_st + g * a.N + n]);
      const float C = to_float(static_cast<const MT*>(a.Cm)[cb + t * a.c_st + g * a.N + n]);
      h[i] = fmaf(hw_exp2(dt * A[i]), h[i], dt * x * B);
      y = fmaf(h[i], C, y);
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) y += __shfl_xor(y, m, 64);
    if (lane == 0) {
      y = fmaf(skip, x, y);
      if (a.z) y *= silu(to_float(static_cast<const MT*>(a.z)[zb + t * a.z_st + d]));
      static_cast<MT*>(a.out)[ob + t * a.o_st + d] = (MT)y;
    }
  }
  if (a.state_out && slot >= 0) {
#pragma unroll
    for (int i = 0; i < kMaxN / 64; ++i)
      if (lane + 64 * i < a.N) a.state_out[(slot * a.D + d) * a.N + lane + 64 * i] = h[i];
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

}  // namespace

template <typename MT>
hipError_t launch_ssm(const SsmArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.B * a.D + 3) / 4;
  if (!grid_fits(blocks, 256)) return hipErrorNotSupported;
  hipLaunchKernelGGL((ssm_kernel<MT>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
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
