// Attention of one new token per sequence over a paged cache.
//
//   s_p = scale q . k_p,  out = sum_p e^(s_p - m) v_p / l,  l = sum_p e^(s_p - m),
//   lse = m + log l,  m = max_p s_p
//
// One workgroup per sequence and query head: its waves take every fourth
// token, each with a running maximum and sum of its own.
#include "gdn_kv.h"

namespace gdn {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

template <typename MT, int FORMAT>
__global__ __launch_bounds__(kWaves * 64) void attend_kernel(AttendArgs a) {
  __shared__ float part[kWaves][256 + 2];
  const int64_t b = blockIdx.x / a.Hq;
  const int h = (int)(blockIdx.x % a.Hq), kh = h / (a.Hq / a.Hk);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const bool mine = lane < a.d / 8;  // lanes that hold channels
  const int64_t reach = a.width << a.page_bits;
  int64_t len = a.lengths[b];
  if (len > reach) len = reach;
  float q[8] = {}, acc[8] = {};
  if (mine) load8<MT, false>(static_cast<const MT*>(a.q) + b * a.q_sb + h * a.q_sh + 8 * lane, q);
  float m = -INFINITY, l = 0.0f;
  for (int64_t p = wave; p < len; p += kWaves) {
    if (a.window && p >= a.sinks && p < len - a.window) continue;
    const int64_t row = kv_row(a.table + b * a.width, a.width, a.pages, a.page_bits, p, a.Hk, kh);
    if (row < 0) continue;
    float x[8] = {};
    float s = 0.0f;
    if (mine) {
      pool8<MT, FORMAT>(a.k_cache, a.k_scales, row, a.d, lane, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(q[i], x[i], s);
    }
    s = wave_sum(s) * a.scale;
    const float n = fmaxf(m, s);
    const float keep = n == -INFINITY ? 1.0f : expf(m - n), e = n == -INFINITY ? 0.0f : expf(s - n);
    m = n;
    l = l * keep + e;
    if (mine) {
      pool8<MT, FORMAT>(a.v_cache, a.v_scales, row, a.d, lane, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(acc[i], keep, e * x[i]);
    }
  }
  if (mine)
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave][8 * lane + i] = acc[i];
  if (lane == 0) {
    part[wave][256] = m;
    part[wave][257] = l;
  }
  __syncthreads();
  if (wave != 0) return;
  float top = -INFINITY, sum = 0.0f, o[8] = {};
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, part[w][256]);
  for (int w = 0; w < kWaves; ++w) {
    const float f = part[w][257] == 0.0f ? 0.0f : expf(part[w][256] - top);
    sum += f * part[w][257];
    if (mine)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += f * part[w][8 * lane + i];
  }
  if (mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = sum == 0.0f ? 0.0f : o[i] / sum;
    store8<MT, false>(static_cast<MT*>(a.out) + b * a.o_sb + h * a.o_sh + 8 * lane, o);
  }
  if (lane == 0 && a.lse) a.lse[b * a.Hq + h] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

template <typename MT, int FORMAT>
hipError_t attend_launch(const AttendArgs& a, hipStream_t stream) {
  const int64_t blocks = a.B * a.Hq;
  if (!grid_fits(blocks, kWaves * 64)) return hipErrorNotSupported;
  hipLaunchKernelGGL((attend_kernel<MT, FORMAT>), dim3((unsigned)blocks), dim3(kWaves * 64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

template <typename MT>
hipError_t launch_attend(const AttendArgs& a, int format, hipStream_t stream) {
  switch (format) {
    case GDN_KV_MXFP8: return attend_launch<MT, GDN_KV_MXFP8>(a, stream);
    case GDN_KV_MXFP4: return attend_launch<MT, GDN_KV_MXFP4>(a, stream);
    default: return attend_launch<MT, sizeof(MT) == 4 ? GDN_KV_F32 : GDN_KV_BF16>(a, stream);
  }
}

template hipError_t launch_attend<float>(const AttendArgs&, int, hipStream_t);
template hipError_t launch_attend<bf16>(const AttendArgs&, int, hipStream_t);

}  // namespace gdn
