// The delta rule's single-token step, the state advanced in place:
//
//   S' = a S (I - beta k^ k^T) + beta v k^T,  o = S' q^
//
// The rows of S are independent: with ks = S_i k^ and qs = S_i q^ (dots over
// dk, both from one read of the row), row i becomes
//
//   S'_i = a S_i + w k^,  w = beta (v_i - a ks)   (erase-free: w = beta v_i)
//   o_i  = a qs + w (k^ q^)                       (exclusive: o_i = a qs)
//
// so a row is read once, kept in registers, and written once: memory-bound on
// the state (8 bytes per entry).  A workgroup takes one head, its waves shares
// of its rows; dk / 4 lanes hold a row, 16 bytes each, and all of a wave's
// rows are in flight together.  128 sequences x 16 heads of 128 x 128: 52-56 us
// for 271 MB, 4.9-5.2 TB/s, the rate of a large copy; one sequence x 12 heads:
// 4.3 us, launch and one chain of loads.
#include "gdn_layer.h"

namespace gdn {
namespace {

// Sum over the LANES (16 or 32) neighbouring lanes of a group, in every lane:
// pairs, quads, eights and sixteens by data-parallel row permutations, then
// the two sixteens by a swizzle.
template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
  auto add = [](float v, int moved) { return v + __builtin_bit_cast(float, moved); };
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0xB1, 0xF, 0xF, true));   // quad: 1 0 3 2
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x4E, 0xF, 0xF, true));   // quad: 2 3 0 1
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x141, 0xF, 0xF, true));  // half row mirrored
  x = add(x, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0x140, 0xF, 0xF, true));  // row mirrored
  if constexpr (LANES == 32) x = add(x, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, x), 0x401F));  // lane ^ 16
  return x;
}

__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
  return fmaf(a[0], b[0], fmaf(a[1], b[1], fmaf(a[2], b[2], a[3] * b[3])));
}

template <typename MT>
__device__ __forceinline__ f32x4 load4(const MT* p) {
  if constexpr (sizeof(MT) == 4) {
    return *reinterpret_cast<const f32x4*>(p);
  } else {
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
  }
}

template <typename MT, int DK, int DV, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void step_kernel(StepArgs a) {
  constexpr int LANES = DK / 4, RPL = 64 / LANES;  // lanes per row, rows per load
  constexpr int ROWS = DV / WAVES, LOADS = ROWS / RPL;
  static_assert(LOADS >= 1, "every wave owns at least one load of rows");
  __shared__ float o_rows[DV];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int sub = lane / LANES, l = lane % LANES;
  const int64_t bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
  const int64_t slot = slot_of(a.index, b, a.slots);
  if (slot < 0) {  // the whole workgroup
    if (a.zero_unused && threadIdx.x < DV) a.out[bh * DV + threadIdx.x] = 0.0f;
    return;
  }
  float* S = a.state + (slot * a.H + h) * (DV * DK) + (wave * ROWS + sub) * DK + l * 4;
  f32x4 s[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) s[i] = *reinterpret_cast<const f32x4*>(S + i * RPL * DK);
  f32x4 k = load4(static_cast<const MT*>(a.k) + bh * DK + l * 4);
  f32x4 q = load4(static_cast<const MT*>(a.q) + bh * DK + l * 4);
  float v[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i)
    v[i] = to_float(static_cast<const MT*>(a.v)[bh * DV + wave * ROWS + i * RPL + sub]);
  const float decay = expf(a.log_alpha[bh]), beta = a.beta[bh];
  const float rk = 1.0f / fmaxf(sqrtf(group_sum<LANES>(dot4(k, k))), kNormEps);
  const float rq = 1.0f / fmaxf(sqrtf(group_sum<LANES>(dot4(q, q))), kNormEps);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    k[e] *= rk;
    q[e] *= rq;
  }
  const float kq = group_sum<LANES>(dot4(k, q));
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const float ks = group_sum<LANES>(dot4(s[i], k)), qs = group_sum<LANES>(dot4(s[i], q));
    const float w = a.erase ? beta * (v[i] - decay * ks) : beta * v[i];
    f32x4 n;
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = fmaf(decay, s[i][e], w * k[e]);
    *reinterpret_cast<f32x4*>(S + i * RPL * DK) = n;
    const float o = a.exclusive ? decay * qs : fmaf(decay, qs, w * kq);
    if (l == 0) o_rows[wave * ROWS + i * RPL + sub] = o;
  }
  __syncthreads();
  // one wave writes the head's readout, DV / 64 channels a lane
  if (wave != 0) return;
  float o[DV / 64];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < DV / 64; ++i) {
    o[i] = o_rows[lane + 64 * i];
    ss = fmaf(o[i], o[i], ss);
  }
  if (a.gate) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) ss += __shfl_xor(ss, m, 64);
    const float inv = 1.0f / sqrtf(ss * (1.0f / DV) + a.norm_eps);
#pragma unroll
    for (int i = 0; i < DV / 64; ++i) {
      const float z = to_float(static_cast<const MT*>(a.gate)[bh * DV + lane + 64 * i]);
      o[i] = a.norm_weight[lane + 64 * i] * (o[i] * inv) * (1.0f / (1.0f + expf(-z)));
    }
  }
#pragma unroll
  for (int i = 0; i < DV / 64; ++i) a.out[bh * DV + lane + 64 * i] = o[i];
}

template <typename MT, int DK, int DV, int WAVES>
hipError_t step_launch(const StepArgs& a, hipStream_t stream) {
  const int64_t blocks = a.B * a.H;
  if (!grid_fits(blocks, WAVES * 64)) return hipErrorNotSupported;
  hipLaunchKernelGGL((step_kernel<MT, DK, DV, WAVES>), dim3((unsigned)blocks), dim3(WAVES * 64), 0, stream, a);
  return hipGetLastError();
}

template <typename MT, int DK>
hipError_t step_for(const StepArgs& a, hipStream_t stream) {
  // few heads: sixteen waves each, for latency (256 heads of 128 x 128: 6.7 us
  // against 8.2); many: four, whose loads in flight (up to 64 KB a workgroup)
  // already keep the memory busy (512 heads: 12.8 us against 13.4)
  if (a.B * a.H < 512)
    return a.dv == 64 ? step_launch<MT, DK, 64, 16>(a, stream) : step_launch<MT, DK, 128, 16>(a, stream);
  return a.dv == 64 ? step_launch<MT, DK, 64, 4>(a, stream) : step_launch<MT, DK, 128, 4>(a, stream);
}

}  // namespace

template <typename MT>
hipError_t launch_step(const StepArgs& a, int dk, hipStream_t stream) {
  return dk == 64 ? step_for<MT, 64>(a, stream) : step_for<MT, 128>(a, stream);
}

template hipError_t launch_step<float>(const StepArgs&, int, hipStream_t);
template hipError_t launch_step<bf16>(const StepArgs&, int, hipStream_t);

}  // namespace gdn
