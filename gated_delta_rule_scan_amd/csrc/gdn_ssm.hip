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
// of matrices: per token, channel and entry a pass needs one exponential
// (quarter rate), the products dt A and dt x B, the update and the readout --
// bound by the vector units, not by memory.  What counts is to take that
// exponential once although the scan over time has to be split over lanes:
//
// A wave takes one channel; lane l takes K consecutive tokens of a tile of
// 64 K.  For every state entry n in turn, it computes its K decays a and
// inputs b (kept in registers), scans them from zero to the lane's end value
// H with P = exp(A sum dt), combines (P, H) over the lanes by a wave-wide
// prefix scan on data-parallel row shifts (the carried state enters through
// lane 0), and runs through the same K registers again from the value that
// enters its lane, adding C h to the K readouts.  The state leaves the tile in
// lane 63.  Tokens behind the sequence's end have dt = 0 and B = C = 0:
// decay 1, no input.
//
// A workgroup takes CH neighbouring channels (CH waves), which share the B
// and C of a tile: those are staged in LDS as fp32, four entries at a time,
// double-buffered, each entry's tokens in the order the lanes read them (16
// bytes a lane, neighbouring lanes in different banks).  Rows of x, dt and z
// come in as CH channels of a token and are turned into a lane's K tokens of
// one channel through whichever half of that buffer is free; the output goes
// back the same way.

constexpr int kMaxN = 256;
constexpr int kGroup = 4;  // state entries staged at a time

template <int CTRL, int ROWS>
__device__ __forceinline__ float shifted(float old, float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false));
}

// (P, H) of each lane becomes that of all lanes up to it (P is spent)
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(float& P, float& H) {
  H = fmaf(P, shifted<CTRL, ROWS>(0.0f, H), H);
  P = P * shifted<CTRL, ROWS>(1.0f, P);
}
__device__ __forceinline__ float wave_scan(float P, float H) {
  scan_step<0x111, 0xF>(P, H);  // from 1, 2, 4, 8 lanes back within a row of 16
  scan_step<0x112, 0xF>(P, H);
  scan_step<0x114, 0xF>(P, H);
  scan_step<0x118, 0xF>(P, H);
  scan_step<0x142, 0xA>(P, H);  // last lane of the row before, into rows 1 and 3
  return fmaf(P, shifted<0x143, 0xC>(0.0f, H), H);  // lane 31, into rows 2 and 3
}

// Where token t of a tile lies in a staged entry: lanes read 16-byte pieces
// j = 0 .. K / 4 - 1 of their K tokens, and a rotation of j by lane keeps the
// 16 lanes of a bank cycle apart.
template <int K>
__device__ __forceinline__ int piece_of(int lane, int j) {
  const int turn = K == 16 ? (lane >> 2) & 3 : K == 8 ? (lane >> 3) & 1 : 0;
  return lane * (K / 4) + (j ^ turn);
}
template <int K>
__device__ __forceinline__ int place_of(int t) {
  return piece_of<K>(t / K, (t % K) / 4) * 4 + t % 4;
}

// CH neighbouring channels of one token row
template <typename MT, int CH>
struct __attribute__((aligned(CH * sizeof(MT) > 16 ? 16 : CH * sizeof(MT)))) Row {
  MT e[CH];
};

template <typename MT, int K, int CH>
__global__ __launch_bounds__(CH * 64, K == 16 ? 2 : 4) void ssm_kernel(SsmArgs a, int tiles_per_group, int row_vec, int bc_vec) {
  constexpr int TT = 64 * K, THREADS = 64 * CH;
  constexpr int ROWS = (TT + THREADS - 1) / THREADS;          // token rows a thread moves per tile and operand
  constexpr int ITEMS = (2 * TT + THREADS - 1) / THREADS;     // (token, B or C) pieces a thread stages per group
  constexpr int HALF = 2 * kGroup * TT;                       // floats of one staging buffer
  static_assert(CH * TT * 4 <= HALF * 4, "a tile of one operand fits a free buffer");
  __shared__ __align__(16) float lds[2 * HALF];               // [2][B, C][kGroup][TT]
  __shared__ float carry[CH * kMaxN];                         // [CH][N]: the states between tiles
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroups are dealt to the eight chiplets in turn; each chiplet takes a
  // run of neighbouring channel tiles, whose rows share cache lines.
  const unsigned nblk = gridDim.x, xcd = blockIdx.x & 7, pos = blockIdx.x >> 3;
  const unsigned blk = xcd * (nblk / 8) + (xcd < (nblk & 7) ? xcd : nblk & 7) + pos;
  const int64_t tiles = (int64_t)tiles_per_group * a.G;
  const int64_t b = blk / tiles;
  const int ct = (int)(blk % tiles), g = ct / tiles_per_group;
  const int64_t per = a.D / a.G, d0 = g * per + (int64_t)(ct % tiles_per_group) * CH;
  const int nch = (int)(g * per + per - d0 < CH ? g * per + per - d0 : CH);
  const int N = (int)a.N;

  int64_t r0 = 0, len = a.T;
  if (a.off) {
    r0 = clamp64(a.off[b], 0, a.T);
    len = clamp64(a.off[b + 1], r0, a.T) - r0;
  }
  auto base = [&](int64_t sb, int64_t st) { return a.off ? r0 * st : b * sb; };
  const MT* x = static_cast<const MT*>(a.x) + base(a.x_sb, a.x_st) + d0;
  const MT* dt = static_cast<const MT*>(a.dt) + base(a.dt_sb, a.dt_st) + d0;
  const MT* z = a.z ? static_cast<const MT*>(a.z) + base(a.z_sb, a.z_st) + d0 : nullptr;
  const MT* Bm = static_cast<const MT*>(a.Bm) + base(a.b_sb, a.b_st) + g * a.N;
  const MT* Cm = static_cast<const MT*>(a.Cm) + base(a.c_sb, a.c_st) + g * a.N;
  MT* out = static_cast<MT*>(a.out) + base(a.o_sb, a.o_st) + d0;
  const int64_t slot = slot_of(a.index, b, a.slots);

  for (int i = tid; i < nch * N; i += THREADS)
    carry[i] = a.state_in && slot >= 0 ? a.state_in[(slot * a.D + d0) * N + i] : 0.0f;

  // ---- staging ----
  auto load_rows = [&](const MT* p, int64_t st, int64_t t0, Row<MT, CH>* r) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int t = tid + i * THREADS;
      if (t < TT && t0 + t < len) {
        if (row_vec) {
          r[i] = *reinterpret_cast<const Row<MT, CH>*>(p + (t0 + t) * st);
        } else {
#pragma unroll
          for (int c = 0; c < CH; ++c) r[i].e[c] = c < nch ? p[(t0 + t) * st + c] : (MT)0.0f;
        }
      } else {
#pragma unroll
        for (int c = 0; c < CH; ++c) r[i].e[c] = (MT)0.0f;
      }
    }
  };
  // rows <-> a lane's tokens, through an LDS buffer of [CH][TT] elements
  auto rows_to_lds = [&](MT* buf, const Row<MT, CH>* r) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int t = tid + i * THREADS;
      if (t < TT) {
#pragma unroll
        for (int c = 0; c < CH; ++c) buf[c * TT + (sizeof(MT) == 4 ? place_of<K>(t) : t)] = r[i].e[c];
      }
    }
  };
  auto own_tokens = [&](MT* buf, MT* v) {
#pragma unroll
    for (int j = 0; j < K / 4; ++j) {
      MT* p = buf + wave * TT + (sizeof(MT) == 4 ? piece_of<K>(lane, j) * 4 : lane * K + j * 4);
      __builtin_memcpy(v + j * 4, __builtin_assume_aligned(p, 4 * sizeof(MT)), 4 * sizeof(MT));
    }
  };
  auto own_tokens_back = [&](MT* buf, const MT* v) {
#pragma unroll
    for (int j = 0; j < K / 4; ++j) {
      MT* p = buf + wave * TT + (sizeof(MT) == 4 ? piece_of<K>(lane, j) * 4 : lane * K + j * 4);
      __builtin_memcpy(__builtin_assume_aligned(p, 4 * sizeof(MT)), v + j * 4, 4 * sizeof(MT));
    }
  };
  struct __attribute__((aligned(4 * sizeof(MT)))) Quad {
    MT e[kGroup];
  };
  auto load_bc = [&](int64_t t0, int n0, Quad* q) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int it = tid + i * THREADS, t = it % TT;
#pragma unroll
      for (int e = 0; e < kGroup; ++e) q[i].e[e] = (MT)0.0f;
      if (it < 2 * TT && t0 + t < len) {
        const MT* p = (it < TT ? Bm + (t0 + t) * a.b_st : Cm + (t0 + t) * a.c_st) + n0;
        if (bc_vec) {
          q[i] = *reinterpret_cast<const Quad*>(p);
        } else {
#pragma unroll
          for (int e = 0; e < kGroup; ++e)
            if (n0 + e < N) q[i].e[e] = p[e];
        }
      }
    }
  };
  auto store_bc = [&](float* buf, const Quad* q) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int it = tid + i * THREADS, t = it % TT;
      if (it < 2 * TT) {
        float* p = buf + (it < TT ? 0 : kGroup * TT) + place_of<K>(t);
#pragma unroll
        for (int e = 0; e < kGroup; ++e) p[e * TT] = to_float(q[i].e[e]);
      }
    }
  };

  const int groups = (N + kGroup - 1) / kGroup;
  const int64_t d = d0 + (wave < nch ? wave : 0);  // idle waves of a partial tile compute, but store nothing
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.skip ? a.skip[d] : 0.0f;
  const float* A = a.A + d * N;

  Quad q[ITEMS];
  Row<MT, CH> rx[ROWS], rd[ROWS], rz[ROWS];
  load_bc(0, 0, q);
  load_rows(x, a.x_st, 0, rx);
  load_rows(dt, a.dt_st, 0, rd);
  store_bc(lds, q);
  int s = 0;  // group s is staged in buffer s & 1
  for (int64_t t0 = 0; t0 < len; t0 += TT) {
    MT* turn = reinterpret_cast<MT*>(lds + ((s + 1) & 1) * HALF);  // the free buffer
    float dts[K], u[K], y[K], total = 0.0f;
    {
      MT v[K];
      rows_to_lds(turn, rx);
      __syncthreads();
      own_tokens(turn, v);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) u[k] = to_float(v[k]);
      rows_to_lds(turn, rd);
      __syncthreads();
      own_tokens(turn, v);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool in = t0 + lane * K + k < len;
        dts[k] = in ? step_size(a, to_float(v[k]), bias) : 0.0f;
        y[k] = skip * u[k];
        u[k] *= dts[k];
        total += dts[k];
      }
    }
    if (z) load_rows(z, a.z_st, t0, rz);
    for (int gr = 0; gr < groups; ++gr, ++s) {
      const bool last = gr + 1 == groups;
      const float* buf = lds + (s & 1) * HALF;
      load_bc(last ? t0 + TT : t0, last ? 0 : (gr + 1) * kGroup, q);  // behind the end: zeros
      if (last) {
        load_rows(x, a.x_st, t0 + TT, rx);
        load_rows(dt, a.dt_st, t0 + TT, rd);
      }
      const int most = N - gr * kGroup < kGroup ? N - gr * kGroup : kGroup;
#pragma unroll 1
      for (int e = 0; e < most; ++e) {
        const int n = gr * kGroup + e;
        const float A2 = A[n] * kLog2e, h0 = carry[wave * N + n];
        float dec[K], in[K];
#pragma unroll
        for (int j = 0; j < K / 4; ++j) {
          const f32x4 B = *reinterpret_cast<const f32x4*>(buf + e * TT + piece_of<K>(lane, j) * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) in[j * 4 + i] = u[j * 4 + i] * B[i];
        }
        float H = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          dec[k] = hw_exp2(dts[k] * A2);
          H = fmaf(dec[k], H, in[k]);
        }
        const float P = hw_exp2(total * A2);
        if (lane == 0) H = fmaf(P, h0, H);
        H = wave_scan(P, H);
        float h = shifted<0x138, 0xF>(h0, H);  // the lane before's; lane 0 starts from the carried state
        if (lane == 63 && wave < nch) carry[wave * N + n] = H;
#pragma unroll
        for (int j = 0; j < K / 4; ++j) {
          const f32x4 C = *reinterpret_cast<const f32x4*>(buf + (kGroup + e) * TT + piece_of<K>(lane, j) * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = j * 4 + i;
            h = fmaf(dec[k], h, in[k]);
            y[k] = fmaf(C[i], h, y[k]);
          }
        }
      }
      store_bc(lds + ((s + 1) & 1) * HALF, q);
      __syncthreads();
    }
    // readouts: gate, and back to rows
    turn = reinterpret_cast<MT*>(lds + ((s + 1) & 1) * HALF);
    MT v[K];
    if (z) {
      rows_to_lds(turn, rz);
      __syncthreads();
      own_tokens(turn, v);
#pragma unroll
      for (int k = 0; k < K; ++k) y[k] *= silu(to_float(v[k]));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = (MT)y[k];
    own_tokens_back(turn, v);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int t = tid + i * THREADS;
      if (t < TT && t0 + t < len) {
        Row<MT, CH> r;
#pragma unroll
        for (int c = 0; c < CH; ++c) r.e[c] = turn[c * TT + (sizeof(MT) == 4 ? place_of<K>(t) : t)];
        MT* p = out + (t0 + t) * a.o_st;
        if (row_vec) {
          *reinterpret_cast<Row<MT, CH>*>(p) = r;
        } else {
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (c < nch) p[c] = r.e[c];
        }
      }
    }
    __syncthreads();
  }
  __syncthreads();
  if (a.state_out && slot >= 0)
    for (int i = tid; i < nch * N; i += THREADS) a.state_out[(slot * a.D + d0) * N + i] = carry[i];
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

template <typename MT, int K, int CH>
hipError_t ssm_launch(const SsmArgs& a, hipStream_t stream) {
  const int64_t per = a.D / a.G, tiles = (per + CH - 1) / CH, blocks = a.B * a.G * tiles;
  if (!grid_fits(blocks, CH * 64) || tiles * a.G > 0x7FFFFFFF) return hipErrorNotSupported;
  auto rows_ok = [&](const void* p, int64_t sb, int64_t st, size_t bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && st * sizeof(MT) % bytes == 0 &&
                  (a.off || a.B == 1 || sb * sizeof(MT) % bytes == 0));
  };
  constexpr size_t row = CH * sizeof(MT) > 16 ? 16 : CH * sizeof(MT), quad = kGroup * sizeof(MT);
  const int row_vec = per % CH == 0 && rows_ok(a.x, a.x_sb, a.x_st, row) && rows_ok(a.dt, a.dt_sb, a.dt_st, row) &&
                      rows_ok(a.z, a.z_sb, a.z_st, row) && rows_ok(a.out, a.o_sb, a.o_st, row);
  const int bc_vec = a.N % kGroup == 0 && rows_ok(a.Bm, a.b_sb, a.b_st, quad) && rows_ok(a.Cm, a.c_sb, a.c_st, quad);
  hipLaunchKernelGGL((ssm_kernel<MT, K, CH>), dim3((unsigned)blocks), dim3(CH * 64), 0, stream, a, (int)tiles,
                     row_vec, bc_vec);
  return hipGetLastError();
}

template <typename MT, int K>
hipError_t ssm_for(const SsmArgs& a, hipStream_t stream) {
  return ssm_launch<MT, K, 8>(a, stream);
}

}  // namespace

template <typename MT>
hipError_t launch_ssm(const SsmArgs& a, hipStream_t stream) {
  // tokens per lane: the fewest whose tile holds an ordinary sequence
  const int64_t T = a.off ? (a.T + a.B - 1) / a.B : a.T;
  if (T <= 256) return ssm_for<MT, 4>(a, stream);
  if (T <= 512) return ssm_for<MT, 8>(a, stream);
  return ssm_for<MT, 16>(a, stream);
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
