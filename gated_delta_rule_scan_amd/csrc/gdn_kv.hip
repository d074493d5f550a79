// Rows of keys and values into a paged cache and back out of it.
//
// A copy, with a block's scale and codes in between where the cache has 8 or 4
// bits: bound by memory on both sides (65520 tokens x 16 heads x 128 from bf16
// into 8 bits 160 us and back 148, 5.1 and 5.5 TB/s, into 4 bits 143 and back 138,
// 4.8 and 4.9; a window of 8 x 4680 tokens x 12 heads out of a cache in bf16 68 us,
// 6.8 TB/s).  A thread moves eight channels of K and the
// same of V; four neighbouring lanes hold a block of 32 channels.  A workgroup
// takes 16 tokens of a few heads, head by head: rows in 8 or 4 bits are parts
// of cache lines, and a wave's lie beside each other in the pool.
#include "gdn_kv.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 2;     // places a thread has under way
constexpr int kPlaces = 2;     // ... and in all
constexpr int kTokenBits = 4;  // tokens of a workgroup

// The scale bytes of a row, which every fourth lane holds, gathered in the
// row's first lane of eight (two bytes) or of each sixteen (four): a lane's
// value from 4, 8 and 12 lanes further in its row of 16.
__device__ __forceinline__ unsigned two_bytes(unsigned s) {
  return s | (unsigned)__builtin_amdgcn_mov_dpp((int)s, 0x104, 0xF, 0xF, true) << 8;
}
__device__ __forceinline__ unsigned four_bytes(unsigned s) {
  const unsigned w = two_bytes(s);
  return w | (unsigned)__builtin_amdgcn_mov_dpp((int)w, 0x108, 0xF, 0xF, true) << 16;
}

// ONCE: pools are read past the caches (see fetch)
template <typename MT, int FORMAT, bool WRITE, bool ALIGNED, bool ONCE>
__global__ __launch_bounds__(kThreads) void kv_kernel(KvArgs a) {
  const unsigned shares = (unsigned)((a.Hk + a.heads - 1) / a.heads);
  const int64_t item = a.first + blockIdx.x / shares;
  const int h0 = (int)(blockIdx.x % shares) * a.heads;
  SeqItem s;
  if (a.off) {
    s = find_packed(a.off, a.B, a.T, (int64_t)1 << a.chunk_bits, item);
  } else {
    s.b = item / a.chunks;
    s.chunk = item % a.chunks;
    s.row0 = 0;
    s.len = a.T;
  }
  // rows behind the last sequence
  const int64_t limit = !WRITE && a.zero_unused && s.b == a.B - 1 && a.off ? a.T - s.row0 : s.len;
  const int64_t t0 = s.chunk << a.chunk_bits;
  if (t0 < 0 || t0 >= limit) return;  // (below zero: rows in front of the first sequence)
  const int lane_bits = __builtin_ctz(a.d) - 3;  // lanes of a row: 8, 16 or 32
  const int heads = a.Hk - h0 < a.heads ? a.Hk - h0 : a.heads;
  const unsigned places = (unsigned)heads << (a.chunk_bits + lane_bits);
  const int64_t first = a.start ? a.start[s.b] : 0;
  const int32_t* table = a.table + s.b * a.width;
  MT* k_rows = static_cast<MT*>(a.k) + (a.off ? 0 : s.b * a.k_sb) + s.row0 * a.k_st;
  MT* v_rows = static_cast<MT*>(a.v) + (a.off ? 0 : s.b * a.v_sb) + s.row0 * a.v_st;

  // places in order of head, token and channels
  for (unsigned i0 = threadIdx.x; i0 < places; i0 += kAtOnce * kThreads) {
    int64_t row[kAtOnce], tok[kAtOnce];
    int c[kAtOnce], h[kAtOnce];
    bool live[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const unsigned i = i0 + u * kThreads;
      c[u] = (int)(i & ((1u << lane_bits) - 1));
      tok[u] = t0 + (i >> lane_bits & ((1u << a.chunk_bits) - 1));
      h[u] = h0 + (int)(i >> (lane_bits + a.chunk_bits));
      live[u] = i < places && tok[u] < limit;
    }
    float x[kAtOnce][2][8];
    const auto rows_at = [&](int u, int j) {
      return j ? v_rows + tok[u] * a.v_st + h[u] * a.v_sh + 8 * c[u] : k_rows + tok[u] * a.k_st + h[u] * a.k_sh + 8 * c[u];
    };
    if constexpr (WRITE)
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (live[u])
#pragma unroll
          for (int j = 0; j < 2; ++j) load8<MT, ALIGNED, true>(rows_at(u, j), x[u][j]);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      row[u] = live[u] && tok[u] < s.len ? kv_row(table, a.width, a.pages, a.page_bits, first + tok[u], a.Hk, h[u]) : -1;
    if constexpr (!WRITE) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (row[u] >= 0) {
          pool8<MT, FORMAT, ONCE>(a.k_cache, a.k_scales, row[u], a.d, c[u], x[u][0]);
          pool8<MT, FORMAT, ONCE>(a.v_cache, a.v_scales, row[u], a.d, c[u], x[u][1]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u][0][e] = x[u][1][e] = 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (row[u] >= 0 || (a.zero_unused && live[u]))
#pragma unroll
          for (int j = 0; j < 2; ++j) store8<MT, ALIGNED>(rows_at(u, j), x[u][j]);
    } else {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        // (the lanes of a row go the same way, so a block's four are all here)
        if (row[u] < 0) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          void* pool = j ? a.v_cache : a.k_cache;
          if constexpr (FORMAT == GDN_KV_F32 || FORMAT == GDN_KV_BF16) {
            store8<MT, true>(static_cast<MT*>(pool) + row[u] * a.d + 8 * c[u], x[u][j]);
          } else {
            const unsigned scale = block_scale<FORMAT>(block_top(x[u][j]));
            unsigned w[2];
            encode8<FORMAT>(x[u][j], scale, w);
            if constexpr (FORMAT == GDN_KV_MXFP8)
              *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + row[u] * a.d + 8 * c[u]) = make_uint2(w[0], w[1]);
            else
              *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(pool) + row[u] * (a.d / 2) + 4 * c[u]) = w[0];
            uint8_t* to = (j ? a.v_scales : a.k_scales) + row[u] * (a.d / 32) + c[u] / 4;
            if (lane_bits == 3) {
              const unsigned two = two_bytes(scale);
              if (c[u] % 8 == 0) *reinterpret_cast<uint16_t*>(to) = (uint16_t)two;
            } else {
              const unsigned four = four_bytes(scale);
              if (c[u] % 16 == 0) *reinterpret_cast<unsigned*>(to) = four;
            }
          }
        }
      }
    }
  }
}

template <typename MT, int FORMAT, bool WRITE, bool ONCE>
hipError_t kv_launch(const KvArgs& given, int64_t items, bool aligned, hipStream_t stream) {
  KvArgs a = given;
  return in_launches(items, (a.Hk + a.heads - 1) / a.heads, kThreads, [&](int64_t first, dim3 blocks) {
    a.first = first;
    if (aligned)
      hipLaunchKernelGGL((kv_kernel<MT, FORMAT, WRITE, true, ONCE>), blocks, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((kv_kernel<MT, FORMAT, WRITE, false, ONCE>), blocks, dim3(kThreads), 0, stream, a);
  });
}

template <typename MT, int FORMAT>
hipError_t kv_for(const KvArgs& a, int64_t items, bool write, bool aligned, hipStream_t stream) {
  if (write) return kv_launch<MT, FORMAT, true, false>(a, items, aligned, stream);
  const int64_t bytes = 2 * (a.off ? a.T : a.B * a.T) * a.Hk * row_bytes(FORMAT, a.d);
  return bytes >= kOnceBytes ? kv_launch<MT, FORMAT, false, true>(a, items, aligned, stream)
                             : kv_launch<MT, FORMAT, false, false>(a, items, aligned, stream);
}

}  // namespace

template <typename MT>
hipError_t launch_kv(const KvArgs& given, int format, bool write, bool aligned, hipStream_t stream) {
  KvArgs a = given;
  // tokens and heads of a workgroup: kPlaces places a thread, of 16 tokens where there are
  a.chunk_bits = 0;
  while (a.chunk_bits < kTokenBits && ((int64_t)1 << a.chunk_bits) < a.T) ++a.chunk_bits;
  a.heads = (kPlaces * kThreads * 8 >> a.chunk_bits) / a.d;
  a.heads = a.heads < 1 ? 1 : a.heads > a.Hk ? a.Hk : a.heads;
  a.chunks = (a.T + ((int64_t)1 << a.chunk_bits) - 1) >> a.chunk_bits;
  const int64_t items = a.off ? (a.T >> a.chunk_bits) + a.B : a.B * a.chunks;
  switch (format) {
    case GDN_KV_MXFP8: return kv_for<MT, GDN_KV_MXFP8>(a, items, write, aligned, stream);
    case GDN_KV_MXFP4: return kv_for<MT, GDN_KV_MXFP4>(a, items, write, aligned, stream);
    default: return kv_for<MT, sizeof(MT) == 4 ? GDN_KV_F32 : GDN_KV_BF16>(a, items, write, aligned, stream);
  }
}

template hipError_t launch_kv<float>(const KvArgs&, int, bool, bool, hipStream_t);
template hipError_t launch_kv<bf16>(const KvArgs&, int, bool, bool, hipStream_t);

}  // namespace gdn
