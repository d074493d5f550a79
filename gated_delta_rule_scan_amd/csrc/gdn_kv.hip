// Rows of keys and values into a paged cache and back out of it.
//
// A copy, with a block's scale and codes in between where the cache has 8 or 4
// bits: memory-bound on both sides.  A thread moves eight channels of K and the
// same of V; four neighbouring lanes hold a block of 32 channels.  A workgroup
// takes a run of one sequence's tokens, all heads: on the rows' side that is
// one contiguous piece, in the pools a piece of a page for every head.
#include "gdn_kv.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename MT, int FORMAT, bool WRITE, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void kv_kernel(KvArgs a) {
  SeqItem s;
  if (a.off) {
    s = find_packed(a.off, a.B, a.T, a.chunk, blockIdx.x);
  } else {
    s.b = blockIdx.x / a.chunks;
    s.chunk = blockIdx.x % a.chunks;
    s.row0 = 0;
    s.len = a.T;
  }
  // rows behind the last sequence
  const int64_t limit = !WRITE && a.zero_unused && s.b == a.B - 1 && a.off ? a.T - s.row0 : s.len;
  const int64_t t0 = s.chunk * a.chunk;
  if (t0 >= limit) return;
  const int tokens = (int)(limit - t0 < a.chunk ? limit - t0 : a.chunk);
  const int lanes = a.d / 8;  // of a row; a multiple of four
  const unsigned per_token = (unsigned)(a.Hk * lanes);
  const int64_t first = a.start ? a.start[s.b] : 0;
  const int32_t* table = a.table + s.b * a.width;
  const int64_t seq_k = a.off ? 0 : s.b * a.k_sb, seq_v = a.off ? 0 : s.b * a.v_sb;
  for (int64_t i = threadIdx.x; i < (int64_t)tokens * per_token; i += kThreads) {
    const unsigned t = (unsigned)(i / per_token), in = (unsigned)(i % per_token);
    const int h = (int)(in / (unsigned)lanes), c = (int)(in % (unsigned)lanes);
    const int64_t tok = t0 + t;
    const int64_t row = tok < s.len ? kv_row(table, a.width, a.pages, a.page_bits, first + tok, a.Hk, h) : -1;
    MT* k = static_cast<MT*>(a.k) + seq_k + (s.row0 + tok) * a.k_st + h * a.k_sh + 8 * c;
    MT* v = static_cast<MT*>(a.v) + seq_v + (s.row0 + tok) * a.v_st + h * a.v_sh + 8 * c;
    float x[2][8];
    if constexpr (WRITE) {
      // (the lanes of a row go the same way, so a block's four are all here)
      if (row < 0) continue;
      load8<MT, ALIGNED>(k, x[0]);
      load8<MT, ALIGNED>(v, x[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        void* pool = j ? a.v_cache : a.k_cache;
        if constexpr (FORMAT == GDN_KV_F32 || FORMAT == GDN_KV_BF16) {
          store8<MT, true>(static_cast<MT*>(pool) + row * a.d + 8 * c, x[j]);
        } else {
          const unsigned scale = block_scale<FORMAT>(block_top(x[j]));
          unsigned w[2];
          encode8<FORMAT>(x[j], scale, w);
          if constexpr (FORMAT == GDN_KV_MXFP8)
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + row * a.d + 8 * c) = make_uint2(w[0], w[1]);
          else
            *reinterpret_cast<unsigned*>(static_cast<uint8_t*>(pool) + row * (a.d / 2) + 4 * c) = w[0];
          if (c % 4 == 0) (j ? a.v_scales : a.k_scales)[row * (a.d / 32) + c / 4] = (uint8_t)scale;
        }
      }
    } else {
      if (row < 0) {
        if (!a.zero_unused) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[0][e] = x[1][e] = 0.0f;
      } else {
        pool8<MT, FORMAT>(a.k_cache, a.k_scales, row, a.d, c, x[0]);
        pool8<MT, FORMAT>(a.v_cache, a.v_scales, row, a.d, c, x[1]);
      }
      store8<MT, ALIGNED>(k, x[0]);
      store8<MT, ALIGNED>(v, x[1]);
    }
  }
}

template <typename MT, int FORMAT, bool WRITE>
hipError_t kv_launch(const KvArgs& a, int64_t items, bool aligned, hipStream_t stream) {
  if (aligned)
    hipLaunchKernelGGL((kv_kernel<MT, FORMAT, WRITE, true>), dim3((unsigned)items), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((kv_kernel<MT, FORMAT, WRITE, false>), dim3((unsigned)items), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename MT, int FORMAT>
hipError_t kv_for(const KvArgs& a, int64_t items, bool write, bool aligned, hipStream_t stream) {
  return write ? kv_launch<MT, FORMAT, true>(a, items, aligned, stream) : kv_launch<MT, FORMAT, false>(a, items, aligned, stream);
}

}  // namespace

template <typename MT>
hipError_t launch_kv(const KvArgs& given, int format, bool write, bool aligned, hipStream_t stream) {
  KvArgs a = given;
  // about eight vectors of K and as many of V a thread
  const int64_t per_token = (int64_t)a.Hk * (a.d / 8);
  a.chunk = (8 * kThreads + per_token - 1) / per_token;
  if (!a.off && a.chunk > a.T) a.chunk = a.T;
  a.chunks = (a.T + a.chunk - 1) / a.chunk;
  const int64_t items = a.off ? a.T / a.chunk + a.B : a.B * a.chunks;
  if (!grid_fits(items, kThreads)) return hipErrorNotSupported;
  switch (format) {
    case GDN_KV_MXFP8: return kv_for<MT, GDN_KV_MXFP8>(a, items, write, aligned, stream);
    case GDN_KV_MXFP4: return kv_for<MT, GDN_KV_MXFP4>(a, items, write, aligned, stream);
    default: return kv_for<MT, sizeof(MT) == 4 ? GDN_KV_F32 : GDN_KV_BF16>(a, items, write, aligned, stream);
  }
}

template hipError_t launch_kv<float>(const KvArgs&, int, bool, bool, hipStream_t);
template hipError_t launch_kv<bf16>(const KvArgs&, int, bool, bool, hipStream_t);

}  // namespace gdn
