// The paged cache's formats: where a token's row lies, and eight of its
// channels as floats to and from what a pool holds.
//
// A block of 32 channels in 8 or 4 bits is 2^e times e4m3 or e2m1 codes, e the
// least integer >= -110 with max|x| <= M 2^e (M = 448 or 6).  With max|x| = m
// 2^f, 1 <= m < 2, and M = 1.75 2^8 (1.5 2^2) that is f - 8 (f - 2), one more
// where m > 1.75 (1.5): read off the bits of max|x|, no division.  x 2^-e is
// exact, so the code's rounding is the only one, and codes times 2^e are exact
// in bf16 and fp32 (down to 2^-119, a normal number in both).
#pragma once

#include "gdn.h"
#include "gdn_layer.h"

namespace gdn {

// Row of a pool in which position `pos` of a sequence lies (its table row), or
// -1: no place.
__device__ __forceinline__ int64_t kv_row(const int32_t* table, int64_t width, int64_t pages, int page_bits, int64_t pos,
                                          int Hk, int h) {
  const int64_t i = pos >> page_bits;
  if (pos < 0 || i >= width) return -1;
  const int64_t page = table[i];
  if (page < 0 || page >= pages) return -1;
  return ((page * Hk + h) << page_bits) + (pos & (((int64_t)1 << page_bits) - 1));
}

// a scale byte s as a float, 2^(s - 127): below the least normal number for 0; 255 is NaN
__device__ __forceinline__ float kv_scale(unsigned s) {
  return __builtin_bit_cast(float, s == 255 ? 0x7FC00000u : s == 0 ? 0x00400000u : s << 23);
}

// Bits of max|x| over 8 channels (NaN and infinities largest), then over the
// four lanes of a quad, which hold a block.
__device__ __forceinline__ unsigned block_top(const float (&x)[8]) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned u = __builtin_bit_cast(unsigned, x[i]) & 0x7FFFFFFFu;
    m = u > m ? u : m;
  }
  const unsigned a = (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true);  // quad: 1 0 3 2
  m = a > m ? a : m;
  const unsigned b = (unsigned)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true);  // quad: 2 3 0 1
  return b > m ? b : m;
}

template <int FORMAT>
__device__ __forceinline__ unsigned block_scale(unsigned top) {
  constexpr unsigned kRoom = FORMAT == GDN_KV_MXFP8 ? 0x600000u : 0x400000u;
  constexpr int kTop = FORMAT == GDN_KV_MXFP8 ? 8 : 2;
  if (top >= 0x7F800000u) return 255;
  const int s = (int)(top >> 23) - kTop + ((top & 0x7FFFFFu) > kRoom ? 1 : 0);
  return s < 17 ? 17 : (unsigned)s;
}

// Eight channels as codes: two words (e4m3) or one (e2m1, in word 0).
template <int FORMAT>
__device__ __forceinline__ void encode8(const float (&x)[8], unsigned scale, unsigned (&w)[2]) {
  const float inv = __builtin_bit_cast(float, (254u - scale) << 23);  // 2^-e, a normal number (byte 255: whatever)
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
  if constexpr (FORMAT == GDN_KV_MXFP8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], c, true);
      w[i] = (unsigned)c;
    }
  } else {
    unsigned c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.0f, 3);
    w[0] = c;
    w[1] = 0;
  }
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int FORMAT>
__device__ __forceinline__ void decode8(const unsigned (&w)[2], float scale, float (&x)[8]) {
  f32x2 p[4];
  if constexpr (FORMAT == GDN_KV_MXFP8) {
    p[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], false);
    p[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], true);
    p[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[1], false);
    p[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[1], true);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 3);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = p[i][0] * scale;
    x[2 * i + 1] = p[i][1] * scale;
  }
}

// A vector that is read `once`: non-temporal.  That is faster where the data
// comes from memory (64 ragged sequences' attention, 1092 MB: 199 us against 212;
// 143 MB out of a cache in 4 bits: 150 against 158) and slower where it waits in
// the cache (fp32 attention over a window, 38 MB: 18.0 against 16.1; 11 MB out of
// a cache in 4 bits: 27.9 against 19.9), so a call that reads less than kOnceBytes
// of a cache does without.
constexpr int64_t kOnceBytes = (int64_t)64 << 20;
template <bool ONCE, typename T>
__device__ __forceinline__ T fetch(const T* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(p);
  else return *p;
}

inline int64_t row_bytes(int format, int d) {
  return format == GDN_KV_F32 ? 4 * d : format == GDN_KV_BF16 ? 2 * d : (format == GDN_KV_MXFP8 ? d : d / 2) + d / 32;
}

// Eight channels of a row, in vectors of 16 bytes; not ALIGNED to them, at any
// address of the type.
template <typename MT, bool ALIGNED>
struct Vec {
  static constexpr int kSize = 16 / sizeof(MT);
  typedef MT type __attribute__((ext_vector_type(16 / sizeof(MT)), aligned(ALIGNED ? 16 : sizeof(MT))));
};

template <typename MT, bool ALIGNED, bool ONCE>
__device__ __forceinline__ void load8(const MT* p, float (&x)[8]) {
  typedef Vec<MT, ALIGNED> V;
#pragma unroll
  for (int i = 0; i < 8; i += V::kSize) {
    const typename V::type v = fetch<ONCE>(reinterpret_cast<const typename V::type*>(p + i));
#pragma unroll
    for (int e = 0; e < V::kSize; ++e) x[i + e] = (float)v[e];
  }
}

template <typename MT, bool ALIGNED>
__device__ __forceinline__ void store8(MT* p, const float (&x)[8]) {
  typedef Vec<MT, ALIGNED> V;
#pragma unroll
  for (int i = 0; i < 8; i += V::kSize) {
    typename V::type v;
#pragma unroll
    for (int e = 0; e < V::kSize; ++e) v[e] = (MT)x[i + e];
    *reinterpret_cast<typename V::type*>(p + i) = v;
  }
}

// Eight channels from 8 * c on of row `row` of a pool, as floats.
template <typename MT, int FORMAT, bool ONCE>
__device__ __forceinline__ void pool8(const void* pool, const uint8_t* scales, int64_t row, int d, int c, float (&x)[8]) {
  if constexpr (FORMAT == GDN_KV_F32 || FORMAT == GDN_KV_BF16) {
    load8<MT, true, ONCE>(static_cast<const MT*>(pool) + row * d + 8 * c, x);
  } else {
    unsigned w[2];
    if constexpr (FORMAT == GDN_KV_MXFP8) {
      typedef unsigned vec __attribute__((ext_vector_type(2)));
      const vec v = fetch<ONCE>(reinterpret_cast<const vec*>(static_cast<const uint8_t*>(pool) + row * d + 8 * c));
      w[0] = v[0];
      w[1] = v[1];
    } else {
      w[0] = fetch<ONCE>(reinterpret_cast<const unsigned*>(static_cast<const uint8_t*>(pool) + row * (d / 2) + 4 * c));
      w[1] = 0;
    }
    decode8<FORMAT>(w, kv_scale(scales[row * (d / 32) + c / 4]), x);
  }
}

}  // namespace gdn
