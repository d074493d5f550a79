// What the layer operators' entry points check their arguments with: byte
// ranges of strided rows and whether two of them meet, sizes, alignment.  Host
// code.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

constexpr int64_t kMost = ((int64_t)1 << 31) - 1;   // B, T (offsets and indices are 32-bit) and D
constexpr int64_t kMostStride = (int64_t)1 << 40;   // elements

inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A set of byte ranges of `len` bytes: one at p + sum_i k_i s[i] for every
// 0 <= k_i < n[i].  Dimensions of one entry are dropped and the others kept
// by rising stride.
struct Rows {
  uintptr_t p = 0;
  int dims = 0;
  int64_t n[3], s[3];
  int64_t len = 0;

  Rows(const void* ptr, int64_t bytes) : p(reinterpret_cast<uintptr_t>(ptr)), len(ptr ? bytes : 0) {}
  Rows& by(int64_t count, int64_t stride_bytes) {
    if (count <= 0) len = 0;
    if (count <= 1) return *this;
    int i = dims++;
    for (; i > 0 && s[i - 1] > stride_bytes; --i) {
      s[i] = s[i - 1];
      n[i] = n[i - 1];
    }
    s[i] = stride_bytes;
    n[i] = count;
    return *this;
  }
  // bytes from the first to behind the last of the first `d` dimensions; -1
  // if that passes what an address holds
  int64_t extent(int d) const {
    int64_t e = len;
    for (int i = 0; i < d; ++i) {
      int64_t m;
      if (__builtin_mul_overflow(n[i] - 1, s[i], &m) || __builtin_add_overflow(e, m, &e) || e > ((int64_t)1 << 56)) return -1;
    }
    return e;
  }
  bool fits() const { return extent(dims) >= 0; }
  bool meets_itself() const {
    for (int i = 0; i < dims; ++i)
      if (s[i] < extent(i)) return true;
    return false;
  }
};

// Whether a and b may share a byte.  Exact for ranges apart and for rows that
// lie beside each other in the rows of one wider buffer; anything else that
// interleaves counts as meeting.
inline bool meet(const Rows& a, const Rows& b) {
  if (a.len == 0 || b.len == 0) return false;
  const uintptr_t ea = a.p + a.extent(a.dims), eb = b.p + b.extent(b.dims);
  if (ea <= b.p || eb <= a.p) return false;
  // Beside each other under the outer dimensions both share: with those all
  // multiples of the smallest (the pitch), the rest of each must lie in its
  // own part of every pitch.
  for (int k = 1; k <= a.dims && k <= b.dims; ++k) {
    const int da = a.dims - k, db = b.dims - k;
    const int64_t pitch = a.s[da];
    if (a.n[da] != b.n[db] || pitch != b.s[db] || pitch <= 0) return true;
    bool multiples = true;
    for (int i = da; i < a.dims; ++i) multiples = multiples && a.s[i] % pitch == 0;
    if (!multiples) continue;
    const int64_t la = a.extent(da), lb = b.extent(db);
    const int64_t apart = b.p >= a.p ? (int64_t)((b.p - a.p) % (uintptr_t)pitch)
                                     : (int64_t)((pitch - (int64_t)((a.p - b.p) % (uintptr_t)pitch)) % pitch);
    if (apart >= la && apart + lb <= pitch) return false;
  }
  return true;
}

inline bool stride_ok(int64_t s) { return s >= 0 && s <= kMostStride; }

inline gdn_status_t launched(hipError_t e) {
  return e == hipSuccess ? GDN_OK : e == hipErrorNotSupported ? GDN_ERR_UNSUPPORTED : GDN_ERR_HIP;
}

inline size_t elem(int32_t dtype) { return dtype == GDN_DTYPE_BF16 ? 2 : 4; }

// rows [B][T] of `len` elements; packed: [T]
inline Rows token_rows(const void* p, int64_t len, size_t es, int64_t B, int64_t sb, int64_t T, int64_t st, bool packed) {
  Rows r(p, len * (int64_t)es);
  r.by(T, st * (int64_t)es);
  if (!packed) r.by(B, sb * (int64_t)es);
  return r;
}

// whether every row starts on 16 bytes
inline bool rows_aligned(const void* p, size_t es, int64_t B, int64_t sb, int64_t T, int64_t st, bool packed) {
  return is_aligned(p, 16) && (T <= 1 || st * es % 16 == 0) && (packed || B <= 1 || sb * es % 16 == 0);
}

inline bool slots_ok(int64_t slots, const int32_t* index, int64_t B) {
  return slots >= 1 && slots <= kMost && (index || slots == B) && is_aligned(index, 4);
}

// in-place or apart
inline bool state_pair_ok(const void* in, const void* out, int64_t bytes) {
  return !in || !out || in == out || !meet(Rows(in, bytes), Rows(out, bytes));
}

}  // namespace gdn
