// Attention of one new token per sequence over a paged cache.
//
//   s_p = scale q . k_p,  out = sum_p e^(s_p - m) v_p / l,  l = sum_p e^(s_p - m),
//   lse = m + log l,  m = max_p s_p
//
// One pass over the keys and values with a running maximum and sum (in powers
// of two), split over the length: bound by reading the cache.  64 sequences of up
// to 8192 tokens, 32 query heads on 8 of 128, bf16: 1092 MB in 178 + 7 us (6.0
// TB/s); one of 131072 tokens in 8 bits: 277 MB in 48 + 4 (5.8 TB/s).  A cache in
// 4 bits is bound by the vector instructions that turn codes into operands: 128
// sequences of up to 8192, 16 query heads on one, 72 MB in 32 us (cached).
// A few short sequences end at the latency of one tile's chain and two launches:
// 1560 tokens of 12 heads 6.5 + 3.3 us.
//
// A wave walks tiles of 32 tokens of one head of the cache and up to 32 query
// heads that share it, in registers alone.  With g = lane / 16, n = lane % 16:
//   S^T = K Q^T  (tokens x queries): lane n of A holds the key of token n (of
//     each half of the tile), group g channels of it; a lane of the result holds
//     the scores of tokens 4g .. 4g+3 with query n.
//   O^T = V^T P^T  (channels x queries): the contraction takes, in group g, just
//     those tokens, so the weights go in as they came out.  A's row n is channel
//     c of the ones that lane n loaded of each of the eight tokens: its values
//     lie in one lane already and need only be put in pairs.
// So keys and values are read as they lie in memory, once, and nothing crosses
// lanes but the maximum over groups.  Query n is the lane's in both results, as
// are its maximum, sum and rescaling.
//
// Rounding: queries and values of 16 bits or fewer enter bf16 products exactly,
// weights as three bf16 terms that add up to them (two are off by 2^-15 at most
// and turn one output in two thousand to its other neighbour, for 1.1 us less of 32.3
// where products bound it: 128 sequences of up to 8192, 16 query heads on one, in
// 4 bits), fp32 queries as three (off by 2^-24 at most); a cache in fp32 goes
// through fp32 products.  Everything else is fp32.
#include "gdn_kv.h"

namespace gdn {
namespace {

constexpr int kTile = 32;          // tokens
constexpr int kWaves = 4;
constexpr int kLeast = kWaves;     // tiles of an item: one a wave
// Sequences are not cut where they have at most 16 tiles (8 heads, 512 tokens: 1
// sequence 9.1 us against 10.5, 32 sequences 10.9 against 16.5; 1024 tokens: 13.7
// against 10.5), or at most 64 and there are workgroups for most compute units
// without (2048 tokens: 8 sequences 22.9 against 15.9, 32 33.1 against 35.5, 128
// 105 against 115).
// Nor from 1024 sequences on: each workgroup of a cut call goes through all
// lengths, which alone keep the card busy (to 4096 tokens, 32 query heads on 8:
// 1024 sequences 1202 against 1886, 4096 4645 against 12664; to 256 tokens in a
// table for 32768: 193 against 859.  One long sequence among short ones would
// rather be cut below that: 32768 among 512 of up to 256, 4 query heads on one,
// 280 against 46; among 2048 281 against 392).
constexpr int kShort = 16, kWhole = 64, kMany = 1024;
// Where they are not cut, eight waves take each (if the registers allow it) for
// up to kFew workgroups or beyond kLong tiles, else four, of which a compute unit
// holds more: 512 tokens, 128 sequences of 8 heads 39 us with eight, 33 with four;
// 64 tokens 20 and 11; 2048 tokens 105 and 113; 24 windows of 793 in fp32 on 4
// heads 15.5 and 15.9.
constexpr int kFew = 128, kLong = 32;
constexpr int kCuts = 4;           // items for every sequence, where there are many of unequal length

// Workgroups of four waves that a compute unit runs at once, by their registers.
constexpr int at_once(int D, int QT, size_t size) {
  return D * QT <= 64 ? (size == 4 ? 3 : 4) : D * QT <= 128 ? (size == 4 ? 2 : 3) : D * QT <= 256 ? (size == 4 ? 1 : 2) : 1;
}

// What of a sequence is visible: [0, sinks) and [lo, len), as `tiles` tiles, the
// first `first` of them from position 0 on, the others from tile `from` on.
struct Seen {
  int64_t len, lo, sinks, tiles, first, from;
};

__device__ __forceinline__ Seen seen_of(const AttendArgs& a, int64_t len) {
  const int64_t reach = a.width << a.page_bits;
  Seen s;
  s.len = len < 0 ? 0 : len > reach ? reach : len;
  s.lo = a.window && s.len > a.window ? s.len - a.window : 0;
  s.sinks = a.sinks < s.lo ? a.sinks : s.lo;
  s.from = s.lo / kTile;
  s.first = (s.sinks + kTile - 1) / kTile;
  if (s.first > s.from) s.first = s.from;
  s.tiles = s.first + (s.len + kTile - 1) / kTile - s.from;
  return s;
}

// Items: runs of C tiles of one sequence, C the least number that leaves at
// most `a.items - B` whole ones; sequence s owns the items floor(before / C) + s
// onwards, `before` the tiles of the sequences before it (as packed batches
// are cut; see find_packed).  Each has one at least.
struct Item {
  int64_t b, chunk, chunks, C;
  int64_t len;
  bool any;  // something to do
};

// Running sum over a wave (modulo 2^32): rows of 16 shifted by 1, 2, 4 and 8,
// then a row's last lane to the next and lane 31 to the upper half.
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned moved(unsigned x) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ unsigned wave_scan(unsigned x) {
  x += moved<0x111, 0xF>(x);
  x += moved<0x112, 0xF>(x);
  x += moved<0x114, 0xF>(x);
  x += moved<0x118, 0xF>(x);
  x += moved<0x142, 0xA>(x);
  x += moved<0x143, 0xC>(x);
  return x;
}

// Lane l's value, the same for the whole wave.
__device__ __forceinline__ int64_t of_lane(int64_t x, int l) {
  const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)x, l), hi = (unsigned)__builtin_amdgcn_readlane((int)(x >> 32), l);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// a / b for a >= 0, b > 0; a division of 64 bits only where it takes one
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((unsigned)a / (unsigned)b) : a / b;
}

// A word that is the same for the whole wave, by a scalar load.
__device__ __forceinline__ int uniform_word(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int*)(uintptr_t)p;
}

__device__ __forceinline__ Item find_item(const AttendArgs& a, int64_t i) {
  const int lane = threadIdx.x & 63;
  if (!a.plan) {  // whole sequences
    Item it;
    it.b = i;
    it.chunk = 0;
    it.chunks = it.C = 1;
    it.len = uniform_word(a.lengths + i);
    it.any = true;
    return it;
  }
  if (a.B == 1) {
    Item it;
    it.b = 0;
    it.chunk = i;
    it.len = uniform_word(a.lengths);
    const int64_t tiles = seen_of(a, it.len).tiles, most = a.items - 1;
    it.C = quotient(tiles + most - 1, most);
    if (it.C < kLeast) it.C = kLeast;
    it.chunks = tiles ? quotient(tiles + it.C - 1, it.C) : 1;
    it.any = i < it.chunks;
    return it;
  }
  const int rounds = (int)((a.B + 63) / 64);
  int64_t total = 0;
  unsigned n = 0, before = 0;  // tiles of the lane's sequence, and before it among these 64
  int64_t len = 0;
  for (int r = 0; r < rounds; ++r) {
    const int64_t b = r * 64 + lane;
    len = b < a.B ? a.lengths[b] : 0;
    n = b < a.B ? (unsigned)seen_of(a, len).tiles : 0;
    before = wave_scan(n) - n;
    total += (int64_t)(unsigned)__builtin_amdgcn_readlane((int)before, 63) + (unsigned)__builtin_amdgcn_readlane((int)n, 63);
  }
  Item it;
  const int64_t most = a.items - a.B;
  it.C = quotient(total + most - 1, most);
  if (it.C < kLeast) it.C = kLeast;
  int64_t run = 0;
  it.b = 0;
  for (int r = 0; r < rounds; ++r) {
    const int64_t b = r * 64 + lane;
    if (rounds > 1) {
      len = b < a.B ? a.lengths[b] : 0;
      n = b < a.B ? (unsigned)seen_of(a, len).tiles : 0;
      before = wave_scan(n) - n;
    }
    const int64_t at = run + before;
    const int64_t first = quotient(at, it.C) + b;
    const unsigned long long in = __ballot(b < a.B && first <= i);
    if (in == 0) break;
    const int l = 63 - __builtin_clzll(in);
    it.b = r * 64 + l;
    it.chunk = i - of_lane(first, l);
    it.len = of_lane(len, l);
    const int64_t tiles = (unsigned)__builtin_amdgcn_readlane((int)n, l);
    it.chunks = tiles ? quotient(tiles + it.C - 1, it.C) : 1;
    if (in != ~0ull) break;
    run += (int64_t)(unsigned)__builtin_amdgcn_readlane((int)before, 63) + (unsigned)__builtin_amdgcn_readlane((int)n, 63);
  }
  it.any = it.chunk < it.chunks;
  return it;
}

__device__ __forceinline__ float over_groups_max(float x) {
  return over_groups(x, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float over_groups_sum(float x) {
  return over_groups(x, [](float a, float b) { return a + b; });
}

constexpr float kMostBf16 = 0x1.FEp127f;

// N words of a pool, aligned to `A` bytes, read ONCE (see fetch) or not.
template <int N, int A, bool ONCE>
__device__ __forceinline__ void words(const uint8_t* p, unsigned (&w)[N]) {
  typedef unsigned vec __attribute__((ext_vector_type(N), aligned(A)));
  const vec v = fetch<ONCE>(reinterpret_cast<const vec*>(p));
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = v[i];
}

// Two channels from codes, as two bf16 values.  The instructions take the
// exponent of `scale` alone, the scale byte as it is: 0 is 2^-127 and 255 NaN.
template <int FORMAT, int AT>  // AT: which pair of the word
__device__ __forceinline__ unsigned two(unsigned w, float scale) {
  if constexpr (FORMAT == GDN_KV_BF16)
    return w;
  else if constexpr (FORMAT == GDN_KV_MXFP8)
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, AT != 0));
  else
    return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, AT));
}

// The geometry of a row of D channels in a format.
template <int FORMAT, int D>
struct Shape {
  static constexpr bool kWide = FORMAT == GDN_KV_F32;
  static constexpr bool kCodes = FORMAT == GDN_KV_MXFP8 || FORMAT == GDN_KV_MXFP4;
  static constexpr int kBits = kWide ? 32 : FORMAT == GDN_KV_BF16 ? 16 : FORMAT == GDN_KV_MXFP8 ? 8 : 4;
  static constexpr int kRow = D * kBits / 8;             // bytes
  static constexpr int kBlocks = D / 32;                 // scale bytes
  static constexpr int kPerWord = 32 / kBits;            // channels
  // keys: a lane loads kRun channels at a time, its group's of every 4 kRun
  static constexpr int kRun = 128 / kBits < D / 4 ? 128 / kBits : D / 4;
  static constexpr int kLoads = D / (4 * kRun);
  static constexpr int kLoadWords = kRun / kPerWord;
  // values: a lane loads kCols channels of a token, kPiece at a time
  static constexpr int kCols = D / 16;
  static constexpr int kPiece = 128 / kBits < kCols ? 128 / kBits : kCols;
  static constexpr int kPieces = kCols / kPiece;
  static constexpr int kPieceBytes = kPiece * kBits / 8;
  static constexpr int kPieceWords = (kPieceBytes + 3) / 4;
  // first channel of the eight (four, in fp32: one of four) that lane group g
  // brings to product m
  static __device__ __forceinline__ int channel(int m, int g) {
    if constexpr (kWide) return m * 16 + g * 4;
    constexpr int per = kRun / 8;
    return (m / per) * 4 * kRun + g * kRun + (m % per) * 8;
  }
  // channel of the output that lane group g holds at (column c, register i)
  static __device__ __forceinline__ int out_channel(int c, int g, int i) {
    return (c / kPiece) * 16 * kPiece + (4 * g + i) * kPiece + c % kPiece;
  }
};

template <typename MT, int FORMAT, int D, int QT, int WAVES, bool ONCE>
__global__ __launch_bounds__(WAVES * 64, WAVES == 8 ? 2 : at_once(D, QT, sizeof(MT))) void attend_kernel(AttendArgs a) {
  typedef Shape<FORMAT, D> F;
  constexpr bool kWide = F::kWide, kCodes = F::kCodes;
  constexpr int kQTerms = kWide || sizeof(MT) == 2 ? 1 : 3, kPTerms = kWide ? 1 : 3;
  __shared__ f32x4 dump[WAVES / 2][QT * F::kCols * 64];
  __shared__ float stat[2][WAVES][QT * 16];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int g = lane >> 4, n = lane & 15;
  const int G = a.Hq / a.Hk, shares = (G + 16 * QT - 1) / (16 * QT);
  const int kh = (int)(blockIdx.x % a.Hk), share = (int)(blockIdx.x / a.Hk % shares);
  const int64_t item = a.first + blockIdx.x / ((unsigned)a.Hk * shares);
  // Page numbers of a tile's halves, from its position, as the table has them:
  // they are looked at where they are used, a tile later (see below).
  struct Pages { int p[2]; };
  auto pages_at = [&](const int32_t* table, int64_t pos) {
    Pages r;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t i = (pos + 16 * s) >> a.page_bits;
      r.p[s] = uniform_word(table + (i < a.width ? i : a.width - 1));
    }
    return r;
  };
  // one sequence, or whole ones, without a window: where the first tile lies does not wait for the length
  const bool known = (a.B == 1 || !a.plan) && !a.window;
  Pages now = {};
  if (known) now = a.plan ? pages_at(a.table, (item * WAVES + wave) * kTile) : pages_at(a.table + item * a.width, wave * kTile);
  const Item it = find_item(a, item);
  if (!it.any) return;
  const int64_t b = it.b;
  const Seen seen = seen_of(a, it.len);
  if (a.plan && it.chunk == 0 && kh == 0 && share == 0 && threadIdx.x == 0) {
    a.plan[2 * b] = (int)item;
    a.plan[2 * b + 1] = (int)it.chunks;
  }

  // queries, by the channels that the keys come in: loaded here, used after the
  // first tile's loads are under way
  const int heads = G - share * 16 * QT < 16 * QT ? G - share * 16 * QT : 16 * QT;  // of this workgroup
  const int head0 = kh * G + share * 16 * QT;
  constexpr int kChans = kWide ? 4 : 8, kProducts = D / (4 * kChans);  // channels of a lane, loads
  MT qr[QT][kProducts][kChans];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const MT* q = static_cast<const MT*>(a.q) + b * a.q_sb + (head0 + (t * 16 + n < heads ? t * 16 + n : 0)) * a.q_sh;
#pragma unroll
    for (int m = 0; m < kProducts; ++m) {
      if (a.q_aligned) {
        __builtin_memcpy(qr[t][m], __builtin_assume_aligned(q + F::channel(m, g), 16), sizeof(qr[t][m]));
      } else {
#pragma unroll
        for (int e = 0; e < kChans; ++e) qr[t][m][e] = q[F::channel(m, g) + e];
      }
    }
  }

  // tiles of this wave: the items of a sequence take turns, a tile a wave
  const int64_t end = seen.tiles, step = it.chunks * WAVES;
  int64_t tile = it.chunk * WAVES + wave;
  const int32_t* table = a.table + b * a.width;
  const uint8_t* pools[2] = {static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache)};
  const int64_t mask = ((int64_t)1 << a.page_bits) - 1;
  const unsigned k_off = n * F::kRow + g * (F::kRun * F::kBits / 8), v_off = 4 * g * F::kRow + n * F::kPieceBytes;

  auto place = [&](int64_t t) { return (t < seen.first ? t : t - seen.first + seen.from) * kTile; };
  auto pages_of = [&](int64_t t) { return pages_at(table, t < end ? place(t) : 0); };
  // (positions beyond the table are beyond the length too)
  auto has_page = [&](const Pages& p, int s) { return p.p[s] >= 0 && p.p[s] < a.pages; };
  // first row in the pools of half s of a tile (page 0 where there is none)
  auto row_of = [&](int64_t t, const Pages& p, int s) {
    const int64_t page = has_page(p, s) ? p.p[s] : 0;
    return ((page * a.Hk + kh) << a.page_bits) + ((place(t) + 16 * s) & mask);
  };

  unsigned kw[2][F::kLoads][F::kLoadWords], vw[8][F::kPieces][F::kPieceWords];
  unsigned ksw[2][kCodes ? (F::kBlocks + 3) / 4 : 1], vsw[2][kCodes ? F::kBlocks : 1];
  auto load_k = [&](int64_t t, const Pages& p) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t row = row_of(t, p, s);
      const uint8_t* base = pools[0] + row * F::kRow;
#pragma unroll
      for (int j = 0; j < F::kLoads; ++j)
        words<F::kLoadWords, F::kLoadWords * 4, ONCE>(base + k_off + j * (4 * F::kRun * F::kBits / 8), kw[s][j]);
      if constexpr (kCodes) {
        const uint8_t* scales = a.k_scales + row * F::kBlocks;
        if constexpr (F::kBlocks == 2) ksw[s][0] = *reinterpret_cast<const uint16_t*>(scales + n * 2);
        else words<F::kBlocks / 4, 4, ONCE>(scales + n * F::kBlocks, ksw[s]);
      }
    }
  };
  auto load_v = [&](int64_t t, const Pages& p) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t row = row_of(t, p, s);
      const uint8_t* base = pools[1] + row * F::kRow;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < F::kPieces; ++j) {
          const uint8_t* at = base + v_off + i * F::kRow + j * 16 * F::kPieceBytes;
          if constexpr (F::kPieceBytes == 2) vw[4 * s + i][j][0] = *reinterpret_cast<const uint16_t*>(at);
          else words<F::kPieceWords, F::kPieceBytes, ONCE>(at, vw[4 * s + i][j]);
        }
      // the scale bytes of tokens 4g .. 4g + 3
      if constexpr (kCodes) words<F::kBlocks, 4, ONCE>(a.v_scales + (row + 4 * g) * F::kBlocks, vsw[s]);
    }
  };

  f32x4 acc[QT][F::kCols];
  float top[QT], sum[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    top[t] = -INFINITY;
    sum[t] = 0.0f;
#pragma unroll
    for (int c = 0; c < F::kCols; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const float scale2 = a.scale * kLog2e;

  Pages next = {};
  if (tile < end) {
    if (!known) now = pages_of(tile);
    load_k(tile, now);
    load_v(tile, now);
    next = pages_of(tile + step);
  }
  bf16x8 qb[kWide ? 1 : QT][kQTerms][kWide ? 1 : kProducts];
  float qw[kWide ? QT : 1][kWide ? kProducts : 1][4];
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int m = 0; m < kProducts; ++m)
#pragma unroll
      for (int e = 0; e < kChans; ++e) {
        float rest = t * 16 + n < heads ? (float)qr[t][m][e] : 0.0f;
        if constexpr (kWide) {
          qw[t][m][e] = rest;
        } else {
#pragma unroll
          for (int k = 0; k < kQTerms; ++k) {
            // (the type's largest where fp32 goes on: infinite first terms leave NaN; the last one carries an infinity)
            const bool beyond = k + 1 < kQTerms && fabsf(rest) > kMostBf16;
            qb[t][k][m][e] = (bf16)(beyond ? copysignf(kMostBf16, rest) : rest);
            rest -= (float)qb[t][k][m][e];
          }
        }
      }
  f32x4 s[QT][2];
  auto scores = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (kWide) {
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          // (four sums, each a chain of a quarter of the products: one chain of all is off by twice as much, 8 sequences of
          // 512 tokens with heads of 128 by 5.4e-7 of the outputs against 2.6e-7, in the same time)
          f32x4 part[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) part[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              part[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, kw[h][m][e]), qw[t][m][e], part[e], 0, 0, 0);
          s[t][h] = (part[0] + part[1]) + (part[2] + part[3]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < QT; ++t) s[t][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < D / 32; ++m) {
          constexpr int per = F::kRun / 8, wpm = 8 / F::kPerWord;  // products of a load, words of a product
          float f = 1.0f;
          if constexpr (kCodes) {
            // the block of channel(m, g): its word and byte
            constexpr int kHalf = F::kRun == 16;  // two groups share a block
            const int at = F::kRun == 16 ? 2 * (m / per) : 4 * (m / per);
            const unsigned byte = (ksw[h][at / 4] >> (8 * (at % 4) + 8 * (kHalf ? g >> 1 : g))) & 255u;
            f = __builtin_bit_cast(float, byte << 23);
          }
          unsigned w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned src = kw[h][m / per][(m % per) * wpm + e * wpm / 4];
            if constexpr (FORMAT == GDN_KV_BF16) w[e] = src;
            else if constexpr (FORMAT == GDN_KV_MXFP8) w[e] = e % 2 ? two<FORMAT, 1>(src, f) : two<FORMAT, 0>(src, f);
            else w[e] = e == 0 ? two<FORMAT, 0>(src, f) : e == 1 ? two<FORMAT, 1>(src, f) : e == 2 ? two<FORMAT, 2>(src, f) : two<FORMAT, 3>(src, f);
          }
          bf16x8 k;
          __builtin_memcpy(&k, w, 16);
#pragma unroll
          for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int x = kQTerms - 1; x >= 0; --x)
              s[t][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, qb[t][x][m], s[t][h], 0, 0, 0);
        }
      }
    }
  };
  // weights of the tile's tokens, and their values added
  auto values = [&]() {
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) s[t][h] *= scale2;
    // a tile that is not visible as a whole: which of the lane's tokens are
    const int64_t p0 = place(tile);
    const bool whole = p0 + kTile <= seen.len && (p0 >= seen.lo || p0 + kTile <= seen.sinks) && has_page(now, 0) && has_page(now, 1);
    unsigned ok = 0xFF;
    if (!whole) {
      asm volatile("");  // (a branch: whole tiles are spared the selections)
      ok = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t p = p0 + 16 * (i / 4) + 4 * g + i % 4;
        if (p < seen.len && (p >= seen.lo || p < seen.sinks) && has_page(now, i / 4)) ok |= 1u << i;
      }
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[t][i / 4][i % 4] = (ok >> i) & 1 ? s[t][i / 4][i % 4] : -INFINITY;
    }
    bf16x8 pb[kWide ? 1 : QT][kPTerms];
    float pw[QT][8];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float x[8], most = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = s[t][i / 4][i % 4];
        most = fmaxf(most, x[i]);
      }
      most = fmaxf(top[t], over_groups_max(most));
      const float ref = most == -INFINITY ? 0.0f : most;
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pw[t][i] = hw_exp2(x[i] - ref);
        part += pw[t][i];
      }
      if (__any(most > top[t])) {
        const float keep = hw_exp2(top[t] - ref);
        sum[t] *= keep;
#pragma unroll
        for (int c = 0; c < F::kCols; ++c) acc[t][c] *= keep;
        top[t] = most;
      }
      sum[t] += part;
      if constexpr (!kWide)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // the first two terms: what is left cut to bf16, or the next below where
          // that is all of it, so that no term of a weight above 2^-100 is zero (an
          // infinite value times each stays infinite) and all of zero are.  Three
          // times eight bits hold all 24.
          float rest = pw[t][i];
#pragma unroll
          for (int k = 0; k < kPTerms; ++k) {
            const unsigned bits = __builtin_bit_cast(unsigned, rest);
            const float cut = __builtin_bit_cast(float, ((bits > 1u ? bits : 1u) - 1u) & 0xFFFF0000u);
            pb[t][k][i] = (bf16)(k + 1 < kPTerms ? cut : rest);
            rest -= cut;
          }
        }
    }
    // values; what is not visible is zero, whatever lies there
    float vs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      vs[i] = 0.0f;
      if constexpr (kCodes) {
        const int block = n * F::kCols / 32;  // of the lane's channels
        const unsigned w = F::kBlocks == 2 ? vsw[i / 4][(i % 4) / 2] >> (16 * (i % 2))
                           : F::kBlocks == 4 ? vsw[i / 4][i % 4]
                                             : block >= 4 ? vsw[i / 4][2 * (i % 4) + 1] : vsw[i / 4][2 * (i % 4)];
        vs[i] = __builtin_bit_cast(float, ((w >> (8 * (block & 3))) & 255u) << 23);
      }
    }
    if (!whole) {
      asm volatile("");
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!((ok >> i) & 1)) {
          vs[i] = 0.0f;
#pragma unroll
          for (int j = 0; j < F::kPieces; ++j)
#pragma unroll
            for (int w = 0; w < F::kPieceWords; ++w) vw[i][j][w] = 0;
        }
    }
    if constexpr (kWide) {
#pragma unroll
      for (int c = 0; c < F::kCols; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int t = 0; t < QT; ++t)
            acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, vw[i][c / F::kPiece][c % F::kPiece]), pw[t][i],
                                                             acc[t][c], 0, 0, 0);
    } else {
#pragma unroll
      for (int c = 0; c < F::kCols; c += 2) {
        unsigned pair[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const unsigned src = vw[i][c / F::kPiece][c % F::kPiece / F::kPerWord];
          const int at = c % F::kPerWord / 2;
          pair[i] = at == 0 ? two<FORMAT, 0>(src, vs[i]) : at == 1 ? two<FORMAT, 1>(src, vs[i]) : at == 2 ? two<FORMAT, 2>(src, vs[i]) : two<FORMAT, 3>(src, vs[i]);
        }
        unsigned even[4], odd[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          even[u] = __builtin_amdgcn_perm(pair[2 * u + 1], pair[2 * u], 0x05040100u);
          odd[u] = __builtin_amdgcn_perm(pair[2 * u + 1], pair[2 * u], 0x07060302u);
        }
        bf16x8 v[2];
        __builtin_memcpy(&v[0], even, 16);
        __builtin_memcpy(&v[1], odd, 16);
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int k = kPTerms - 1; k >= 0; --k)
              acc[t][c + o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[o], pb[t][k], acc[t][c + o], 0, 0, 0);
      }
    }
  };
  // The next tile's keys set out as soon as this one's are used, its values
  // likewise, each without a branch: where one of the two might not have set
  // out, waiting for one would be waiting for both.
  if (tile < end) {
    while (tile + step < end) {
      scores();
      load_k(tile + step, next);
      values();
      load_v(tile + step, next);
      // scalar loads come back in any order, so a wait for one is a wait for
      // all: the next ones set out here, and have come by when they are used
      tile += step;
      now = next;
      next = pages_of(tile + step);
    }
    scores();
    values();
  }

  // the waves' parts, brought to one maximum and added by twos
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    sum[t] = over_groups_sum(sum[t]);
    if (g == 0) {
      stat[0][wave][t * 16 + n] = top[t];
      stat[1][wave][t * 16 + n] = sum[t];
    }
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float most = -INFINITY, all = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) most = fmaxf(most, stat[0][w][t * 16 + n]);
    const float ref = most == -INFINITY ? 0.0f : most;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) all += hw_exp2(stat[0][w][t * 16 + n] - ref) * stat[1][w][t * 16 + n];
    const float f = hw_exp2(top[t] - ref);
#pragma unroll
    for (int c = 0; c < F::kCols; ++c) acc[t][c] *= f;
    top[t] = most;
    sum[t] = all;
  }
#pragma unroll
  for (int half = WAVES / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int c = 0; c < F::kCols; ++c) dump[wave - half][(t * F::kCols + c) * 64 + lane] = acc[t][c];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int c = 0; c < F::kCols; ++c) acc[t][c] += dump[wave][(t * F::kCols + c) * 64 + lane];
    if (half > 1) __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    if (t * 16 + n >= heads) continue;
    const int h = head0 + t * 16 + n;
    if (it.chunks > 1) {
      float* to = a.parts + (item * a.Hq + h) * D;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < F::kCols; ++c) to[F::out_channel(c, g, i)] = acc[t][c][i];
      if (g == 0) {
        a.stats[2 * (item * a.Hq + h)] = top[t];
        a.stats[2 * (item * a.Hq + h) + 1] = sum[t];
      }
    } else {
      // (zero, whatever 2^-inf made of the values)
      const bool none = sum[t] == 0.0f;
      const float inv = 1.0f / sum[t];
      MT* to = static_cast<MT*>(a.out) + b * a.o_sb + h * a.o_sh;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < F::kCols; ++c) to[F::out_channel(c, g, i)] = (MT)(none ? 0.0f : acc[t][c][i] * inv);
      if (g == 0 && a.lse) a.lse[b * a.Hq + h] = none ? -INFINITY : (top[t] + log2f(sum[t])) * 0.6931471805599453f;
    }
  }
}

// The items of a sequence that was split, joined: a workgroup per sequence and
// query head, its waves every eighth item, D / 64 channels a lane; a lane
// works out the weight of one of 64 items.  A chain of load latencies: the
// values' loads are under way before the maxima are known.
constexpr int kJoinWaves = 8;

template <typename MT, int D>
__global__ __launch_bounds__(kJoinWaves * 64) void join_kernel(AttendArgs a) {
  constexpr int N = D / 64, U = 64 / kJoinWaves;
  __shared__ float part[kJoinWaves][D];
  const int64_t b = a.first + blockIdx.x / a.Hq;
  const int h = (int)(blockIdx.x % a.Hq);
  const int first = a.plan[2 * b], chunks = a.plan[2 * b + 1];
  if (chunks == 1) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const float* stats = a.stats + 2 * ((int64_t)first * a.Hq + h);
  const float* parts = a.parts + ((int64_t)first * a.Hq + h) * D + lane * N;
  float v[U][N];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = base + wave + u * kJoinWaves;
      if (c < chunks) {
        __builtin_memcpy(v[u], __builtin_assume_aligned(parts + (int64_t)c * a.Hq * D, N * 4), N * 4);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[u][i] = 0.0f;
      }
    }
  };
  load(0);
  float most = -INFINITY;
  for (int c = lane; c < chunks; c += 64) most = fmaxf(most, stats[2 * (int64_t)c * a.Hq]);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) most = fmaxf(most, __shfl_xor(most, m, 64));
  const float ref = most == -INFINITY ? 0.0f : most;
  float sum = 0.0f, o[N] = {};
  for (int base = 0; base < chunks; base += 64) {
    float f = 0.0f;
    if (base + lane < chunks) {
      const float* s = stats + 2 * (int64_t)(base + lane) * a.Hq;
      f = hw_exp2(s[0] - ref);
      sum = fmaf(f, s[1], sum);
    }
    float w[U][N];
    __builtin_memcpy(w, v, sizeof(w));
    if (base + 64 < chunks) load(base + 64);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float k = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), wave + u * kJoinWaves));
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fmaf(k, w[u][i], o[i]);
    }
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, 64);
#pragma unroll
  for (int i = 0; i < N; ++i) part[wave][lane * N + i] = o[i];
  __syncthreads();
  const bool none = sum == 0.0f;
  const float inv = 1.0f / sum;
  if (threadIdx.x < D) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) x += part[w][threadIdx.x];
    static_cast<MT*>(a.out)[b * a.o_sb + h * a.o_sh + threadIdx.x] = (MT)(none ? 0.0f : x * inv);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[b * a.Hq + h] = none ? -INFINITY : (most + log2f(sum)) * 0.6931471805599453f;
}

template <typename MT, int FORMAT, int D, int QT>
hipError_t attend_launch(const AttendArgs& given, hipStream_t stream) {
  AttendArgs a = given;
  const int64_t shares = (a.Hq / a.Hk + 16 * QT - 1) / (16 * QT);
  const auto launch = [&](auto kernel, int waves) {
    return in_launches(a.items, a.Hk * shares, waves * 64, [&](int64_t first, dim3 blocks) {
      a.first = first;
      hipLaunchKernelGGL(kernel, blocks, dim3(waves * 64), 0, stream, a);
    });
  };
  if constexpr (D < 256 && D * QT * sizeof(MT) <= 512)
    if (!a.plan && a.tiles > kWaves && (a.items * a.Hk * shares <= kFew || a.tiles > kLong))
      return launch(attend_kernel<MT, FORMAT, D, QT, 8, false>, 8);
  const hipError_t e = a.plan && a.once ? launch(attend_kernel<MT, FORMAT, D, QT, kWaves, true>, kWaves)
                                        : launch(attend_kernel<MT, FORMAT, D, QT, kWaves, false>, kWaves);
  if (e != hipSuccess || !a.plan) return e;
  return in_launches(a.B, a.Hq, kJoinWaves * 64, [&](int64_t first, dim3 blocks) {
    a.first = first;
    hipLaunchKernelGGL((join_kernel<MT, D>), blocks, dim3(kJoinWaves * 64), 0, stream, a);
  });
}

// 32 query heads a workgroup where more than 16 share a head of the cache; 16
// with fp32 rows of 256 channels, whose registers do not hold more
template <typename MT, int FORMAT, int D>
hipError_t attend_by_heads(const AttendArgs& a, hipStream_t stream) {
  if constexpr (sizeof(MT) == 4 && D == 256)
    return attend_launch<MT, FORMAT, D, 1>(a, stream);
  else
    return a.Hq / a.Hk <= 16 ? attend_launch<MT, FORMAT, D, 1>(a, stream) : attend_launch<MT, FORMAT, D, 2>(a, stream);
}

template <typename MT, int FORMAT>
hipError_t attend_for(const AttendArgs& a, hipStream_t stream) {
  return a.d == 64    ? attend_by_heads<MT, FORMAT, 64>(a, stream)
         : a.d == 128 ? attend_by_heads<MT, FORMAT, 128>(a, stream)
                      : attend_by_heads<MT, FORMAT, 256>(a, stream);
}

size_t padded(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

AttendPlan attend_plan(int64_t B, int64_t Hq, int64_t Hk, int64_t d, bool half, int64_t reach, int64_t window, int64_t sinks) {
  AttendPlan p = {};
  const int64_t G = Hq / Hk;
  const int QT = G <= 16 || (!half && d == 256) ? 1 : 2;
  const int64_t shares = (G + 16 * QT - 1) / (16 * QT);
  // tiles that a sequence can have
  int64_t most = reach;
  if (window && window + sinks < reach) most = window + sinks + 2 * kTile;
  const int64_t tiles = (most + kTile - 1) / kTile;
  // not cut: one kernel and no workspace
  if (B >= kMany || tiles <= kShort || (tiles <= kWhole && B * Hk * shares >= 3 * tiles)) {
    p.items = B;
    return p;
  }
  // as many as run at once, each sequence's last one counted; or where those
  // are few for every sequence, more, in several turns
  const int64_t slots = 256 * at_once((int)d, QT, half ? 2 : 4) / (Hk * shares);
  int64_t whole = slots >= 2 * B ? slots - B : kCuts * B;
  // no more than all of them make
  const int64_t all = (tiles + kLeast - 1) / kLeast;
  if (all < (whole + B - 1) / B) whole = all * B;
  p.items = whole + B;
  p.plan_bytes = padded((size_t)B * 8);
  p.parts_bytes = padded((size_t)p.items * Hq * d * 4);
  p.total_bytes = p.plan_bytes + p.parts_bytes + padded((size_t)p.items * Hq * 8);
  return p;
}

template <typename MT>
hipError_t launch_attend(const AttendArgs& given, int format, hipStream_t stream) {
  AttendArgs a = given;
  // (what can be visible: how much is, only the device knows)
  const int64_t reach = a.width << a.page_bits, tokens = a.window && a.window + a.sinks < reach ? a.window + a.sinks : reach;
  a.tiles = (tokens + kTile - 1) / kTile;
  a.once = 2 * a.B * tokens >= kOnceBytes / (a.Hk * row_bytes(format, a.d));
  switch (format) {
    case GDN_KV_MXFP8: return attend_for<MT, GDN_KV_MXFP8>(a, stream);
    case GDN_KV_MXFP4: return attend_for<MT, GDN_KV_MXFP4>(a, stream);
    default: return attend_for<MT, sizeof(MT) == 4 ? GDN_KV_F32 : GDN_KV_BF16>(a, stream);
  }
}

template hipError_t launch_attend<float>(const AttendArgs&, int, hipStream_t);
template hipError_t launch_attend<bf16>(const AttendArgs&, int, hipStream_t);

}  // namespace gdn
