// C entry points of the layer operators (short causal convolution, selective
// scan, rotary positions, single-token steps): argument validation and
// dispatch.  Everything here is host code; validation finishes before
// anything is enqueued, so a rejected call leaves every buffer untouched.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "gdn.h"
#include "gdn_layer.h"

namespace gdn {
namespace {

constexpr int64_t kMost = ((int64_t)1 << 31) - 1;   // B, T (offsets and indices are 32-bit) and D
constexpr int64_t kMostStride = (int64_t)1 << 40;   // elements

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

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
bool meet(const Rows& a, const Rows& b) {
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

bool stride_ok(int64_t s) { return s >= 0 && s <= kMostStride; }

gdn_status_t launched(hipError_t e) {
  return e == hipSuccess ? GDN_OK : e == hipErrorNotSupported ? GDN_ERR_UNSUPPORTED : GDN_ERR_HIP;
}

size_t elem(int32_t dtype) { return dtype == GDN_DTYPE_BF16 ? 2 : 4; }

// rows [B][T] of `len` elements; packed: [T]
Rows token_rows(const void* p, int64_t len, size_t es, int64_t B, int64_t sb, int64_t T, int64_t st, bool packed) {
  Rows r(p, len * (int64_t)es);
  r.by(T, st * (int64_t)es);
  if (!packed) r.by(B, sb * (int64_t)es);
  return r;
}

// whether every row starts on 16 bytes
bool rows_aligned(const void* p, size_t es, int64_t B, int64_t sb, int64_t T, int64_t st, bool packed) {
  return is_aligned(p, 16) && (T <= 1 || st * es % 16 == 0) && (packed || B <= 1 || sb * es % 16 == 0);
}

bool slots_ok(int64_t slots, const int32_t* index, int64_t B) {
  return slots >= 1 && slots <= kMost && (index || slots == B) && is_aligned(index, 4);
}

// in-place or apart
bool state_pair_ok(const void* in, const void* out, int64_t bytes) {
  return !in || !out || in == out || !meet(Rows(in, bytes), Rows(out, bytes));
}

gdn_status_t conv_check(const gdn_conv_problem_t* p, bool step, const void* x, const float* weight, const float* bias,
                        const void* state_in, const void* state_out, const void* out, ConvArgs* a, bool* aligned) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->B, T = step ? 1 : p->T, D = p->D;
  const int32_t* off = step ? nullptr : p->seq_offsets;
  if (B < 1 || B > kMost || T < 0 || T > kMost || D < 1 || D > kMost) return GDN_ERR_INVALID_ARGUMENT;
  if (p->activation != GDN_ACT_NONE && p->activation != GDN_ACT_SILU) return GDN_ERR_INVALID_ARGUMENT;
  if (p->options & ~GDN_LAYER_OPT_ZERO_UNUSED) return GDN_ERR_INVALID_ARGUMENT;
  if (p->dtype != GDN_DTYPE_F32 && p->dtype != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED;
  if (p->width < 2 || p->width > 4) return GDN_ERR_UNSUPPORTED;
  const int64_t x_st = step ? 0 : p->x_stride_t, o_st = step ? 0 : p->out_stride_t;
  if (!stride_ok(p->x_stride_b) || !stride_ok(x_st) || !stride_ok(p->out_stride_b) || !stride_ok(o_st))
    return GDN_ERR_INVALID_ARGUMENT;
  const bool state = step || state_in || state_out;
  if (state ? !slots_ok(p->slots, p->state_index, B) : !is_aligned(p->state_index, 4)) return GDN_ERR_INVALID_ARGUMENT;
  if (!weight || (T > 0 && (!x || !out)) || (step && !state_out)) return GDN_ERR_INVALID_ARGUMENT;
  const size_t es = elem(p->dtype);
  if (!is_aligned(x, es) || !is_aligned(out, es) || !is_aligned(state_in, es) || !is_aligned(state_out, es) ||
      !is_aligned(weight, 4) || !is_aligned(bias, 4) || !is_aligned(off, 4))
    return GDN_ERR_INVALID_ARGUMENT;
  const Rows r_x = token_rows(x, D, es, B, p->x_stride_b, T, x_st, off);
  const Rows r_o = token_rows(out, D, es, B, p->out_stride_b, T, o_st, off);
  const Rows r_s = Rows(state ? (state_in ? state_in : state_out) : nullptr, (p->width - 1) * D * (int64_t)es)
                       .by(state ? p->slots : 1, (p->width - 1) * D * (int64_t)es);
  if (!r_x.fits() || !r_o.fits() || !r_s.fits()) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t sbytes = state ? r_s.extent(r_s.dims) : 0;
  const Rows ins[] = {r_x, Rows(weight, D * p->width * 4), Rows(bias, D * 4), Rows(off, (B + 1) * 4),
                      Rows(p->state_index, B * 4)};
  if (r_o.meets_itself()) return GDN_ERR_INVALID_ARGUMENT;
  for (const Rows& r : ins)
    if (meet(r_o, r) || meet(Rows(state_out, sbytes), r)) return GDN_ERR_INVALID_ARGUMENT;
  if (meet(r_o, Rows(state_in, sbytes)) || meet(r_o, Rows(state_out, sbytes))) return GDN_ERR_INVALID_ARGUMENT;
  if (!state_pair_ok(state_in, state_out, sbytes)) return GDN_ERR_INVALID_ARGUMENT;
  memset(a, 0, sizeof(*a));
  a->x = x; a->weight = weight; a->bias = bias; a->state_in = state_in; a->state_out = const_cast<void*>(state_out);
  a->out = const_cast<void*>(out);
  a->off = off; a->index = p->state_index;
  a->B = B; a->T = T; a->D = D; a->slots = p->slots;
  a->x_sb = p->x_stride_b; a->x_st = x_st; a->o_sb = p->out_stride_b; a->o_st = o_st;
  a->silu = p->activation == GDN_ACT_SILU;
  a->zero_unused = (p->options & GDN_LAYER_OPT_ZERO_UNUSED) != 0;
  *aligned = D * es % 16 == 0 && is_aligned(state_in, 16) && is_aligned(state_out, 16) &&
             rows_aligned(x, es, B, p->x_stride_b, T, x_st, off) && rows_aligned(out, es, B, p->out_stride_b, T, o_st, off);
  return GDN_OK;
}

// the sizes and options alone
gdn_status_t ssm_sizes(const gdn_ssm_problem_t* p, bool step) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->B, T = step ? 1 : p->T, D = p->D, N = p->N, G = p->G;
  if (B < 1 || B > kMost || T < 0 || T > kMost || D < 1 || D > kMost || N < 1 || G < 1 || G > D || D % G != 0)
    return GDN_ERR_INVALID_ARGUMENT;
  if (p->options & ~(GDN_SSM_OPT_SOFTPLUS | GDN_LAYER_OPT_ZERO_UNUSED)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->dtype != GDN_DTYPE_F32 && p->dtype != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED;
  if (N > 256) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status_t ssm_check(const gdn_ssm_problem_t* p, bool step, const void* x, const void* dt, const float* A,
                       const void* Bm, const void* Cm, const float* state_in, const float* state_out, const void* out,
                       SsmArgs* a) {
  const gdn_status_t sizes = ssm_sizes(p, step);
  if (sizes != GDN_OK) return sizes;
  const int64_t B = p->B, T = step ? 1 : p->T, D = p->D, N = p->N, G = p->G;
  const int32_t* off = step ? nullptr : p->seq_offsets;
  const int64_t sb[6] = {p->x_stride_b, p->dt_stride_b, p->b_stride_b, p->c_stride_b, p->out_stride_b,
                         p->z ? p->z_stride_b : 0};
  int64_t st[6] = {p->x_stride_t, p->dt_stride_t, p->b_stride_t, p->c_stride_t, p->out_stride_t, p->z ? p->z_stride_t : 0};
  for (int i = 0; i < 6; ++i) {
    if (T <= 1) st[i] = 0;  // no other token
    if (!stride_ok(sb[i]) || !stride_ok(st[i])) return GDN_ERR_INVALID_ARGUMENT;
    if (st[i] >= (int64_t)1 << 26) return GDN_ERR_UNSUPPORTED;  // some tokens' rows within 32-bit byte offsets
  }
  const bool state = step || state_in || state_out;
  if (state ? !slots_ok(p->slots, p->state_index, B) : !is_aligned(p->state_index, 4)) return GDN_ERR_INVALID_ARGUMENT;
  if (!A || (T > 0 && (!x || !dt || !Bm || !Cm || !out)) || (step && !state_out)) return GDN_ERR_INVALID_ARGUMENT;
  const size_t es = elem(p->dtype);
  const void* typed[] = {x, dt, Bm, Cm, out, p->z};
  for (const void* q : typed)
    if (!is_aligned(q, es)) return GDN_ERR_INVALID_ARGUMENT;
  const void* words[] = {A, p->dt_bias, p->skip, state_in, state_out, off};
  for (const void* q : words)
    if (!is_aligned(q, 4)) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t len[6] = {D, D, G * N, G * N, D, D};
  const Rows r_o = token_rows(out, D, es, B, sb[4], T, st[4], off);
  const Rows r_s = Rows(state ? (state_in ? state_in : state_out) : nullptr, D * N * 4).by(state ? p->slots : 1, D * N * 4);
  if (!r_o.fits() || !r_s.fits() || r_o.meets_itself()) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t sbytes = state ? r_s.extent(r_s.dims) : 0;
  const Rows so(state_out, sbytes);
  SsmPlan plan = {};
  if (!step) plan = ssm_plan(B, T, D, N, G, off != nullptr);
  const Rows ws(plan.split ? p->workspace : nullptr, (int64_t)plan.total_bytes);
  if (plan.split) {
    if (!p->workspace || !is_aligned(p->workspace, 256)) return GDN_ERR_INVALID_ARGUMENT;
    if (p->workspace_bytes < plan.total_bytes) return GDN_ERR_WORKSPACE_TOO_SMALL;
  }
  for (int i = 0; i < 6; ++i) {
    if (i == 4) continue;
    const Rows r = token_rows(typed[i], len[i], es, B, sb[i], T, st[i], off);
    if (!r.fits() || meet(r_o, r) || meet(so, r) || meet(ws, r)) return GDN_ERR_INVALID_ARGUMENT;
  }
  if (meet(ws, r_o) || meet(ws, so) || meet(ws, Rows(state_in, sbytes))) return GDN_ERR_INVALID_ARGUMENT;
  const Rows ins[] = {Rows(A, D * N * 4), Rows(p->dt_bias, D * 4), Rows(p->skip, D * 4), Rows(off, (B + 1) * 4),
                      Rows(p->state_index, B * 4)};
  for (const Rows& r : ins)
    if (meet(r_o, r) || meet(so, r) || meet(ws, r)) return GDN_ERR_INVALID_ARGUMENT;
  if (meet(r_o, Rows(state_in, sbytes)) || meet(r_o, so)) return GDN_ERR_INVALID_ARGUMENT;
  if (!state_pair_ok(state_in, state_out, sbytes)) return GDN_ERR_INVALID_ARGUMENT;
  memset(a, 0, sizeof(*a));
  a->chunk = plan.chunk; a->chunks = plan.chunks;
  if (plan.split) {
    a->ends = static_cast<float*>(p->workspace);
    a->steps = reinterpret_cast<float*>(static_cast<unsigned char*>(p->workspace) + plan.ends_bytes);
  }
  a->x = x; a->dt = dt; a->A = A; a->Bm = Bm; a->Cm = Cm; a->z = p->z; a->dt_bias = p->dt_bias; a->skip = p->skip;
  a->state_in = state_in; a->state_out = const_cast<float*>(state_out); a->out = const_cast<void*>(out);
  a->off = off; a->index = p->state_index;
  a->B = B; a->T = T; a->D = D; a->N = N; a->G = G; a->slots = p->slots;
  a->x_sb = sb[0]; a->dt_sb = sb[1]; a->b_sb = sb[2]; a->c_sb = sb[3]; a->o_sb = sb[4]; a->z_sb = sb[5];
  a->x_st = st[0]; a->dt_st = st[1]; a->b_st = st[2]; a->c_st = st[3]; a->o_st = st[4]; a->z_st = st[5];
  a->softplus = (p->options & GDN_SSM_OPT_SOFTPLUS) != 0;
  a->zero_unused = (p->options & GDN_LAYER_OPT_ZERO_UNUSED) != 0;
  a->vec4 = N % 4 == 0 && is_aligned(A, 16) && is_aligned(state_in, 16) && is_aligned(state_out, 16);
  return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status_t gdn_conv_forward(const gdn_conv_problem_t* p, const void* x, const float* weight,
                                         const float* bias, const void* state_in, void* state_out, void* out) {
  ConvArgs a;
  bool aligned = false;
  const gdn_status_t st = conv_check(p, false, x, weight, bias, state_in, state_out, out, &a, &aligned);
  if (st != GDN_OK) return st;
  if (a.T == 0 && !state_out) return GDN_OK;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_conv<bf16>(a, p->width, aligned, stream)
                                             : launch_conv<float>(a, p->width, aligned, stream));
}

extern "C" gdn_status_t gdn_conv_step(const gdn_conv_problem_t* p, const void* x, const float* weight, const float* bias,
                                      void* state, void* out) {
  ConvArgs a;
  bool aligned = false;
  const gdn_status_t st = conv_check(p, true, x, weight, bias, nullptr, state, out, &a, &aligned);
  if (st != GDN_OK) return st;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_conv_step<bf16>(a, p->width, aligned, stream)
                                             : launch_conv_step<float>(a, p->width, aligned, stream));
}

extern "C" size_t gdn_ssm_workspace_bytes(const gdn_ssm_problem_t* p) {
  if (ssm_sizes(p, false) != GDN_OK) return 0;
  return ssm_plan(p->B, p->T, p->D, p->N, p->G, p->seq_offsets != nullptr).total_bytes;
}

extern "C" gdn_status_t gdn_ssm_forward(const gdn_ssm_problem_t* p, const void* x, const void* dt, const float* A,
                                        const void* Bm, const void* Cm, const float* state_in, float* state_out,
                                        void* out) {
  SsmArgs a;
  const gdn_status_t st = ssm_check(p, false, x, dt, A, Bm, Cm, state_in, state_out, out, &a);
  if (st != GDN_OK) return st;
  if (a.T == 0 && !state_out) return GDN_OK;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_ssm<bf16>(a, stream) : launch_ssm<float>(a, stream));
}

extern "C" gdn_status_t gdn_ssm_step(const gdn_ssm_problem_t* p, const void* x, const void* dt, const float* A,
                                     const void* Bm, const void* Cm, float* state, void* out) {
  SsmArgs a;
  const gdn_status_t st = ssm_check(p, true, x, dt, A, Bm, Cm, nullptr, state, out, &a);
  if (st != GDN_OK) return st;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_ssm_step<bf16>(a, stream) : launch_ssm_step<float>(a, stream));
}

extern "C" gdn_status_t gdn_rotary(const gdn_rotary_problem_t* p, const void* q, const void* k, const double* inv_freq,
                                   const void* positions, void* q_out, void* k_out) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->B, T = p->T;
  if (B < 1 || B > kMost || T < 0 || T > kMost || p->Hq < 1 || p->Hk < 0 || p->d < 1) return GDN_ERR_INVALID_ARGUMENT;
  if (p->options & ~(GDN_ROTARY_OPT_INTERLEAVED | GDN_ROTARY_OPT_INVERSE)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->rot < 2 || p->rot % 2 != 0 || p->rot > p->d) return GDN_ERR_INVALID_ARGUMENT;
  if (p->position_bits != 0 && p->position_bits != 32 && p->position_bits != 64) return GDN_ERR_INVALID_ARGUMENT;
  if (p->axes < 1 || p->axes > 4 || (p->position_bits == 0 && p->axes != 1)) return GDN_ERR_INVALID_ARGUMENT;
  if (!isfinite(p->scale)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->position0 < -((int64_t)1 << 52) || p->position0 > ((int64_t)1 << 52)) return GDN_ERR_INVALID_ARGUMENT;
  RotaryArgs a;
  memset(&a, 0, sizeof(a));
  int64_t pairs = 0;
  for (int i = 0; i < p->axes; ++i) {
    const int64_t n = p->axes == 1 ? p->rot / 2 : p->section[i];
    if (n < 0 || n > p->rot) return GDN_ERR_INVALID_ARGUMENT;
    pairs += n;
    a.edge[i] = (int)pairs;
  }
  if (pairs != p->rot / 2) return GDN_ERR_INVALID_ARGUMENT;
  if (p->dtype != GDN_DTYPE_F32 && p->dtype != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED;
  if (p->d > 256 || p->Hq > 65536 || p->Hk > 65536) return GDN_ERR_UNSUPPORTED;
  const int64_t strides[4][3] = {{p->q_stride_b, p->q_stride_t, p->q_stride_h},
                                 {p->k_stride_b, p->k_stride_t, p->k_stride_h},
                                 {p->q_out_stride_b, p->q_out_stride_t, p->q_out_stride_h},
                                 {p->k_out_stride_b, p->k_out_stride_t, p->k_out_stride_h}};
  const void* ptr[4] = {q, p->Hk ? k : nullptr, q_out, p->Hk ? k_out : nullptr};
  if (T == 0) return GDN_OK;
  if (!q || !q_out || !inv_freq || (p->Hk && (!k || !k_out)) || (p->position_bits && !positions))
    return GDN_ERR_INVALID_ARGUMENT;
  const size_t es = elem(p->dtype);
  if (!is_aligned(inv_freq, 8) || (p->position_bits && !is_aligned(positions, p->position_bits / 8)))
    return GDN_ERR_INVALID_ARGUMENT;
  constexpr int kOperands = 4;
  const int V = (int)(16 / es);
  bool vec = p->rot % (2 * V) == 0 && p->d % V == 0;
  Rows rows[kOperands] = {Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0)};
  for (int i = 0; i < kOperands; ++i) {
    if (!ptr[i]) continue;
    const int64_t H = (i & 1) ? p->Hk : p->Hq;
    if (!is_aligned(ptr[i], es)) return GDN_ERR_INVALID_ARGUMENT;
    vec = vec && is_aligned(ptr[i], 16);
    const int64_t n[3] = {B, T, H};
    Rows r(ptr[i], p->d * (int64_t)es);
    for (int j = 2; j >= 0; --j) {
      if (!stride_ok(strides[i][j])) return GDN_ERR_INVALID_ARGUMENT;
      r.by(n[j], strides[i][j] * (int64_t)es);
      if (n[j] > 1 && strides[i][j] % V != 0) vec = false;
    }
    if (!r.fits()) return GDN_ERR_INVALID_ARGUMENT;
    rows[i] = r;
  }
  if (B > kMost / (T > 0 ? T : 1)) return GDN_ERR_UNSUPPORTED;
  a.tokens = B * T;
  const Rows others[] = {Rows(inv_freq, p->rot / 2 * 8),
                         Rows(p->position_bits ? positions : nullptr, p->axes * a.tokens * (p->position_bits / 8))};
  for (int o = 2; o < kOperands; ++o) {
    if (!ptr[o]) continue;
    if (rows[o].meets_itself()) return GDN_ERR_INVALID_ARGUMENT;
    for (const Rows& r : others)
      if (meet(rows[o], r)) return GDN_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < 2; ++i) {
      if (!ptr[i]) continue;
      // in place: the same head at the same address
      const bool same = i == o - 2 && ptr[i] == ptr[o] && (B <= 1 || strides[i][0] == strides[o][0]) &&
                        (T <= 1 || strides[i][1] == strides[o][1]) &&
                        (((o & 1) ? p->Hk : p->Hq) <= 1 || strides[i][2] == strides[o][2]);
      if (same) {
        if (o == 2) a.in_place_q = 1;
        else a.in_place_k = 1;
      } else if (meet(rows[o], rows[i])) {
        return GDN_ERR_INVALID_ARGUMENT;
      }
    }
  }
  if (meet(rows[2], rows[3])) return GDN_ERR_INVALID_ARGUMENT;
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out; a.freq = inv_freq; a.pos = positions;
  a.B = B; a.T = T; a.position0 = p->position0;
  a.q_sb = strides[0][0]; a.q_st = strides[0][1]; a.q_sh = strides[0][2];
  a.k_sb = strides[1][0]; a.k_st = strides[1][1]; a.k_sh = strides[1][2];
  a.qo_sb = strides[2][0]; a.qo_st = strides[2][1]; a.qo_sh = strides[2][2];
  a.ko_sb = strides[3][0]; a.ko_st = strides[3][1]; a.ko_sh = strides[3][2];
  a.Hq = (int)p->Hq; a.Hk = (int)p->Hk; a.d = (int)p->d; a.rot = (int)p->rot;
  a.bits = p->position_bits; a.axes = p->axes;
  a.interleaved = (p->options & GDN_ROTARY_OPT_INTERLEAVED) != 0;
  a.inverse = (p->options & GDN_ROTARY_OPT_INVERSE) != 0;
  a.scale = p->scale;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_rotary<bf16>(a, vec, stream) : launch_rotary<float>(a, vec, stream));
}

extern "C" gdn_status_t gdn_step(const gdn_step_problem_t* p, const void* q, const void* k, const void* v,
                                 const float* log_alpha, const float* beta, float* state, float* out) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->B, H = p->H, dk = p->dk, dv = p->dv;
  if (B < 1 || B > kMost || H < 1 || H > kMost || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARGUMENT;
  if (p->options & ~(GDN_OPT_NO_ERASE | GDN_OPT_EXCLUSIVE_FORWARD | GDN_LAYER_OPT_ZERO_UNUSED)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->gate && (!p->norm_weight || !(p->norm_eps >= 0.f) || !(p->norm_eps <= 3.4e38f))) return GDN_ERR_INVALID_ARGUMENT;
  if (p->dtype != GDN_DTYPE_F32 && p->dtype != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED;
  if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return GDN_ERR_UNSUPPORTED;
  if (B > kMost / H) return GDN_ERR_UNSUPPORTED;
  if (!slots_ok(p->slots, p->state_index, B)) return GDN_ERR_INVALID_ARGUMENT;
  if (!q || !k || !v || !log_alpha || !beta || !state || !out) return GDN_ERR_INVALID_ARGUMENT;
  const void* vecs[] = {q, k, v, state, p->gate};
  for (const void* x : vecs)
    if (!is_aligned(x, 16)) return GDN_ERR_INVALID_ARGUMENT;
  const void* words[] = {log_alpha, beta, out, p->gate ? p->norm_weight : nullptr};
  for (const void* x : words)
    if (!is_aligned(x, 4)) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t es = (int64_t)elem(p->dtype);
  const Rows r_s = Rows(state, H * dv * dk * 4).by(p->slots, H * dv * dk * 4);
  if (!r_s.fits()) return GDN_ERR_INVALID_ARGUMENT;
  const Rows so(state, r_s.extent(r_s.dims)), r_o(out, B * H * dv * 4);
  const Rows ins[] = {Rows(q, B * H * dk * es), Rows(k, B * H * dk * es), Rows(v, B * H * dv * es),
                      Rows(log_alpha, B * H * 4), Rows(beta, B * H * 4), Rows(p->state_index, B * 4),
                      Rows(p->gate, B * H * dv * es), Rows(p->gate ? p->norm_weight : nullptr, dv * 4)};
  for (const Rows& r : ins)
    if (meet(r_o, r) || meet(so, r)) return GDN_ERR_INVALID_ARGUMENT;
  if (meet(r_o, so)) return GDN_ERR_INVALID_ARGUMENT;
  StepArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v; a.log_alpha = log_alpha; a.beta = beta; a.state = state; a.out = out;
  a.index = p->state_index; a.gate = p->gate; a.norm_weight = p->gate ? p->norm_weight : nullptr; a.norm_eps = p->norm_eps;
  a.B = B; a.H = H; a.slots = p->slots; a.dv = (int)dv;
  a.erase = (p->options & GDN_OPT_NO_ERASE) ? 0 : 1;
  a.exclusive = (p->options & GDN_OPT_EXCLUSIVE_FORWARD) != 0;
  a.zero_unused = (p->options & GDN_LAYER_OPT_ZERO_UNUSED) != 0;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_step<bf16>(a, (int)dk, stream) : launch_step<float>(a, (int)dk, stream));
}
