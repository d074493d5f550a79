// C entry points of what a hybrid model runs beside its recurrent layers (the
// paged cache, a new token's attention over it, the seam between two blocks):
// argument validation and dispatch.  Everything here is host code; validation
// finishes before anything is enqueued, so a rejected call leaves every buffer
// untouched.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "gdn.h"
#include "gdn_layer.h"
#include "gdn_rows.h"

namespace gdn {
namespace {

constexpr int64_t kMostHeads = 65536;

bool quantised(int32_t format) { return format == GDN_KV_MXFP8 || format == GDN_KV_MXFP4; }

// sizes of a cache, its formats, and the type of the rows beside it
gdn_status_t cache_sizes(int64_t B, int64_t Hk, int64_t d, int64_t pages, int64_t page, int64_t width, int32_t dtype,
                         int32_t format) {
  if (B < 1 || B > kMost || Hk < 1 || d < 1 || pages < 1 || pages > kMost || page < 1 || width < 1 || width > kMost)
    return GDN_ERR_INVALID_ARGUMENT;
  if (format < GDN_KV_F32 || format > GDN_KV_MXFP4) return GDN_ERR_INVALID_ARGUMENT;
  if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED;
  // a pool that is not quantised holds the rows' own type
  if (!quantised(format) && (format == GDN_KV_F32) != (dtype == GDN_DTYPE_F32)) return GDN_ERR_UNSUPPORTED;
  if (Hk > kMostHeads || (d != 64 && d != 128 && d != 256)) return GDN_ERR_UNSUPPORTED;
  if (page < 16 || page > 1024 || (page & (page - 1)) != 0) return GDN_ERR_UNSUPPORTED;
  if (B > kMost / width) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int log2_of(int64_t page) { return __builtin_ctzll((unsigned long long)page); }

int64_t code_bytes(int32_t format, int64_t d) {
  return format == GDN_KV_F32 ? 4 * d : format == GDN_KV_BF16 ? 2 * d : format == GDN_KV_MXFP8 ? d : d / 2;
}

// a pool and its scales as ranges; false: too large, misaligned or missing
bool pool_ranges(const void* pool, const void* scales, int64_t pages, int64_t Hk, int64_t page, int64_t d, int32_t format,
                 Rows* r) {
  if (!pool || !is_aligned(pool, 16)) return false;
  const int64_t rows = Hk * page;
  r[0] = Rows(pool, rows * code_bytes(format, d)).by(pages, rows * code_bytes(format, d));
  r[1] = Rows(nullptr, 0);
  if (quantised(format)) {
    if (!scales || !is_aligned(scales, 4)) return false;
    r[1] = Rows(scales, rows * (d / 32)).by(pages, rows * (d / 32));
  }
  if (!r[0].fits() || !r[1].fits()) return false;
  // (one range each)
  r[0] = Rows(pool, r[0].extent(r[0].dims));
  if (r[1].len) r[1] = Rows(scales, r[1].extent(r[1].dims));
  return true;
}

gdn_status_t kv_call(const gdn_kv_problem_t* p, bool write, const void* k, const void* v, const void* k_cache,
                     const void* v_cache, const void* k_scales, const void* v_scales) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->B, T = p->T, Hk = p->Hk, d = p->d;
  if (T < 0 || T > kMost) return GDN_ERR_INVALID_ARGUMENT;
  if (p->options & ~(write ? 0 : (int32_t)GDN_LAYER_OPT_ZERO_UNUSED)) return GDN_ERR_INVALID_ARGUMENT;
  const gdn_status_t sizes = cache_sizes(B, Hk, d, p->pages, p->page, p->table_width, p->dtype, p->format);
  if (sizes != GDN_OK) return sizes;
  if (!p->seq_offsets && B > kMost / (T > 0 ? T : 1)) return GDN_ERR_UNSUPPORTED;
  if (!p->page_table || !is_aligned(p->page_table, 4) || !is_aligned(p->start, 4) || !is_aligned(p->seq_offsets, 4))
    return GDN_ERR_INVALID_ARGUMENT;
  Rows pools[4] = {Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0)};
  if (!pool_ranges(k_cache, k_scales, p->pages, Hk, p->page, d, p->format, pools) ||
      !pool_ranges(v_cache, v_scales, p->pages, Hk, p->page, d, p->format, pools + 2))
    return GDN_ERR_INVALID_ARGUMENT;
  if (T == 0) return GDN_OK;
  const int64_t es = (int64_t)elem(p->dtype);
  const void* ptr[2] = {k, v};
  const int64_t strides[2][3] = {{p->k_stride_b, p->k_stride_t, p->k_stride_h}, {p->v_stride_b, p->v_stride_t, p->v_stride_h}};
  const int64_t count[3] = {p->seq_offsets ? 1 : B, T, Hk};
  Rows rows[2] = {Rows(nullptr, 0), Rows(nullptr, 0)};
  bool aligned = true;
  for (int i = 0; i < 2; ++i) {
    if (!ptr[i] || !is_aligned(ptr[i], es)) return GDN_ERR_INVALID_ARGUMENT;
    aligned = aligned && is_aligned(ptr[i], 16);
    Rows r(ptr[i], d * es);
    for (int j = 2; j >= 0; --j) {
      if (count[j] <= 1) continue;
      if (!stride_ok(strides[i][j])) return GDN_ERR_INVALID_ARGUMENT;
      r.by(count[j], strides[i][j] * es);
      if (strides[i][j] * es % 16 != 0) aligned = false;
    }
    if (!r.fits()) return GDN_ERR_INVALID_ARGUMENT;
    rows[i] = r;
  }
  const Rows tables[] = {Rows(p->page_table, B * p->table_width * 4), Rows(p->start, B * 4),
                         Rows(p->seq_offsets, (B + 1) * 4)};
  if (write) {
    for (int i = 0; i < 4; ++i) {
      for (int j = i + 1; j < 4; ++j)
        if (meet(pools[i], pools[j])) return GDN_ERR_INVALID_ARGUMENT;
      for (const Rows& t : tables)
        if (meet(pools[i], t)) return GDN_ERR_INVALID_ARGUMENT;
      if (meet(pools[i], rows[0]) || meet(pools[i], rows[1])) return GDN_ERR_INVALID_ARGUMENT;
    }
  } else {
    if (meet(rows[0], rows[1])) return GDN_ERR_INVALID_ARGUMENT;
    for (const Rows& r : rows) {
      if (r.meets_itself()) return GDN_ERR_INVALID_ARGUMENT;
      for (const Rows& t : tables)
        if (meet(r, t)) return GDN_ERR_INVALID_ARGUMENT;
      for (const Rows& t : pools)
        if (meet(r, t)) return GDN_ERR_INVALID_ARGUMENT;
    }
  }
  KvArgs a;
  memset(&a, 0, sizeof(a));
  a.k = const_cast<void*>(k); a.v = const_cast<void*>(v);
  a.k_cache = const_cast<void*>(k_cache); a.v_cache = const_cast<void*>(v_cache);
  a.k_scales = static_cast<uint8_t*>(const_cast<void*>(k_scales));
  a.v_scales = static_cast<uint8_t*>(const_cast<void*>(v_scales));
  a.off = p->seq_offsets; a.table = p->page_table; a.start = p->start;
  a.B = B; a.T = T; a.width = p->table_width; a.pages = p->pages;
  a.k_sb = strides[0][0]; a.k_st = strides[0][1]; a.k_sh = strides[0][2];
  a.v_sb = strides[1][0]; a.v_st = strides[1][1]; a.v_sh = strides[1][2];
  a.Hk = (int)Hk; a.d = (int)d; a.page_bits = log2_of(p->page);
  a.zero_unused = (p->options & GDN_LAYER_OPT_ZERO_UNUSED) != 0;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_kv<bf16>(a, p->format, write, aligned, stream)
                                             : launch_kv<float>(a, p->format, write, aligned, stream));
}

gdn_status_t attention_sizes(const gdn_attention_problem_t* p) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  if (p->Hq < 1 || p->window < 0 || p->window > kMost || p->sinks < 0 || p->sinks > kMost) return GDN_ERR_INVALID_ARGUMENT;
  const gdn_status_t sizes = cache_sizes(p->B, p->Hk, p->d, p->pages, p->page, p->table_width, p->dtype, p->format);
  if (sizes != GDN_OK) return sizes;
  if (p->Hq % p->Hk != 0) return GDN_ERR_INVALID_ARGUMENT;
  if (p->Hq > kMostHeads || p->B > kMost / p->Hq) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

AttendPlan plan_of(const gdn_attention_problem_t* p) {
  return attend_plan(p->B, p->Hq, p->Hk, p->d, p->dtype == GDN_DTYPE_BF16, p->table_width * p->page, p->window, p->window ? p->sinks : 0);
}

gdn_status_t norm_sizes(const gdn_norm_problem_t* p) {
  if (!p) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->B, T = p->T, D = p->D;
  if (B < 1 || B > kMost || T < 0 || T > kMost || D < 1) return GDN_ERR_INVALID_ARGUMENT;
  if (p->options & ~GDN_LAYER_OPT_ZERO_UNUSED) return GDN_ERR_INVALID_ARGUMENT;
  if (!isfinite(p->residual_scale) || !(p->eps >= 0.f) || !(p->eps <= 3.4e38f)) return GDN_ERR_INVALID_ARGUMENT;
  if (p->gate && p->gate_stride_b != 0 && p->gate_stride_b != D) return GDN_ERR_INVALID_ARGUMENT;
  if (p->dtype != GDN_DTYPE_F32 && p->dtype != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED;
  if (D > 16384 || (!p->seq_offsets && B > kMost / (T > 0 ? T : 1))) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

size_t norm_parts_bytes(const gdn_norm_problem_t* p, int sums) {
  const NormPlan plan = norm_plan(p->B, p->T, p->D, p->dtype == GDN_DTYPE_BF16, p->seq_offsets != nullptr, true);
  return (size_t)plan.items * sums * p->D * 4;
}

gdn_status_t norm_call(const gdn_norm_problem_t* p, bool backward, const void* x, const void* y, const void* h,
                       const void* n, const void* dx, const void* dy, float* dgate, float* dpost, float* dweight) {
  const gdn_status_t sizes = norm_sizes(p);
  if (sizes != GDN_OK) return sizes;
  const int64_t B = p->B, T = p->T, D = p->D, es = (int64_t)elem(p->dtype);
  const int32_t* off = p->seq_offsets;
  if ((p->gate || p->post_weight) && T > 0 && !y) return GDN_ERR_INVALID_ARGUMENT;
  if ((n != nullptr) != (p->weight != nullptr) && T > 0) return GDN_ERR_INVALID_ARGUMENT;
  if (backward) {
    if ((dy && !y) || (dgate && !p->gate) || (dpost && !p->post_weight) || (dweight && !p->weight)) return GDN_ERR_INVALID_ARGUMENT;
  } else if (!h && !n && T > 0) {
    return GDN_ERR_INVALID_ARGUMENT;
  }
  if (T > 0 && !x) return GDN_ERR_INVALID_ARGUMENT;
  const void* ptr[6] = {x, y, h, n, dx, dy};
  const int64_t sb[6] = {p->x_stride_b, p->y_stride_b, p->h_stride_b, p->n_stride_b, p->dx_stride_b, p->dy_stride_b};
  const int64_t st[6] = {p->x_stride_t, p->y_stride_t, p->h_stride_t, p->n_stride_t, p->dx_stride_t, p->dy_stride_t};
  Rows rows[6] = {Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0)};
  bool aligned = D * es % 16 == 0;
  for (int i = 0; i < 6; ++i) {
    if (!ptr[i]) continue;
    if (!is_aligned(ptr[i], es) || !stride_ok(sb[i]) || !stride_ok(st[i])) return GDN_ERR_INVALID_ARGUMENT;
    rows[i] = token_rows(ptr[i], D, es, B, sb[i], T, st[i], off);
    if (!rows[i].fits()) return GDN_ERR_INVALID_ARGUMENT;
    aligned = aligned && rows_aligned(ptr[i], es, B, sb[i], T, st[i], off);
  }
  const void* words[] = {p->gate, p->post_weight, p->weight, dgate, dpost, dweight, off};
  for (const void* q : words)
    if (!is_aligned(q, 4)) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t gate_bytes = (p->gate_stride_b ? B : 1) * D * 4;
  const int sums = (dgate ? 1 : 0) + (dpost ? 1 : 0) + (dweight ? 1 : 0);
  size_t need = 0;
  if (backward && sums) {
    need = norm_parts_bytes(p, sums);
    if (need && (!p->workspace || !is_aligned(p->workspace, 256))) return GDN_ERR_INVALID_ARGUMENT;
    if (p->workspace_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
  }
  // what is written, and what else there is
  const Rows params[] = {Rows(p->gate, gate_bytes), Rows(p->post_weight, D * 4), Rows(p->weight, D * 4),
                         Rows(off, (B + 1) * 4)};
  const Rows written[] = {backward ? rows[4] : rows[2], backward ? rows[5] : rows[3], Rows(dgate, gate_bytes),
                          Rows(dpost, D * 4), Rows(dweight, D * 4), Rows(need ? p->workspace : nullptr, (int64_t)need)};
  const int in_place = backward ? 2 : 0;  // the row that the first output may be
  for (int o = 0; o < 6; ++o) {
    if (written[o].meets_itself()) return GDN_ERR_INVALID_ARGUMENT;
    for (int i = o + 1; i < 6; ++i)
      if (meet(written[o], written[i])) return GDN_ERR_INVALID_ARGUMENT;
    for (const Rows& r : params)
      if (meet(written[o], r)) return GDN_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < (backward ? 4 : 2); ++i) {
      const int first = backward ? 4 : 2;
      const bool same = o == 0 && i == in_place && ptr[i] && ptr[i] == ptr[first] && (off || B <= 1 || sb[i] == sb[first]) &&
                        (T <= 1 || st[i] == st[first]);
      if (!same && meet(written[o], rows[i])) return GDN_ERR_INVALID_ARGUMENT;
    }
  }
  if (T == 0 && !(backward && sums)) return GDN_OK;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.y = y; a.h = const_cast<void*>(h); a.n = const_cast<void*>(n);
  a.dx = const_cast<void*>(dx); a.dy = const_cast<void*>(dy);
  a.gate = p->gate; a.post = p->post_weight; a.weight = p->weight; a.off = off;
  a.B = B; a.T = T; a.D = D;
  a.x_sb = sb[0]; a.y_sb = sb[1]; a.h_sb = sb[2]; a.n_sb = sb[3]; a.dx_sb = sb[4]; a.dy_sb = sb[5];
  a.x_st = st[0]; a.y_st = st[1]; a.h_st = st[2]; a.n_st = st[3]; a.dx_st = st[4]; a.dy_st = st[5];
  a.gate_sb = p->gate_stride_b; a.alpha = p->residual_scale; a.eps = p->eps;
  a.zero_unused = (p->options & GDN_LAYER_OPT_ZERO_UNUSED) != 0;
  const NormPlan plan = norm_plan(B, T, D, p->dtype == GDN_DTYPE_BF16, off != nullptr, backward);
  a.chunk = plan.chunk; a.chunks = plan.chunks; a.items = plan.items;
  a.parts = static_cast<float*>(p->workspace);
  a.sums = sums; a.dgate = dgate; a.dpost = dpost; a.dweight = dweight;
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  const bool half = p->dtype == GDN_DTYPE_BF16;
  if (backward) return launched(half ? launch_norm_back<bf16>(a, aligned, stream) : launch_norm_back<float>(a, aligned, stream));
  return launched(half ? launch_norm<bf16>(a, aligned, stream) : launch_norm<float>(a, aligned, stream));
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status_t gdn_kv_write(const gdn_kv_problem_t* p, const void* k, const void* v, void* k_cache, void* v_cache,
                                     void* k_scales, void* v_scales) {
  return kv_call(p, true, k, v, k_cache, v_cache, k_scales, v_scales);
}

extern "C" gdn_status_t gdn_kv_read(const gdn_kv_problem_t* p, const void* k_cache, const void* v_cache,
                                    const void* k_scales, const void* v_scales, void* k, void* v) {
  return kv_call(p, false, k, v, k_cache, v_cache, k_scales, v_scales);
}

extern "C" size_t gdn_attention_workspace_bytes(const gdn_attention_problem_t* p) {
  if (attention_sizes(p) != GDN_OK) return 0;
  return plan_of(p).total_bytes;
}

extern "C" gdn_status_t gdn_attention_step(const gdn_attention_problem_t* p, const void* q, const void* k_cache,
                                           const void* v_cache, const void* k_scales, const void* v_scales, void* out,
                                           float* lse) {
  const gdn_status_t sizes = attention_sizes(p);
  if (sizes != GDN_OK) return sizes;
  if (!isfinite(p->scale)) return GDN_ERR_INVALID_ARGUMENT;
  const int64_t B = p->B, d = p->d, es = (int64_t)elem(p->dtype);
  if (!q || !out || !p->page_table || !p->lengths) return GDN_ERR_INVALID_ARGUMENT;
  if (!is_aligned(q, es) || !is_aligned(out, es) || !is_aligned(lse, 4) || !is_aligned(p->page_table, 4) ||
      !is_aligned(p->lengths, 4))
    return GDN_ERR_INVALID_ARGUMENT;
  const int64_t strides[4] = {p->q_stride_b, p->q_stride_h, p->out_stride_b, p->out_stride_h};
  for (const int64_t s : strides)
    if (!stride_ok(s)) return GDN_ERR_INVALID_ARGUMENT;
  Rows pools[4] = {Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0), Rows(nullptr, 0)};
  if (!pool_ranges(k_cache, k_scales, p->pages, p->Hk, p->page, d, p->format, pools) ||
      !pool_ranges(v_cache, v_scales, p->pages, p->Hk, p->page, d, p->format, pools + 2))
    return GDN_ERR_INVALID_ARGUMENT;
  const Rows r_q = Rows(q, d * es).by(p->Hq, p->q_stride_h * es).by(B, p->q_stride_b * es);
  const Rows r_o = Rows(out, d * es).by(p->Hq, p->out_stride_h * es).by(B, p->out_stride_b * es);
  if (!r_q.fits() || !r_o.fits() || r_o.meets_itself()) return GDN_ERR_INVALID_ARGUMENT;
  const Rows r_l(lse, B * p->Hq * 4);
  const AttendPlan plan = plan_of(p);
  const size_t need = plan.total_bytes;
  if (need && (!p->workspace || !is_aligned(p->workspace, 256))) return GDN_ERR_INVALID_ARGUMENT;
  if (p->workspace_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
  const Rows written[] = {r_o, r_l, Rows(need ? p->workspace : nullptr, (int64_t)need)};
  const Rows read[] = {r_q, pools[0], pools[1], pools[2], pools[3], Rows(p->page_table, B * p->table_width * 4),
                       Rows(p->lengths, B * 4)};
  for (int o = 0; o < 3; ++o) {
    for (int i = o + 1; i < 3; ++i)
      if (meet(written[o], written[i])) return GDN_ERR_INVALID_ARGUMENT;
    for (const Rows& r : read)
      if (meet(written[o], r)) return GDN_ERR_INVALID_ARGUMENT;
  }
  AttendArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scales = static_cast<const uint8_t*>(k_scales); a.v_scales = static_cast<const uint8_t*>(v_scales);
  a.out = out; a.lse = lse; a.table = p->page_table; a.lengths = p->lengths;
  a.B = B; a.width = p->table_width; a.pages = p->pages;
  a.q_sb = p->q_stride_b; a.q_sh = p->q_stride_h; a.o_sb = p->out_stride_b; a.o_sh = p->out_stride_h;
  a.window = p->window; a.sinks = p->sinks;
  a.Hq = (int)p->Hq; a.Hk = (int)p->Hk; a.d = (int)d; a.page_bits = log2_of(p->page); a.scale = p->scale;
  a.q_aligned = is_aligned(q, 16) && (p->Hq <= 1 || p->q_stride_h * es % 16 == 0) && (B <= 1 || p->q_stride_b * es % 16 == 0);
  a.items = plan.items;
  if (need) {
    unsigned char* ws = static_cast<unsigned char*>(p->workspace);
    a.plan = reinterpret_cast<int32_t*>(ws);
    a.parts = reinterpret_cast<float*>(ws + plan.plan_bytes);
    a.stats = reinterpret_cast<float*>(ws + plan.plan_bytes + plan.parts_bytes);
  }
  hipStream_t stream = static_cast<hipStream_t>(p->stream);
  return launched(p->dtype == GDN_DTYPE_BF16 ? launch_attend<bf16>(a, p->format, stream)
                                             : launch_attend<float>(a, p->format, stream));
}

extern "C" gdn_status_t gdn_norm_forward(const gdn_norm_problem_t* p, const void* x, const void* y, void* h, void* n) {
  return norm_call(p, false, x, y, h, n, nullptr, nullptr, nullptr, nullptr, nullptr);
}

extern "C" size_t gdn_norm_workspace_bytes(const gdn_norm_problem_t* p) {
  if (norm_sizes(p) != GDN_OK) return 0;
  return norm_parts_bytes(p, (p->gate ? 1 : 0) + (p->post_weight ? 1 : 0) + (p->weight ? 1 : 0));
}

extern "C" gdn_status_t gdn_norm_backward(const gdn_norm_problem_t* p, const void* x, const void* y, const void* dh,
                                          const void* dn, void* dx, void* dy, float* dgate, float* dpost_weight,
                                          float* dweight) {
  return norm_call(p, true, x, y, dh, dn, dx, dy, dgate, dpost_weight, dweight);
}
