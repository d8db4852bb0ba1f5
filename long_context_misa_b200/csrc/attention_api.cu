// C ABI of the attention side: argument validation and dispatch.
// Declarations and semantics: include/misa_attention.h.
#include <algorithm>
#include <cmath>

#include "api_common.h"
#include "attention.h"

namespace {

using namespace misa::api;

misa_status check_kv(const misa_kv *c) {
  if (!c) return fail(MISA_ERR_INVALID, "kv is NULL");
  if (!c->k || !c->v || !c->seq_len) return fail(MISA_ERR_INVALID, "kv k/v/seq_len is NULL");
  if (c->dtype != MISA_KEY_BF16 && c->dtype != MISA_KEY_FP8_E4M3)
    return fail(MISA_ERR_INVALID, "unknown cache dtype %d", c->dtype);
  const bool fp8 = c->dtype == MISA_KEY_FP8_E4M3;
  if (fp8 != (c->k_scale != nullptr) || fp8 != (c->v_scale != nullptr))
    return fail(MISA_ERR_INVALID, "k_scale and v_scale must be non-NULL exactly for e4m3 caches");
  if (c->d != 64 && c->d != 128) return fail(MISA_ERR_UNSUPPORTED, "d=%d unsupported (64 or 128)", c->d);
  if (c->n_seq < 1 || c->L_cap < 1) return fail(MISA_ERR_INVALID, "n_seq=%d L_cap=%d must be >= 1", c->n_seq, c->L_cap);
  if (c->H_kv < 1) return fail(MISA_ERR_INVALID, "H_kv=%d must be >= 1", c->H_kv);
  if (c->H_kv > MISA_MAX_H) return fail(MISA_ERR_UNSUPPORTED, "H_kv=%d above %d", c->H_kv, MISA_MAX_H);
  if (c->L_cap > MISA_MAX_L) return fail(MISA_ERR_UNSUPPORTED, "L_cap=%d above %d", c->L_cap, MISA_MAX_L);
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(MISA_ERR_INVALID, "k and v must be 16-byte aligned");
  return MISA_OK;
}

misa_status check_rope(const misa_rope *r, int d) {
  if (!r || !r->phase) return fail(MISA_ERR_INVALID, "rope or its phase table is NULL");
  if (r->layout != MISA_ROPE_HALF && r->layout != MISA_ROPE_INTERLEAVED)
    return fail(MISA_ERR_INVALID, "unknown rope layout %d", r->layout);
  if (r->rot < 2 || r->rot % 2) return fail(MISA_ERR_INVALID, "rot=%d must be even and >= 2", r->rot);
  if (r->first < 0 || r->rot > d - r->first)
    return fail(MISA_ERR_INVALID, "rotated elements [%d, %d + %d) outside a row of %d", r->first, r->first, r->rot, d);
  if (!std::isfinite(r->amplitude)) return fail(MISA_ERR_INVALID, "rope amplitude is not finite");
  return MISA_OK;
}

// Whether [n][H] rows of d elements with these strides do not meet: one of the
// two axes steps over all of the other's rows.
bool apart(int64_t row, int n, int64_t head, int H, int d) {
  auto size = [](int64_t x) { return x < 0 ? -x : x; };
  const int64_t r = size(row), h = size(head);
  const bool rows_out = (n < 2 || r >= (H < 2 ? d : h * (H - 1) + d)) && (H < 2 || h >= d);
  const bool heads_out = (H < 2 || h >= (n < 2 ? d : r * (n - 1) + d)) && (n < 2 || r >= d);
  return rows_out || heads_out;
}

// [n][H] rows of d bytes: strides not negative, extents of 1 where they repeat
// the same memory.
struct Rows {
  int64_t at, row, head, n, H, d;
  Rows(const uint16_t *p, int64_t row_, int64_t head_, int n_, int H_, int d_)
      : at((int64_t)(intptr_t)p), row(2 * row_), head(2 * head_), n(row_ ? n_ : 1), H(head_ ? H_ : 1), d(2 * (int64_t)d_) {
    if (row < 0) at += row * (n - 1), row = -row;
    if (head < 0) at += head * (H - 1), head = -head;
    if (n == 1) row = 0;
    if (H == 1) head = 0;
  }
  int64_t row_span() const { return head * (H - 1) + d; }
  int64_t span() const { return row * (n - 1) + row_span(); }
};

// The whole numbers k of [lo, hi] with -below < off + k step < above; step > 0,
// or 0 with lo == hi == 0.
struct Range {
  int64_t lo, hi;
};
Range within(int64_t off, int64_t step, int64_t below, int64_t above, int64_t lo, int64_t hi) {
  if (step == 0) return off > -below && off < above ? Range{0, 0} : Range{0, -1};
  auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
  return {std::max(lo, floor_div(-below - off, step) + 1), std::min(hi, -floor_div(off - above, step) - 1)};
}

// Whether a row of a and one of b share memory, b's first row `off` behind a's.
bool rows_meet(const Rows &a, const Rows &b, int64_t off) {
  for (int64_t p = 0; p < a.H; ++p) {
    const Range q = within(off - p * a.head, b.head, b.d, a.d, 0, b.H - 1);
    if (q.lo <= q.hi) return true;
  }
  return false;
}

// Whether two sets of rows share memory: exactly, so that interleaved slices of
// one projection are told from rows that meet.
bool meet(const Rows &a, const Rows &b) {
  const int64_t off = b.at - a.at;
  if (off >= a.span() || -off >= b.span()) return false;
  if (a.row == b.row || a.n == 1 || b.n == 1) {  // rows k = j - i apart
    const int64_t row = a.n == 1 ? b.row : a.row;
    const Range k = within(off, row, b.row_span(), a.row_span(), 1 - a.n, b.n - 1);
    for (int64_t i = k.lo; i <= k.hi; ++i)
      if (rows_meet(a, b, off + i * row)) return true;
    return false;
  }
  for (int64_t i = 0; i < a.n; ++i) {
    const Range j = within(off - i * a.row, b.row, b.row_span(), a.row_span(), 0, b.n - 1);
    for (int64_t x = j.lo; x <= j.hi; ++x)
      if (rows_meet(a, b, off - i * a.row + x * b.row)) return true;
  }
  return false;
}

// Whether two arrays of n 16-bit elements share memory.
bool overlap16(const uint16_t *a, const uint16_t *b, int64_t n) { return a < b + n && b < a + n; }

// Whether two arrays of bytes do.
bool share(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

misa::KvView view(const misa_kv *c) {
  misa::KvView v;
  v.k = static_cast<uint8_t *>(c->k);
  v.v = static_cast<uint8_t *>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.seq_len = c->seq_len;
  v.status = c->status;
  v.n_seq = c->n_seq;
  v.L_cap = c->L_cap;
  v.H_kv = c->H_kv;
  v.d = c->d;
  v.fp8 = c->dtype == MISA_KEY_FP8_E4M3;
  return v;
}

misa::RopeView view(const misa_rope *r) {
  if (!r) return {nullptr, 0, 0, 0, 1.f};
  return {r->phase, r->rot, r->first, r->layout == MISA_ROPE_INTERLEAVED, r->amplitude};
}

misa_status check_attend(const misa_kv *kv, const misa_attend_queries *qs, int32_t k, int32_t n_draft) {
  misa_status st = check_kv(kv);
  if (st != MISA_OK) return st;
  if (!qs) return fail(MISA_ERR_INVALID, "queries is NULL");
  if (qs->n_q < 0 || qs->n_q > 65535) return fail(MISA_ERR_INVALID, "n_q=%d outside [0, 65535]", qs->n_q);
  if (qs->H < 1 || qs->H % kv->H_kv)
    return fail(MISA_ERR_INVALID, "H=%d is not a positive multiple of H_kv=%d", qs->H, kv->H_kv);
  if (qs->H > MISA_MAX_H) return fail(MISA_ERR_UNSUPPORTED, "H=%d above %d", qs->H, MISA_MAX_H);
  if (k < 0) return fail(MISA_ERR_INVALID, "k=%d < 0", k);
  if (k > MISA_MAX_L) return fail(MISA_ERR_UNSUPPORTED, "k=%d above %d", k, MISA_MAX_L);
  if (n_draft < 0) return fail(MISA_ERR_INVALID, "draft n=%d < 0", n_draft);
  if (n_draft > MISA_MAX_DRAFT) return fail(MISA_ERR_UNSUPPORTED, "draft n=%d above %d", n_draft, MISA_MAX_DRAFT);
  return MISA_OK;
}

}  // namespace

extern "C" {

misa_status misa_rope_phases(uint64_t *phases, int32_t rot, double base, int32_t scaling, double factor,
                             double orig_len, double beta_fast, double beta_slow) {
  if (!phases) return fail(MISA_ERR_INVALID, "phases is NULL");
  if (rot < 2 || rot % 2) return fail(MISA_ERR_INVALID, "rot=%d must be even and >= 2", rot);
  if (!(base > 0) || !std::isfinite(base)) return fail(MISA_ERR_INVALID, "base must be positive and finite");
  if (scaling < MISA_ROPE_NONE || scaling > MISA_ROPE_YARN) return fail(MISA_ERR_INVALID, "unknown scaling %d", scaling);
  if (scaling != MISA_ROPE_NONE && (!(factor > 0) || !std::isfinite(factor)))
    return fail(MISA_ERR_INVALID, "factor must be positive and finite");
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == MISA_ROPE_NTK && rot > 2) base *= std::pow(factor, (double)rot / (rot - 2));
  double lo = 0, hi = 0;
  if (scaling == MISA_ROPE_YARN) {
    if (!(orig_len > 0) || !std::isfinite(orig_len)) return fail(MISA_ERR_INVALID, "orig_len must be positive and finite");
    if (!(beta_slow > 0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast))
      return fail(MISA_ERR_INVALID, "beta_fast >= beta_slow > 0 violated");
    if (base == 1.0) return fail(MISA_ERR_INVALID, "base 1 has no ramp");
    // the pair that turns `turns` times in orig_len positions
    auto pair_of = [&](double turns) { return rot * std::log(orig_len / (turns * two_pi)) / (2 * std::log(base)); };
    lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair_of(beta_slow)), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == MISA_ROPE_LINEAR) f /= factor;
    if (scaling == MISA_ROPE_YARN) {
      const double r = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1 - r) + f / factor * r;
    }
    if (!std::isfinite(f)) return fail(MISA_ERR_INVALID, "pair %d has no finite frequency", i);
    // turns per position, their fraction in 2^-64 steps (the product with a
    // position wraps over whole turns)
    const long double turns = (long double)f / 6.283185307179586476925286766559L;
    const long double frac = turns - floorl(turns);
    const long double steps = floorl(frac * 18446744073709551616.0L + 0.5L);
    phases[i] = steps >= 18446744073709551616.0L ? 0 : (uint64_t)steps;
  }
  return MISA_OK;
}

misa_status misa_apply_rope(const misa_rope *rope, const misa_rope_rows *groups, int32_t n_groups,
                            misa_stream stream) {
  NvtxRange nvtx("misa_apply_rope");
  misa_status st;
  if (!groups) return fail(MISA_ERR_INVALID, "groups is NULL");
  if (n_groups < 1 || n_groups > MISA_MAX_ROPE_GROUPS)
    return fail(MISA_ERR_INVALID, "n_groups=%d outside [1, %d]", n_groups, MISA_MAX_ROPE_GROUPS);
  for (int i = 0; i < n_groups; ++i) {
    const misa_rope_rows &g = groups[i];
    if (g.n < 0 || g.H < 0 || g.d < 1) return fail(MISA_ERR_INVALID, "group %d: n=%d H=%d d=%d", i, g.n, g.H, g.d);
    if (g.d > 1024) return fail(MISA_ERR_UNSUPPORTED, "group %d: d=%d above 1024", i, g.d);
    if ((st = check_rope(rope, g.d)) != MISA_OK) return st;
    if (g.n == 0 || g.H == 0) continue;  // nothing to read or write
    if (!g.x || !g.y || !g.pos) return fail(MISA_ERR_INVALID, "group %d: x/y/pos is NULL", i);
    if (g.x == g.y && (g.x_row != g.y_row || g.x_head != g.y_head))
      return fail(MISA_ERR_INVALID, "group %d: in place needs equal strides", i);
    if (!apart(g.y_row, g.n, g.y_head, g.H, g.d)) return fail(MISA_ERR_INVALID, "group %d: rows of y overlap", i);
    const Rows x(g.x, g.x_row, g.x_head, g.n, g.H, g.d), y(g.y, g.y_row, g.y_head, g.n, g.H, g.d);
    if (g.x != g.y && meet(x, y)) return fail(MISA_ERR_INVALID, "group %d: rows of y overlap rows of x", i);
    for (int j = 0; j < i; ++j) {
      const misa_rope_rows &o = groups[j];
      if (o.n == 0 || o.H == 0) continue;
      const Rows ox(o.x, o.x_row, o.x_head, o.n, o.H, o.d), oy(o.y, o.y_row, o.y_head, o.n, o.H, o.d);
      if (meet(y, oy) || meet(y, ox) || meet(x, oy))
        return fail(MISA_ERR_INVALID, "groups %d and %d: one writes what the other takes", j, i);
    }
  }
  if (injected_failure("misa_apply_rope", &st)) return st;
  const cudaError_t e = misa::launch_rope(view(rope), groups, n_groups, stream);
  return e == cudaSuccess ? MISA_OK : cuda_fail(e, "misa_apply_rope");
}

misa_status misa_append_kv(const misa_kv *kv, const misa_new_kv *new_kv, const int32_t *new_pos, int32_t count,
                           const misa_rope *rope, const int32_t *rope_pos, int32_t commit, misa_stream stream) {
  NvtxRange nvtx("misa_append_kv");
  misa_status st = check_kv(kv);
  if (st != MISA_OK) return st;
  if (rope && (st = check_rope(rope, kv->d)) != MISA_OK) return st;
  if (count < 1 || count > kv->L_cap) return fail(MISA_ERR_INVALID, "count=%d outside [1, L_cap=%d]", count, kv->L_cap);
  if (!new_kv || !new_kv->k || !new_kv->v || !new_pos) return fail(MISA_ERR_INVALID, "new_kv/k/v/new_pos is NULL");
  if (commit && new_pos != kv->seq_len && misa::overlap(new_pos, kv->n_seq, kv->seq_len, kv->n_seq))
    return fail(MISA_ERR_INVALID, "new_pos overlaps seq_len");
  if (rope_pos && !rope) return fail(MISA_ERR_INVALID, "rope_pos without rope");
  const int64_t strides[6] = {new_kv->k_seq, new_kv->k_tok, new_kv->k_head, new_kv->v_seq, new_kv->v_tok, new_kv->v_head};
  for (const int64_t x : strides)
    if (x % 8) return fail(MISA_ERR_INVALID, "new_kv strides must be multiples of 8 elements");
  if (!aligned16(new_kv->k) || !aligned16(new_kv->v)) return fail(MISA_ERR_INVALID, "new_kv k and v must be 16-byte aligned");
  if (injected_failure("misa_append_kv", &st)) return st;
  const cudaError_t e = misa::launch_append_kv(view(kv), *new_kv, new_pos, count, view(rope), rope_pos, commit != 0, stream);
  return e == cudaSuccess ? MISA_OK : cuda_fail(e, "misa_append_kv");
}

misa_status misa_read_kv(const misa_kv *kv, const int32_t *seq, const int32_t *tok, int32_t n, int32_t k,
                         uint16_t *k_out, uint16_t *v_out, misa_stream stream) {
  NvtxRange nvtx("misa_read_kv");
  misa_status st = check_kv(kv);
  if (st != MISA_OK) return st;
  if (n < 0 || k < 1) return fail(MISA_ERR_INVALID, "n=%d k=%d", n, k);
  if (k > MISA_MAX_L) return fail(MISA_ERR_UNSUPPORTED, "k=%d above %d", k, MISA_MAX_L);
  if (n > 0 && !k_out && !v_out) return fail(MISA_ERR_INVALID, "k_out and v_out are both NULL");
  if (n > 0 && (!seq || !tok)) return fail(MISA_ERR_INVALID, "seq/tok is NULL");
  if (!aligned16(k_out) || !aligned16(v_out)) return fail(MISA_ERR_INVALID, "k_out and v_out must be 16-byte aligned");
  if (k_out && v_out && overlap16(k_out, v_out, (int64_t)n * k * kv->H_kv * kv->d))
    return fail(MISA_ERR_INVALID, "k_out and v_out overlap");
  if (injected_failure("misa_read_kv", &st)) return st;
  const cudaError_t e = misa::launch_read_kv(view(kv), seq, tok, n, k, k_out, v_out, stream);
  return e == cudaSuccess ? MISA_OK : cuda_fail(e, "misa_read_kv");
}

size_t misa_attend_workspace_bytes(const misa_kv *kv, const misa_attend_queries *qs, int32_t k, int32_t n_draft) {
  if (check_attend(kv, qs, k, n_draft) != MISA_OK) return 0;
  return misa::attend_ws_bytes(view(kv), qs->n_q, qs->H, k, n_draft);
}

misa_status misa_attend(const misa_kv *kv, const misa_attend_queries *qs, const int32_t *topk, int32_t k,
                        const misa_draft *draft, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                        misa_stream stream) {
  NvtxRange nvtx("misa_attend");
  misa_status st = check_attend(kv, qs, k, draft ? draft->n : 0);
  if (st != MISA_OK) return st;
  const bool any = qs->n_q > 0;  // an empty batch has no memory to point to
  if (topk ? k < 1 : any && k > 0) return fail(MISA_ERR_INVALID, "k=%d %s a list", k, topk ? "with" : "without");
  if (draft && (draft->n < 1 || (any && (!draft->start || !draft->mask))))
    return fail(MISA_ERR_INVALID, "draft n=%d, start or mask NULL", draft->n);
  if (any && (!qs->q || !qs->q_seq || !qs->q_pos || !out))
    return fail(MISA_ERR_INVALID, "q/q_seq/q_pos/out is NULL");
  if (any && overlap16(qs->q, out, (int64_t)qs->n_q * qs->H * kv->d))
    return fail(MISA_ERR_INVALID, "out overlaps q");
  if (!std::isfinite(qs->scale)) return fail(MISA_ERR_INVALID, "scale is not finite");
  if (!aligned16(qs->q) || !aligned16(out)) return fail(MISA_ERR_INVALID, "q and out must be 16-byte aligned");
  const size_t need = misa::attend_ws_bytes(view(kv), qs->n_q, qs->H, k, draft ? draft->n : 0);
  if (ws_bytes < need) return fail(MISA_ERR_WORKSPACE, "workspace %zu bytes, need %zu", ws_bytes, need);
  if (need > 0 && (!ws || !aligned16(ws))) return fail(MISA_ERR_INVALID, "workspace NULL or not 16-byte aligned");
  const size_t n_lse = (size_t)qs->n_q * qs->H, n_row = n_lse * kv->d * 2;
  if (share(lse, n_lse * 4, qs->q, n_row) || share(lse, n_lse * 4, out, n_row))
    return fail(MISA_ERR_INVALID, "lse overlaps q or out");
  if (share(ws, need, qs->q, n_row) || share(ws, need, out, n_row) || share(ws, need, lse, n_lse * 4))
    return fail(MISA_ERR_INVALID, "the workspace overlaps q, out or lse");
  if (injected_failure("misa_attend", &st)) return st;
  misa::AttendView a;
  a.q = qs->q;
  a.q_seq = qs->q_seq;
  a.q_pos = qs->q_pos;
  a.n_q = qs->n_q;
  a.H = qs->H;
  a.scale = qs->scale;
  a.topk = topk;
  a.k = k;
  a.draft_start = draft ? draft->start : nullptr;
  a.draft_mask = draft ? draft->mask : nullptr;
  a.n_draft = draft ? draft->n : 0;
  a.out = out;
  a.lse = lse;
  const cudaError_t e = misa::launch_attend(view(kv), a, ws, stream);
  return e == cudaSuccess ? MISA_OK : cuda_fail(e, "misa_attend");
}

}  // extern "C"
