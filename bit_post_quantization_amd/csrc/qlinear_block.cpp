// C ABI of a conditioned block's operators (declared in include/qlinear.h):
// argument checks, the division of the caller's workspace, and the launches.
#include "../../include/qlinear.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ql_block.h"

namespace ql {
ql_status set_error(ql_status st, const char* msg);
}

namespace {

ql_status fail(ql_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return ql::set_error(st, buf);
}

ql_status ok() { return ql::set_error(QL_OK, ""); }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int t) { return t == QL_F32 || t == QL_BF16; }
int64_t size_of(int t) { return t == QL_BF16 ? 2 : 4; }
int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

ql_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need > 0 && !ws) return fail(QL_ERR_ARG, "workspace is NULL");
  if (!aligned(ws, 16)) return fail(QL_ERR_ARG, "workspace must be 16-byte aligned");
  if (have < need)
    return fail(QL_ERR_ARG, "workspace holds %lld bytes, the call needs %lld", (long long)have,
                (long long)need);
  return QL_OK;
}

#define QL_CHECK(expr)            \
  do {                            \
    const ql_status st_ = (expr); \
    if (st_ != QL_OK) return st_; \
  } while (0)

// -------------------------------------------------------------- 4-bit rows ----

constexpr int kMaxFewRows = 1 << 20;

ql_status check_rows4(const ql_rows4* d) {
  if (!d) return fail(QL_ERR_ARG, "descriptor is NULL");
  if (d->N < 1) return fail(QL_ERR_ARG, "N = %d must be >= 1", d->N);
  if (d->N > 1 << 22) return fail(QL_ERR_UNSUPPORTED, "N = %d: at most %d", d->N, 1 << 22);
  if (d->K < 16 || d->K > 65536 || d->K % 16 != 0)
    return fail(QL_ERR_ARG, "K = %d must be a multiple of 16 in [16, 65536]", d->K);
  if (d->group != 32 && d->group != 64 && d->group != 128)
    return fail(QL_ERR_ARG, "group = %d must be 32, 64 or 128", d->group);
  if (!dtype_ok(d->x_dtype)) return fail(QL_ERR_ARG, "bad x_dtype %d", (int)d->x_dtype);
  if (!dtype_ok(d->s_dtype)) return fail(QL_ERR_ARG, "bad s_dtype %d", (int)d->s_dtype);
  if (d->act != QL_ACT_NONE && d->act != QL_ACT_SILU)
    return fail(QL_ERR_ARG, "bad act %d", (int)d->act);
  if ((int64_t)d->N * d->K >= (int64_t)1 << 34)
    return fail(QL_ERR_UNSUPPORTED, "N * K of 2^34 or more (N = %d, K = %d)", d->N, d->K);
  return QL_OK;
}

ql_status check_few_rows(int32_t M) {
  if (M < 0) return fail(QL_ERR_ARG, "M = %d must be >= 0", M);
  if (M > kMaxFewRows) return fail(QL_ERR_UNSUPPORTED, "M = %d exceeds %d rows", M, kMaxFewRows);
  return QL_OK;
}

ql_status check_packed(const ql_rows4* d, const void* packed) {
  if (!packed) return fail(QL_ERR_ARG, "packed is NULL");
  if (!aligned(packed, 16)) return fail(QL_ERR_ARG, "packed must be 16-byte aligned");
  return QL_OK;
}

// ------------------------------------------------------------------- views ----

// A tensor by heads of B x L x H rows of dim elements. Strides of an extent of
// one are not looked at. unit: bytes that its start and strides are multiples of.
ql_status check_view(const char* name, const ql_heads_view* t, int64_t B, int64_t L, int64_t H,
                     int dim, int64_t size, int64_t unit, bool out) {
  if (!t || !t->p) return fail(QL_ERR_ARG, "%s is NULL", name);
  if (!aligned(t->p, unit))
    return fail(QL_ERR_ARG, "%s does not start at a multiple of %lld bytes", name, (long long)unit);
  struct Axis {
    int64_t stride, n;
  } axis[3] = {{t->batch, B}, {t->row, L}, {t->head, H}};
  for (const Axis& a : axis) {
    if (a.n <= 1) continue;
    if (a.stride < 0) return fail(QL_ERR_ARG, "%s: stride %lld is negative", name, (long long)a.stride);
    if (a.stride * size % unit != 0)
      return fail(QL_ERR_ARG, "%s: stride %lld is no multiple of %lld bytes", name,
                  (long long)a.stride, (long long)unit);
    if (a.stride > ((int64_t)1 << 40))
      return fail(QL_ERR_UNSUPPORTED, "%s: stride %lld", name, (long long)a.stride);
  }
  if (!out) return QL_OK;
  // rows of an output do not share elements: by rising stride, each axis steps over all
  // that the axes before it span
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (axis[j].stride > axis[j + 1].stride) {
        const Axis x = axis[j];
        axis[j] = axis[j + 1];
        axis[j + 1] = x;
      }
  __int128 span = dim;
  for (const Axis& a : axis) {
    if (a.n <= 1) continue;
    if (a.stride < span)
      return fail(QL_ERR_ARG, "%s: rows overlap (stride %lld)", name, (long long)a.stride);
    span += (__int128)(a.n - 1) * a.stride;
  }
  return QL_OK;
}

// Strides of an extent of one are not used with an index above 0, whatever they are.
ql_heads_view view(const ql_heads_view* t) { return t ? *t : ql_heads_view{nullptr, 0, 0, 0}; }

// ------------------------------------------------------------------- heads ----

ql_status check_heads(const ql_heads* d) {
  if (!d) return fail(QL_ERR_ARG, "descriptor is NULL");
  if (d->batch < 0 || d->positions < 0)
    return fail(QL_ERR_ARG, "batch = %d and positions = %d must be >= 0", d->batch, d->positions);
  if ((int64_t)d->batch * d->positions >= 1 << 24)
    return fail(QL_ERR_UNSUPPORTED, "batch = %d times positions = %d: less than 2^24", d->batch,
                d->positions);
  if (d->q_heads < 0 || d->k_heads < 0 || d->v_heads < 0)
    return fail(QL_ERR_ARG, "heads = (%d, %d, %d) must be >= 0", d->q_heads, d->k_heads, d->v_heads);
  const int64_t heads = (int64_t)d->q_heads + d->k_heads + d->v_heads;
  if (heads < 1) return fail(QL_ERR_ARG, "no heads");
  if (heads > 4096) return fail(QL_ERR_UNSUPPORTED, "%lld heads: at most 4096", (long long)heads);
  if (d->dim < 8 || d->dim % 8 != 0)
    return fail(QL_ERR_ARG, "dim = %d must be a positive multiple of 8", d->dim);
  if (d->dim > 160) return fail(QL_ERR_UNSUPPORTED, "dim = %d: at most 160", d->dim);
  if (!dtype_ok(d->x_dtype)) return fail(QL_ERR_ARG, "bad x_dtype %d", (int)d->x_dtype);
  if (!dtype_ok(d->y_dtype)) return fail(QL_ERR_ARG, "bad y_dtype %d", (int)d->y_dtype);
  if (!dtype_ok(d->w_dtype)) return fail(QL_ERR_ARG, "bad w_dtype %d", (int)d->w_dtype);
  if (d->norm != QL_HEADS_NONE && d->norm != QL_HEADS_RMS)
    return fail(QL_ERR_ARG, "bad norm %d", (int)d->norm);
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps))
    return fail(QL_ERR_ARG, "eps = %g must be positive and finite", (double)d->eps);
  if (d->norm == QL_HEADS_NONE && (d->gamma_q || d->gamma_k))
    return fail(QL_ERR_ARG, "gamma_q or gamma_k without a norm");
  if (!aligned(d->gamma_q, size_of(d->w_dtype)) || !aligned(d->gamma_k, size_of(d->w_dtype)))
    return fail(QL_ERR_ARG, "gamma_q or gamma_k is not element-aligned");
  if (d->n_axes < 0 || d->n_axes > QL_MAX_AXES)
    return fail(QL_ERR_ARG, "n_axes = %d must be in [0, %d]", d->n_axes, QL_MAX_AXES);
  int64_t sum = 0;
  for (int i = 0; i < d->n_axes; ++i) {
    if (d->axis_dims[i] < 2 || d->axis_dims[i] % 2)
      return fail(QL_ERR_ARG, "axis_dims[%d] = %d must be even and >= 2", i, d->axis_dims[i]);
    sum += d->axis_dims[i];
  }
  if (sum > d->dim)
    return fail(QL_ERR_ARG, "axis_dims add up to %lld, more than dim = %d", (long long)sum, d->dim);
  if (d->pairs != QL_PAIRS_ADJACENT && d->pairs != QL_PAIRS_HALVES)
    return fail(QL_ERR_ARG, "bad pairs %d", (int)d->pairs);
  if (d->pos_dtype != QL_POS_I32 && d->pos_dtype != QL_POS_F32)
    return fail(QL_ERR_ARG, "bad pos_dtype %d", (int)d->pos_dtype);
  return QL_OK;
}

ql_status check_turns(const ql_heads* d, const void* pos, int64_t pos_batch) {
  if (d->n_axes == 0) return QL_OK;
  if (!d->freqs || !aligned(d->freqs, 8))
    return fail(QL_ERR_ARG, "freqs is NULL or not 8-byte aligned");
  if (!pos || !aligned(pos, 4)) return fail(QL_ERR_ARG, "pos is NULL or not 4-byte aligned");
  if (pos_batch < 0) return fail(QL_ERR_ARG, "pos: batch stride %lld is negative", (long long)pos_batch);
  return QL_OK;
}

// x or dx: rows of all heads.
ql_status check_rows(const ql_heads* d, const char* name, const void* p, int64_t batch, int64_t row,
                     bool out) {
  const ql_heads_view t = {const_cast<void*>(p), batch, row, 0};
  const int width = (d->q_heads + d->k_heads + d->v_heads) * d->dim;
  if (d->positions > 1 && row < width)
    return fail(QL_ERR_ARG, "%s: row stride %lld is less than a row of %d", name, (long long)row, width);
  return check_view(name, &t, d->batch, d->positions, 1, width, size_of(d->x_dtype),
                    size_of(d->x_dtype), out);
}

ql_status check_parts(const ql_heads* d, const ql_heads_view* const (&y)[3], bool out) {
  static const char* const names[2][3] = {{"dq", "dk", "dv"}, {"q", "k", "v"}};
  const int heads[3] = {d->q_heads, d->k_heads, d->v_heads};
  for (int i = 0; i < 3; ++i)
    if (heads[i] > 0)
      QL_CHECK(check_view(names[out][i], y[i], d->batch, d->positions, heads[i], d->dim,
                          size_of(d->y_dtype), size_of(d->y_dtype), out));
  return QL_OK;
}

bool whole(const void* p, int64_t size, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2,
           int64_t s2) {
  return aligned(p, 16) && (n0 <= 1 || s0 * size % 16 == 0) && (n1 <= 1 || s1 * size % 16 == 0) &&
         (n2 <= 1 || s2 * size % 16 == 0);
}

ql::HeadsArgs heads_args(const ql_heads* d, const void* x, int64_t xb, int64_t xr, const void* pos,
                         int64_t pb, const ql_heads_view* const (&y)[3]) {
  ql::HeadsArgs a{};
  a.x = x;
  a.xb = xb;
  a.xr = xr;
  a.pos = pos;
  a.pb = pb;
  a.heads[0] = d->q_heads;
  a.heads[1] = d->k_heads;
  a.heads[2] = d->v_heads;
  const int64_t xs = size_of(d->x_dtype), ys = size_of(d->y_dtype);
  a.vec = whole(x, xs, d->batch, xb, d->positions, xr, 1, 0);
  for (int i = 0; i < 3; ++i) {
    a.y[i] = a.heads[i] > 0 ? view(y[i]) : ql_heads_view{nullptr, 0, 0, 0};
    if (a.heads[i] > 0)
      a.vec = a.vec && whole(a.y[i].p, ys, d->batch, a.y[i].batch, d->positions, a.y[i].row,
                             a.heads[i], a.y[i].head);
  }
  a.gamma[0] = d->gamma_q;
  a.gamma[1] = d->gamma_k;
  a.freqs = d->freqs;
  a.B = d->batch;
  a.L = d->positions;
  a.D = d->dim;
  a.n_axes = d->n_axes;
  for (int i = 0; i < d->n_axes; ++i) a.half[i] = d->axis_dims[i] / 2;
  a.eps = d->eps;
  a.rms = d->norm == QL_HEADS_RMS;
  a.halves = d->pairs == QL_PAIRS_HALVES;
  a.pos_f32 = d->pos_dtype == QL_POS_F32;
  a.x_bf16 = d->x_dtype == QL_BF16;
  a.y_bf16 = d->y_dtype == QL_BF16;
  a.w_bf16 = d->w_dtype == QL_BF16;
  return a;
}

int heads_groups(const ql_heads* d) {
  return ql::heads_grad_groups((int64_t)d->batch * d->positions);
}

int64_t heads_ws(const ql_heads* d) {
  if (d->norm == QL_HEADS_NONE) return 0;
  return (int64_t)heads_groups(d) * 2 * d->dim * 4;
}

// --------------------------------------------------------------- attention ----

float base2(float scale) { return (float)((double)scale * 1.4426950408889634074); }

ql_status check_attn(const ql_attn* d) {
  if (!d) return fail(QL_ERR_ARG, "descriptor is NULL");
  if (d->batch < 0 || d->q_len < 0 || d->k_len < 0)
    return fail(QL_ERR_ARG, "batch = %d, q_len = %d and k_len = %d must be >= 0", d->batch,
                d->q_len, d->k_len);
  if (d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads != 0)
    return fail(QL_ERR_ARG, "heads = %d must be a positive multiple of kv_heads = %d", d->heads,
                d->kv_heads);
  if (d->dim < 8 || d->dim % 8 != 0)
    return fail(QL_ERR_ARG, "dim = %d must be a positive multiple of 8", d->dim);
  if (d->dim > 160) return fail(QL_ERR_UNSUPPORTED, "dim = %d: at most 160", d->dim);
  if (!dtype_ok(d->dtype)) return fail(QL_ERR_ARG, "bad dtype %d", (int)d->dtype);
  // the kernels multiply with scale log2(e)
  if (!(d->scale > 0.0f) || !std::isfinite(base2(d->scale)))
    return fail(QL_ERR_ARG, "scale = %g must be positive and less than 2^128 / log2(e)",
                (double)d->scale);
  typedef __int128 wide;
  if ((wide)d->batch * d->heads * d->q_len >= (wide)1 << 31 ||
      (wide)d->batch * d->kv_heads * d->k_len >= (wide)1 << 31 ||
      (wide)d->q_len * (d->heads / d->kv_heads) >= (wide)1 << 30 || d->k_len > 1 << 30)
    return fail(QL_ERR_UNSUPPORTED,
                "batch = %d, heads = %d (%d), q_len = %d, k_len = %d: 2^31 rows or more", d->batch,
                d->heads, d->kv_heads, d->q_len, d->k_len);
  if (!aligned(d->k_lens, 4)) return fail(QL_ERR_ARG, "k_lens must be 4-byte aligned");
  if (d->k_mask && d->batch > 1 && d->mask_batch < 0)
    return fail(QL_ERR_ARG, "mask_batch = %lld is negative", (long long)d->mask_batch);
  // workgroups of one launch
  const ql::AttnPlan p = ql::attn_plan(*d);
  const wide bh = (wide)d->batch * d->kv_heads, most = 1 << 23;
  if (bh * p.row_tiles * p.splits > most || bh * p.q_tiles > most ||
      bh * p.key_tiles * p.k_splits > most)
    return fail(QL_ERR_UNSUPPORTED, "batch = %d, heads = %d (%d), q_len = %d, k_len = %d exceed one launch",
                d->batch, d->heads, d->kv_heads, d->q_len, d->k_len);
  return QL_OK;
}

ql_status attn_view(const ql_attn* d, const char* name, const ql_heads_view* t, bool keys, bool out) {
  return check_view(name, t, d->batch, keys ? d->k_len : d->q_len, keys ? d->kv_heads : d->heads,
                    d->dim, size_of(d->dtype), 16, out);
}

ql::AttnArgs attn_args(const ql_attn* d) {
  ql::AttnArgs a{};
  a.lens = d->k_lens;
  a.mask = d->k_mask;
  a.mask_batch = d->mask_batch;
  a.B = d->batch;
  a.H = d->heads;
  a.Hk = d->kv_heads;
  a.G = d->heads / d->kv_heads;
  a.Lq = d->q_len;
  a.Lk = d->k_len;
  a.D = d->dim;
  a.R = a.Lq * a.G;
  // Neighbouring heads lie in the same lines of memory; but sequences differ in length, and
  // every XCD is to have its share of all of them: at least four units each.
  a.unit = 1;
  while (a.unit < 8 && a.Hk % (2 * a.unit) == 0 && (int64_t)a.B * a.Hk / (2 * a.unit) % 8 == 0 &&
         (int64_t)a.B * a.Hk / (2 * a.unit) >= 32)
    a.unit *= 2;
  a.scale = d->scale;
  a.scale2 = base2(d->scale);
  a.bf16 = d->dtype == QL_BF16;
  return a;
}

// Whether n rows of a tensor lie within 32-bit offsets of the first, g heads side by side.
bool near(const ql_heads_view& t, int64_t n, int64_t g, int64_t size) {
  return t.row * size * (n / g) + t.head * size * g < (int64_t)1 << 32;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

namespace ql {

// Rows and keys by tiles, and how many workgroups share a long axis where few tiles of
// the other one are there. The sizes are those of k_attn.hip's kernels. How many workgroups
// splitting aims at is a compromise; us at each aim, heads of 128 in bf16 unless said:
//   forward, 512: 8 x 1 query, 4096 keys, 32 heads on 8: 39 at 256, 36 at 512, 43 at 768;
//     2 x 512 queries, 2048 keys, 16 heads of 72: 37 at 256, 34 at 512, 41 at 1024; but
//     256 queries, 4608 keys, 16 heads: 28 at 256, 33 at 512, 40 at 1024
//   few keys, workgroups that go through several tiles of rows, 512: 16 x 1024 queries, up to
//     120 keys, 16 heads of 72: 35 at 256, 33 at 512, 37 at 768
//   forward, waves that share the keys (fp32, up to 64 rows), one a compute unit for heads past 96
//     and two for others, 2 x 1 query, 4096 keys at 256, 512 and 768: 16 heads of 64 31 31 41, of
//     72 41 40 52; 8 of 128 38 46 46, of 160 47 56 56; 4 x 1, 4608 keys, 16 of 64: 56 52 57
//   few keys: up to which heads they stay in LDS (else its tiles follow each other), 16 x 1024
//     queries, kept/not at 77 keys, at 120: bf16, 16 heads of 72 28/38, 31/39; 8 of 128 22/26,
//     26/27; of 136 32/33, 42/33 (4 x 4096 queries, 77 keys: 30/34); of 160, where keeping spills,
//     37/36, 45/36; fp32, at 77 keys, 8 of 72 59/64; of 96 65/75; of 128 82/77
//   gradient, bf16, 512: 2 x 8190 queries, 512 and 156 keys, 16 heads on 8: 377 at 256, 280
//     at 512; fp32, 256: 8 x 256 queries, 77 keys, 16 heads of 72: 71 at 256, 78 at 512
AttnPlan attn_plan(const ql_attn& d) {
  AttnPlan p{};
  const int64_t G = d.heads / d.kv_heads, R = d.q_len * G, bh = (int64_t)d.batch * d.kv_heads;
  const int64_t n = (int64_t)d.batch * d.heads * d.q_len;
  const bool bf16 = d.dtype == QL_BF16;
  p.narrow = !bf16 && R <= 64;
  p.row_tiles = ceil_div(R, p.narrow ? 64 : 128);
  const int64_t tiles = ceil_div(d.k_len, 64);
  const int64_t base = bh * p.row_tiles;
  int64_t s = base > 0 ? (p.narrow && d.dim > 96 ? 256 : 512) / base : 1;
  const int64_t most = tiles / (p.narrow ? 2 : 4);
  s = s < most ? s : most;
  p.splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  if (!p.narrow && p.splits == 1 && d.k_len <= 128 && d.dim <= (bf16 ? 128 : 96)) {
    const int64_t each = base / 512;
    p.per_group = (int)(each < 1 ? 1 : each > p.row_tiles ? p.row_tiles : each);
  }
  p.forward_bytes = p.splits > 1 ? up16(p.splits * n * d.dim * 4) + up16(p.splits * n * 4) : 0;

  p.q_tiles = ceil_div(R, 128);
  p.key_tiles = ceil_div(d.k_len, 128);
  const int64_t kbase = bh * p.key_tiles;
  s = kbase > 0 ? (bf16 ? 512 : 256) / kbase : 1;
  const int64_t kmost = ceil_div(R, 32) / (bf16 ? 8 : 2);
  s = s < kmost ? s : kmost;
  p.k_splits = (int)(s < 1 ? 1 : s > 64 ? 64 : s);
  p.grad_bytes = up16(n * 4);
  if (p.k_splits > 1)
    p.grad_bytes += up16(kbase * p.k_splits * 256 * d.dim * 4);
  return p;
}

namespace {
int blocks16(int D) {
  const int n = (D + 15) / 16;
  return n <= 2 ? 2 : n <= 4 ? 4 : n <= 6 ? n : n <= 8 ? 8 : 10;
}
}  // namespace

hipError_t launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int dc = blocks16(a.D);
#define QL_ATTN_GO(T, DC) \
  if (dc == DC && a.bf16 == (sizeof(#T) == sizeof("bf16"))) return attn_forward_##T##_##DC(a, p, s);
  QL_ATTN_UNITS(QL_ATTN_GO)
#undef QL_ATTN_GO
  return hipErrorInvalidValue;
}

hipError_t launch_attn_grad(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int dc = blocks16(a.D);
#define QL_ATTN_GO(T, DC) \
  if (dc == DC && a.bf16 == (sizeof(#T) == sizeof("bf16"))) return attn_grad_##T##_##DC(a, p, s);
  QL_ATTN_UNITS(QL_ATTN_GO)
#undef QL_ATTN_GO
  return hipErrorInvalidValue;
}

}  // namespace ql

#define QL_LAUNCH(expr, what)                                                      \
  do {                                                                             \
    const hipError_t e_ = (expr);                                                  \
    if (e_ != hipSuccess)                                                          \
      return fail(e_ == hipErrorOutOfMemory ? QL_ERR_OOM : QL_ERR_HIP, "%s: %s",   \
                  what, hipGetErrorString(e_));                                    \
  } while (0)

extern "C" {

ql_status qlinear_rows4_bytes(const ql_rows4* d, int64_t* bytes) {
  QL_CHECK(check_rows4(d));
  if (!bytes) return fail(QL_ERR_ARG, "bytes is NULL");
  *bytes = ql::rows4_layout(*d).bytes;
  return ok();
}

ql_status qlinear_rows4_pack(const ql_rows4* d, const int8_t* codes, const void* scales,
                             void* packed, void* stream) {
  QL_CHECK(check_rows4(d));
  QL_CHECK(check_packed(d, packed));
  if (!codes || !scales) return fail(QL_ERR_ARG, "codes or scales is NULL");
  if (!aligned(scales, size_of(d->s_dtype)))
    return fail(QL_ERR_ARG, "scales is not element-aligned");
  QL_LAUNCH(ql::launch_rows4_pack(*d, codes, scales, packed, reinterpret_cast<hipStream_t>(stream)),
            "packing 4-bit weights");
  return ok();
}

ql_status qlinear_rows4_quantize(const ql_rows4* d, const void* W, ql_dtype w_dtype, void* packed,
                                 void* stream) {
  QL_CHECK(check_rows4(d));
  QL_CHECK(check_packed(d, packed));
  if (!dtype_ok(w_dtype)) return fail(QL_ERR_ARG, "bad w_dtype %d", (int)w_dtype);
  if (!W || !aligned(W, size_of(w_dtype)))
    return fail(QL_ERR_ARG, "W is NULL or not element-aligned");
  QL_LAUNCH(ql::launch_rows4_quantize(*d, W, w_dtype == QL_BF16, packed,
                                      reinterpret_cast<hipStream_t>(stream)),
            "quantizing 4-bit weights");
  return ok();
}

ql_status qlinear_rows4_unpack(const ql_rows4* d, int8_t* codes, void* scales, void* stream) {
  QL_CHECK(check_rows4(d));
  QL_CHECK(check_packed(d, d->packed));
  if (!aligned(scales, size_of(d->s_dtype)))
    return fail(QL_ERR_ARG, "scales is not element-aligned");
  if (!codes && !scales) return ok();
  QL_LAUNCH(ql::launch_rows4_unpack(*d, codes, scales, reinterpret_cast<hipStream_t>(stream)),
            "unpacking 4-bit weights");
  return ok();
}

ql_status qlinear_rows4_workspace(const ql_rows4* d, int32_t M, int64_t* bytes) {
  QL_CHECK(check_rows4(d));
  QL_CHECK(check_few_rows(M));
  if (!bytes) return fail(QL_ERR_ARG, "bytes is NULL");
  *bytes = ql::rows4_ws(*d, M).bytes;
  return ok();
}

ql_status qlinear_rows4(const ql_rows4* d, const void* X, int64_t ldx, int32_t M, float* Y,
                        int64_t ldy, void* workspace, int64_t workspace_bytes, void* stream) {
  QL_CHECK(check_rows4(d));
  QL_CHECK(check_few_rows(M));
  if (M == 0) return ok();  // empty tensors may carry NULL data pointers
  QL_CHECK(check_packed(d, d->packed));
  if (!aligned(d->bias, 4)) return fail(QL_ERR_ARG, "bias must be 4-byte aligned");
  if (!X || !Y) return fail(QL_ERR_ARG, "X or Y is NULL");
  if (!aligned(X, size_of(d->x_dtype)) || !aligned(Y, 4))
    return fail(QL_ERR_ARG, "X or Y is not element-aligned");
  if (ldx < d->K || ldy < d->N)
    return fail(QL_ERR_ARG, "ldx = %lld or ldy = %lld is less than its row", (long long)ldx,
                (long long)ldy);
  if (X == Y) return fail(QL_ERR_ARG, "Y is X");
  const ql::Rows4Ws w = ql::rows4_ws(*d, M);
  QL_CHECK(check_workspace(workspace, workspace_bytes, w.bytes));
  const ql::Rows4Layout l = ql::rows4_layout(*d);
  ql::Rows4Args a{};
  a.codes = reinterpret_cast<const ql::Rows4Piece*>(d->packed);
  a.scales = reinterpret_cast<const char*>(d->packed) + l.scales;
  a.bias = d->bias;
  a.X = X;
  a.ldx = ldx;
  a.Y = Y;
  a.ldy = ldy;
  a.digits = reinterpret_cast<char*>(workspace);
  a.worths = reinterpret_cast<float*>(a.digits + w.worths);
  a.part = reinterpret_cast<float*>(a.digits + w.part);
  a.M = M;
  a.N = d->N;
  a.K = d->K;
  a.units = l.units;
  a.tiles = l.tiles;
  a.group = d->group;
  a.x_bf16 = d->x_dtype == QL_BF16;
  a.s_bf16 = d->s_dtype == QL_BF16;
  a.silu = d->act == QL_ACT_SILU;
  a.x_vec = aligned(X, 16) && ldx * size_of(d->x_dtype) % 16 == 0;
  QL_LAUNCH(ql::launch_rows4(a, reinterpret_cast<hipStream_t>(stream)), "launching 4-bit rows");
  return ok();
}

ql_status qlinear_heads_workspace(const ql_heads* d, int64_t* bytes) {
  QL_CHECK(check_heads(d));
  if (!bytes) return fail(QL_ERR_ARG, "bytes is NULL");
  *bytes = heads_ws(d);
  return ok();
}

ql_status qlinear_heads(const ql_heads* d, const void* x, int64_t x_batch, int64_t x_row,
                        const void* pos, int64_t pos_batch, const ql_heads_view* q,
                        const ql_heads_view* k, const ql_heads_view* v, void* stream) {
  QL_CHECK(check_heads(d));
  if (d->batch == 0 || d->positions == 0) return ok();
  QL_CHECK(check_rows(d, "x", x, x_batch, x_row, false));
  QL_CHECK(check_turns(d, pos, pos_batch));
  const ql_heads_view* const y[3] = {q, k, v};
  QL_CHECK(check_parts(d, y, true));
  const ql::HeadsArgs a = heads_args(d, x, x_batch, x_row, pos, pos_batch, y);
  for (int i = 0; i < 3; ++i)
    if (a.y[i].p && (a.y[i].p == x || a.y[i].p == a.y[(i + 1) % 3].p))
      return fail(QL_ERR_ARG, "q, k, v and x must differ");
  QL_LAUNCH(ql::launch_heads(a, reinterpret_cast<hipStream_t>(stream)), "launching the heads' norms");
  return ok();
}

ql_status qlinear_heads_grad(const ql_heads* d, const ql_heads_view* dq, const ql_heads_view* dk,
                             const ql_heads_view* dv, const void* x, int64_t x_batch,
                             int64_t x_row, const void* pos, int64_t pos_batch, void* dx,
                             int64_t dx_batch, int64_t dx_row, void* dgamma_q, void* dgamma_k,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  QL_CHECK(check_heads(d));
  const int64_t ws = size_of(d->w_dtype);
  if (!aligned(dgamma_q, ws) || !aligned(dgamma_k, ws))
    return fail(QL_ERR_ARG, "dgamma_q or dgamma_k is not element-aligned");
  if (d->norm == QL_HEADS_NONE && (dgamma_q || dgamma_k))
    return fail(QL_ERR_ARG, "dgamma_q or dgamma_k without a norm");
  ql::HeadsArgs a{};
  const ql_heads_view* const y[3] = {dq, dk, dv};
  if (d->batch > 0 && d->positions > 0) {
    QL_CHECK(check_rows(d, "x", x, x_batch, x_row, false));
    QL_CHECK(check_rows(d, "dx", dx, dx_batch, dx_row, true));
    QL_CHECK(check_turns(d, pos, pos_batch));
    QL_CHECK(check_parts(d, y, false));
    QL_CHECK(check_workspace(workspace, workspace_bytes, heads_ws(d)));
    a = heads_args(d, x, x_batch, x_row, pos, pos_batch, y);
    a.vec = a.vec && whole(dx, size_of(d->x_dtype), d->batch, dx_batch, d->positions, dx_row, 1, 0);
    if (dx == x || (dx == a.y[0].p || dx == a.y[1].p || dx == a.y[2].p))
      return fail(QL_ERR_ARG, "dx must differ from x, dq, dk and dv");
  } else {
    a = heads_args(d, nullptr, 0, 0, nullptr, 0, {nullptr, nullptr, nullptr});
  }
  const void* const g[2] = {dgamma_q, dgamma_k};  // written without positions too
  for (int i = 0; i < 2; ++i)
    if (g[i] && (g[i] == g[1 - i] || g[i] == d->gamma_q || g[i] == d->gamma_k || g[i] == dx))
      return fail(QL_ERR_ARG, "dgamma_q and dgamma_k must differ from each other, the gammas and dx");
  a.dx = dx;
  a.db = dx_batch;
  a.dr = dx_row;
  a.dgamma[0] = dgamma_q;
  a.dgamma[1] = dgamma_k;
  a.groups = heads_groups(d);
  a.part = dgamma_q || dgamma_k ? reinterpret_cast<float*>(workspace) : nullptr;
  QL_LAUNCH(ql::launch_heads_grad(a, reinterpret_cast<hipStream_t>(stream)),
            "launching the heads' gradient");
  return ok();
}

ql_status qlinear_attention_workspace(const ql_attn* d, int32_t grad, int64_t* bytes) {
  QL_CHECK(check_attn(d));
  if (!bytes) return fail(QL_ERR_ARG, "bytes is NULL");
  if (grad != 0 && grad != 1) return fail(QL_ERR_ARG, "grad = %d must be 0 or 1", grad);
  const ql::AttnPlan p = ql::attn_plan(*d);
  *bytes = grad ? p.grad_bytes : p.forward_bytes;
  return ok();
}

ql_status qlinear_attention(const ql_attn* d, const ql_heads_view* q, const ql_heads_view* k,
                            const ql_heads_view* v, const ql_heads_view* out, float* lse,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  QL_CHECK(check_attn(d));
  if (d->batch == 0 || d->q_len == 0) return ok();
  QL_CHECK(attn_view(d, "q", q, false, false));
  QL_CHECK(attn_view(d, "out", out, false, true));
  if (d->k_len > 0) {  // empty tensors may carry NULL pointers
    QL_CHECK(attn_view(d, "k", k, true, false));
    QL_CHECK(attn_view(d, "v", v, true, false));
    if (out->p == k->p || out->p == v->p) return fail(QL_ERR_ARG, "out is k or v");
  }
  if (out->p == q->p) return fail(QL_ERR_ARG, "out is q");
  if (!aligned(lse, 4)) return fail(QL_ERR_ARG, "lse must be 4-byte aligned");
  const ql::AttnPlan p = ql::attn_plan(*d);
  QL_CHECK(check_workspace(workspace, workspace_bytes, p.forward_bytes));
  ql::AttnArgs a = attn_args(d);
  a.q = view(q);
  a.k = view(k);
  a.v = view(v);
  a.o = view(out);
  a.lse = lse;
  const int64_t size = size_of(d->dtype);
  a.near_keys = near(a.k, 128, 1, size) && near(a.v, 128, 1, size);
  a.row_tiles = p.row_tiles;
  a.per_group = p.per_group;
  a.splits = p.splits;
  if (p.splits > 1) {
    const int64_t n = (int64_t)d->batch * d->heads * d->q_len;
    a.part = reinterpret_cast<float*>(workspace);
    a.part_lse = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                          up16(p.splits * n * d->dim * 4));
  }
  QL_LAUNCH(ql::launch_attn(a, p, reinterpret_cast<hipStream_t>(stream)), "launching attention");
  return ok();
}

ql_status qlinear_attention_grad(const ql_attn* d, const ql_heads_view* dout,
                                 const ql_heads_view* q, const ql_heads_view* k,
                                 const ql_heads_view* v, const ql_heads_view* out,
                                 const float* lse, const ql_heads_view* dq,
                                 const ql_heads_view* dk, const ql_heads_view* dv, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  QL_CHECK(check_attn(d));
  if (d->batch == 0 || (d->q_len == 0 && d->k_len == 0)) return ok();
  if (d->q_len > 0) {  // empty tensors may carry NULL pointers
    QL_CHECK(attn_view(d, "dout", dout, false, false));
    QL_CHECK(attn_view(d, "q", q, false, false));
    QL_CHECK(attn_view(d, "out", out, false, false));
    QL_CHECK(attn_view(d, "dq", dq, false, true));
    if (!lse || !aligned(lse, 4)) return fail(QL_ERR_ARG, "lse is NULL or not 4-byte aligned");
  }
  if (d->k_len > 0) {
    QL_CHECK(attn_view(d, "k", k, true, false));
    QL_CHECK(attn_view(d, "v", v, true, false));
    QL_CHECK(attn_view(d, "dk", dk, true, true));
    QL_CHECK(attn_view(d, "dv", dv, true, true));
  }
  const bool rows = d->q_len > 0, keys = d->k_len > 0;
  const void* const in[5] = {rows ? dout->p : nullptr, rows ? q->p : nullptr,
                             rows ? out->p : nullptr, keys ? k->p : nullptr, keys ? v->p : nullptr};
  const void* const to[3] = {rows ? dq->p : nullptr, keys ? dk->p : nullptr, keys ? dv->p : nullptr};
  for (int i = 0; i < 3; ++i) {
    if (!to[i]) continue;
    for (const void* p : in)
      if (p == to[i]) return fail(QL_ERR_ARG, "dq, dk and dv must differ from what is read");
    if (to[i] == to[(i + 1) % 3]) return fail(QL_ERR_ARG, "dq, dk and dv must differ");
  }
  const ql::AttnPlan p = ql::attn_plan(*d);
  QL_CHECK(check_workspace(workspace, workspace_bytes, p.grad_bytes));
  ql::AttnArgs a = attn_args(d);
  a.dout = view(dout);
  a.q = view(q);
  a.k = view(k);
  a.v = view(v);
  a.o = view(out);
  a.lse = const_cast<float*>(lse);
  a.dq = view(dq);
  a.dk = view(dk);
  a.dv = view(dv);
  const int64_t size = size_of(d->dtype);
  a.near_keys = near(a.k, 128, 1, size) && near(a.v, 128, 1, size);
  a.near_rows = 32 % a.G == 0 && near(a.q, 32, a.G, size) && near(a.dout, 32, a.G, size);
  a.delta = reinterpret_cast<float*>(workspace);
  a.part = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                    up16((int64_t)d->batch * d->heads * d->q_len * 4));
  QL_LAUNCH(ql::launch_attn_grad(a, p, reinterpret_cast<hipStream_t>(stream)),
            "launching the attention's gradient");
  return ok();
}

}  // extern "C"
