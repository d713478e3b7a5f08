// C ABI of the operators beside the layer (declared in include/qlinear.h):
// argument checks, the division of the caller's workspace, and the launches.
#include "../../include/qlinear.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "ql_ops.h"

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

ql_status hip_fail(hipError_t e, const char* what) {
  return fail(e == hipErrorOutOfMemory ? QL_ERR_OOM : QL_ERR_HIP, "%s: %s", what,
              hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(ql_dtype t) { return t == QL_F32 || t == QL_BF16; }
size_t size_of(ql_dtype t) { return t == QL_BF16 ? 2 : 4; }

ql_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need > 0 && !ws) return fail(QL_ERR_ARG, "workspace is NULL");
  if (!aligned(ws, 16)) return fail(QL_ERR_ARG, "workspace must be 16-byte aligned");
  if (have < need)
    return fail(QL_ERR_ARG, "workspace holds %lld bytes, the call needs %lld", (long long)have,
                (long long)need);
  return QL_OK;
}

// ---------------------------------------------------------------- adapters ----

constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 65535;
constexpr int kMaxRows = 1 << 23;

ql_status check_grid(const ql_lora* d, int rows, int32_t n_requests, bool grad) {
  if (ql::lora_fits(rows, n_requests, d->N, grad)) return QL_OK;
  return fail(QL_ERR_UNSUPPORTED, "%d rows of %d requests with N = %d exceed one launch", rows,
              n_requests, d->N);
}

ql_status check_lora(const ql_lora* d, int32_t M, int32_t n_requests) {
  if (!d) return fail(QL_ERR_ARG, "adapter descriptor is NULL");
  if (d->N < 1) return fail(QL_ERR_ARG, "N = %d must be >= 1", d->N);
  if (d->K < 16 || d->K > 65536 || d->K % 16 != 0)
    return fail(QL_ERR_ARG, "K = %d must be a multiple of 16 in [16, 65536]", d->K);
  if (d->rank < 1) return fail(QL_ERR_ARG, "rank = %d must be >= 1", d->rank);
  if (d->rank > kMaxRank)
    return fail(QL_ERR_UNSUPPORTED, "rank = %d: at most %d", d->rank, kMaxRank);
  if (d->n_adapters < 1) return fail(QL_ERR_ARG, "n_adapters = %d must be >= 1", d->n_adapters);
  if (d->n_adapters > kMaxAdapters)
    return fail(QL_ERR_UNSUPPORTED, "n_adapters = %d: at most %d", d->n_adapters, kMaxAdapters);
  if (!dtype_ok(d->x_dtype)) return fail(QL_ERR_ARG, "bad x_dtype %d", (int)d->x_dtype);
  if (!dtype_ok(d->w_dtype)) return fail(QL_ERR_ARG, "bad w_dtype %d", (int)d->w_dtype);
  if (M < 0) return fail(QL_ERR_ARG, "M = %d must be >= 0", M);
  if (M > kMaxRows) return fail(QL_ERR_UNSUPPORTED, "M = %d exceeds %d rows", M, kMaxRows);
  if (n_requests < (M > 0 ? 1 : 0))  // a batch without rows may be one without requests
    return fail(QL_ERR_ARG, "n_requests = %d must be >= %d", n_requests, M > 0 ? 1 : 0);
  if (n_requests > kMaxRows)
    return fail(QL_ERR_UNSUPPORTED, "n_requests = %d exceeds %d", n_requests, kMaxRows);
  if ((int64_t)d->N * d->rank >= (int64_t)1 << 31)
    return fail(QL_ERR_UNSUPPORTED, "B_a of 2^31 elements or more (N = %d, rank = %d)", d->N, d->rank);
  return QL_OK;
}

ql_status check_lora_pointers(const ql_lora* d, const ql_requests* q) {
  if (!d->A || !d->B) return fail(QL_ERR_ARG, "A or B is NULL");
  if (!aligned(d->A, 16)) return fail(QL_ERR_ARG, "A must be 16-byte aligned");
  if (!aligned(d->B, size_of(d->w_dtype))) return fail(QL_ERR_ARG, "B is not element-aligned");
  if (!q->row_offsets || !q->adapter)
    return fail(QL_ERR_ARG, "row_offsets or adapter is NULL");
  if (!aligned(d->scales, 4) || !aligned(d->ranks, 4) || !aligned(q->row_offsets, 4) ||
      !aligned(q->adapter, 4))
    return fail(QL_ERR_ARG, "scales, ranks, row_offsets and adapter must be 4-byte aligned");
  return QL_OK;
}

int split_len(int D, int splits) {
  const int len = (D + splits - 1) / splits;
  return (len + ql::kDsStep - 1) / ql::kDsStep * ql::kDsStep;
}

// Workspace of the backward call: the partial sums of dS, then the slots of
// dA and dB and their adapters.
struct GradWs {
  int s_splits, x_splits, y_splits, x_slots, y_slots;
  int64_t ds, da, db, aid, bid, total;
};
GradWs grad_ws(const ql_lora* d, int32_t M, int32_t n) {
  GradWs w;
  if (n < 1) n = 1;
  w.s_splits = ql::lora_ds_splits(M, n, d->N);
  w.x_splits = ql::lora_x_splits(M, d->K);
  w.y_splits = ql::lora_y_splits(M, n, d->N);
  w.x_slots = w.x_splits + n - 1;
  w.y_slots = w.y_splits + n - 1;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 15) / 16 * 16;
    return here;
  };
  w.ds = take((int64_t)w.s_splits * M * d->rank * 4);
  w.da = take((int64_t)w.x_slots * d->K * d->rank * 4);
  w.db = take((int64_t)w.y_slots * d->N * d->rank * 4);
  w.aid = take((int64_t)w.x_slots * 4);
  w.bid = take((int64_t)w.y_slots * 4);
  w.total = at;
  return w;
}

ql::Requests requests(const ql_lora* d, const ql_requests* q, int rows) {
  return ql::Requests{q->row_offsets, q->adapter, q->n_requests, rows, d->n_adapters};
}

// ------------------------------------------------------------------- norm ----

ql_status check_norm(const ql_norm* d) {
  if (!d) return fail(QL_ERR_ARG, "norm descriptor is NULL");
  if (d->batch < 0 || d->positions < 0)
    return fail(QL_ERR_ARG, "batch = %d and positions = %d must be >= 0", d->batch, d->positions);
  if (d->positions > 1 << 30)
    return fail(QL_ERR_UNSUPPORTED, "positions = %d: at most 1073741824", d->positions);
  if (d->channels < 1 || d->groups < 1 || d->channels % d->groups != 0)
    return fail(QL_ERR_ARG, "channels = %d must be a positive multiple of groups = %d", d->channels,
                d->groups);
  if (d->batch > 65535) return fail(QL_ERR_UNSUPPORTED, "batch = %d: at most 65535", d->batch);
  if (d->channels > 8192 || d->groups > 2048)
    return fail(QL_ERR_UNSUPPORTED, "channels = %d, groups = %d: at most 8192 and 2048",
                d->channels, d->groups);
  if ((int64_t)d->batch * d->groups > 1 << 22)
    return fail(QL_ERR_UNSUPPORTED, "batch = %d times groups = %d: at most 4194304", d->batch,
                d->groups);
  if (!dtype_ok(d->x_dtype)) return fail(QL_ERR_ARG, "bad x_dtype %d", (int)d->x_dtype);
  if (!dtype_ok(d->w_dtype)) return fail(QL_ERR_ARG, "bad w_dtype %d", (int)d->w_dtype);
  if (d->act != QL_ACT_NONE && d->act != QL_ACT_SILU)
    return fail(QL_ERR_ARG, "bad act %d", (int)d->act);
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps))
    return fail(QL_ERR_ARG, "eps = %g must be positive and finite", (double)d->eps);
  if (!aligned(d->gamma, size_of(d->w_dtype)) || !aligned(d->beta, size_of(d->w_dtype)))
    return fail(QL_ERR_ARG, "gamma or beta is not element-aligned");
  return QL_OK;
}

ql_status check_image(const ql_norm* d, const char* name, const void* p, int64_t batch, int64_t row) {
  if (!p) return fail(QL_ERR_ARG, "%s is NULL", name);
  if (!aligned(p, size_of(d->x_dtype))) return fail(QL_ERR_ARG, "%s is not element-aligned", name);
  if (row < d->channels)
    return fail(QL_ERR_ARG, "%s: row stride %lld is less than channels = %d", name, (long long)row,
                d->channels);
  if (batch < 0) return fail(QL_ERR_ARG, "%s: batch stride %lld is negative", name, (long long)batch);
  return QL_OK;
}

// Two images of an output must not share an element: workgroups of both would
// write it. They share one where d batch strides and some row strides, d < batch,
// come within `channels` of each other.
ql_status check_apart(const ql_norm* d, const char* name, int64_t batch, int64_t row) {
  typedef __int128 wide;
  const wide last = d->positions - 1;
  bool apart = d->batch == 1 || (wide)batch >= last * row + d->channels ||  // one after another
               (batch >= d->channels && row >= (wide)(d->batch - 1) * batch + d->channels);
  if (!apart && batch >= d->channels) {  // neither contains the other: image by image
    apart = true;
    for (int32_t i = 1; apart && i < d->batch; ++i) {
      const wide q = (wide)i * batch / row, r = (wide)i * batch % row;
      apart = !(q <= last && r < d->channels) && !(q + 1 <= last && row - r < d->channels);
    }
  }
  if (apart) return QL_OK;
  return fail(QL_ERR_ARG, "%s: images overlap (batch stride %lld, row stride %lld)", name,
              (long long)batch, (long long)row);
}

int64_t norm_ws(const ql_norm* d, bool grad) {
  return ql::norm_ws_bytes(d->batch, d->positions, d->channels, d->groups,
                           (int)size_of(d->x_dtype), grad);
}

ql::NormArgs norm_args(const ql_norm* d) {
  ql::NormArgs a{};
  a.gamma = d->gamma;
  a.beta = d->beta;
  a.B = d->batch;
  a.L = d->positions;
  a.C = d->channels;
  a.G = d->groups;
  a.eps = d->eps;
  a.act = d->act;
  a.x_bf16 = d->x_dtype == QL_BF16;
  a.w_bf16 = d->w_dtype == QL_BF16;
  return a;
}

ql_status check_grads(const ql_grad* table, int32_t n, int64_t units, const double* partials) {
  if (n < 0 || units < 0)
    return fail(QL_ERR_ARG, "n = %d and units = %lld must be >= 0", n, (long long)units);
  if (n == 0 && units != 0) return fail(QL_ERR_ARG, "units = %lld without tensors", (long long)units);
  if (n > 0 && !table) return fail(QL_ERR_ARG, "table is NULL");
  if (!partials) return fail(QL_ERR_ARG, "partials is NULL");
  if (!aligned(table, 8) || !aligned(partials, 8))
    return fail(QL_ERR_ARG, "table and partials must be 8-byte aligned");
  return QL_OK;
}

}  // namespace

#define QL_CHECK(expr)               \
  do {                               \
    const ql_status st_ = (expr);    \
    if (st_ != QL_OK) return st_;    \
  } while (0)
#define QL_LAUNCH(expr, what)                        \
  do {                                               \
    const hipError_t e_ = (expr);                    \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

extern "C" {

ql_status qlinear_lora_workspace(const ql_lora* d, int32_t M, int32_t n_requests, int32_t cfg,
                                 int32_t grad, int64_t* bytes) {
  QL_CHECK(check_lora(d, M, n_requests));
  if (!bytes) return fail(QL_ERR_ARG, "bytes is NULL");
  if (cfg != 0 && cfg != 1) return fail(QL_ERR_ARG, "cfg = %d must be 0 or 1", cfg);
  if (grad != 0 && grad != 1) return fail(QL_ERR_ARG, "grad = %d must be 0 or 1", grad);
  QL_CHECK(check_grid(d, cfg && !grad ? M / 2 : M, n_requests, grad != 0));
  *bytes = grad ? grad_ws(d, M, n_requests).total
                : ql::lora_forward_ws(cfg ? M / 2 : M, n_requests, d->N, d->rank,
                                      d->w_dtype == QL_BF16);
  return ok();
}

ql_status qlinear_lora(const ql_lora* d, const void* X, int64_t ldx, int32_t M,
                       const ql_requests* q, int32_t cfg, float w, const float* base, int64_t ldb,
                       float* Y, int64_t ldy, float* S, void* workspace, int64_t workspace_bytes,
                       void* stream) {
  if (!q) return fail(QL_ERR_ARG, "requests is NULL");
  QL_CHECK(check_lora(d, M, q->n_requests));
  if (cfg != 0 && cfg != 1) return fail(QL_ERR_ARG, "cfg = %d must be 0 or 1", cfg);
  if (cfg && (M % 2)) return fail(QL_ERR_ARG, "M = %d must be even with cfg = 1", M);
  if (M == 0) return ok();  // empty tensors may carry NULL data pointers
  QL_CHECK(check_lora_pointers(d, q));
  if (!X || !Y) return fail(QL_ERR_ARG, "X or Y is NULL");
  if (!aligned(X, size_of(d->x_dtype))) return fail(QL_ERR_ARG, "X is not element-aligned");
  if (!aligned(Y, 4) || !aligned(base, 4) || !aligned(S, 4))
    return fail(QL_ERR_ARG, "base, Y and S must be 4-byte aligned");
  if (ldx < d->K) return fail(QL_ERR_ARG, "ldx = %lld is less than K = %d", (long long)ldx, d->K);
  if (ldy < d->N || (base && ldb < d->N))
    return fail(QL_ERR_ARG, "ldy = %lld or ldb = %lld is less than N = %d", (long long)ldy,
                (long long)ldb, d->N);
  if (base == Y && ldb != ldy)
    return fail(QL_ERR_ARG, "base is Y with another row stride (%lld, %lld)", (long long)ldb,
                (long long)ldy);
  ql::ForwardArgs a{};
  a.halves = cfg ? 2 : 1;
  a.q = requests(d, q, M / a.halves);
  QL_CHECK(check_grid(d, a.q.rows, q->n_requests, false));
  QL_CHECK(check_workspace(workspace, workspace_bytes,
                           ql::lora_forward_ws(a.q.rows, q->n_requests, d->N, d->rank,
                                               d->w_dtype == QL_BF16)));
  a.X = X;
  a.ldx = ldx;
  a.A = d->A;
  a.B = d->B;
  a.scales = d->scales;
  a.ranks = d->ranks;
  a.N = d->N;
  a.K = d->K;
  a.rank = d->rank;
  a.w = w;
  a.base = base;
  a.Y = Y;
  a.ldb = ldb;
  a.ldy = ldy;
  a.S = S;
  a.ws = workspace;
  a.x_bf16 = d->x_dtype == QL_BF16;
  a.w_bf16 = d->w_dtype == QL_BF16;
  QL_LAUNCH(ql::launch_lora_forward(a, reinterpret_cast<hipStream_t>(stream)),
            "launching the adapters");
  return ok();
}

ql_status qlinear_lora_grad(const ql_lora* d, const void* X, int64_t ldx, int32_t M,
                            const ql_requests* q, const float* S, const float* dY, int64_t lddy,
                            void* dX, int64_t lddx, void* dA, void* dB, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  if (!q) return fail(QL_ERR_ARG, "requests is NULL");
  QL_CHECK(check_lora(d, M, q->n_requests));
  const size_t xs = size_of(d->x_dtype), wsz = size_of(d->w_dtype);
  if (!aligned(dX, xs) || !aligned(dA, wsz) || !aligned(dB, wsz))
    return fail(QL_ERR_ARG, "dX, dA or dB is not element-aligned");
  if (M > 0) {  // empty tensors may carry NULL data pointers
    QL_CHECK(check_lora_pointers(d, q));
    if (!X || !S || !dY) return fail(QL_ERR_ARG, "X, S or dY is NULL");
    if (!aligned(X, xs) || !aligned(S, 4) || !aligned(dY, 4))
      return fail(QL_ERR_ARG, "X, S or dY is not element-aligned");
    if (ldx < d->K || lddy < d->N || (dX && lddx < d->K))
      return fail(QL_ERR_ARG, "ldx = %lld, lddy = %lld or lddx = %lld is less than its row",
                  (long long)ldx, (long long)lddy, (long long)lddx);
  }
  QL_CHECK(check_grid(d, M, q->n_requests, true));
  const GradWs w = grad_ws(d, M, q->n_requests);
  if (M > 0) {
    QL_CHECK(check_workspace(workspace, workspace_bytes, w.total));
    if ((dA && (dA == dB || dA == dX)) || (dB && dB == dX))
      return fail(QL_ERR_ARG, "dX, dA and dB must differ");
  }
  char* ws = reinterpret_cast<char*>(workspace);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool w_bf16 = d->w_dtype == QL_BF16;
  ql::OuterArgs x{}, y{};
  ql::DsArgs a{};
  x.rank = y.rank = d->rank;
  x.w_bf16 = y.w_bf16 = w_bf16;
  x.p_bf16 = d->x_dtype == QL_BF16;
  if (M > 0) {
    x.q = y.q = a.q = requests(d, q, M);
    x.ranks = y.ranks = a.ranks = d->ranks;
  }
  if (M > 0 && (dX || dA)) {
    a.dY = dY;
    a.ldy = lddy;
    a.B = d->B;
    a.scales = d->scales;
    a.N = d->N;
    a.rank = d->rank;
    a.splits = w.s_splits;
    a.split_len = split_len(d->N, w.s_splits);
    a.part = reinterpret_cast<float*>(ws + w.ds);
    a.tall = ql::lora_ds_tall(M, q->n_requests);
    x.P = X;
    x.ldp = ldx;
    x.part = a.part;
    x.q_splits = w.s_splits;
    x.A = d->A;
    x.D = d->K;
    x.dX = dX;
    x.lddx = lddx;
    x.out = reinterpret_cast<float*>(ws + w.da);
    x.slot_id = reinterpret_cast<int32_t*>(ws + w.aid);
    x.splits = w.x_splits;
    x.row_len = (M + w.x_splits - 1) / w.x_splits;
  }
  if (M > 0 && dB) {
    y.P = dY;
    y.ldp = lddy;
    y.part = S;
    y.q_splits = 1;
    y.D = d->N;
    y.out = reinterpret_cast<float*>(ws + w.db);
    y.slot_id = reinterpret_cast<int32_t*>(ws + w.bid);
    y.splits = w.y_splits;
    y.row_len = (M + w.y_splits - 1) / w.y_splits;
  }
  if (a.part || y.out) QL_LAUNCH(ql::launch_lora_grad_y(a, y, s), "launching dS and dB");
  if (x.out) QL_LAUNCH(ql::launch_lora_grad_x(x, s), "launching dA and dX");
  if (dA || dB) {
    ql::SlotSumArgs sa{}, sb{};
    sa.n_adapters = sb.n_adapters = d->n_adapters;
    sa.rank = sb.rank = d->rank;
    sa.ranks = sb.ranks = M > 0 ? d->ranks : nullptr;
    sa.w_bf16 = sb.w_bf16 = w_bf16;
    sa.slots = M > 0 ? w.x_slots : 0;
    sb.slots = M > 0 ? w.y_slots : 0;
    sa.part = x.out;
    sa.slot_id = x.slot_id;
    sa.D = d->K;
    sa.out = dA;  // dS has the scale already
    sa.transposed = true;
    sb.part = y.out;
    sb.slot_id = y.slot_id;
    sb.D = d->N;
    sb.scales = M > 0 ? d->scales : nullptr;
    sb.out = dB;
    QL_LAUNCH(ql::launch_lora_slot_sum(sa, sb, s), "launching the sums of dA and dB");
  }
  return ok();
}

ql_status qlinear_group_norm_workspace(const ql_norm* d, int32_t grad, int64_t* bytes) {
  QL_CHECK(check_norm(d));
  if (!bytes) return fail(QL_ERR_ARG, "bytes is NULL");
  if (grad != 0 && grad != 1) return fail(QL_ERR_ARG, "grad = %d must be 0 or 1", grad);
  const bool empty = d->batch == 0 || d->positions == 0;
  *bytes = empty ? 0 : norm_ws(d, grad != 0);
  return ok();
}

ql_status qlinear_group_norm(const ql_norm* d, const void* x, int64_t x_batch, int64_t x_row,
                             void* y, int64_t y_batch, int64_t y_row, float* mean, float* rstd,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  QL_CHECK(check_norm(d));
  if (d->batch == 0) return ok();
  if (d->positions > 0) {  // empty tensors may carry NULL pointers
    QL_CHECK(check_image(d, "x", x, x_batch, x_row));
    QL_CHECK(check_image(d, "y", y, y_batch, y_row));
  }
  if (!aligned(mean, 4) || !aligned(rstd, 4))
    return fail(QL_ERR_ARG, "mean and rstd must be 4-byte aligned");
  if (d->positions > 0) {
    if (x == y && (x_batch != y_batch || x_row != y_row))
      return fail(QL_ERR_ARG, "y is x with other strides");
    QL_CHECK(check_workspace(workspace, workspace_bytes, norm_ws(d, false)));
    QL_CHECK(check_apart(d, "y", y_batch, y_row));
  } else if (!mean && !rstd) {
    return ok();
  }
  ql::NormArgs a = norm_args(d);
  a.x = x;
  a.xb = x_batch;
  a.xr = x_row;
  a.y = y;
  a.yb = y_batch;
  a.yr = y_row;
  a.mean = mean;
  a.rstd = rstd;
  a.ws = workspace;
  QL_LAUNCH(ql::launch_group_norm(a, reinterpret_cast<hipStream_t>(stream)),
            "launching group norm");
  return ok();
}

ql_status qlinear_group_norm_grad(const ql_norm* d, const void* dy, int64_t dy_batch,
                                  int64_t dy_row, const void* x, int64_t x_batch, int64_t x_row,
                                  const float* mean, const float* rstd, void* dx, int64_t dx_batch,
                                  int64_t dx_row, void* dgamma, void* dbeta, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  QL_CHECK(check_norm(d));
  const size_t ws = size_of(d->w_dtype);
  if (!aligned(dgamma, ws) || !aligned(dbeta, ws))
    return fail(QL_ERR_ARG, "dgamma or dbeta is not element-aligned");
  ql::NormArgs a = norm_args(d);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  if (d->batch > 0 && d->positions > 0) {
    QL_CHECK(check_image(d, "dy", dy, dy_batch, dy_row));
    QL_CHECK(check_image(d, "x", x, x_batch, x_row));
    QL_CHECK(check_image(d, "dx", dx, dx_batch, dx_row));
    if (!mean || !rstd) return fail(QL_ERR_ARG, "mean or rstd is NULL");
    if (!aligned(mean, 4) || !aligned(rstd, 4))
      return fail(QL_ERR_ARG, "mean and rstd must be 4-byte aligned");
    if ((dx == dy && (dx_batch != dy_batch || dx_row != dy_row)) ||
        (dx == x && (dx_batch != x_batch || dx_row != x_row)))
      return fail(QL_ERR_ARG, "dx is dy or x with other strides");
    QL_CHECK(check_workspace(workspace, workspace_bytes, norm_ws(d, true)));
    QL_CHECK(check_apart(d, "dx", dx_batch, dx_row));
    // some workgroups write them while others still read gamma and beta
    if ((dgamma && (dgamma == dbeta || dgamma == d->gamma || dgamma == d->beta)) ||
        (dbeta && (dbeta == d->gamma || dbeta == d->beta)))
      return fail(QL_ERR_ARG, "dgamma and dbeta must differ from each other, gamma and beta");
  }
  a.dy = dy;
  a.dyb = dy_batch;
  a.dyr = dy_row;
  a.x = x;
  a.xb = x_batch;
  a.xr = x_row;
  a.y = dx;
  a.yb = dx_batch;
  a.yr = dx_row;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.ws = workspace;
  QL_LAUNCH(ql::launch_group_norm_grad(a, reinterpret_cast<hipStream_t>(stream)),
            "launching the group norm's gradient");
  return ok();
}

ql_status qlinear_grad_norm(const ql_grad* table, int32_t n, int64_t units, double* partials,
                            void* stream) {
  QL_CHECK(check_grads(table, n, units, partials));
  QL_LAUNCH(ql::launch_grad_norm(table, n, units, partials, reinterpret_cast<hipStream_t>(stream)),
            "launching the gradient norm");
  return ok();
}

ql_status qlinear_grad_clip(const ql_grad* table, int32_t n, int64_t units, const double* partials,
                            float max_norm, float* norm, void* stream) {
  QL_CHECK(check_grads(table, n, units, partials));
  if (!norm || !aligned(norm, 4)) return fail(QL_ERR_ARG, "norm is NULL or not 4-byte aligned");
  if (!(max_norm >= 0.0f)) return fail(QL_ERR_ARG, "max_norm = %g must be >= 0", (double)max_norm);
  QL_LAUNCH(ql::launch_grad_clip(table, n, units, partials, max_norm, norm,
                                 reinterpret_cast<hipStream_t>(stream)),
            "launching the gradient clipping");
  return ok();
}

}  // extern "C"
