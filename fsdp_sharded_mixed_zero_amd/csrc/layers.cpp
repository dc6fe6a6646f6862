// Host side of the token-table and norm calls (zero_layers.h): the argument
// checks of every call. The kernels and their launches are in layers.hip.
#include "layers_internal.h"

#include <cmath>

using zero::fail;

namespace {

size_t type_bytes(int32_t type) { return type == ZERO_BF16 ? 2 : type == ZERO_I64 ? 8 : 4; }
bool float_type(int32_t type) { return type == ZERO_BF16 || type == ZERO_F32; }

// One array of a call: rows of `cols` elements, `stride` elements apart.
struct View {
  const char* name;
  const void* p;
  int64_t rows, cols, stride;
  size_t size;       // of an element
  bool written;

  bool empty() const { return p == nullptr || rows == 0 || cols == 0; }
  uintptr_t lo() const { return uintptr_t(p); }
  uintptr_t hi() const { return lo() + (uintptr_t(rows - 1) * uintptr_t(stride) + uintptr_t(cols)) * size; }
};

bool same(const View& a, const View& b) {
  return a.p == b.p && a.size == b.size && a.rows == b.rows && a.cols == b.cols && (a.stride == b.stride || a.rows == 1);
}

// Whether two arrays share a byte. Columns of one larger array (the same stride
// in bytes) lie apart although their ranges meet.
bool overlap(const View& a, const View& b) {
  if (a.empty() || b.empty() || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  const uintptr_t sa = uintptr_t(a.stride) * a.size, sb = uintptr_t(b.stride) * b.size;
  const uintptr_t ca = uintptr_t(a.cols) * a.size, cb = uintptr_t(b.cols) * b.size;
  if (a.rows > 1 && b.rows > 1 && sa == sb && ca <= sa && cb <= sa) {
    const uintptr_t d = b.lo() >= a.lo() ? (b.lo() - a.lo()) % sa : (sa - (a.lo() - b.lo()) % sa) % sa;
    return d < ca || d + cb > sa;
  }
  return true;
}

// Address, alignment and stride of one array that has elements.
int check_view(const View& v, const char* who) {
  if (v.rows == 0 || v.cols == 0) return ZERO_OK;
  if (v.p == nullptr) return fail(ZERO_EINVAL, "%s: %s is NULL", who, v.name);
  if (uintptr_t(v.p) & (v.size - 1)) return fail(ZERO_EINVAL, "%s: %s is misaligned", who, v.name);
  if (v.stride < 0 || (v.written && v.rows > 1 && v.stride < v.cols))
    return fail(ZERO_EINVAL, "%s: stride %lld of %s, whose rows have %lld elements", who, (long long)v.stride, v.name,
                (long long)v.cols);
  if (v.rows > 1 && v.stride > (int64_t(1) << 40) / v.rows)
    return fail(ZERO_EINVAL, "%s: %s spans more than 2^40 elements", who, v.name);
  return ZERO_OK;
}

// Every array of a call; `may` lists pairs (written, other) that may be one and
// the same array.
int check_views(const View* v, int n, const int (*may)[2], int n_may, const char* who) {
  for (int i = 0; i < n; ++i)
    if (int rc = check_view(v[i], who)) return rc;
  for (int i = 0; i < n; ++i) {
    if (!v[i].written) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || (v[j].written && j < i) || !overlap(v[i], v[j])) continue;
      bool allowed = false;
      for (int k = 0; k < n_may && !allowed; ++k)
        allowed = ((may[k][0] == i && may[k][1] == j) || (may[k][0] == j && may[k][1] == i)) && same(v[i], v[j]);
      if (!allowed) return fail(ZERO_EINVAL, "%s: %s overlaps %s", who, v[i].name, v[j].name);
    }
  }
  return ZERO_OK;
}

bool sizes_fit(int64_t n, int64_t dim) {
  return n >= 0 && n <= ZERO_LAYER_ROWS && dim >= 1 && dim <= ZERO_LAYER_DIM && n * dim <= ZERO_LAYER_ELEMS;
}

int check_sizes(int64_t n, int64_t dim, const char* who) {
  if (n < 0 || n > ZERO_LAYER_ROWS) return fail(ZERO_EINVAL, "%s: n = %lld outside [0, %d]", who, (long long)n, ZERO_LAYER_ROWS);
  if (dim < 1 || dim > ZERO_LAYER_DIM)
    return fail(ZERO_EINVAL, "%s: dim = %lld outside [1, %d]", who, (long long)dim, ZERO_LAYER_DIM);
  if (n * dim > ZERO_LAYER_ELEMS)
    return fail(ZERO_EINVAL, "%s: %lld rows of %lld elements, more than 2^35 together", who, (long long)n, (long long)dim);
  return ZERO_OK;
}

int check_rows(int64_t rows, const char* who) {
  if (rows < 1 || rows > ZERO_LAYER_ROWS)
    return fail(ZERO_EINVAL, "%s: rows = %lld outside [1, %d]", who, (long long)rows, ZERO_LAYER_ROWS);
  return ZERO_OK;
}

int check_scale(double scale, const char* who) {
  if (!std::isfinite(float(scale))) return fail(ZERO_EINVAL, "%s: the scale %g is not a finite fp32 number", who, scale);
  return ZERO_OK;
}

int check_token_type(int32_t type, const char* who) {
  if (type != ZERO_I32 && type != ZERO_I64) return fail(ZERO_EINVAL, "%s: unknown token type %d", who, type);
  return ZERO_OK;
}

int check_types(const int32_t* types, int n, const char* who) {
  for (int i = 0; i < n; ++i)
    if (!float_type(types[i])) return fail(ZERO_EINVAL, "%s: unknown element type %d", who, types[i]);
  return ZERO_OK;
}

}  // namespace

extern "C" int zero_embedding(const void* tokens, int32_t token_type, int64_t n, const void* table, int32_t table_type,
                              int64_t rows, int64_t dim, double scale, void* out, int32_t out_type, int64_t out_stride,
                              hipStream_t stream) {
  static const char* who = "zero_embedding";
  const int32_t types[2] = {table_type, out_type};
  if (int rc = check_token_type(token_type, who)) return rc;
  if (int rc = check_types(types, 2, who)) return rc;
  if (int rc = check_sizes(n, dim, who)) return rc;
  if (int rc = check_rows(rows, who)) return rc;
  if (int rc = check_scale(scale, who)) return rc;
  if (n == 0) return zero::ok();
  const View v[3] = {{"out", out, n, dim, out_stride, type_bytes(out_type), true},
                     {"the tokens", tokens, 1, n, n, type_bytes(token_type), false},
                     {"the table", table, 1, rows * dim, rows * dim, type_bytes(table_type), false}};
  if (int rc = check_views(v, 3, nullptr, 0, who)) return rc;
  return zero::launch_embedding(tokens, token_type == ZERO_I64, n, table, table_type, rows, dim, float(scale), out,
                                out_type, out_stride, stream, who);
}

extern "C" size_t zero_token_order_bytes(int64_t n, int64_t rows) {
  if (n < 0 || n > ZERO_LAYER_ROWS || rows < 1 || rows > ZERO_LAYER_ROWS) return 0;
  return size_t(zero::Order(n).words) * sizeof(int32_t);
}

extern "C" int zero_token_order(const void* tokens, int32_t token_type, int64_t n, int64_t rows, void* order,
                                size_t order_bytes, hipStream_t stream) {
  static const char* who = "zero_token_order";
  if (int rc = check_token_type(token_type, who)) return rc;
  if (int rc = check_sizes(n, 1, who)) return rc;
  if (int rc = check_rows(rows, who)) return rc;
  if (order == nullptr) return fail(ZERO_EINVAL, "%s: the order is NULL", who);
  if (uintptr_t(order) & 15) return fail(ZERO_EINVAL, "%s: the order is not 16-byte aligned", who);
  const size_t need = zero_token_order_bytes(n, rows);
  if (order_bytes < need) return fail(ZERO_EINVAL, "%s: order of %zu bytes, need %zu", who, order_bytes, need);
  const View v[2] = {{"the order", order, 1, int64_t(need), int64_t(need), 1, true},
                     {"the tokens", tokens, 1, n, n, type_bytes(token_type), false}};
  if (int rc = check_views(v, 2, nullptr, 0, who)) return rc;
  return zero::launch_token_order(tokens, token_type == ZERO_I64, n, rows, static_cast<int32_t*>(order), stream, who);
}

extern "C" size_t zero_embedding_grad_workspace_bytes(int64_t n, int64_t dim) {
  if (!sizes_fit(n, dim)) return 0;
  // never less than for fewer tokens, whose pieces are shorter
  const int64_t pieces = std::max<int64_t>({1, zero::embedding_pieces(n), zero::embedding_pieces(std::min(n, zero::kShortPieces))});
  return size_t(pieces) * 2 * size_t((dim + 3) / 4 * 4) * sizeof(float);
}

extern "C" int zero_embedding_grad(const void* order, int64_t n, int64_t rows, int64_t dim, const void* d_out,
                                   int32_t out_type, int64_t out_stride, double scale, void* grad, int32_t grad_type,
                                   int64_t first, int64_t count, int32_t accumulate, void* workspace, size_t ws_bytes,
                                   hipStream_t stream) {
  static const char* who = "zero_embedding_grad";
  const int32_t types[2] = {out_type, grad_type};
  if (int rc = check_types(types, 2, who)) return rc;
  if (int rc = check_sizes(n, dim, who)) return rc;
  if (int rc = check_rows(rows, who)) return rc;
  if (int rc = check_scale(scale, who)) return rc;
  const int64_t total = rows * dim;
  if (first < 0 || count < 0 || first > total || count > total - first)
    return fail(ZERO_EINVAL, "%s: elements [%lld, +%lld) of a table of %lld", who, (long long)first, (long long)count,
                (long long)total);
  if (count > ZERO_LAYER_ELEMS)
    return fail(ZERO_EINVAL, "%s: a part of %lld elements, more than 2^35", who, (long long)count);
  if (order == nullptr || workspace == nullptr) return fail(ZERO_EINVAL, "%s: NULL order or workspace", who);
  if ((uintptr_t(order) | uintptr_t(workspace)) & 15)
    return fail(ZERO_EINVAL, "%s: order or workspace is not 16-byte aligned", who);
  const size_t need = zero_embedding_grad_workspace_bytes(n, dim), order_need = zero_token_order_bytes(n, rows);
  if (ws_bytes < need) return fail(ZERO_EINVAL, "%s: workspace of %zu bytes, need %zu", who, ws_bytes, need);
  const View v[4] = {{"grad", grad, 1, count, count, type_bytes(grad_type), true},
                     {"the workspace", workspace, 1, int64_t(need), int64_t(need), 1, true},
                     {"d_out", d_out, n, dim, out_stride, type_bytes(out_type), false},
                     {"the order", order, 1, int64_t(order_need), int64_t(order_need), 1, false}};
  if (int rc = check_views(v, 4, nullptr, 0, who)) return rc;
  if (count == 0) return zero::ok();
  return zero::launch_embedding_grad(static_cast<const int32_t*>(order), n, rows, dim, d_out, out_type, out_stride,
                                     float(scale), grad, grad_type, first, count, accumulate != 0,
                                     static_cast<float*>(workspace), stream, who);
}

extern "C" int zero_norm(const zero_norm_args* args, hipStream_t stream) {
  static const char* who = "zero_norm";
  if (args == nullptr) return fail(ZERO_EINVAL, "%s: NULL arguments", who);
  const zero_norm_args& a = *args;
  const int32_t types[2] = {a.type, a.weight_type};
  if (int rc = check_types(types, 2, who)) return rc;
  if (int rc = check_sizes(a.n, a.dim, who)) return rc;
  if (!(a.eps >= 0.0) || !std::isfinite(float(a.eps))) return fail(ZERO_EINVAL, "%s: invalid eps %g", who, a.eps);
  if ((a.residual == nullptr) != (a.total == nullptr))
    return fail(ZERO_EINVAL, "%s: one of residual and total is NULL", who);
  if (a.n == 0) return zero::ok();
  const size_t e = type_bytes(a.type), w = type_bytes(a.weight_type);
  const auto some = [&](const void* p, int64_t k) { return p == nullptr ? 0 : k; };
  const View v[8] = {{"y", a.y, a.n, a.dim, a.y_stride, e, true},
                     {"total", a.total, some(a.total, a.n), a.dim, a.total_stride, e, true},
                     {"mean", a.mean, 1, some(a.mean, a.n), a.n, 4, true},
                     {"rstd", a.rstd, 1, some(a.rstd, a.n), a.n, 4, true},
                     {"x", a.x, a.n, a.dim, a.x_stride, e, false},
                     {"residual", a.residual, some(a.residual, a.n), a.dim, a.residual_stride, e, false},
                     {"weight", a.weight, 1, some(a.weight, a.dim), a.dim, w, false},
                     {"bias", a.bias, 1, some(a.bias, a.dim), a.dim, w, false}};
  static const int may[3][2] = {{0, 4}, {1, 4}, {1, 5}};
  if (int rc = check_views(v, 8, may, 3, who)) return rc;
  return zero::launch_norm(a, stream, who);
}

extern "C" size_t zero_norm_grad_workspace_bytes(int64_t n, int64_t dim) {
  if (!sizes_fit(n, dim)) return 0;
  return size_t(zero::norm_grad_blocks(n, dim)) * 2 * size_t((dim + 3) / 4 * 4) * sizeof(float);
}

extern "C" int zero_norm_grad(const zero_norm_grad_args* args, void* workspace, size_t ws_bytes, hipStream_t stream) {
  static const char* who = "zero_norm_grad";
  if (args == nullptr) return fail(ZERO_EINVAL, "%s: NULL arguments", who);
  const zero_norm_grad_args& a = *args;
  const int32_t types[3] = {a.type, a.weight_type, a.grad_type};
  if (int rc = check_types(types, 3, who)) return rc;
  if (int rc = check_sizes(a.n, a.dim, who)) return rc;
  if (a.d_x == nullptr && a.d_weight == nullptr && a.d_bias == nullptr)
    return fail(ZERO_EINVAL, "%s: no output is asked for", who);
  if (a.d_total != nullptr && a.d_x == nullptr) return fail(ZERO_EINVAL, "%s: d_total without d_x", who);
  const bool sums = a.d_weight != nullptr || a.d_bias != nullptr;
  const size_t need = sums ? zero_norm_grad_workspace_bytes(a.n, a.dim) : 0;
  if (sums) {
    if (workspace == nullptr) return fail(ZERO_EINVAL, "%s: NULL workspace", who);
    if (uintptr_t(workspace) & 15) return fail(ZERO_EINVAL, "%s: the workspace is not 16-byte aligned", who);
    if (ws_bytes < need) return fail(ZERO_EINVAL, "%s: workspace of %zu bytes, need %zu", who, ws_bytes, need);
  }
  const size_t e = type_bytes(a.type), w = type_bytes(a.weight_type), g = type_bytes(a.grad_type);
  const auto some = [&](const void* p, int64_t k) { return p == nullptr ? 0 : k; };
  const View v[10] = {{"d_x", a.d_x, some(a.d_x, a.n), a.dim, a.d_x_stride, e, true},
                      {"d_weight", a.d_weight, 1, some(a.d_weight, a.dim), a.dim, g, true},
                      {"d_bias", a.d_bias, 1, some(a.d_bias, a.dim), a.dim, g, true},
                      {"the workspace", workspace, 1, int64_t(need), int64_t(need), 1, true},
                      {"d_y", a.d_y, a.n, a.dim, a.d_y_stride, e, false},
                      {"x", a.x, a.n, a.dim, a.x_stride, e, false},
                      {"d_total", a.d_total, some(a.d_total, a.n), a.dim, a.d_total_stride, e, false},
                      {"mean", a.mean, 1, a.rms ? 0 : a.n, a.n, 4, false},
                      {"rstd", a.rstd, 1, a.n, a.n, 4, false},
                      {"weight", a.weight, 1, some(a.weight, a.dim), a.dim, w, false}};
  static const int may[3][2] = {{0, 4}, {0, 5}, {0, 6}};
  if (int rc = check_views(v, 10, may, 3, who)) return rc;
  if (a.n == 0 && (!sums || a.accumulate)) return zero::ok();
  return zero::launch_norm_grad(a, static_cast<float*>(workspace), stream, who);
}
