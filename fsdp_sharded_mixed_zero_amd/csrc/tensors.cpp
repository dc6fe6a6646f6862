// Host side of the tensor-list calls (zero_tensors.h): the list, its table's
// layout, the argument checks of every call and the hyperparameter constants.
// The kernels and their launches are in tensors.hip.
#include "tensors_internal.h"

#include <algorithm>
#include <cmath>
#include <new>

using zero::fail;

namespace {

// Elements and tensors of a list: its units, at most 2^30 + 2^25, fit 32 bits.
constexpr int64_t kMaxTotal = int64_t(1) << 40;
constexpr int32_t kMaxTensors = 1 << 24;

struct Range {
  uintptr_t lo, hi;
  int32_t tensor;
};

bool misaligned(const void* p, uintptr_t n) { return (uintptr_t(p) & (n - 1)) != 0; }

// Whether [p, p + n) meets one of the sorted, disjoint ranges.
bool meets(const std::vector<std::pair<uintptr_t, uintptr_t>>& owned, const void* p, uintptr_t n) {
  const uintptr_t lo = uintptr_t(p), hi = lo + n;
  const auto it = std::upper_bound(owned.begin(), owned.end(), lo,
                                   [](uintptr_t v, const std::pair<uintptr_t, uintptr_t>& r) { return v < r.second; });
  return it != owned.end() && it->first < hi;   // the first range that ends after lo
}

size_t type_bytes(int32_t type) { return type == ZERO_BF16 ? 2 : 4; }

// The handle is bound to a table on the current device.
int check_bound(zero_tensors_t h, const char* who) {
  if (h->table == nullptr) return fail(ZERO_EINVAL, "%s: the list has no table (zero_tensors_upload)", who);
  int dev = -1;
  if (int rc = zero::current_device(&dev, who)) return rc;
  if (dev != h->device)
    return fail(ZERO_EINVAL, "%s: the list's table is on device %d, the current device is %d", who, h->device, dev);
  return ZERO_OK;
}

// The bytes between the first and the last of some arrays. Where they meet none
// of the list's buffers, no single array does: one search instead of one each
// (700 gradients of one flat buffer: a call of 10 us instead of 16).
struct Hull {
  uintptr_t lo = ~uintptr_t(0), hi = 0;
  void add(const void* p, uintptr_t n) {
    lo = std::min(lo, uintptr_t(p));
    hi = std::max(hi, uintptr_t(p) + n);
  }
  bool meets_none_of(const std::vector<std::pair<uintptr_t, uintptr_t>>& owned) const {
    return hi == 0 || !meets(owned, reinterpret_cast<const void*>(lo), hi - lo);
  }
};

// The gradients' alignment and, with `written`, that none lies in a buffer the call writes.
int check_grads(zero_tensors_t h, const void* const* grads, bool written, const char* who) {
  const uintptr_t size = type_bytes(h->grad_type);
  Hull hull;
  for (size_t i = 0; i < h->t.size(); ++i) {
    if (grads[i] == nullptr || h->t[i].len == 0) continue;
    if (misaligned(grads[i], size)) return fail(ZERO_EINVAL, "%s: the gradient of tensor %zu is misaligned", who, i);
    hull.add(grads[i], size * uintptr_t(h->t[i].len));
  }
  if (!written || hull.meets_none_of(h->owned)) return ZERO_OK;
  for (size_t i = 0; i < h->t.size(); ++i)
    if (grads[i] != nullptr && h->t[i].len > 0 && meets(h->owned, grads[i], size * uintptr_t(h->t[i].len)))
      return fail(ZERO_EINVAL, "%s: the gradient of tensor %zu overlaps a buffer of the list", who, i);
  return ZERO_OK;
}

// Whether the ranges, in any order, are disjoint; sorts them unless each starts
// where the one before it ends or later.
bool disjoint(std::vector<std::pair<uintptr_t, uintptr_t>>& r) {
  const auto apart = [&] {
    for (size_t k = 0; k + 1 < r.size(); ++k)
      if (r[k].second > r[k + 1].first) return false;
    return true;
  };
  if (apart()) return true;
  std::sort(r.begin(), r.end());
  return apart();
}

}  // namespace

extern "C" int zero_tensors(const zero_tensor* tensors, int32_t n, int32_t param_type, int32_t grad_type,
                            int32_t state_bits, zero_tensors_t* out) {
  static const char* who = "zero_tensors";
  if (tensors == nullptr || out == nullptr) return fail(ZERO_EINVAL, "%s: NULL argument", who);
  if (n < 1 || n > kMaxTensors) return fail(ZERO_EINVAL, "%s: n must be >= 1 and <= 2^24 (got %d)", who, n);
  for (int32_t type : {param_type, grad_type})
    if (type != ZERO_BF16 && type != ZERO_F32) return fail(ZERO_EINVAL, "%s: unknown element type %d", who, type);
  if (state_bits != 32 && state_bits != 8) return fail(ZERO_EINVAL, "%s: state_bits must be 32 or 8", who);
  zero_tensors_s* h = nullptr;
  try {
    h = new zero_tensors_s;
    h->param_type = param_type;
    h->grad_type = grad_type;
    h->state_bits = state_bits;
    h->t.assign(tensors, tensors + n);
    for (auto& f : h->first) f.resize(size_t(n) + 1);
    h->partial.assign(size_t(n) + 1, 0);
    std::vector<Range> ranges;
    ranges.reserve(size_t(n) * 6);
    const bool wide = state_bits == 32, own_master = param_type == ZERO_F32;
    int64_t total = 0, units = 0, chunks = 0;
    int rc = ZERO_OK;
    for (int32_t i = 0; i < n && rc == ZERO_OK; ++i) {
      const zero_tensor& t = tensors[i];
      h->first[0][size_t(i)] = int32_t(units);
      h->first[1][size_t(i)] = int32_t(chunks);
      if (t.len < 0 || t.len > kMaxTotal || total + t.len > kMaxTotal) {
        rc = fail(ZERO_EINVAL, "%s: length %lld of tensor %d is below 0, or the total beyond 2^40", who,
                  (long long)t.len, i);
        break;
      }
      if (t.group < 0 || t.group >= ZERO_TENSOR_GROUPS) {
        rc = fail(ZERO_EINVAL, "%s: group %d of tensor %d outside [0, %d)", who, t.group, i, ZERO_TENSOR_GROUPS);
        break;
      }
      h->top_group = std::max(h->top_group, t.group);
      total += t.len;
      h->partial[size_t(i) + 1] = h->partial[size_t(i)] + (t.len % zero::kUnitElems != 0);
      const int64_t lead = wide && t.len > 0 ? zero::line_phase(uintptr_t(own_master ? t.param : t.master)) : 0;
      units += (lead + t.len + zero::kUnitElems - 1) / zero::kUnitElems;
      chunks += (t.len + zero::kSqChunk - 1) / zero::kSqChunk;
      if (t.len == 0) continue;
      if (own_master && t.master != nullptr)
        rc = fail(ZERO_EINVAL, "%s: tensor %d has fp32 parameters and a master", who, i);
      if (wide && (t.m_scale != nullptr || t.v_scale != nullptr))
        rc = fail(ZERO_EINVAL, "%s: tensor %d has a 32-bit state and scales", who, i);
      const int64_t blocks = (t.len + ZERO_STATE8_BLOCK - 1) / ZERO_STATE8_BLOCK;
      const size_t state = wide ? 4 : 1;
      const struct { const void* p; size_t align, bytes; const char* name; bool used; } buf[6] = {
          {t.param, type_bytes(param_type), type_bytes(param_type) * size_t(t.len), "param", true},
          {t.master, 4, 4 * size_t(t.len), "master", !own_master},
          {t.m, state, state * size_t(t.len), "m", true},
          {t.v, state, state * size_t(t.len), "v", true},
          {t.m_scale, 4, 4 * size_t(blocks), "m_scale", !wide},
          {t.v_scale, 4, 4 * size_t(blocks), "v_scale", !wide}};
      for (const auto& b : buf) {
        if (!b.used || rc != ZERO_OK) continue;
        if (b.p == nullptr || misaligned(b.p, b.align)) {
          rc = fail(ZERO_EINVAL, "%s: %s of tensor %d is %s", who, b.name, i, b.p ? "misaligned" : "NULL");
          break;
        }
        ranges.push_back({uintptr_t(b.p), uintptr_t(b.p) + b.bytes, i});
      }
    }
    h->first[0][size_t(n)] = int32_t(units);
    h->first[1][size_t(n)] = int32_t(chunks);
    for (int k = 0; k < 2; ++k)
      while (((int64_t(h->first[k].back()) - 1) >> h->shift[k]) >= zero::kSlots) ++h->shift[k];
    if (rc == ZERO_OK) {
      std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
      for (size_t k = 0; k + 1 < ranges.size() && rc == ZERO_OK; ++k)
        if (ranges[k].hi > ranges[k + 1].lo)
          rc = fail(ZERO_EINVAL, "%s: buffers of tensors %d and %d overlap", who, ranges[k].tensor,
                    ranges[k + 1].tensor);
    }
    if (rc != ZERO_OK) {
      delete h;
      return rc;
    }
    for (const Range& r : ranges) {   // neighbours joined: the searches stay short
      if (!h->owned.empty() && h->owned.back().second == r.lo)
        h->owned.back().second = r.hi;
      else
        h->owned.emplace_back(r.lo, r.hi);
    }
  } catch (...) {
    delete h;
    return fail(ZERO_ENOMEM, "%s: out of host memory", who);
  }
  *out = h;
  return zero::ok();
}

extern "C" void zero_tensors_free(zero_tensors_t h) { delete h; }

extern "C" size_t zero_tensors_table_bytes(zero_tensors_t h) {
  return h == nullptr ? 0 : zero::Table(int32_t(h->t.size())).bytes;
}

extern "C" int zero_tensors_upload(zero_tensors_t h, void* d_table, size_t bytes, hipStream_t stream) {
  static const char* who = "zero_tensors_upload";
  if (h == nullptr || d_table == nullptr) return fail(ZERO_EINVAL, "%s: NULL handle or table", who);
  if (misaligned(d_table, 16)) return fail(ZERO_EINVAL, "%s: the table is not 16-byte aligned", who);
  const size_t need = zero_tensors_table_bytes(h);
  if (bytes < need) return fail(ZERO_EINVAL, "%s: table of %zu bytes, need %zu", who, bytes, need);
  if (meets(h->owned, d_table, need)) return fail(ZERO_EINVAL, "%s: the table overlaps a buffer of the list", who);
  int dev = -1;
  if (int rc = zero::current_device(&dev, who)) return rc;
  try {
    if (int rc = zero::launch_upload(h, d_table, stream, who)) return rc;
  } catch (...) {
    return fail(ZERO_ENOMEM, "%s: out of host memory", who);
  }
  h->table = d_table;
  h->device = dev;
  return zero::ok();
}

extern "C" size_t zero_tensors_sqnorm_workspace_bytes(zero_tensors_t h) {
  return h == nullptr ? 0 : std::max<size_t>(1, size_t(h->first[1].back())) * sizeof(double);
}

extern "C" int zero_tensors_sqnorm(zero_tensors_t h, const void* const* grads, double* d_out, int32_t accumulate,
                                   void* d_workspace, size_t ws_bytes, hipStream_t stream) {
  static const char* who = "zero_tensors_sqnorm";
  if (h == nullptr || grads == nullptr) return fail(ZERO_EINVAL, "%s: NULL handle or gradient array", who);
  if (d_out == nullptr || d_workspace == nullptr) return fail(ZERO_EINVAL, "%s: NULL output or workspace", who);
  if (misaligned(d_out, 8) || misaligned(d_workspace, 8))
    return fail(ZERO_EINVAL, "%s: output or workspace is not 8-byte aligned", who);
  const size_t need = zero_tensors_sqnorm_workspace_bytes(h);
  if (ws_bytes < need) return fail(ZERO_EINVAL, "%s: workspace of %zu bytes, need %zu", who, ws_bytes, need);
  if (int rc = check_grads(h, grads, false, who)) return rc;
  if (int rc = check_bound(h, who)) return rc;
  return zero::launch_sqnorm(h, grads, d_out, accumulate ? 1 : 0, static_cast<double*>(d_workspace), stream, who);
}

extern "C" int zero_tensors_adamw_step(zero_tensors_t h, const void* const* grads, const zero_adamw_hparams* groups,
                                       int32_t n_groups, const double* d_rank_sqnorms, int32_t n_ranks,
                                       hipStream_t stream) {
  static const char* who = "zero_tensors_adamw_step";
  if (h == nullptr || grads == nullptr || groups == nullptr)
    return fail(ZERO_EINVAL, "%s: NULL handle, gradient array or hyperparameters", who);
  if (n_groups < 1 || n_groups > ZERO_TENSOR_GROUPS)
    return fail(ZERO_EINVAL, "%s: %d groups, outside [1, %d]", who, n_groups, ZERO_TENSOR_GROUPS);
  if (h->top_group >= n_groups)
    return fail(ZERO_EINVAL, "%s: %d groups given, the list uses group %d", who, n_groups, h->top_group);
  zero::StepConst c{};
  for (int32_t k = 0; k < n_groups; ++k) {
    const zero_adamw_hparams& hp = groups[k];
    if (int rc = zero::check_adamw_hparams(&hp, who)) return rc;
    if (hp.max_norm != groups[0].max_norm || hp.clip_eps != groups[0].clip_eps)
      return fail(ZERO_EINVAL, "%s: max_norm and clip_eps differ between groups", who);
    const double t = double(hp.step);
    const double bc1 = 1.0 - std::pow(hp.beta1, t), bc2 = 1.0 - std::pow(hp.beta2, t);
    c.g[k] = {float(hp.beta1), float(1.0 - hp.beta1), float(hp.beta2), float(1.0 - hp.beta2),
              float(hp.lr * hp.weight_decay), float(hp.lr / bc1), float(1.0 / std::sqrt(bc2)), float(hp.eps)};
    zero::adamw_exact_constants(&hp, &c.x[k]);
  }
  const bool clip = groups[0].max_norm > 0.0;
  if (clip && (d_rank_sqnorms == nullptr || n_ranks < 1))
    return fail(ZERO_EINVAL, "%s: clipping needs the ranks' sums of squares", who);
  if (clip && misaligned(d_rank_sqnorms, 8)) return fail(ZERO_EINVAL, "%s: misaligned sums of squares", who);
  c.rank_sq = d_rank_sqnorms;
  c.n_ranks = clip ? n_ranks : 0;
  c.clip_on = clip ? 1 : 0;
  c.max_norm = groups[0].max_norm;
  c.clip_eps = groups[0].clip_eps;
  if (int rc = check_grads(h, grads, true, who)) return rc;
  if (int rc = check_bound(h, who)) return rc;
  return zero::launch_adamw(h, grads, c, stream, who);
}

// The arrays of an import (read) or export (written), and its launch.
static int state8(zero_tensors_t h, bool import, const float* const* m, const float* const* v, hipStream_t stream,
                  const char* who) {
  if (h == nullptr || m == nullptr || v == nullptr) return fail(ZERO_EINVAL, "%s: NULL argument", who);
  if (h->state_bits != 8) return fail(ZERO_EINVAL, "%s: the list's state is 32-bit already", who);
  try {
    Hull hull[2];
    for (size_t i = 0; i < h->t.size(); ++i) {
      const uintptr_t bytes = 4 * uintptr_t(h->t[i].len);
      if (bytes == 0 || (m[i] == nullptr && v[i] == nullptr)) continue;
      if (m[i] == nullptr || v[i] == nullptr) return fail(ZERO_EINVAL, "%s: one array of tensor %zu is NULL", who, i);
      if (misaligned(m[i], 4) || misaligned(v[i], 4))
        return fail(ZERO_EINVAL, "%s: an array of tensor %zu is misaligned", who, i);
      hull[0].add(m[i], bytes);
      hull[1].add(v[i], bytes);
    }
    for (int k = 0; k < 2; ++k) {
      const float* const* x = k == 0 ? m : v;
      if (hull[k].meets_none_of(h->owned)) continue;
      for (size_t i = 0; i < h->t.size(); ++i)
        if (x[i] != nullptr && h->t[i].len > 0 && meets(h->owned, x[i], 4 * uintptr_t(h->t[i].len)))
          return fail(ZERO_EINVAL, "%s: an array of tensor %zu overlaps a buffer of the list", who, i);
    }
    if (!import) {   // the m arrays, then the v arrays, each lot in list order as a rule
      std::vector<std::pair<uintptr_t, uintptr_t>> out;
      out.reserve(2 * h->t.size());
      const bool v_first = hull[1].lo < hull[0].lo;
      for (const float* const* x : {v_first ? v : m, v_first ? m : v})
        for (size_t i = 0; i < h->t.size(); ++i)
          if (x[i] != nullptr && h->t[i].len > 0)
            out.emplace_back(uintptr_t(x[i]), uintptr_t(x[i]) + 4 * uintptr_t(h->t[i].len));
      if (!disjoint(out)) return fail(ZERO_EINVAL, "%s: two exported arrays overlap", who);
    }
  } catch (...) {
    return fail(ZERO_ENOMEM, "%s: out of host memory", who);
  }
  if (int rc = check_bound(h, who)) return rc;
  return zero::launch_state8(h, import, m, v, stream, who);
}

extern "C" int zero_tensors_state_import(zero_tensors_t h, const float* const* m, const float* const* v,
                                         hipStream_t stream) {
  return state8(h, true, m, v, stream, "zero_tensors_state_import");
}

extern "C" int zero_tensors_state_export(zero_tensors_t h, float* const* m, float* const* v, hipStream_t stream) {
  return state8(h, false, m, v, stream, "zero_tensors_state_export");
}
