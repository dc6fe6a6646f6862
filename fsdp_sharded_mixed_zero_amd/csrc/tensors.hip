// Kernels of the tensor-list calls (zero_tensors.h) and their launches. Part
// of device.hip, after kernels.hip.
//
//   tensors_upload_kernel   the list's table, out of the kernel arguments
//   tensors_sqnorm_kernel   one partial sum of squares per unit
//   tensors_adamw_kernel    clip + AdamW + parameter cast, 32-bit state
//   tensors_adamw8_kernel   the same with the moments in 8 bits
//   tensors_import_kernel, tensors_export_kernel
//                           fp32 moments <-> the 8-bit state
//
// A unit of work is 1024 consecutive elements of one tensor, four 8-bit
// blocks, and belongs to one wave. A launch carries the gradient pointers of
// up to 384 tensors in its arguments; everything that does not change from
// step to step is in the list's device table.
#include <cstring>

#include "tensors_internal.h"

namespace {

using zero::GroupConst;
using zero::kUnitElems;
using zero::StepConst;

constexpr int kListThreads = 256;                       // four waves, four units
constexpr int kListWaves = kListThreads / 64;
constexpr int64_t kListMaxUnits = int64_t(1) << 24;     // units per launch: 2^30 work-items

// What a launch covers: units [u0, u1), which lie in tensors [t0, t0 + n).
struct ListRange {
  const int32_t* first;
  const zero_tensor* rec;
  int32_t t0, n;
  int32_t u0, u1;
};

struct SqArgs {
  ListRange l;
  double* partial;
  const void* grads[ZERO_TENSORS_PER_LAUNCH];
};

struct StepArgs {
  ListRange l;
  StepConst c;
  const void* grads[ZERO_TENSORS_PER_LAUNCH];
};

constexpr int kStatePerLaunch = 224;
struct State8Args {
  ListRange l;
  const float* m[kStatePerLaunch];
  const float* v[kStatePerLaunch];
};

constexpr int kUploadWords = 960;
struct UploadArgs {
  uint32_t* dst;
  int32_t n;
  uint32_t w[kUploadWords];
};
static_assert(sizeof(SqArgs) <= 4096 && sizeof(StepArgs) <= 4096 && sizeof(State8Args) <= 4096 &&
                  sizeof(UploadArgs) <= 4096,
              "kernel arguments fit the 4 KiB segment");

// ------------------------------------------------------- finding the tensor

// The tensor that holds unit u: the last t of the launch with first[t] <= u.
// Each round the 64 lanes probe 64 evenly spaced entries and count those at or
// below u (the counts ascend), so 384 tensors take two rounds.
__device__ __forceinline__ int find_tensor(const ListRange& l, int u) {
  int lo = l.t0, span = l.n;
  const int lane = threadIdx.x & 63;
  while (span > 1) {
    const int stride = (span + 63) >> 6;
    const int k = lane * stride;
    const bool below = k < span && l.first[lo + k] <= u;
    const int top = (__popcll(__ballot(below)) - 1) * stride;
    lo += top;
    span = span - top < stride ? span - top : stride;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// This wave's unit, or -1 past the launch's last.
__device__ __forceinline__ int my_unit(const ListRange& l) {
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int64_t u = int64_t(l.u0) + int64_t(blockIdx.x) * kListWaves + wave;
  return u < l.u1 ? int(u) : -1;
}

// ------------------------------------------------- four elements of a tensor
//
// A lane owns elements e .. e + 3 of a block (e = 4 * lane), of which the first
// `cnt` exist (cnt < 4 at a tensor's end only). Tensors start at any element,
// so the vector accesses are declared with their element's alignment: the
// hardware takes them at any address.

typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 bf16x4_any __attribute__((aligned(2)));
typedef unsigned int bytes4_any __attribute__((aligned(1)));

__device__ __forceinline__ f32x4 load4(const float* p, int cnt) {
  if (cnt >= 4) return *reinterpret_cast<const f32x4_any*>(p);
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < cnt; ++k) r[k] = p[k];
  return r;
}

__device__ __forceinline__ f32x4 load4(const uint16_t* p, int cnt) {
  u32x2 w = {0u, 0u};
  if (cnt >= 4) {
    w = *reinterpret_cast<const bf16x4_any*>(p);
  } else {
    if (cnt > 0) w[0] = p[0];
    if (cnt > 1) w[0] |= uint32_t(p[1]) << 16;
    if (cnt > 2) w[1] = p[2];
  }
  return f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
}

__device__ __forceinline__ uint32_t load4(const uint8_t* p, int cnt) {
  if (cnt >= 4) return *reinterpret_cast<const bytes4_any*>(p);
  uint32_t w = 0;
  for (int k = 0; k < cnt; ++k) w |= uint32_t(p[k]) << (8 * k);
  return w;
}

__device__ __forceinline__ void store4(float* p, int cnt, f32x4 x) {
  if (cnt >= 4) {
    *reinterpret_cast<f32x4_any*>(p) = x;
  } else {
    for (int k = 0; k < cnt; ++k) p[k] = x[k];
  }
}

__device__ __forceinline__ void store4(uint16_t* p, int cnt, f32x4 x) {
  const u32x2 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  if (cnt >= 4) {
    *reinterpret_cast<bf16x4_any*>(p) = w;
  } else {
    if (cnt > 0) p[0] = uint16_t(w[0]);
    if (cnt > 1) p[1] = uint16_t(w[0] >> 16);
    if (cnt > 2) p[2] = uint16_t(w[1]);
  }
}

__device__ __forceinline__ void store4(uint8_t* p, int cnt, uint32_t w) {
  if (cnt >= 4) {
    *reinterpret_cast<bytes4_any*>(p) = w;
  } else {
    for (int k = 0; k < cnt; ++k) p[k] = uint8_t(w >> (8 * k));
  }
}

// Elements of a tensor of `len` from e on, at most 4, at least 0.
__device__ __forceinline__ int count4(int64_t len, int64_t e) {
  const int64_t n = len - e;
  return n >= 4 ? 4 : n > 0 ? int(n) : 0;
}

// ------------------------------------------------------------- 8-bit moments

__device__ __forceinline__ f32x4 e4m3_values(uint32_t w) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
  return f32x4{a[0], a[1], b[0], b[1]};
}

// The nearest e4m3 values (ties to even), one byte each; a NaN or a value
// beyond 464 gives the NaN.
__device__ __forceinline__ uint32_t e4m3_bytes(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// x to fp32 with all of its low bits folded into one sticky bit (rounding to
// odd at 21 significant bits): rounding the result to the 4 bits of an e4m3
// value then gives the correct rounding of x, ties and all.
__device__ __forceinline__ float sticky_f32(double x) {
  const uint64_t b = uint64_t(__double_as_longlong(x));
  const uint64_t hi = (b >> 32) | (uint32_t(b) != 0u ? 1u : 0u);
  return float(__longlong_as_double((long long)(hi << 32)));
}

// The largest x of the wave (x >= 0).
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x = fmaxf(x, __shfl_xor(x, off, 64));
  return x;
}

// x, or 0 where it is NaN or +infinity.
__device__ __forceinline__ float finite_or_0(float x) { return x < __builtin_inff() ? x : 0.f; }

constexpr float kE4M3Max = 448.f;
// The smallest maxima that scales are formed from: 448 / max stays finite, and
// the root's maximum comes from a square that is normal in fp32.
constexpr float kLeastMax = 0x1p-100f, kLeastRoot = 0x1p-63f;

// One block of the 8-bit state: this lane's four moments m, v (fp64) to bytes.
// y[k] = sqrt(v[k]) in units of the block's scale, for the update.
struct Block8 {
  uint32_t m, v;
  float m_scale, v_scale;
  float y[4];
};

__device__ __forceinline__ Block8 block_to_8bit(const double m[4], const double v[4]) {
  float am = 0.f, av = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    am = fmaxf(am, finite_or_0(fabsf(float(m[k]))));
    av = fmaxf(av, finite_or_0(float(v[k])));
  }
  am = fmaxf(wave_max(am), kLeastMax);
  const float as = fmaxf(sqrtf(wave_max(av)), kLeastRoot);
  Block8 r;
  r.m_scale = am / kE4M3Max;
  r.v_scale = as / kE4M3Max;
  const double im = double(kE4M3Max / am), is = double(kE4M3Max / as), is2 = is * is;
  r.m = e4m3_bytes(sticky_f32(m[0] * im), sticky_f32(m[1] * im), sticky_f32(m[2] * im), sticky_f32(m[3] * im));
  // The root in fp32 is off by less than 2^-22; where the 8-bit values of
  // y * (1 - 2^-21) and y * (1 + 2^-21) differ, a border lies between them and
  // the squares decide in fp64.
  double w[4];
  float lo[4], hi[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = v[k] * is2;
    r.y[k] = sqrtf(float(w[k]));
    const float y = v[k] > 0.0 ? fmaxf(r.y[k], 0x1p-9f) : r.y[k];   // not below the least e4m3 value
    lo[k] = y * (1.f - 0x1p-21f);
    hi[k] = y * (1.f + 0x1p-21f);
  }
  uint32_t down = e4m3_bytes(lo[0], lo[1], lo[2], lo[3]);
  const uint32_t up = e4m3_bytes(hi[0], hi[1], hi[2], hi[3]);
  if (down != up) {
    const f32x4 a = e4m3_values(down), b = e4m3_values(up);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t byte = 0xFFu << (8 * k);
      if (((down ^ up) & byte) == 0) continue;
      const double mid = 0.5 * (double(a[k]) + double(b[k]));
      const bool even = ((down >> (8 * k)) & 1u) == 0;
      if (w[k] > mid * mid || (w[k] == mid * mid && !even)) down = (down & ~byte) | (up & byte);
    }
  }
  r.v = down;
  return r;
}

// ------------------------------------------------------------------ kernels

__global__ __launch_bounds__(256) void tensors_upload_kernel(const UploadArgs a) {
  for (int i = threadIdx.x; i < a.n; i += 256) a.dst[i] = a.w[i];
}

template <typename G>
__global__ __launch_bounds__(kListThreads) void tensors_sqnorm_kernel(const SqArgs a) {
  const int u = my_unit(a.l);
  if (u < 0) return;
  const int t = find_tensor(a.l, u), lane = threadIdx.x & 63;
  const G* g = static_cast<const G*>(a.grads[t - a.l.t0]);
  double acc = 0.0;
  if (g != nullptr) {
    const int64_t len = a.l.rec[t].len, base = int64_t(u - a.l.first[t]) * kUnitElems;
#pragma unroll
    for (int k = 0; k < zero::kUnitBlocks; ++k) {
      const int64_t e = base + k * ZERO_STATE8_BLOCK + 4 * lane;
      acc = sq4(load4(g + e, count4(len, e)), acc);
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) acc += __shfl_xor(acc, off, 64);
  if (lane == 0) a.partial[u] = acc;
}

// The clip coefficient, in the flat updates' order.
__device__ __forceinline__ double list_clip(const StepConst& c) {
  AdamWArgs a{};
  a.clip_on = c.clip_on;
  a.n_ranks = c.n_ranks;
  a.rank_sq = c.rank_sq;
  a.max_norm = c.max_norm;
  a.clip_eps = c.clip_eps;
  return clip_coefficient(a);
}

// The update of one element in fp64 (adamw_exact, with a group's constants).
__device__ __forceinline__ void exact_update(const zero::AdamWExact& x, double c, float g, float& p, float& m,
                                             float& v) {
  const double gh = c * double(g);
  const double m1 = x.beta1 * double(m) + x.omb1 * gh;
  const double v1 = x.beta2 * double(v) + x.omb2 * (gh * gh);
  const double denom = sqrt(v1) / x.sqrt_bc2 + x.eps;
  p = float(double(p) * x.decay - x.step_size * (m1 / denom));
  m = float(m1);
  v = float(v1);
}

// P: uint16_t (bf16 parameters and an fp32 master) or float (its own master).
template <typename P, typename G>
__global__ __launch_bounds__(kListThreads) void tensors_adamw_kernel(const StepArgs a) {
  const int u = my_unit(a.l);
  if (u < 0) return;
  const int t = find_tensor(a.l, u), lane = threadIdx.x & 63;
  const G* g = static_cast<const G*>(a.grads[t - a.l.t0]);
  if (g == nullptr) return;
  const zero_tensor& r = a.l.rec[t];
  const int64_t len = r.len, base = int64_t(u - a.l.first[t]) * kUnitElems;
  constexpr bool kOwnMaster = sizeof(P) == 4;
  P* param = static_cast<P*>(r.param);
  float* master = kOwnMaster ? static_cast<float*>(r.param) : r.master;
  float *ms = static_cast<float*>(r.m), *vs = static_cast<float*>(r.v);
  const int group = r.group;
  AdamWArgs k{};
  k.beta1 = a.c.g[group].beta1;
  k.omb1 = a.c.g[group].omb1;
  k.beta2 = a.c.g[group].beta2;
  k.omb2 = a.c.g[group].omb2;
  k.lr_wd = a.c.g[group].lr_wd;
  k.step_size = a.c.g[group].step_size;
  k.inv_sqrt_bc2 = a.c.g[group].inv_sqrt_bc2;
  k.eps = a.c.g[group].eps;
  const double c64 = list_clip(a.c);
  const float c = float(c64);
#pragma unroll 1
  for (int b = 0; b < zero::kUnitBlocks; ++b) {
    const int64_t e = base + b * ZERO_STATE8_BLOCK + 4 * lane;
    const int cnt = count4(len, e);
    if (cnt == 0) break;
    const f32x4 g4 = load4(g + e, cnt);
    f32x4 p4 = load4(master + e, cnt), m4 = load4(ms + e, cnt), v4 = load4(vs + e, cnt);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float p1, m1, v1;
      float p = p4[i], m = m4[i], v = v4[i];
      if (adamw_fast(k, c, g4[i], p, m, v, p1, m1, v1)) {
        exact_update(a.c.x[group], c64, g4[i], p, m, v);
        p1 = p, m1 = m, v1 = v;
      }
      p4[i] = p1, m4[i] = m1, v4[i] = v1;
    }
    store4(master + e, cnt, p4);
    store4(ms + e, cnt, m4);
    store4(vs + e, cnt, v4);
    if constexpr (!kOwnMaster) store4(param + e, cnt, p4);
  }
}

template <typename P, typename G>
__global__ __launch_bounds__(kListThreads) void tensors_adamw8_kernel(const StepArgs a) {
  const int u = my_unit(a.l);
  if (u < 0) return;
  const int t = find_tensor(a.l, u), lane = threadIdx.x & 63;
  const G* g = static_cast<const G*>(a.grads[t - a.l.t0]);
  if (g == nullptr) return;
  const zero_tensor& r = a.l.rec[t];
  const int64_t len = r.len, base = int64_t(u - a.l.first[t]) * kUnitElems;
  constexpr bool kOwnMaster = sizeof(P) == 4;
  P* param = static_cast<P*>(r.param);
  float* master = kOwnMaster ? static_cast<float*>(r.param) : r.master;
  uint8_t *ms = static_cast<uint8_t*>(r.m), *vs = static_cast<uint8_t*>(r.v);
  const GroupConst& k = a.c.g[r.group];
  const zero::AdamWExact& x = a.c.x[r.group];
  const double c = list_clip(a.c);
#pragma unroll 1
  for (int b = 0; b < zero::kUnitBlocks; ++b) {
    const int64_t e0 = base + b * ZERO_STATE8_BLOCK, e = e0 + 4 * lane, block = e0 / ZERO_STATE8_BLOCK;
    if (e0 >= len) break;   // uniform: the whole wave takes part in the block's maxima
    const int cnt = count4(len, e);
    const f32x4 g4 = load4(g + e, cnt);
    f32x4 p4 = load4(master + e, cnt);
    const f32x4 m8 = e4m3_values(load4(ms + e, cnt)), s8 = e4m3_values(load4(vs + e, cnt));
    const double m_scale = double(r.m_scale[block]), v_scale = double(r.v_scale[block]);
    double m[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // elements past the end are zeros here and leave the maxima alone
      const double gh = c * double(g4[i]), s = double(s8[i]) * v_scale;
      m[i] = x.beta1 * (double(m8[i]) * m_scale) + x.omb1 * gh;
      v[i] = x.beta2 * (s * s) + x.omb2 * (gh * gh);
    }
    const Block8 q = block_to_8bit(m, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float denom = fmaf(q.y[i] * q.v_scale, k.inv_sqrt_bc2, k.eps);
      p4[i] = fmaf(-k.step_size, float(m[i]) / denom, fmaf(-k.lr_wd, p4[i], p4[i]));
    }
    store4(master + e, cnt, p4);
    if constexpr (!kOwnMaster) store4(param + e, cnt, p4);
    store4(ms + e, cnt, q.m);
    store4(vs + e, cnt, q.v);
    if (lane == 0) {
      r.m_scale[block] = q.m_scale;
      r.v_scale[block] = q.v_scale;
    }
  }
}

__global__ __launch_bounds__(kListThreads) void tensors_import_kernel(const State8Args a) {
  const int u = my_unit(a.l);
  if (u < 0) return;
  const int t = find_tensor(a.l, u), lane = threadIdx.x & 63;
  const float *m32 = a.m[t - a.l.t0], *v32 = a.v[t - a.l.t0];
  if (m32 == nullptr) return;
  const zero_tensor& r = a.l.rec[t];
  const int64_t len = r.len, base = int64_t(u - a.l.first[t]) * kUnitElems;
#pragma unroll 1
  for (int b = 0; b < zero::kUnitBlocks; ++b) {
    const int64_t e0 = base + b * ZERO_STATE8_BLOCK, e = e0 + 4 * lane, block = e0 / ZERO_STATE8_BLOCK;
    if (e0 >= len) break;
    const int cnt = count4(len, e);
    const f32x4 m4 = load4(m32 + e, cnt), v4 = load4(v32 + e, cnt);
    const double m[4] = {m4[0], m4[1], m4[2], m4[3]}, v[4] = {v4[0], v4[1], v4[2], v4[3]};
    const Block8 q = block_to_8bit(m, v);
    store4(static_cast<uint8_t*>(r.m) + e, cnt, q.m);
    store4(static_cast<uint8_t*>(r.v) + e, cnt, q.v);
    if (lane == 0) {
      r.m_scale[block] = q.m_scale;
      r.v_scale[block] = q.v_scale;
    }
  }
}

__global__ __launch_bounds__(kListThreads) void tensors_export_kernel(const State8Args a) {
  const int u = my_unit(a.l);
  if (u < 0) return;
  const int t = find_tensor(a.l, u), lane = threadIdx.x & 63;
  float *m32 = const_cast<float*>(a.m[t - a.l.t0]), *v32 = const_cast<float*>(a.v[t - a.l.t0]);
  if (m32 == nullptr) return;
  const zero_tensor& r = a.l.rec[t];
  const int64_t len = r.len, base = int64_t(u - a.l.first[t]) * kUnitElems;
#pragma unroll 1
  for (int b = 0; b < zero::kUnitBlocks; ++b) {
    const int64_t e = base + b * ZERO_STATE8_BLOCK + 4 * lane, block = e / ZERO_STATE8_BLOCK;
    const int cnt = count4(len, e);
    if (cnt == 0) break;
    const f32x4 m8 = e4m3_values(load4(static_cast<const uint8_t*>(r.m) + e, cnt));
    const f32x4 s8 = e4m3_values(load4(static_cast<const uint8_t*>(r.v) + e, cnt));
    const float m_scale = r.m_scale[block];
    const double v_scale = double(r.v_scale[block]), v_scale2 = v_scale * v_scale;
    f32x4 m4, v4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m4[i] = m8[i] * m_scale;
      v4[i] = float(double(s8[i] * s8[i]) * v_scale2);   // the square of an e4m3 value is exact
    }
    store4(m32 + e, cnt, m4);
    store4(v32 + e, cnt, v4);
  }
}

// ----------------------------------------------------------------- launches

int launched(const char* who) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(ZERO_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  return zero::ok();
}

// Calls go(range) for ranges that cover the list's units: at most per_launch
// tensors and kListMaxUnits units each.
template <typename F>
int for_ranges(const zero_tensors_s* h, int per_launch, F go) {
  const int32_t n = int32_t(h->t.size());
  const int32_t* first = static_cast<const int32_t*>(h->table);
  const zero_tensor* rec =
      reinterpret_cast<const zero_tensor*>(static_cast<const char*>(h->table) + zero::table_records_at(n));
  for (int32_t t0 = 0; t0 < n; t0 += per_launch) {
    const int32_t t1 = std::min(n, t0 + per_launch);
    const int64_t end = h->first[size_t(t1)];
    for (int64_t u = h->first[size_t(t0)]; u < end; u += kListMaxUnits) {
      const ListRange l{first, rec, t0, t1 - t0, int32_t(u), int32_t(std::min(end, u + kListMaxUnits))};
      if (int rc = go(l)) return rc;
    }
  }
  return zero::ok();
}

dim3 list_grid(const ListRange& l) { return dim3(unsigned((l.u1 - l.u0 + kListWaves - 1) / kListWaves)); }

template <typename P, typename G>
void launch_step(bool wide, const StepArgs& a, hipStream_t stream) {
  if (wide)
    hipLaunchKernelGGL((tensors_adamw_kernel<P, G>), list_grid(a.l), dim3(kListThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((tensors_adamw8_kernel<P, G>), list_grid(a.l), dim3(kListThreads), 0, stream, a);
}

}  // namespace

namespace zero {

int current_device(int* dev, const char* who) {
  const hipError_t e = hipGetDevice(dev);
  if (e != hipSuccess) return fail(ZERO_EHIP, "%s: hipGetDevice: %s", who, hipGetErrorString(e));
  return ZERO_OK;
}

int launch_upload(const zero_tensors_s* h, void* table, hipStream_t stream, const char* who) {
  const int32_t n = int32_t(h->t.size());
  std::vector<uint32_t> words(table_bytes(n) / 4, 0u);
  std::memcpy(words.data(), h->first.data(), h->first.size() * sizeof(int32_t));
  std::memcpy(words.data() + table_records_at(n) / 4, h->t.data(), h->t.size() * sizeof(zero_tensor));
  for (size_t at = 0; at < words.size(); at += kUploadWords) {
    UploadArgs a;
    a.dst = static_cast<uint32_t*>(table) + at;
    a.n = int32_t(std::min<size_t>(kUploadWords, words.size() - at));
    std::memcpy(a.w, words.data() + at, size_t(a.n) * 4);
    hipLaunchKernelGGL(tensors_upload_kernel, dim3(1), dim3(256), 0, stream, a);
    if (int rc = launched(who)) return rc;
  }
  return ok();
}

int launch_sqnorm(const zero_tensors_s* h, const void* const* grads, double* out, int32_t accumulate, double* ws,
                  hipStream_t stream, const char* who) {
  const int rc = for_ranges(h, ZERO_TENSORS_PER_LAUNCH, [&](const ListRange& l) {
    SqArgs a;
    a.l = l;
    a.partial = ws;
    std::copy(grads + l.t0, grads + l.t0 + l.n, a.grads);
    if (h->grad_type == ZERO_BF16)
      hipLaunchKernelGGL(tensors_sqnorm_kernel<uint16_t>, list_grid(l), dim3(kListThreads), 0, stream, a);
    else
      hipLaunchKernelGGL(tensors_sqnorm_kernel<float>, list_grid(l), dim3(kListThreads), 0, stream, a);
    return launched(who);
  });
  return rc ? rc : zero_sum_partials(ws, h->first.back(), out, accumulate, stream);
}

int launch_adamw(const zero_tensors_s* h, const void* const* grads, const StepConst& c, hipStream_t stream,
                 const char* who) {
  return for_ranges(h, ZERO_TENSORS_PER_LAUNCH, [&](const ListRange& l) {
    StepArgs a;
    a.l = l;
    a.c = c;
    std::copy(grads + l.t0, grads + l.t0 + l.n, a.grads);
    const bool wide = h->state_bits == 32, bf16 = h->grad_type == ZERO_BF16;
    if (h->param_type == ZERO_BF16)
      bf16 ? launch_step<uint16_t, uint16_t>(wide, a, stream) : launch_step<uint16_t, float>(wide, a, stream);
    else
      bf16 ? launch_step<float, uint16_t>(wide, a, stream) : launch_step<float, float>(wide, a, stream);
    return launched(who);
  });
}

int launch_state8(const zero_tensors_s* h, bool import, const float* const* m, const float* const* v,
                  hipStream_t stream, const char* who) {
  return for_ranges(h, kStatePerLaunch, [&](const ListRange& l) {
    State8Args a;
    a.l = l;
    std::copy(m + l.t0, m + l.t0 + l.n, a.m);
    std::copy(v + l.t0, v + l.t0 + l.n, a.v);
    if (import)
      hipLaunchKernelGGL(tensors_import_kernel, list_grid(l), dim3(kListThreads), 0, stream, a);
    else
      hipLaunchKernelGGL(tensors_export_kernel, list_grid(l), dim3(kListThreads), 0, stream, a);
    return launched(who);
  });
}

}  // namespace zero
