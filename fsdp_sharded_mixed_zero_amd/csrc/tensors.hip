// Kernels of the tensor-list calls (zero_tensors.h) and their launches. Part
// of device.hip, after kernels.hip.
//
//   tensors_upload_kernel   the list's table, out of the kernel arguments
//   tensors_sqnorm_kernel   one partial sum of squares per four chunks
//   tensors_adamw_kernel    clip + AdamW + parameter cast, 32-bit state
//   tensors_adamw8_kernel   the same with the moments in 8 bits
//   tensors_import_kernel, tensors_export_kernel
//                           fp32 moments <-> the 8-bit state
//
// Every element is read and written once and takes a few dozen instructions,
// so the kernels are bound by HBM on long lists (5.7 to 6.4 TB/s, a plain copy
// reaching 6.25) and by the launch on short ones (5 us). What a list adds to a
// flat array is to find a wave's tensor, which costs memory latency: the work
// is cut into units of 1024 consecutive elements of one tensor (four 8-bit
// blocks; chunks of 4096 for the norm), and a running count of them is searched
// from a slot near the answer. A launch carries the gradients' addresses in its
// arguments, as 32-bit steps for up to 768 tensors; everything that does not
// change from step to step is in the device table.
// Times below are medians of one MI355X, the kernel alone unless a call is named.
#include <cstring>

#include "tensors_internal.h"

namespace {

using zero::GroupConst;
using zero::kSqChunk;
using zero::kUnitElems;
using zero::StepConst;

// One wave a block: a wave's registers are free for the next unit as soon as it
// ends (256 threads: the 8-bit step over 119 M elements 403 us against 382).
constexpr int kListThreads = 64;
constexpr int kSqListWaves = 4, kSqListThreads = 64 * kSqListWaves;
constexpr int64_t kListMaxUnits = int64_t(1) << 23;     // units per launch: at most 2^31 work-items

// What a launch covers: units [u0, u1) (chunks, for the norm), which lie in
// tensors [t0, t0 + n); first[t]: tensor t's first one; slot: where the search
// for unit u begins, at u >> shift.
struct ListRange {
  const int32_t *first, *slot;
  const zero_tensor* rec;
  int32_t t0, n;
  int32_t u0, u1;
  int32_t n_all, shift;
};

// Addresses of a launch's N tensors: steps of 2^shift bytes from the lowest one
// (their common alignment), so that twice as many fit the arguments as with
// pointers. A launch ends before a tensor that would need more than 32 bits.
constexpr uint32_t kNoTensor = 0xFFFFFFFFu;
template <int N>
struct Addresses {
  uintptr_t base;
  uint32_t shift;
  uint32_t step[N];

  template <typename T>
  __device__ __forceinline__ T* at(int i) const {
    const uint32_t s = step[i];
    return s == kNoTensor ? nullptr : reinterpret_cast<T*>(base + (uintptr_t(s) << shift));
  }
};

// base: the first chunk of the first block, at most l.u0; the chunks from there
// to l.u0 are another launch's, which left their sum in partial[0].
struct SqArgs {
  ListRange l;
  int32_t base;
  double* partial;
  Addresses<ZERO_TENSORS_PER_LAUNCH> grads;
};

struct StepArgs {
  ListRange l;
  StepConst c;
  Addresses<ZERO_TENSORS_PER_LAUNCH> grads;
};

constexpr int kStatePerLaunch = 480;
struct State8Args {
  ListRange l;
  Addresses<kStatePerLaunch> m, v;
};

constexpr int kUploadWords = 960;
struct UploadArgs {
  uint32_t* dst;
  int32_t n;
  uint32_t w[kUploadWords];
};
static_assert(sizeof(SqArgs) <= 4096 && sizeof(StepArgs) <= 4096 &&
                  sizeof(State8Args) <= 4096 && sizeof(UploadArgs) <= 4096,
              "kernel arguments fit the 4 KiB segment");

// ------------------------------------------------------- finding the tensor

// A value at a wave-uniform address that the kernel does not write, read by a
// scalar load (the compiler cannot know that the stores leave it alone).
template <typename T>
__device__ __forceinline__ T uniform_load(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

// The tensor that holds unit u, the last t with first[t] <= u, and in *start
// its first unit. The 64 lanes compare 64 consecutive entries, from the slot's
// tensor on, as often as all of them are at or below u (the counts ascend).
// (64 entries spaced over a launch's tensors, then the rest between two of them,
// touch a cache line a lane: the 32-bit step over 868 tensors 544 us against 535
// when the slots were chosen; with what came after them it takes 522.)
__device__ __forceinline__ int find_tensor(const ListRange& l, int u, int* start) {
  int lo = l.n_all <= 64 ? 0 : uniform_load(l.slot + (u >> l.shift));
  const int lane = threadIdx.x & 63;
  for (;;) {
    const int x = lo + lane <= l.n_all ? l.first[lo + lane] : 0x7FFFFFFF;
    const int below = __popcll(__ballot(x <= u));   // at least 1; lane 63's entry is the next round's first
    *start = __builtin_amdgcn_readlane(x, below - 1);
    if (below < 64) return __builtin_amdgcn_readfirstlane(lo + below - 1);
    lo += 63;
  }
}

// What a wave works on: its tensor, its unit's first element, how many elements
// the tensor has from there on, and the block of the unit it takes if it takes
// only one.
struct Unit {
  int t;
  int64_t base, rest;
  int block;
};

// Blocks go round the 8 XCDs one by one; in this order an XCD gets runs of
// kXcdRun consecutive units, whose neighbours' cache lines then meet in one L2
// (8-bit step over tensors packed without gaps, fp32 gradients: 391 us in
// dispatch order, 380 in runs of 32; the import 212 and 203; aligned tensors
// gain up to 3 %). The blocks after the last whole round keep their order.
constexpr int kXcds = 8, kXcdRun = 32;
__device__ __forceinline__ int block_in_runs() {
  const int b = int(blockIdx.x), whole = int(gridDim.x) / (kXcds * kXcdRun) * (kXcds * kXcdRun);
  if (b >= whole) return b;
  const int xcd = b % kXcds, i = b / kXcds;
  return (i / kXcdRun * kXcds + xcd) * kXcdRun + i % kXcdRun;
}

// The wave's unit, which WAVES waves share (1, 2 or 4), the same number of
// blocks each.
template <int WAVES>
__device__ __forceinline__ Unit my_unit(const ListRange& l) {
  const int u = l.u0 + (WAVES > 1 ? int(blockIdx.x) / WAVES : block_in_runs());
  Unit w;
  w.block = int(blockIdx.x) % WAVES * (zero::kUnitBlocks / WAVES);
  int start;
  w.t = find_tensor(l, u, &start);
  w.base = int64_t(u - start) * kUnitElems;
  w.rest = uniform_load(&l.rec[w.t].len) - w.base;
  return w;
}

// ------------------------------------------------- four elements of a tensor
//
// A lane owns elements 4 * lane .. 4 * lane + 3 of each block, of which the
// first `cnt` exist (cnt < 4 at a tensor's end only). Tensors start at any
// element, so the vector accesses are declared with their element's
// alignment: the hardware takes them at any address. Everything is read and
// written once, so the accesses are non-temporal (cached ones: the 32-bit step
// 20 % slower, the 8-bit step 10 %), except the loads of bytes, whose lines two
// instructions share where a tensor starts off a boundary (24.3 M elements so:
// 70.9 us cached, 81.3 us non-temporal; 119 M on boundaries: 363 and 358). The
// pointers are marked global: one that comes out of memory would be a flat one.

#define ZERO_GLOBAL __attribute__((address_space(1)))

typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 bf16x4_any __attribute__((aligned(2)));
typedef u32x4 words4_any __attribute__((aligned(2)));
typedef unsigned int bytes4_any __attribute__((aligned(1)));

template <typename V>
__device__ __forceinline__ V stream_load(const void* p) {
  return __builtin_nontemporal_load((const ZERO_GLOBAL V*)p);
}

template <typename V>
__device__ __forceinline__ void stream_store(void* p, V x) {
  __builtin_nontemporal_store(x, (ZERO_GLOBAL V*)p);
}

__device__ __forceinline__ f32x4 widen(u32x2 w) { return f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])}; }
__device__ __forceinline__ f32x4 widen(f32x4 w) { return w; }

__device__ __forceinline__ f32x4 load4(const float* p, int cnt) {
  if (cnt >= 4) return stream_load<f32x4_any>(p);
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < cnt) r[k] = p[k];
  return r;
}

__device__ __forceinline__ u32x2 load4(const uint16_t* p, int cnt) {
  if (cnt >= 4) return stream_load<bf16x4_any>(p);
  u32x2 w = {0u, 0u};
  if (cnt > 0) w[0] = p[0];
  if (cnt > 1) w[0] |= uint32_t(p[1]) << 16;
  if (cnt > 2) w[1] = p[2];
  return w;
}

__device__ __forceinline__ uint32_t load4(const uint8_t* p, int cnt) {
  if (cnt >= 4) return *(const ZERO_GLOBAL bytes4_any*)p;
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < cnt) w |= uint32_t(p[k]) << (8 * k);
  return w;
}

__device__ __forceinline__ void store4(float* p, int cnt, f32x4 x) {
  if (cnt >= 4) {
    stream_store<f32x4_any>(p, x);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < cnt) p[k] = x[k];
  }
}

__device__ __forceinline__ void store4(uint16_t* p, int cnt, f32x4 x) {
  const u32x2 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  if (cnt >= 4) {
    stream_store<bf16x4_any>(p, w);
  } else {
    if (cnt > 0) p[0] = uint16_t(w[0]);
    if (cnt > 1) p[1] = uint16_t(w[0] >> 16);
    if (cnt > 2) p[2] = uint16_t(w[1]);
  }
}

__device__ __forceinline__ void store4(uint8_t* p, int cnt, uint32_t w) {
  if (cnt >= 4) {
    stream_store<bytes4_any>(p, w);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < cnt) p[k] = uint8_t(w >> (8 * k));
  }
}

// The same of the elements [lo, cnt) of the four at p: lo > 0 where a unit
// begins before its tensor.
template <typename T>
__device__ __forceinline__ auto load4(const T* p, int lo, int cnt) {
  auto x = load4(p, lo == 0 ? cnt : 0);
  if (lo != 0) {
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      if (k < lo || k >= cnt) continue;
      if constexpr (sizeof(T) == 2) x[k >> 1] |= uint32_t(p[k]) << (16 * (k & 1));
      else x[k] = p[k];
    }
  }
  return x;
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int lo, int cnt, f32x4 x) {
  if (lo == 0) {
    store4(p, cnt, x);
  } else {
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      if (k < lo || k >= cnt) continue;
      if constexpr (sizeof(T) == 2) p[k] = to_bf16(x[k]);
      else p[k] = x[k];
    }
  }
}

// Of the `rest` elements from a block's first on, how many this lane's four hold.
__device__ __forceinline__ int count4(int64_t rest) {
  const int64_t n = rest - 4 * int(threadIdx.x & 63);
  return n >= 4 ? 4 : n > 0 ? int(n) : 0;
}

// ------------------------------------------------------------- 8-bit moments

constexpr int kBlocks = zero::kUnitBlocks;
constexpr int kBlock = ZERO_STATE8_BLOCK;

__device__ __forceinline__ f32x4 e4m3_values(uint32_t w) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
  return f32x4{a[0], a[1], b[0], b[1]};
}

// The nearest e4m3 values (ties to even), one byte each; a NaN or a value
// beyond 464 gives the NaN.
__device__ __forceinline__ uint32_t e4m3_bytes(f32x4 x) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true));
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8(int(byte), 0); }

template <typename T>
__device__ __forceinline__ float pick(const T& x, int k) {
  return k == 0 ? x[0] : k == 1 ? x[1] : k == 2 ? x[2] : x[3];
}

// Bytes `down` and `up` of values just below and just above four exact ones:
// where they differ, a border lies between, and exact(k) (the exact value's
// magnitude, or its square with SQ) decides in fp64; a tie goes to the even byte.
template <bool SQ, typename F>
__device__ __forceinline__ uint32_t decide(uint32_t down, uint32_t up, F exact) {
  for (uint32_t diff = down ^ up; diff != 0;) {
    const int k = (__ffs(int(diff)) - 1) >> 3;
    const uint32_t byte = 0xFFu << (8 * k);
    const uint32_t lo = (down >> (8 * k)) & 0xFFu, hi = (up >> (8 * k)) & 0xFFu;
    double mid = 0.5 * (fabs(double(e4m3_value(lo))) + fabs(double(e4m3_value(hi))));
    if (SQ) mid *= mid;
    const double z = exact(k);
    if (z > mid || (z == mid && (lo & 1u))) down = (down & ~byte) | (up & byte);
    diff &= ~byte;
  }
  return down;
}

// The fp32 values that are rounded to bytes are off by at most 2^-22 of
// themselves: the bytes of x * (1 - 2^-21) and x * (1 + 2^-21) agree unless a
// border is that near (one element in 10^5). Roots of zero are not rare where
// rows get no gradients, and v_bytes looks at each of them again.
constexpr float kBelow = 1.f - 0x1p-21f, kAbove = 1.f + 0x1p-21f;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(x), CTRL, 0xF, 0xF, true));
}

__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Lane of block b's maximum of |m| after block_maxima (kind 0), or of v (kind 1).
__device__ __forceinline__ constexpr int lane_of(int b, int kind) {
  return 16 * (b == 1 ? 2 : b == 2 ? 1 : b) + 8 * kind;
}

// Wave-wide maxima of eight non-negative floats (as bits, which order alike)
// per lane: am[b] and av[b] of four blocks. Each exchange folds two values'
// halves into one register, so eight reductions take 21 instructions and end
// with the maximum of block b in the eight lanes from lane_of(b, kind) on.
__device__ __forceinline__ uint32_t block_maxima(const uint32_t am[4], const uint32_t av[4]) {
  uint32_t r[4], s[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // low half-wave: the pair's first, high half: its second
    const uint32_t x = i < 2 ? am[2 * i] : av[2 * i - 4], y = i < 2 ? am[2 * i + 1] : av[2 * i - 3];
    const auto sw = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    r[i] = max_u(sw[0], sw[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // even rows: the pair's first register, odd rows: its second
    const auto sw = __builtin_amdgcn_permlane16_swap(r[2 * i], r[2 * i + 1], false, false);
    s[i] = max_u(sw[0], sw[1]);
  }
  const uint32_t a = max_u(s[0], dpp<0x128>(s[0])), b = max_u(s[1], dpp<0x128>(s[1]));   // row_ror:8
  uint32_t x = (threadIdx.x & 8) ? b : a;
  x = max_u(x, dpp<0x141>(x));   // row_half_mirror
  x = max_u(x, dpp<0x4E>(x));    // quad_perm [2, 3, 0, 1]
  return max_u(x, dpp<0xB1>(x)); // quad_perm [1, 0, 3, 2]
}

// The largest |m| and v of this lane's four. NaN is ignored (fmaxf).
__device__ __forceinline__ void lane_maxima(const float m[4], const float v[4], uint32_t& am, uint32_t& av) {
  am = __float_as_uint(fmaxf(fmaxf(fmaxf(fabsf(m[0]), fabsf(m[1])), fmaxf(fabsf(m[2]), fabsf(m[3]))), 0.f));
  av = __float_as_uint(fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), 0.f));
}

__device__ __forceinline__ float finite_or_0(float x) { return x < __builtin_inff() ? x : 0.f; }

constexpr float kE4M3Max = 448.f;
// The smallest maxima that scales are formed from: 448 / max stays finite, and
// the root's maximum comes from a square that is normal in fp32.
constexpr float kLeastMax = 0x1p-100f, kLeastRoot = 0x1p-63f;

__device__ __forceinline__ float lane_f32(float x, int lane) {
  return __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(x)), lane)));
}

// Scales of up to four blocks, every lane holding those of its own eight-lane
// group (lane_of); scale = max / 448, up = 448 / max.
struct Scales {
  float scale, up;
};

// m, v: this lane's moments of NB blocks as fp32. Writes the scales of the
// blocks that exist.
template <int NB>
__device__ __forceinline__ Scales block_scales(const float m[NB][4], const float v[NB][4], float* m_scale,
                                               float* v_scale, int64_t block0, int64_t n_blocks) {
  uint32_t am[kBlocks] = {}, av[kBlocks] = {};
#pragma unroll
  for (int b = 0; b < NB; ++b) lane_maxima(m[b], v[b], am[b], av[b]);
  uint32_t top = block_maxima(am, av);
  if (__any(top >= 0x7F800000u)) {   // an infinite moment: the maxima again, without it
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float fm[4], fv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        fm[k] = finite_or_0(fabsf(m[b][k]));
        fv[k] = finite_or_0(v[b][k]);
      }
      lane_maxima(fm, fv, am[b], av[b]);
    }
    top = block_maxima(am, av);
  }
  const int lane = threadIdx.x & 63;
  const bool root = lane & 8;
  const float x = __uint_as_float(top);
  const float t = root ? fmaxf(sqrtf(x), kLeastRoot) : fmaxf(x, kLeastMax);
  const Scales s{t / kE4M3Max, kE4M3Max / t};
  const int row = lane >> 4, b = row == 1 ? 2 : row == 2 ? 1 : row;
  const int64_t block = block0 + b;
  if ((lane & 7) == 0 && b < NB && block < n_blocks) ((ZERO_GLOBAL float*)(root ? v_scale : m_scale))[block] = s.scale;
  return s;
}

// m, in units of the scale, to bytes. mf: fp32 of m; exact(k): the fp64 m[k].
template <typename F>
__device__ __forceinline__ uint32_t m_bytes(const float mf[4], float up, F exact) {
  f32x4 lo, hi;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float y = mf[k] * up;
    lo[k] = y * kBelow;
    hi[k] = y * kAbove;
  }
  const uint32_t down = e4m3_bytes(lo), above = e4m3_bytes(hi);
  return decide<false>(down, above, [&](int j) { return fabs(exact(j)) * double(up); });
}

// sqrt(v), in units of the scale, to bytes; y[k]: that root in fp32, for the
// update, off by up to 2^-63 units where its square is subnormal. vf: fp32 of
// v; exact(k): the fp64 v[k], which every zero byte asks for, and every element
// of a block of tiny roots or of zeros only. In the step it comes from memory
// again: 24.3 M elements take 72 us, 98 with half of the blocks zero and 131
// with all of them (119 M, fp32 gradients: 361, 563, 787).
template <typename F>
__device__ __forceinline__ uint32_t v_bytes(const float vf[4], float up, float y[4], F exact) {
  const auto square = [&](int j) { return exact(j) * (double(up) * double(up)); };
  f32x4 lo, hi;
  if (up < 0x1p52f) {
    // vf * up^2, rounded three times, then the root within one unit in the
    // last place: off by less than 2^-22. Where vf is subnormal the root is
    // under 2^-11 units, half of the least byte's border.
    const float up2 = up * up;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __builtin_amdgcn_sqrtf(vf[k] * up2);
  } else {   // a block whose largest root is under 2^-43: up^2 may pass fp32, vf may be subnormal
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __builtin_amdgcn_sqrtf(float(square(k)));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lo[k] = y[k] * kBelow;
    hi[k] = y[k] * kAbove;
  }
  const uint32_t below = e4m3_bytes(lo), above = e4m3_bytes(hi);
  uint32_t bytes = decide<true>(below, above, square);
  // a zero byte (0x80 in `zeros`): a root above zero is stored as the least value
  for (uint32_t zeros = (bytes - 0x01010101u) & ~bytes & 0x80808080u; zeros != 0; zeros &= zeros - 1) {
    const int k = (__ffs(int(zeros)) - 1) >> 3;
    if (((bytes >> (8 * k)) & 0xFFu) == 0 && exact(k) > 0.0) bytes |= 1u << (8 * k);
  }
  return bytes;
}

// ------------------------------------------------------------------ kernels

__global__ __launch_bounds__(256) void tensors_upload_kernel(const UploadArgs a) {
  for (int i = threadIdx.x; i < a.n; i += 256) a.dst[i] = a.w[i];
}

// Sums of squares. A wave takes a chunk of 4096 elements of one tensor, a lane
// 16 bytes of it at a time: VE elements. Bound by the reads: 119 M bf16
// gradients in 37 us, 6.4 TB/s, and 4 us for the final sum over the partials;
// 24.3 M fp32 20 us a call. (In chunks of 2048 and 1024, where finding the
// tensor takes most of a wave's life, 47 and 62 us a call against 45. One block
// and one launch instead of two gain 1 us up to some 60 thousand elements and
// lose from 90 thousand on, where one CU squares them in fp64: left out.)
template <typename G>
struct SqChunk {
  static constexpr int VE = 16 / sizeof(G), NV = kSqChunk / (64 * VE);
  u32x4 x[NV];
  G end;   // one of the elements after the last whole 16 bytes

  // The chunk's values from g on, of which `rest` exist (none with g null).
  __device__ __forceinline__ void load(const G* g, int64_t rest) {
    const int lane = threadIdx.x & 63;
    const int n = g == nullptr ? 0 : rest < kSqChunk ? int(rest) : kSqChunk;
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      const int e = (b * 64 + lane) * VE;
      x[b] = u32x4{0u, 0u, 0u, 0u};
      if (e + VE <= n) x[b] = stream_load<words4_any>(g + e);
    }
    end = G(0);
    if (lane < n % VE) end = *(const ZERO_GLOBAL G*)(g + (n - n % VE + lane));
  }

  __device__ __forceinline__ double add(double acc) const {
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      if constexpr (sizeof(G) == 2) acc = sq8(x[b], acc);
      else acc = sq4(__builtin_bit_cast(f32x4, x[b]), acc);
    }
    if constexpr (sizeof(G) == 2) return sq1(end, acc);
    else return fma(double(end), double(end), acc);
  }
};

// One wave per chunk, one partial per block, summed wave by wave. Where a launch
// begins inside a block's chunks, the first wave, which has none, takes the sum
// of the ones before: the block then adds the same values in the same order as
// if one launch held them all.
template <typename G>
__global__ __launch_bounds__(kSqListThreads) void tensors_sqnorm_kernel(const SqArgs a) {
  const int64_t u = a.base + int64_t(blockIdx.x) * kSqListWaves + (threadIdx.x >> 6);
  double acc = 0.0;
  if (u < a.l.u0) {
    if (threadIdx.x == 0) acc = a.partial[0];
  } else if (u < a.l.u1) {
    int start;
    const int t = find_tensor(a.l, __builtin_amdgcn_readfirstlane(int(u)), &start);
    const int64_t base = (u - start) * kSqChunk;
    const G* g = a.grads.template at<const G>(t - a.l.t0);
    SqChunk<G> x;
    x.load(g == nullptr ? g : g + base, uniform_load(&a.l.rec[t].len) - base);
    acc = x.add(acc);
  }
  const double s = block_sum<kSqListThreads>(acc);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = s;
}

// The clip coefficient, in the flat updates' order. Up to 64 sums are read
// eight at a time by scalar loads (one at a time: a chain of memory latencies;
// a lane each and v_readlane: three times the instructions, 576 us against 543
// for the 32-bit step over 119 M elements).
__device__ __forceinline__ double list_clip(const StepConst& c) {
  if (!c.clip_on) return 1.0;
  if (c.n_ranks > 64) {
    AdamWArgs a{};
    a.clip_on = 1;
    a.n_ranks = c.n_ranks;
    a.rank_sq = c.rank_sq;
    a.max_norm = c.max_norm;
    a.clip_eps = c.clip_eps;
    return clip_coefficient(a);
  }
  double G = 0.0;
  int r = 0;
  for (; r + 8 <= c.n_ranks; r += 8) {
    double x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = uniform_load(c.rank_sq + r + k);
#pragma unroll
    for (int k = 0; k < 8; ++k) G += x[k];
  }
  for (; r < c.n_ranks; ++r) G += uniform_load(c.rank_sq + r);
  const double ratio = c.max_norm / (sqrt(G) + c.clip_eps);
  return ratio >= 1.0 ? 1.0 : ratio;   // a NaN ratio stays NaN
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

// The 8-bit state from block b0 of a unit on: this lane's first byte of each
// moment, the tensor's scales, the block's index and the number of blocks.
struct State8 {
  uint8_t *m, *v;
  float *m_scale, *v_scale;
  int64_t block0, n_blocks;
};

__device__ __forceinline__ State8 state8_of(const ListRange& l, const Unit& w, int b0) {
  const zero_tensor* r = l.rec + w.t;
  const int64_t e = w.base + b0 * kBlock + 4 * int(threadIdx.x & 63);
  return State8{static_cast<uint8_t*>(uniform_load(&r->m)) + e, static_cast<uint8_t*>(uniform_load(&r->v)) + e,
                uniform_load(&r->m_scale), uniform_load(&r->v_scale), w.base / kBlock + b0,
                (w.base + w.rest + kBlock - 1) / kBlock};
}

// The stored scales of NB blocks: of m in lanes 0-3, of the roots in lanes 4-7.
template <int NB>
__device__ __forceinline__ float old_scales(const State8& s) {
  const int lane = threadIdx.x & 63;
  const int64_t block = s.block0 + (lane & 3);
  if (lane >= 8 || (lane & 3) >= NB || block >= s.n_blocks) return 0.f;
  return ((const ZERO_GLOBAL float*)(lane < 4 ? s.m_scale : s.v_scale))[block];
}

// Calls work.run<NB, FULL>(b): NB blocks from b on, of which all are full, or some
// reach beyond the tensor's end. A wave takes its blocks at once, except that the
// four of a partial unit come in turn: a second copy of the code for four would
// not fit the instruction cache beside the first (8-bit step of 24.3 M elements
// 67 us instead of 63).
template <int WAVES, typename W>
__device__ __forceinline__ void over_unit(const Unit& w, const W& work) {
  constexpr int NB = kBlocks / WAVES;
  const int64_t rest = w.rest - w.block * kBlock;
  if (NB > 1 && rest >= NB * kBlock) {
    work.template run<NB, true>(w.block);
  } else if constexpr (NB < kBlocks) {
    if (rest > 0) work.template run<NB, false>(w.block);
  } else {
#pragma unroll 1
    for (int b = 0; b * kBlock < rest; ++b) work.template run<1, false>(b);
  }
}

// The 32-bit step, one wave to a block of 256 elements (four blocks a wave:
// 574 us against 563 when that was chosen). P: uint16_t (bf16 parameters and an
// fp32 master) or float (its own master). Bound by HBM: 119 M elements in
// 522 us, 6.4 TB/s, with no byte read or written twice. The blocks lie by the
// master's 128-byte lines (line_phase): with blocks by the tensor's first
// element, waves on different XCDs write parts of the same lines, and tensors
// packed without gaps take 730 us instead of 555.
template <typename P, typename G>
__global__ __launch_bounds__(kListThreads) void tensors_adamw_kernel(const StepArgs a) {
  const Unit w = my_unit<4>(a.l);
  const zero_tensor* r = a.l.rec + w.t;
  P* param = static_cast<P*>(uniform_load(&r->param));
  float* master = sizeof(P) == 4 ? reinterpret_cast<float*>(param) : uniform_load(&r->master);
  const int lead = zero::line_phase(uintptr_t(master));
  const int64_t e0 = w.base + w.block * kBlock - lead, rest = w.base + w.rest - e0;   // the block's first element
  const G* g = a.grads.template at<const G>(w.t - a.l.t0);
  if (g == nullptr || rest <= 0) return;
  const int lane = threadIdx.x & 63;
  const int64_t e = e0 + 4 * lane;
  const int lo = e < 0 ? e > -4 ? int(-e) : 4 : 0, cnt = e <= -4 ? 0 : count4(rest);
  float *ms = static_cast<float*>(uniform_load(&r->m)) + e, *vs = static_cast<float*>(uniform_load(&r->v)) + e;
  g += e;
  param += e;
  master += e;
  const f32x4 g4 = widen(load4(g, lo, cnt));
  f32x4 p4 = load4(master, lo, cnt), m4 = load4(ms, lo, cnt), v4 = load4(vs, lo, cnt);
  const int group = uniform_load(&r->group);
  const GroupConst& k = a.c.g[group];
  AdamWArgs q{};
  q.beta1 = k.beta1, q.omb1 = k.omb1, q.beta2 = k.beta2, q.omb2 = k.omb2;
  q.lr_wd = k.lr_wd, q.step_size = k.step_size, q.inv_sqrt_bc2 = k.inv_sqrt_bc2, q.eps = k.eps;
  const double c64 = list_clip(a.c);
  const float c = float(c64);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float p1, m1, v1;
    float p = p4[i], m = m4[i], v = v4[i];
    if (adamw_fast(q, c, g4[i], p, m, v, p1, m1, v1)) {
      exact_update(a.c.x[group], c64, g4[i], p, m, v);
      p1 = p, m1 = m, v1 = v;
    }
    p4[i] = p1, m4[i] = m1, v4[i] = v1;
  }
  store4(master, lo, cnt, p4);
  store4(ms, lo, cnt, m4);
  store4(vs, lo, cnt, v4);
  if constexpr (sizeof(P) == 2) store4(param, lo, cnt, p4);
}

// A value loaded once more: the address passes through an empty asm statement,
// so the compiler cannot keep what was loaded from it before.
template <typename T>
__device__ __forceinline__ T reload(const T* p) {
  asm volatile("" : "+v"(p));
  return *(const ZERO_GLOBAL T*)p;
}

// The 8-bit step's fp32 root is off by up to 2^-75 (a subnormal square of a
// moment) and by up to 2^-63 units of the block's scale: a denominator below
// 2^25 of either takes the update in fp64. With eps = 1e-8 that begins at
// blocks whose largest root passes 10^5.
constexpr float kLeastDenom = 0x1p-50f, kLeastUnits = 0x1p-38f;

__device__ __forceinline__ float grad_value(uint16_t g) { return __uint_as_float(uint32_t(g) << 16); }
__device__ __forceinline__ float grad_value(float g) { return g; }

// The 8-bit step of NB blocks from b0 on in one wave: all loads first, then
// the moments in fp64, the blocks' maxima together, then block by block the
// bytes and the update. Four blocks share the eight reductions and keep 16
// loads in flight a lane (one block a wave: 418 us for 119 M elements, two 372,
// four 382, but 24.3 M in 99, 89 and 86 us). Bound by HBM: 119 M elements with
// fp32 gradients in 354 us a call, 6.1 TB/s, 24.3 M packed without gaps in
// 65 us, 6.0 TB/s; some 850 vector instructions per 1024 elements hide under it.
template <typename P, typename G>
struct AdamW8 {
  const ListRange& l;
  const StepConst& step;
  const Unit& w;
  const G* grad;

  template <int NB, bool FULL>
  __device__ __forceinline__ void run(int b0) const {
    const int lane = threadIdx.x & 63;
    const zero_tensor* r = l.rec + w.t;
    const int64_t e = w.base + b0 * kBlock + 4 * lane;
    P* param = static_cast<P*>(uniform_load(&r->param)) + e;
    float* master = sizeof(P) == 4 ? reinterpret_cast<float*>(param) : uniform_load(&r->master) + e;
    const State8 st = state8_of(l, w, b0);
    const G* g = grad + e;
    int cnt[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) cnt[b] = FULL ? 4 : count4(w.rest - (b0 + b) * kBlock);
    decltype(load4(g, 4)) g4[NB];
    f32x4 p4[NB];
    uint32_t m8[NB], s8[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      g4[b] = load4(g + b * kBlock, cnt[b]);
      p4[b] = load4(master + b * kBlock, cnt[b]);
      m8[b] = load4(st.m + b * kBlock, cnt[b]);
      s8[b] = load4(st.v + b * kBlock, cnt[b]);
    }
    const float old = old_scales<NB>(st);
    const int group = uniform_load(&r->group);
    const GroupConst& k = step.g[group];
    const zero::AdamWExact& x = step.x[group];
    const double c = list_clip(step), c1 = x.omb1 * c, c2 = x.omb2 * (c * c);
    // beta1 * M * scale + (1 - beta1) * c * g and beta2 * (S * scale)^2 + (1 - beta2) * (c * g)^2
    const auto first = [&](int b, float value, float gk) {
      const double scaled = x.beta1 * double(lane_f32(old, b));
      return fma(double(value), scaled, c1 * double(gk));
    };
    const auto second = [&](int b, float value, float gk) {
      const double s = double(lane_f32(old, 4 + b)), gd = double(gk);
      return fma(double(value * value), x.beta2 * (s * s), c2 * (gd * gd));   // an e4m3 value's square is exact
    };
    float mf[NB][4], vf[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const f32x4 mv = e4m3_values(m8[b]), sv = e4m3_values(s8[b]), gv = widen(g4[b]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mf[b][i] = float(first(b, mv[i], gv[i]));
        vf[b][i] = float(second(b, sv[i], gv[i]));
      }
      __builtin_amdgcn_sched_barrier(0);   // block by block: all four interleaved take 40 registers more
    }
    const Scales s = block_scales<NB>(mf, vf, st.m_scale, st.v_scale, st.block0, st.n_blocks);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // An element's moments again in fp64, where a byte hangs on them: from
      // memory, so that the gradients and bytes need no registers until here
      // (137 to 149 without this, about 100 with it: four waves a SIMD, not three).
      const auto exact_m = [&](int j) {
        const int at = b * kBlock + j;
        return j < cnt[b] ? first(b, e4m3_value(reload(st.m + at)), grad_value(reload(g + at))) : 0.0;
      };
      const auto exact_v = [&](int j) {
        const int at = b * kBlock + j;
        return j < cnt[b] ? second(b, e4m3_value(reload(st.v + at)), grad_value(reload(g + at))) : 0.0;
      };
      const uint32_t mb = m_bytes(mf[b], lane_f32(s.up, lane_of(b, 0)), exact_m);
      float y[4];
      const uint32_t vb = v_bytes(vf[b], lane_f32(s.up, lane_of(b, 1)), y, exact_v);
      const float v_scale = lane_f32(s.scale, lane_of(b, 1));
      const float least = fmaxf(kLeastDenom, v_scale * kLeastUnits) * k.inv_sqrt_bc2;
      uint32_t tiny = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float denom = fmaf(y[i] * v_scale, k.inv_sqrt_bc2, k.eps);
        const float q = mf[b][i] * __builtin_amdgcn_rcpf(denom);   // the reciprocal within one unit in the last place
        if (denom < least) tiny |= 1u << i;
        p4[b][i] = fmaf(-k.step_size, q, fmaf(-k.lr_wd, p4[b][i], p4[b][i]));
      }
      for (tiny &= (1u << cnt[b]) - 1u; tiny != 0; tiny &= tiny - 1) {
        const int j = __ffs(int(tiny)) - 1;
        const double denom = sqrt(exact_v(j)) / x.sqrt_bc2 + x.eps;
        const float p = float(double(reload(master + b * kBlock + j)) * x.decay - x.step_size * (exact_m(j) / denom));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i == j) p4[b][i] = p;
      }
      store4(master + b * kBlock, cnt[b], p4[b]);
      if constexpr (sizeof(P) == 2) store4(param + b * kBlock, cnt[b], p4[b]);
      store4(st.m + b * kBlock, cnt[b], mb);
      store4(st.v + b * kBlock, cnt[b], vb);
    }
  }
};

template <typename P, typename G, int WAVES>
__global__ __launch_bounds__(kListThreads) void tensors_adamw8_kernel(const StepArgs a) {
  const Unit w = my_unit<WAVES>(a.l);
  const G* g = a.grads.template at<const G>(w.t - a.l.t0);
  if (g != nullptr) over_unit<WAVES>(w, AdamW8<P, G>{a.l, a.c, w, g});
}

// The conversions of NB blocks from b0 on, with the step's rounding and layout.
// Bound by HBM: the import of 105 M elements takes 170 us, 6.2 TB/s; the export of
// 24.3 M into arrays off 128-byte lines 42.5 us, 5.7 TB/s (4 % more bytes
// written than asked for: both ends' waves write the lines they share).
struct Import8 {
  const ListRange& l;
  const Unit& w;
  const float *m32, *v32;

  template <int NB, bool FULL>
  __device__ __forceinline__ void run(int b0) const {
    const int64_t e = w.base + b0 * kBlock + 4 * int(threadIdx.x & 63);
    const State8 st = state8_of(l, w, b0);
    int cnt[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) cnt[b] = FULL ? 4 : count4(w.rest - (b0 + b) * kBlock);
    float m[NB][4], v[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const f32x4 m4 = load4(m32 + e + b * kBlock, cnt[b]), v4 = load4(v32 + e + b * kBlock, cnt[b]);
#pragma unroll
      for (int i = 0; i < 4; ++i) m[b][i] = m4[i], v[b][i] = v4[i];
    }
    const Scales s = block_scales<NB>(m, v, st.m_scale, st.v_scale, st.block0, st.n_blocks);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float y[4];
      store4(st.m + b * kBlock, cnt[b],
             m_bytes(m[b], lane_f32(s.up, lane_of(b, 0)), [&](int j) { return double(pick(m[b], j)); }));
      store4(st.v + b * kBlock, cnt[b],
             v_bytes(v[b], lane_f32(s.up, lane_of(b, 1)), y, [&](int j) { return double(pick(v[b], j)); }));
    }
  }
};

template <int WAVES>
__global__ __launch_bounds__(kListThreads) void tensors_import_kernel(const State8Args a) {
  const Unit w = my_unit<WAVES>(a.l);
  const float *m32 = a.m.at<const float>(w.t - a.l.t0), *v32 = a.v.at<const float>(w.t - a.l.t0);
  if (m32 != nullptr) over_unit<WAVES>(w, Import8{a.l, w, m32, v32});
}

struct Export8 {
  const ListRange& l;
  const Unit& w;
  float *m32, *v32;

  template <int NB, bool FULL>
  __device__ __forceinline__ void run(int b0) const {
    const int64_t e = w.base + b0 * kBlock + 4 * int(threadIdx.x & 63);
    const State8 st = state8_of(l, w, b0);
    int cnt[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) cnt[b] = FULL ? 4 : count4(w.rest - (b0 + b) * kBlock);
    uint32_t m8[NB], s8[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      m8[b] = load4(st.m + b * kBlock, cnt[b]);
      s8[b] = load4(st.v + b * kBlock, cnt[b]);
    }
    const float old = old_scales<NB>(st);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const f32x4 m = e4m3_values(m8[b]), root = e4m3_values(s8[b]);
      const float m_scale = lane_f32(old, b);
      const double s = double(lane_f32(old, 4 + b)), s2 = s * s;
      f32x4 m4, v4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m4[i] = m[i] * m_scale;
        v4[i] = float(double(root[i] * root[i]) * s2);   // an e4m3 value's square is exact
      }
      store4(m32 + e + b * kBlock, cnt[b], m4);
      store4(v32 + e + b * kBlock, cnt[b], v4);
    }
  }
};

template <int WAVES>
__global__ __launch_bounds__(kListThreads) void tensors_export_kernel(const State8Args a) {
  const Unit w = my_unit<WAVES>(a.l);
  float *m32 = a.m.at<float>(w.t - a.l.t0), *v32 = a.v.at<float>(w.t - a.l.t0);
  if (m32 != nullptr) over_unit<WAVES>(w, Export8{a.l, w, m32, v32});
}

// ----------------------------------------------------------------- launches

int launched(const char* who) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(ZERO_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  return zero::ok();
}

// The lowest and the highest address of some tensors, and the bits in which
// any of them differ.
struct Window {
  uintptr_t lo = ~uintptr_t(0), hi = 0, differ = 0;

  int shift() const { return differ == 0 ? 0 : __builtin_ctzll(differ); }

  // Whether p joins without taking the window beyond 32-bit steps.
  bool take(const void* p) {
    if (p == nullptr) return true;
    Window w = *this;
    if (hi != 0) w.differ |= uintptr_t(p) ^ lo;
    w.lo = std::min(lo, uintptr_t(p));
    w.hi = std::max(hi, uintptr_t(p));
    if (((w.hi - w.lo) >> w.shift()) >= kNoTensor) return false;
    *this = w;
    return true;
  }

  template <int N>
  void write(Addresses<N>* out, const void* const* p, int n) const {
    out->base = lo;
    out->shift = uint32_t(shift());
    for (int i = 0; i < n; ++i)
      out->step[i] = p[i] == nullptr ? kNoTensor : uint32_t((uintptr_t(p[i]) - lo) >> out->shift);
  }
};

// Calls go(range) for ranges that cover the list's units (chunks): tensors of one
// run of `most`, as far as fits(t) lets tensor t join the ones before it, and
// kListMaxUnits units each. restart() begins a new set of tensors. The runs
// begin at multiples of `most`, wherever the ranges between them end.
template <typename R, typename F, typename Go>
int for_ranges(const zero_tensors_s* h, bool chunks, int most, R restart, F fits, Go go) {
  const int32_t n = int32_t(h->t.size());
  const zero::Table at(n);
  const char* table = static_cast<const char*>(h->table);
  const int kind = chunks ? 1 : 0;
  const std::vector<int32_t>& counts = h->first[kind];
  ListRange l;
  l.first = reinterpret_cast<const int32_t*>(table + at.first[kind]);
  l.slot = reinterpret_cast<const int32_t*>(table + at.slot[kind]);
  l.rec = reinterpret_cast<const zero_tensor*>(table + at.records);
  l.n_all = n;
  l.shift = h->shift[kind];
  for (int32_t t0 = 0; t0 < n;) {
    restart();
    int32_t t1 = t0;
    while (t1 < n && (t1 == t0 || t1 % most != 0) && (h->t[size_t(t1)].len == 0 || fits(t1))) ++t1;
    const int64_t end = counts[size_t(t1)];
    for (int64_t u = counts[size_t(t0)]; u < end; u += kListMaxUnits) {
      l.t0 = t0, l.n = t1 - t0, l.u0 = int32_t(u), l.u1 = int32_t(std::min(end, u + kListMaxUnits));
      if (int rc = go(l)) return rc;
    }
    t0 = t1;
  }
  return zero::ok();
}

// for_ranges over the gradients' addresses, which go into args->grads.
template <typename A, typename Go>
int for_gradients(const zero_tensors_s* h, bool chunks, const void* const* grads, A* args, Go go) {
  Window w;
  return for_ranges(
      h, chunks, ZERO_TENSORS_PER_LAUNCH, [&] { w = Window(); }, [&](int32_t t) { return w.take(grads[t]); },
      [&](const ListRange& l) {
        args->l = l;
        w.write(&args->grads, grads + l.t0, l.n);
        return go();
      });
}

// Waves that share a unit: four up to kFourWaveUnits, where they are too few to
// fill the chip (8-bit step over 90 units 5.4 us, with two waves 7.1, with one
// 10); two up to kTwoWaveUnits (over 1536 units 7.3 us, with four 8.1, with one
// 8.1), and where so many tensors end inside a unit that the partial units,
// whose blocks one wave takes in turn, set the time (700 tensors of 8000
// elements 21.3 us, with one wave 26.3; of 17243, 12.4 and 14.7; but of 30001,
// 32.2 and 29.8); else one (2048 units 8.4 us, with two 8.7; 24 thousand 63 and 68).
constexpr int64_t kFourWaveUnits = 1024, kTwoWaveUnits = 1792, kUnitsPerPartial = 20;
int waves_of(const zero_tensors_s* h, const ListRange& l) {
  const int64_t units = l.u1 - l.u0;
  if (units <= kFourWaveUnits) return 4;
  const int64_t partial = h->partial[size_t(l.t0) + size_t(l.n)] - h->partial[size_t(l.t0)];
  return units <= kTwoWaveUnits || units <= kUnitsPerPartial * partial ? 2 : 1;
}

// Launches kernel(args), `waves` waves per unit. lds: bytes of LDS a block asks
// for (and does not use), which limits the waves of a CU.
#define ZERO_LIST_LAUNCH(kernel, waves, lds, args, stream)                                                \
  hipLaunchKernelGGL((kernel), dim3(unsigned((args).l.u1 - (args).l.u0) * unsigned(waves)), dim3(kListThreads), \
                     lds, stream, args)

// LDS of the conversions' blocks, against too many waves in flight: with
// 10 KiB, 16 to a CU, the import takes 195 us instead of 204 (119 M elements)
// and the export the same 194; with fp32 arrays that do not start on 128-byte
// lines, whose ends two waves write, the export takes 45.5 us with 16 KiB
// against 50.4 (24.3 M; 215 us against 194 on lines).
constexpr unsigned kConvertLds = 10 << 10, kConvertLdsOffLines = 16 << 10;

// The same of the 32-bit step's: 20 waves to a CU instead of 32 (119 M elements,
// bf16 gradients 527 us without and 520 us, fp32 569 and 560; 24.3 M, 111.5 and
// 110.3).
constexpr unsigned kStep32Lds = 8 << 10;

// LDS of the 8-bit step's blocks in long launches with fp32 gradients, against
// too many waves in flight: by the kernel's registers a CU holds 16; with 16 KiB,
// 10. By the elements of 100 equal tensors, with and without it: 2^25.9, 174 us
// and 168; 2^26.1, 204 and 205; 2^26.5, 278 and 285; 2^27, 387 and 404. Lists of
// several shapes at 84 to 119 M elements gain 1 % in the mean (-3 to 4 %). With
// bf16 gradients, 12 waves gained nothing over the same lists (within 3 %).
constexpr int64_t kLongUnits = int64_t(1) << 16;
template <typename G>
unsigned step8_lds(const ListRange& l) {
  return sizeof(G) == 2 || l.u1 - l.u0 <= kLongUnits ? 0u : 16u << 10;
}

template <typename P, typename G>
void launch_step(const zero_tensors_s* h, const StepArgs& a, hipStream_t stream) {
  const int waves = h->state_bits == 32 ? 0 : waves_of(h, a.l);
  if (waves == 0)
    ZERO_LIST_LAUNCH((tensors_adamw_kernel<P, G>), 4, kStep32Lds, a, stream);
  else if (waves == 4)
    ZERO_LIST_LAUNCH((tensors_adamw8_kernel<P, G, 4>), 4, 0, a, stream);
  else if (waves == 2)
    ZERO_LIST_LAUNCH((tensors_adamw8_kernel<P, G, 2>), 2, 0, a, stream);
  else
    ZERO_LIST_LAUNCH((tensors_adamw8_kernel<P, G, 1>), 1, step8_lds<G>(a.l), a, stream);
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
  const Table at(n);
  std::vector<uint32_t> words(at.bytes / 4, 0u);
  for (int k = 0; k < 2; ++k) {
    const std::vector<int32_t>& first = h->first[k];
    std::memcpy(words.data() + at.first[k] / 4, first.data(), first.size() * sizeof(int32_t));
    int32_t t = 0;
    for (int64_t s = 0; s < kSlots && (s << h->shift[k]) < first.back(); ++s) {
      while (first[size_t(t) + 1] <= (s << h->shift[k])) ++t;
      words[at.slot[k] / 4 + size_t(s)] = uint32_t(t);
    }
  }
  std::memcpy(words.data() + at.records / 4, h->t.data(), h->t.size() * sizeof(zero_tensor));
  for (size_t w = 0; w < words.size(); w += kUploadWords) {
    UploadArgs a;
    a.dst = static_cast<uint32_t*>(table) + w;
    a.n = int32_t(std::min<size_t>(kUploadWords, words.size() - w));
    std::memcpy(a.w, words.data() + w, size_t(a.n) * 4);
    hipLaunchKernelGGL(tensors_upload_kernel, dim3(1), dim3(256), 0, stream, a);
    if (int rc = launched(who)) return rc;
  }
  return ok();
}

int launch_sqnorm(const zero_tensors_s* h, const void* const* grads, double* out, int32_t accumulate, double* ws,
                  hipStream_t stream, const char* who) {
  SqArgs a;
  // The blocks hold four chunks each, counted from the first one of the launch's
  // run of tensors: the lengths alone say which chunks share a block, also where
  // the addresses end a launch between them.
  const std::vector<int32_t>& counts = h->first[1];
  int32_t run = -1;
  int64_t first = 0, n = 0;   // partial sums before the run, and all so far
  const int rc = for_gradients(h, true, grads, &a, [&] {
    if (a.l.t0 / ZERO_TENSORS_PER_LAUNCH != run) {
      run = a.l.t0 / ZERO_TENSORS_PER_LAUNCH;
      first = n;
    }
    const int64_t begin = counts[size_t(run) * ZERO_TENSORS_PER_LAUNCH];
    const int64_t group = (a.l.u0 - begin) / kSqListWaves;
    a.base = int32_t(begin + group * kSqListWaves);
    const int64_t blocks = (a.l.u1 - a.base + kSqListWaves - 1) / kSqListWaves;
    a.partial = ws + first + group;
    n = first + group + blocks;
    if (h->grad_type == ZERO_BF16)
      hipLaunchKernelGGL(tensors_sqnorm_kernel<uint16_t>, dim3(unsigned(blocks)), dim3(kSqListThreads), 0, stream, a);
    else
      hipLaunchKernelGGL(tensors_sqnorm_kernel<float>, dim3(unsigned(blocks)), dim3(kSqListThreads), 0, stream, a);
    return launched(who);
  });
  return rc ? rc : zero_sum_partials(ws, n, out, accumulate, stream);
}

int launch_adamw(const zero_tensors_s* h, const void* const* grads, const StepConst& c, hipStream_t stream,
                   const char* who) {
  StepArgs a;
  a.c = c;
  return for_gradients(h, false, grads, &a, [&] {
    const bool bf16 = h->grad_type == ZERO_BF16;
    if (h->param_type == ZERO_BF16)
      bf16 ? launch_step<uint16_t, uint16_t>(h, a, stream) : launch_step<uint16_t, float>(h, a, stream);
    else
      bf16 ? launch_step<float, uint16_t>(h, a, stream) : launch_step<float, float>(h, a, stream);
    return launched(who);
  });
}

int launch_state8(const zero_tensors_s* h, bool import, const float* const* m, const float* const* v,
                    hipStream_t stream, const char* who) {
  State8Args a;
  Window wm, wv;
  uintptr_t low = 0;
  const auto p = [](const float* const* x) { return reinterpret_cast<const void* const*>(x); };
  return for_ranges(
      h, false, kStatePerLaunch, [&] { wm = wv = Window(), low = 0; },
      [&](int32_t t) {
        low |= uintptr_t(m[t]) | uintptr_t(v[t]);
        return wm.take(m[t]) && wv.take(v[t]);
      },
      [&](const ListRange& l) {
        a.l = l;
        wm.write(&a.m, p(m) + l.t0, l.n);
        wv.write(&a.v, p(v) + l.t0, l.n);
        const unsigned lds = import || low % 128 == 0 ? kConvertLds : kConvertLdsOffLines;
        const int waves = waves_of(h, l);
        if (import && waves == 4)
          ZERO_LIST_LAUNCH(tensors_import_kernel<4>, 4, 0, a, stream);
        else if (import && waves == 2)
          ZERO_LIST_LAUNCH(tensors_import_kernel<2>, 2, 0, a, stream);
        else if (import)
          ZERO_LIST_LAUNCH(tensors_import_kernel<1>, 1, lds, a, stream);
        else if (waves == 4)
          ZERO_LIST_LAUNCH(tensors_export_kernel<4>, 4, 0, a, stream);
        else if (waves == 2)
          ZERO_LIST_LAUNCH(tensors_export_kernel<2>, 2, 0, a, stream);
        else
          ZERO_LIST_LAUNCH(tensors_export_kernel<1>, 1, lds, a, stream);
        return launched(who);
      });
}

}  // namespace zero
