// Kernels of the token-table and norm calls (zero_layers.h) and their launches.
// Part of device.hip, after tensors.hip.
//
//   embedding_kernel         rows of a table, scaled
//   order_rank_kernel        the sort of few tokens, by counting
//   order_split_kernel       of some thousand, a range of rows a block
//   order_count_kernel, order_scan_kernel, order_scatter_kernel
//                            one pass of the sort of many tokens
//   embedding_grad_kernel    sums of pieces of the sorted tokens, and zeros for
//                            the rows without one
//   embedding_join_kernel    the sums of runs that several pieces share
//   embedding_grad_few_kernel  both in one launch
//   norm_kernel, norm_long_kernel
//                            the norm of rows in registers, and of longer ones
//   norm_grad_kernel, norm_grad_few_kernel, norm_grad_long_kernel,
//   norm_grad_columns_kernel, norm_grad_join_kernel
//                            its gradient
//
// All of them do a few operations per byte, so long ones are bound by HBM (this library's
// copy of 0.5 GB reaches 6.2 TB/s, a fill 6.6) and short ones by their launches
// (2.4 us of the GPU's time each at least, 3.2 us of the host's). What is read or
// written once is not kept in the caches (cached stores: the norm of 16384 x 8192 97 us
// instead of 94, its gradient over 16384 x 2944 79 instead of 75); weights, tokens and
// partial sums are. Times are those of one MI355X: of a call among others, or of a
// kernel where one is named.
#include <type_traits>

#include "layers_internal.h"

namespace {

using zero::kSortBits;
using zero::kSortBlock;
using zero::kSortDigits;
using zero::kSortItems;
using zero::kSortThreads;
using zero::grad_threads;
using zero::NormShape;
using zero::Order;

// ------------------------------------------------------- E elements of a row
//
// A row is cut into vectors of E elements, one a lane. Its last lane takes the
// row's last E elements, of which the first `lo` are the neighbour's: so every
// lane's load is one instruction that no branch guards (a guarded one has to wait
// for those before it), also of a lane with nothing to do, whose lo is E. Rows
// start at any element, so the accesses are declared with their element's
// alignment: the hardware takes them at any address. Rows shorter than a vector go
// with E = 1.

struct Span {
  int col, lo;         // elements [col + lo, col + E) of the row are the lane's
};
template <int E>
__device__ __forceinline__ Span span_of(int vector, int dim) {
  const int over = max(0, vector * E + E - dim);
  return {vector * E - over, min(over, E)};
}

template <int E, typename T> struct Words;
template <> struct Words<8, uint16_t> { u32x4 w; };
template <> struct Words<4, uint16_t> { u32x2 w; };
template <> struct Words<1, uint16_t> { uint16_t w; };
template <> struct Words<4, float> { f32x4 w; };
template <> struct Words<8, float> { f32x4 w, w2; };
template <> struct Words<1, float> { float w; };

template <typename V>
__device__ __forceinline__ V plain_load(const void* p) { return *(const ZERO_GLOBAL V*)p; }
template <typename V>
__device__ __forceinline__ void plain_store(void* p, V x) { *(ZERO_GLOBAL V*)p = x; }

// The E elements at p; STREAM: not kept in the caches.
template <int E, bool STREAM, typename T>
__device__ __forceinline__ Words<E, T> load_vector(const T* p) {
  Words<E, T> r;
  if constexpr (E == 1) {
    r.w = STREAM ? stream_load<T>(p) : plain_load<T>(p);
  } else if constexpr (sizeof(T) == 2 && E == 8) {
    r.w = STREAM ? stream_load<words4_any>(p) : plain_load<words4_any>(p);
  } else if constexpr (sizeof(T) == 2) {
    r.w = STREAM ? stream_load<bf16x4_any>(p) : plain_load<bf16x4_any>(p);
  } else {
    r.w = STREAM ? stream_load<f32x4_any>(p) : plain_load<f32x4_any>(p);
    if constexpr (E == 8) r.w2 = STREAM ? stream_load<f32x4_any>(p + 4) : plain_load<f32x4_any>(p + 4);
  }
  return r;
}

template <int E, bool STREAM, typename T>
__device__ __forceinline__ void store_vector(T* p, const Words<E, T>& r) {
  const auto put = [](void* to, auto any, auto x) {
    if constexpr (STREAM) stream_store<decltype(any)>(to, x);
    else plain_store<decltype(any)>(to, x);
  };
  if constexpr (E == 1) put(p, T(), r.w);
  else if constexpr (sizeof(T) == 2 && E == 8) put(p, words4_any(), r.w);
  else if constexpr (sizeof(T) == 2) put(p, bf16x4_any(), r.w);
  else put(p, f32x4_any(), r.w);
  if constexpr (sizeof(T) == 4 && E == 8) put(p + 4, f32x4_any(), r.w2);
}

template <int E, typename T>
__device__ __forceinline__ void widen(const Words<E, T>& r, float (&x)[E]) {
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if constexpr (E == 1 && sizeof(T) == 2) x[k] = bf16_lo(r.w);
    else if constexpr (E == 1) x[k] = r.w;
    else if constexpr (sizeof(T) == 2) x[k] = (k & 1) ? bf16_hi(r.w[k >> 1]) : bf16_lo(r.w[k >> 1]);
    else if constexpr (E == 8) x[k] = k < 4 ? r.w[k & 3] : r.w2[k & 3];
    else x[k] = r.w[k];
  }
}

// x rounded to the type.
template <int E, typename T>
__device__ __forceinline__ Words<E, T> narrow(const float (&x)[E]) {
  Words<E, T> r;
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if constexpr (E == 1 && sizeof(T) == 2) r.w = to_bf16(x[k]);
    else if constexpr (E == 1) r.w = x[k];
    else if constexpr (sizeof(T) == 2) { if ((k & 1) == 0) r.w[k >> 1] = pack_bf16x2(x[k], x[k + 1]); }
    else if constexpr (E == 8) { if (k < 4) r.w[k & 3] = x[k]; else r.w2[k & 3] = x[k]; }
    else r.w[k] = x[k];
  }
  return r;
}

// The elements [lo, hi) of the E at p, zeros beside them.
template <int E, typename T>
__device__ __forceinline__ Words<E, T> load_some(const T* p, int lo, int hi) {
  Words<E, T> r{};
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if (k < lo || k >= hi) continue;
    if constexpr (E == 1) r.w = p[k];
    else if constexpr (sizeof(T) == 2) r.w[k >> 1] |= uint32_t(p[k]) << (16 * (k & 1));
    else r.w[k] = p[k];
  }
  return r;
}

template <int E, typename T>
__device__ __forceinline__ void store_some(T* p, int lo, int hi, const Words<E, T>& r) {
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if (k < lo || k >= hi) continue;
    if constexpr (E == 1) p[k] = r.w;
    else if constexpr (sizeof(T) == 2) p[k] = uint16_t(r.w[k >> 1] >> (16 * (k & 1)));
    else if constexpr (E == 8) p[k] = k < 4 ? r.w[k & 3] : r.w2[k & 3];
    else p[k] = r.w[k];
  }
}

// The lane's vector of the row at p, the neighbour's elements included.
template <int E, bool STREAM = true, typename T>
__device__ __forceinline__ Words<E, T> load_row(const T* p, const Span& s) {
  return load_vector<E, STREAM>(p + s.col);
}

template <int E, bool STREAM = true, typename T>
__device__ __forceinline__ void store_row(T* p, const Span& s, const Words<E, T>& r) {
  if (s.lo == 0) store_vector<E, STREAM>(p + s.col, r);
  else store_some<E, T>(p + s.col, s.lo, E, r);
}

// The neighbour's elements zeroed.
template <int E>
__device__ __forceinline__ void only_own(const Span& s, float (&x)[E]) {
  if (s.lo > 0)
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = k < s.lo ? 0.f : x[k];
}

// ------------------------------------------------------------------- lookup

// A token's row, or `rows` for one outside the table.
template <typename I>
__device__ __forceinline__ int table_row(I token, int rows) {
  return token >= 0 && token < I(rows) ? int(token) : rows;
}

// A wave takes a tile of 64 vectors of four rows: the rows are known to the whole wave
// (scalar loads), and four loads are in flight. 16384 rows of 4096 fp32, to bf16: 41 us,
// 5.2 TB/s of what has to move; bound by HBM.
constexpr int kLookupRows = 4;

template <typename I, typename T, typename O, int E>
__global__ __launch_bounds__(256) void embedding_kernel(const I* __restrict__ tokens, int n, const T* __restrict__ table,
                                                        int rows, int dim, int tiles, float scale, O* __restrict__ out,
                                                        int64_t stride) {
  const uint32_t w = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = int64_t(w / uint32_t(tiles)) * kLookupRows;
  if (t0 >= n) return;
  const Span s = span_of<E>(int(w % uint32_t(tiles)) * 64 + int(threadIdx.x & 63), dim);
  int row[kLookupRows];
  Words<E, T> x[kLookupRows];
#pragma unroll
  for (int k = 0; k < kLookupRows; ++k) row[k] = table_row(uniform_load(tokens + min(t0 + k, int64_t(n - 1))), rows);
#pragma unroll
  for (int k = 0; k < kLookupRows; ++k)
    x[k] = load_row<E, false>(table + int64_t(row[k] < rows ? row[k] : 0) * dim, s);
#pragma unroll
  for (int k = 0; k < kLookupRows; ++k) {
    if (t0 + k >= n) break;
    float v[E];
    widen<E, T>(x[k], v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = row[k] < rows ? v[e] * scale : 0.f;
    store_row<E>(out + (t0 + k) * stride, s, narrow<E, O>(v));
  }
}

// --------------------------------------------------------------------- sort

// Few tokens: a token's place is the number of tokens before it, those of lower
// rows and those of its own row at lower positions: n^2 comparisons. Row numbers
// are exact in fp32, where a comparison and its count are two instructions that
// need no wait between them: the difference clamped to [0, 1], and the sum. A
// block takes 32 tokens, two in each of 16 lanes; its 64 such groups take a part
// of the tokens to compare with each, from LDS. 512 tokens 3.9 us, 8192 8.5 us, bound by
// the comparisons from some 4000 on (compared and counted as integers 12.4 us: each
// comparison's mask takes two idle cycles to reach the count). Passes over digits take
// 18 us at 12288 tokens, this 16; beyond 4096 only tables too long for
// order_split_kernel come here.
constexpr int kRankThreads = 1024, kRankParts = kRankThreads / 16, kRankEach = 32;
static_assert(ZERO_LAYER_ROWS < 1 << 24, "rows and counts are exact in fp32");

template <typename I>
__global__ __launch_bounds__(kRankThreads) void order_rank_kernel(const I* __restrict__ tokens, int n, int rows,
                                                                  int32_t* __restrict__ row, int32_t* __restrict__ pos) {
  __shared__ alignas(16) float key[zero::kRankTokens + 4 * kRankParts];
  __shared__ float part[kRankThreads / 64][kRankEach];
  const int t = threadIdx.x, lane = t & 63;
  // a group's part: whole fours of tokens
  const int each = ((n + kRankParts - 1) / kRankParts + 3) / 4 * 4;
  constexpr int kLoads = int(zero::kRankTokens) / kRankThreads;
  I token[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k)       // not guarded one by one: all are on their way at once
    if (k * kRankThreads < n) token[k] = tokens[min(k * kRankThreads + t, n - 1)];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = k * kRankThreads + t;
    if (i < each * kRankParts) key[i] = i < n ? float(table_row(token[k], rows)) : 0x1p30f;
  }
  __syncthreads();
  const int i0 = int(blockIdx.x) * kRankEach;
  const int i[2] = {i0 + (t & 15), i0 + 16 + (t & 15)};
  const float mine[2] = {i[0] < n ? key[i[0]] : 0.f, i[1] < n ? key[i[1]] : 0.f};
  const int j0 = (t >> 4) * each, j1 = j0 + each;
  // before the block's tokens an equal row counts, behind them it does not
  const int before = min(max(i0, j0), j1), behind = max(min(i0 + kRankEach, j1), before);
  float place[2] = {0.f, 0.f};
  const auto count = [&](int from, int to, auto limit) {       // limit: of token h against the one at j
#pragma unroll 4
    for (int j = from; j < to; j += 4) {
      const f32x4 k = *reinterpret_cast<const f32x4*>(&key[j]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) place[h] += __builtin_amdgcn_fmed3f(limit(h, j + e) - k[e], 0.f, 1.f);
    }
  };
  const float after[2] = {mine[0] + 1.f, mine[1] + 1.f};
  count(j0, before, [&](int h, int) { return after[h]; });
  count(before, behind, [&](int h, int j) { return j < i[h] ? after[h] : mine[h]; });
  count(behind, j1, [&](int h, int) { return mine[h]; });
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    place[h] += __shfl_xor(place[h], 16, 64);
    place[h] += __shfl_xor(place[h], 32, 64);
    if (lane < 16) part[t >> 6][h * 16 + lane] = place[h];
  }
  __syncthreads();
  if (t < kRankEach && i0 + t < n) {
    float at = 0.f;
#pragma unroll
    for (int k = 0; k < kRankThreads / 64; ++k) at += part[k][t];
    row[int(at)] = int(key[i0 + t]);
    pos[int(at)] = i0 + t;
  }
}

// Some thousand tokens: each of up to 256 blocks takes `each` consecutive rows, reads all
// tokens and keeps those of its rows; they go behind the tokens of lower rows, which it
// counts. One launch, and no counts between blocks. A wave's tokens are consecutive: it
// lists those that are kept, ranks them 64 at a time among those of their row (lanes
// with the same bits), and the block sorts them in LDS and stores them in order.
// us for 50257 rows, and where one block has all tokens (150 rows): 6000 tokens 5.9 and
// 8.9, 8192 6.3 and 10.3, 12288 8.2 and 15.4, 16384 9.2 and 18.1; by counting 4096 5.6,
// 8192 8.5, 12288 16; in passes 16384 18. Bound by the reading and listing of all tokens
// by every block. 32768 tokens 16.3 and 36.4, in passes 19.5: left to these. Rows beyond
// 512 a block go the other ways. Stored unsorted, 16384 tokens of one block took 28.
constexpr int64_t kSplitFrom = 4096, kSplitTokens = 16384;
constexpr int kSplitThreads = 1024, kSplitWaves = kSplitThreads / 64, kSplitBlocks = 256, kSplitEach = 512;
static_assert(kSplitEach <= 1 << 16 && kSplitTokens <= 1 << 16, "16 bits each in a list's entry");

// The lower 32 bits of a token, all ones where it has more: larger than any row, as a
// negative one is.
__device__ __forceinline__ uint32_t low_word(int32_t token) { return uint32_t(token); }
__device__ __forceinline__ uint32_t low_word(int64_t token) {
  return uint32_t(uint64_t(token) >> 32) == 0 ? uint32_t(token) : ~0u;
}

template <typename I, int N>
__global__ __launch_bounds__(kSplitThreads) void order_split_kernel(const I* __restrict__ tokens, int n, int rows, int each,
                                                                    int bits, int32_t* __restrict__ row_out,
                                                                    int32_t* __restrict__ pos_out) {
  __shared__ uint32_t list[kSplitWaves][64 * N];         // the wave's tokens that are the block's: position and row - lo
  __shared__ uint32_t seen[kSplitWaves][kSplitEach / 2]; // how many of a row, two in a word; then where they begin
  __shared__ int32_t lower_sum[kSplitWaves], wave_sum[kSplitWaves];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lo = int(blockIdx.x) * each, first = wave * 64 * N;
  I x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = tokens[min(first + k * 64 + lane, n - 1)];
  for (int k = t; k < kSplitWaves * kSplitEach / 2; k += kSplitThreads) (&seen[0][0])[k] = 0;
  int lower = 0, mine = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int left = min(max(n - first - k * 64, 0), 64);
    const uint64_t valid = left == 0 ? 0 : ~uint64_t(0) >> (64 - left);
    const uint32_t r = min(low_word(x[k]), uint32_t(rows)), key = r - uint32_t(lo);
    lower += __popcll(__ballot(r < uint32_t(lo)) & valid);
    const uint64_t there = __ballot(key < uint32_t(each)) & valid;
    if (there == 0) continue;
    if ((there >> lane) & 1)
      list[wave][mine + __popcll(there & ((uint64_t(1) << lane) - 1))] = key << 16 | uint32_t(first + k * 64 + lane);
    mine += __popcll(there);
  }
  if (lane == 0) lower_sum[wave] = lower;
  __syncthreads();
  uint32_t at[N];
  constexpr int kAtOnce = 2;
#pragma unroll
  for (int k0 = 0; k0 < N; k0 += kAtOnce) {
    if (k0 * 64 >= mine) continue;
    uint32_t d[kAtOnce], like[kAtOnce][2];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int i = (k0 + k) * 64 + lane;
      d[k] = list[wave][min(i, mine - 1)] >> 16;
      const uint64_t there = __ballot(i < mine);
      like[k][0] = uint32_t(there);
      like[k][1] = uint32_t(there >> 32);
    }
    for (int b = 0; b < bits; ++b) {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const uint32_t bit = -(d[k] >> b & 1);           // of all lanes those with the same one
        const uint64_t m = __ballot(bit != 0);
        like[k][0] &= ~(uint32_t(m) ^ bit);
        like[k][1] &= ~(uint32_t(m >> 32) ^ bit);
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t before = __builtin_amdgcn_mbcnt_hi(like[k][1], __builtin_amdgcn_mbcnt_lo(like[k][0], 0));
      // a wave's accesses to LDS are in order: what is read are the tokens of the earlier steps
      at[k0 + k] = (seen[wave][d[k] / 2] >> (d[k] % 2 * 16) & 0xffff) + before;
      __builtin_amdgcn_wave_barrier();
      if (before == 0 && (k0 + k) * 64 + lane < mine)
        atomicAdd(&seen[wave][d[k] / 2], uint32_t(__popc(like[k][0]) + __popc(like[k][1])) << (d[k] % 2 * 16));
      __builtin_amdgcn_wave_barrier();
    }
  }
  __syncthreads();
  // a row a thread
  using Half = uint16_t __attribute__((may_alias));
  const auto half = [&](int w, uint32_t d) -> Half& { return reinterpret_cast<Half*>(seen[w])[d]; };
  int total = 0;
  if (t < each)
#pragma unroll
    for (int w = 0; w < kSplitWaves; ++w) total += half(w, t);
  int up = total;
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(up, off, 64);
    if (lane >= off) up += y;
  }
  if (lane == 63) wave_sum[wave] = up;
  __syncthreads();
  int below = 0;
#pragma unroll
  for (int w = 0; w < kSplitWaves; ++w) below += lower_sum[w];
  if (t < each) {
    int begin = up - total;
    for (int w = 0; w < wave; ++w) begin += wave_sum[w];
#pragma unroll
    for (int w = 0; w < kSplitWaves; ++w) {
      const int c = half(w, t);
      half(w, t) = uint16_t(begin);
      begin += c;
    }
  }
  int count = 0;
#pragma unroll
  for (int w = 0; w < kSplitWaves; ++w) count += wave_sum[w];
  uint32_t v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k * 64 < mine) v[k] = list[wave][min(k * 64 + lane, mine - 1)];
  }
  __syncthreads();
  // sorted in LDS, so that what is stored is consecutive
  uint32_t* const sorted = &list[0][0];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (k * 64 + lane < mine) sorted[half(wave, v[k] >> 16) + at[k]] = v[k];
  }
  __syncthreads();
  for (int i = t; i < count; i += kSplitThreads) {
    const uint32_t x = sorted[i];
    row_out[below + i] = lo + int(x >> 16);
    pos_out[below + i] = int(x & 0xffff);
  }
}

// Many tokens: passes over the row numbers' digits of up to 9 bits from the
// lowest on, each of which keeps the order of equal digits. A pass counts the
// digits of every block's 2048 tokens, then places every token behind those of
// lower digits, those of earlier blocks and those before it in its block. Two passes
// for up to 2^18 - 1 rows: 32768 tokens 19 us, four launches' latencies; 2^20 48 us.
struct SortArgs {
  const void* in;          // tokens in the first pass, rows in later ones
  const int32_t* pos_in;   // of later ones
  int32_t n, rows, shift, bits, blocks, scanned;
  int32_t *row_out, *pos_out;
  int32_t* digits;
};

template <typename I>
__global__ __launch_bounds__(kSortThreads) void order_count_kernel(SortArgs a) {
  __shared__ int32_t count[kSortDigits];
  const int t = threadIdx.x, first = int(blockIdx.x) * kSortBlock;
  const I* in = static_cast<const I*>(a.in);
  I x[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) x[k] = in[min(first + k * kSortThreads + t, a.n - 1)];
  for (int k = t; k < kSortDigits; k += kSortThreads) count[k] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    if (first + k * kSortThreads + t >= a.n) continue;
    const int r = table_row(x[k], a.rows);
    atomicAdd(&count[(r >> a.shift) & ((1 << a.bits) - 1)], 1);
  }
  __syncthreads();
  for (int k = t; k < kSortDigits; k += kSortThreads) a.digits[int64_t(blockIdx.x) * kSortDigits + k] = count[k];
}

// Many blocks: every block's counts become those of the blocks before it, and a row
// behind them the totals: 64 digits a block, its 16 waves a part of the rows each.
// (Every block adding up all rows by itself: 107 us for 2^20 tokens instead of 48, 14 ms
// for 16 million instead of 0.46; with fewer than 112 blocks it is a launch more, 31 us
// instead of 29 for 200000.)
constexpr int kScanWaves = 16, kScanBlocks = 112;
__global__ __launch_bounds__(64 * kScanWaves) void order_scan_kernel(int32_t* digits, int blocks) {
  __shared__ int32_t sum[kScanWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, each = (blocks + kScanWaves - 1) / kScanWaves;
  const int from = min(wave * each, blocks), to = min(from + each, blocks);
  int32_t* d = digits + int(blockIdx.x) * 64 + lane;
  int s = 0;
#pragma unroll 8
  for (int b = from; b < to; ++b) s += d[int64_t(b) * kSortDigits];
  sum[wave][lane] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += sum[w][lane];
  if (wave == kScanWaves - 1) d[int64_t(blocks) * kSortDigits] = before + s;
#pragma unroll 8
  for (int b = from; b < to; ++b) {
    const int c = d[int64_t(b) * kSortDigits];
    d[int64_t(b) * kSortDigits] = before;
    before += c;
  }
}

template <typename I, bool FIRST>
__global__ __launch_bounds__(kSortThreads) void order_scatter_kernel(SortArgs a) {
  constexpr int kWaves = kSortThreads / 64;
  __shared__ int32_t base[kSortDigits];             // where the block's tokens of a digit begin
  __shared__ int32_t seen[kWaves][kSortDigits];     // then: where the wave's do
  __shared__ int32_t wave_sum[kWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int n_digits = 1 << a.bits;
  // a wave's tokens are consecutive: 64 at a time, each one's rank among those of its digit
  const int first = int(blockIdx.x) * kSortBlock + wave * 64 * kSortItems;
  const I* in = static_cast<const I*>(a.in);
  I x[kSortItems];
  int row[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = min(first + k * 64 + lane, a.n - 1);
    x[k] = in[i];
    pos[k] = FIRST ? i : a.pos_in[i];
  }
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) row[k] = first + k * 64 + lane < a.n ? table_row(x[k], a.rows) : -1;
  for (int k = t; k < kWaves * kSortDigits; k += kSortThreads) (&seen[0][0])[k] = 0;
  // a digit a thread: all blocks' tokens of lower digits, and the earlier blocks' of its own
  static_assert(kSortThreads == kSortDigits, "a digit a thread");
  int total = 0, before = 0;
  constexpr int kAtOnce = 16;
  if (a.scanned) {
    total = a.digits[int64_t(a.blocks) * kSortDigits + t];
    before = a.digits[int64_t(blockIdx.x) * kSortDigits + t];
  }
  for (int b0 = a.scanned ? a.blocks : 0; b0 < a.blocks; b0 += kAtOnce) {
    int c[kAtOnce];
#pragma unroll
    for (int b = 0; b < kAtOnce; ++b) c[b] = a.digits[int64_t(min(b0 + b, a.blocks - 1)) * kSortDigits + t];
#pragma unroll
    for (int b = 0; b < kAtOnce; ++b) {
      // by selection: a branch would put each load behind it
      total += c[b] & (b0 + b < a.blocks ? -1 : 0);
      before += c[b] & (b0 + b < int(blockIdx.x) ? -1 : 0);
    }
  }
  int up = total;
  for (int off = 1; off < 64; off <<= 1) {
    const int x = __shfl_up(up, off, 64);
    if (lane >= off) up += x;
  }
  if (lane == 63) wave_sum[wave] = up;
  __syncthreads();
  int lower = up - total;
  for (int w = 0; w < wave; ++w) lower += wave_sum[w];
  base[t] = lower + before;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const bool there = row[k] >= 0;
    const int d = there ? (row[k] >> a.shift) & (n_digits - 1) : 0;
    uint64_t like = __ballot(there);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t m = __ballot((d >> b) & 1);
      like &= ((d >> b) & 1) ? m : ~m;
    }
    const int lower_lanes = __popcll(like & ((uint64_t(1) << lane) - 1));
    if (there) {
      rank[k] = seen[wave][d] + lower_lanes;     // a wave's accesses to LDS are in order
    }
    __builtin_amdgcn_wave_barrier();
    if (there && lower_lanes == 0) seen[wave][d] += __popcll(like);
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int d = t; d < n_digits; d += kSortThreads) {
    int at = base[d];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int c = seen[w][d];
      seen[w][d] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    if (row[k] < 0) continue;
    const int d = (row[k] >> a.shift) & (n_digits - 1);
    const int at = seen[wave][d] + rank[k];
    a.row_out[at] = row[k];
    a.pos_out[at] = pos[k];
  }
}

// ---------------------------------------------------- the table's gradient

struct EmbeddingGradArgs {
  const int32_t *row, *pos;  // the rows of tokens outside the table lie past row_hi
  const void* d_out;
  void* grad;
  float* ws;                 // [pieces][2][dim4]: sums of a run's middle or end, and of its beginning
  int64_t stride, first, count;
  float scale;
  int32_t n, dim, dim4, tiles, pieces, piece;
  int32_t row_lo, row_hi;    // rows that the part touches
  int32_t sum_blocks;
};

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef i32x8 i32x8_any __attribute__((aligned(4)));

__device__ __forceinline__ i32x8 load8(const int32_t* p) {
  return *(const __attribute__((address_space(4))) i32x8_any*)p;
}

// grad's elements of row r at the lane's span. Where the part begins or ends inside
// the row, only those of the lane's elements that lie in it.
template <int E, typename G>
__device__ __forceinline__ Words<E, G> read_grad(const EmbeddingGradArgs& a, int r, const Span& s) {
  const int64_t base = int64_t(r) * a.dim - a.first;      // grad's index of the row's first element
  const G* g = static_cast<const G*>(a.grad) + base;
  if (base >= 0 && base + a.dim <= a.count) return load_row<E>(g, s);
  const int lo = int(max(int64_t(s.lo), -base - s.col)), hi = int(min(int64_t(E), a.count - base - s.col));
  return load_some<E, G>(g + s.col, lo, hi);
}

template <int E, typename G>
__device__ __forceinline__ void write_grad(const EmbeddingGradArgs& a, int r, const Span& s, const Words<E, G>& w) {
  const int64_t base = int64_t(r) * a.dim - a.first;
  G* g = static_cast<G*>(a.grad) + base;
  if (base >= 0 && base + a.dim <= a.count) {
    store_row<E>(g, s, w);
    return;
  }
  const int lo = int(max(int64_t(s.lo), -base - s.col)), hi = int(min(int64_t(E), a.count - base - s.col));
  store_some<E, G>(g + s.col, lo, hi, w);
}

template <int E, typename G, bool ADD>
__device__ __forceinline__ void write_sum(const EmbeddingGradArgs& a, int r, const Span& s, const Words<E, G>& old,
                                          const float (&sum)[E]) {
  float v[E];
  if constexpr (ADD) {
    widen<E, G>(old, v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(sum[e], a.scale, v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = sum[e] * a.scale;
  }
  write_grad<E, G>(a, r, s, narrow<E, G>(v));
}

// The first of the n sorted rows at or above r, or n: 64 compared at a time, their
// spacing divided by 64 each round.
__device__ __forceinline__ int first_at(const int32_t* row, int n, int r) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = n;                 // it is in [lo, lo + len]
  while (len > 0) {
    const int step = (len + 63) >> 6;
    const int last = row[lo + min((lane + 1) * step, len) - 1];    // of the lane's rows
    const int below = __popcll(__ballot(last < r));                // so many lanes' rows lie below r
    if (below == 64) return lo + len;
    len = __builtin_amdgcn_readfirstlane(min(step, len - below * step));
    lo = __builtin_amdgcn_readfirstlane(lo + below * step);
    if (step == 1) return lo;
  }
  return lo;
}

// Of the rows [r0, r1), at most 64, those that are not among the sorted ones, a
// bit each: between the first sorted one and the last, every lane looks for its own.
__device__ __forceinline__ uint64_t rows_without(const int32_t* row, int n, int r0, int r1) {
  const int mine = r0 + int(threadIdx.x & 63);
  const int from = first_at(row, n, r0), to = first_at(row, n, r1);
  int lo = from, hi = to;
  while (__ballot(lo < hi)) {
    const int mid = (lo + hi) >> 1;
    const int x = row[min(mid, n - 1)];
    const bool up = lo < hi && x < mine;
    hi = lo < hi && !up ? mid : hi;
    lo = up ? mid + 1 : lo;
  }
  const bool there = lo < to && row[max(min(lo, n - 1), 0)] == mine;
  return __ballot(mine < r1 && !there);
}

constexpr int kFillRows = 4;       // rows that a wave looks for and clears
constexpr int64_t kFewTokens = 96;
constexpr int kBatch = 8;          // rows that a wave loads before it adds them

// The sums of the sorted tokens [i0, i1), a piece, at the lane's span: of a run that
// lies in the piece to grad, of a run that goes on beyond it to put(1, sum), of one
// that began before it to put(0, sum).
template <typename T, typename G, int E, bool ADD, typename Put>
__device__ __forceinline__ void sum_piece(const EmbeddingGradArgs& a, int i0, int i1, const Span& s, const Put& put) {
  // rows and positions by eights: the arrays go on that far behind their last entry
  i32x8 r8 = load8(a.row + i0), p8 = load8(a.pos + i0);
  const int prior = uniform_load(a.row + max(i0 - 1, 0)), r_last = uniform_load(a.row + i1 - 1);
  if (r_last < a.row_lo || r8[0] >= a.row_hi) return;
  bool head = i0 > 0 && prior == r8[0];      // the run at hand began in an earlier piece
  float sum[E] = {};
  for (int i = i0; i < i1; i += kBatch) {
    if (i > i0) {
      r8 = load8(a.row + i);
      p8 = load8(a.pos + i);
    }
    const int r9 = uniform_load(a.row + i + kBatch);
    int r[kBatch + 1];
    Words<E, T> x[kBatch];
    Words<E, G> old[ADD ? kBatch : 1];
#pragma unroll
    for (int k = 0; k <= kBatch; ++k) r[k] = i + k >= a.n ? -1 : k < kBatch ? r8[k % kBatch] : r9;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      // a row that is there, also where the order is not one of these tokens
      const uint32_t p = i + k < i1 && r[k] >= a.row_lo && r[k] < a.row_hi ? min(uint32_t(p8[k]), uint32_t(a.n - 1)) : 0u;
      x[k] = load_row<E>(static_cast<const T*>(a.d_out) + int64_t(p) * a.stride, s);
    }
    if constexpr (ADD) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i + k < i1 && r[k] != r[k + 1] && r[k] >= a.row_lo && r[k] < a.row_hi) old[k] = read_grad<E, G>(a, r[k], s);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i + k >= i1) break;
      float v[E];
      widen<E, T>(x[k], v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += v[e];
      const bool end = r[k] != r[k + 1];
      if (!end && i + k + 1 < i1) continue;
      if (r[k] >= a.row_lo && r[k] < a.row_hi) {
        if (head || !end) put(head ? 0 : 1, sum);
        else write_sum<E, G, ADD>(a, r[k], s, old[ADD ? k : 0], sum);
      }
      head = false;
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] = 0.f;
    }
  }
}

// Of the run that begins in the piece and goes on beyond it: its row, in *r, and how
// many pieces more it reaches; 0 where there is none, or none in the part.
__device__ __forceinline__ int pieces_beyond(const EmbeddingGradArgs& a, int piece, int* r) {
  const int i0 = piece * a.piece, i1 = i0 + a.piece;
  if (i1 >= a.n) return 0;
  *r = uniform_load(a.row + i1);
  const int end = uniform_load(a.row + i1 - 1), begin = uniform_load(a.row + i0),
            prior = uniform_load(a.row + max(i0 - 1, 0));
  if (end != *r || *r < a.row_lo || *r >= a.row_hi) return 0;
  if (i0 > 0 && begin == *r && prior == *r) return 0;      // began earlier
  // the pieces whose first token goes on with the run: 64 compared at a time
  for (int more = 0;;) {
    const int64_t i = int64_t(piece + 1 + more + int(threadIdx.x & 63)) * a.piece;
    const uint64_t on = __ballot(i < a.n && a.row[i < a.n ? i : 0] == *r);
    if (on != ~uint64_t(0)) return more + __builtin_ctzll(~on);
    more += 64;
  }
}

// sum += what the pieces [from, to) have left of a run that began before them, read
// eight at a time.
template <int E>
__device__ __forceinline__ void add_pieces(const EmbeddingGradArgs& a, float (&sum)[E], int from, int to, const Span& s) {
  constexpr int N = 8;
  for (int j = from; j < to; j += N) {
    Words<E, float> x[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
      x[k] = load_row<E, false>(a.ws + int64_t(min(j + k, to - 1)) * 2 * a.dim4, s);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float v[E];
      widen<E, float>(x[k], v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += j + k < to ? v[e] : 0.f;
    }
  }
}

template <int E, typename G>
__device__ __forceinline__ void clear_rows(const EmbeddingGradArgs& a, uint32_t w, int lane) {
  const int r0 = a.row_lo + int(w / uint32_t(a.tiles)) * kFillRows, r1 = min(r0 + kFillRows, a.row_hi);
  if (r0 >= r1) return;
  const Span s = span_of<E>(int(w % uint32_t(a.tiles)) * 64 + lane, a.dim);
  for (uint64_t absent = rows_without(a.row, a.n, r0, r1); absent != 0; absent &= absent - 1)
    write_grad<E, G>(a, r0 + __builtin_ctzll(absent), s, Words<E, G>{});
}

// Many tokens: a wave a piece and a tile of 64 vectors, its sums of shared runs in
// the workspace for embedding_join_kernel; eight rows are on their way at a time, with
// grad's old values where they are added to. So every wave has the same number of rows
// to add, however the tokens are spread, and no atomics decide an order. The blocks
// behind those write zeros, four rows and a tile a wave (the search for a token costs
// one row a wave 140 us, and 16 rows a wave, farther apart than the memory likes, 82 us
// instead of 73, for 8192 tokens of 50257 rows of 2944). That gradient in bf16 takes 53 us,
// 6.2 TB/s; 32768 tokens added to 4000 fp32 rows of 8192 32 us, 4.5 TB/s.
template <typename T, typename G, int E, bool ADD>
__global__ __launch_bounds__(256) void embedding_grad_kernel(const EmbeddingGradArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (!ADD && int(blockIdx.x) >= a.sum_blocks) {
    clear_rows<E, G>(a, (blockIdx.x - a.sum_blocks) * 4 + wave, lane);
    return;
  }
  const uint32_t w = blockIdx.x * 4 + wave;
  const int piece = int(w / uint32_t(a.tiles));
  if (piece >= a.pieces) return;
  const Span s = span_of<E>(int(w % uint32_t(a.tiles)) * 64 + lane, a.dim);
  const int i0 = piece * a.piece;
  sum_piece<T, G, E, ADD>(a, i0, min(i0 + a.piece, a.n), s, [&](int which, const float (&sum)[E]) {
    store_row<E, false>(a.ws + (int64_t(piece) * 2 + which) * a.dim4, s, narrow<E, float>(sum));
  });
}

// The runs that several pieces share: a block for the one that begins in a piece and
// four tiles, a wave a tile. A run over more than kAlone pieces (half of a batch on one
// row, as one that is padded with a real token has it) is left to the blocks of its
// first four pieces, which take one of the four tiles each, their waves a quarter of
// the pieces. Four vectors of fp32 whatever the gradient's type: so many more waves.
// (A block for four pieces instead of four tiles waits for the longest of their runs:
// 10 us instead of 7 at 32768 tokens, 8192 wide.)
constexpr int kJoinTiles = 4, kAlone = 64;

template <typename G, int E, bool ADD>
__global__ __launch_bounds__(64 * kJoinTiles) void embedding_join_kernel(const EmbeddingGradArgs a) {
  __shared__ float part[kJoinTiles][64 * E];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t across = uint32_t(a.tiles + kJoinTiles - 1) / kJoinTiles;
  const int piece = int(blockIdx.x / across), tile0 = int(blockIdx.x % across) * kJoinTiles;
  // a run begins in the piece and goes on; or one that began at most three pieces before is a long one, as the
  // token far behind tells. All of it read at once: most blocks have nothing to do.
  const int64_t i0 = int64_t(piece) * a.piece, i1 = i0 + a.piece, far = i0 + int64_t(kAlone - kJoinTiles) * a.piece;
  const int prior = uniform_load(a.row + max(i0 - 1, int64_t(0))), first = uniform_load(a.row + i0),
            end = uniform_load(a.row + min(i1, int64_t(a.n)) - 1), next = uniform_load(a.row + min(i1, int64_t(a.n) - 1)),
            distant = uniform_load(a.row + min(far, int64_t(a.n) - 1));
  const bool earlier = piece > 0 && prior == first;
  if (i1 >= a.n || end != next || next < a.row_lo || next >= a.row_hi) return;
  if (earlier && first == next && (far >= a.n || prior != distant)) return;
  int r = 0, begin = piece, more = 0;
  if (!(earlier && first == next)) {
    more = pieces_beyond(a, piece, &r);
  } else {
    for (int q = 1; q < kJoinTiles && q <= piece && more == 0; ++q) {
      begin = piece - q;
      more = pieces_beyond(a, begin, &r);
      if (more < q) more = 0;         // a run that ends before this piece
    }
    if (more <= kAlone) return;
  }
  if (more == 0) return;
  const bool alone = more <= kAlone;
  const int tile = tile0 + (alone ? wave : piece - begin);
  if (tile >= a.tiles && !alone) return;
  const bool there = tile < a.tiles && (alone || wave == 0);
  const Span s = span_of<E>(min(tile, a.tiles - 1) * 64 + lane, a.dim);
  Words<E, G> old{};
  if constexpr (ADD) {
    if (there) old = read_grad<E, G>(a, r, s);
  }
  float sum[E];
  widen<E, float>(load_row<E, false>(a.ws + (int64_t(begin) * 2 + 1) * a.dim4, s), sum);
  if (alone) {
    add_pieces<E>(a, sum, begin + 1, begin + 1 + more, s);
  } else {
    const int each = (more + kJoinTiles - 1) / kJoinTiles;
    float some[E] = {};
    add_pieces<E>(a, some, begin + 1 + min(wave * each, more), begin + 1 + min((wave + 1) * each, more), s);
#pragma unroll
    for (int e = 0; e < E; ++e) part[wave][e * 64 + lane] = some[e];
    __syncthreads();
    for (int k = 0; k < kJoinTiles; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += part[k][e * 64 + lane];
  }
  if (there) write_sum<E, G, ADD>(a, r, s, old, sum);
}

constexpr int kWide = 16;

// Few tokens: a block a tile, a wave a sixteenth of the tokens, and the sums of
// shared runs in LDS: one launch instead of two.
template <typename T, typename G, int E, bool ADD>
__global__ __launch_bounds__(64 * kWide) void embedding_grad_few_kernel(const EmbeddingGradArgs a) {
  __shared__ float part[kWide][2][64 * E];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (!ADD && int(blockIdx.x) >= a.sum_blocks) {
    clear_rows<E, G>(a, (blockIdx.x - a.sum_blocks) * kWide + wave, lane);
    return;
  }
  const Span s = span_of<E>(int(blockIdx.x) * 64 + lane, a.dim);
  if (wave < a.pieces)
    sum_piece<T, G, E, ADD>(a, wave * a.piece, min((wave + 1) * a.piece, a.n), s, [&](int which, const float (&sum)[E]) {
#pragma unroll
      for (int e = 0; e < E; ++e) part[wave][which][e * 64 + lane] = sum[e];
    });
  __syncthreads();
  int r = 0;
  const int more = wave < a.pieces ? pieces_beyond(a, wave, &r) : 0;
  if (more == 0) return;
  Words<E, G> old{};
  if constexpr (ADD) old = read_grad<E, G>(a, r, s);
  float sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = part[wave][1][e * 64 + lane];
  for (int j = 1; j <= more; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] += part[wave + j][0][e * 64 + lane];
  write_sum<E, G, ADD>(a, r, s, old, sum);
}

// --------------------------------------------------------------------- norm

// E elements of a vector; ones or zeros where there is none.
template <int E, typename W>
__device__ __forceinline__ Words<E, W> load_weight(const void* w, const Span& s, float none) {
  if (w != nullptr) return load_row<E, false>(static_cast<const W*>(w), s);
  float x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = none;
  return narrow<E, W>(x);
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// The sum over aligned groups of LANES lanes, in every lane and in the same
// order for all: pairs, fours, eights, sixteens by moves within a row of 16
// lanes, then the rows and the halves of the wave by swaps.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  static_assert(LANES == 16 || LANES == 32 || LANES == 64, "a row of lanes, two, or the wave");
  x = dpp_add<0xB1>(x);       // quad_perm [1, 0, 3, 2]
  x = dpp_add<0x4E>(x);       // quad_perm [2, 3, 0, 1]
  x = dpp_add<0x141>(x);      // row_half_mirror
  x = dpp_add<0x140>(x);      // row_mirror
  if constexpr (LANES >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (LANES == 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return x;
}

// The sums of K values over the TPR threads that share a row, in every one of
// them. With TPR above 64 every thread of the block has to call it, and lds holds
// 2 * K * (waves of the block) values, half of which a call takes (`turn`, 0 and 1
// in turn), so one barrier a call suffices. LEAN: 16 waves' sums are read a lane each,
// not all by every thread, which takes 16 registers more.
template <int TPR, int K, bool LEAN = false>
__device__ __forceinline__ void row_sum(float (&x)[K], float* lds, int turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = lanes_sum<(TPR < 64 ? TPR : 64)>(x[k]);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    float* s = lds + turn * K * int(blockDim.x / 64);
    const int wave = threadIdx.x / 64, first = wave / kWaves * kWaves;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[wave * K + k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (LEAN && kWaves == 16) {
        x[k] = lanes_sum<16>(s[(threadIdx.x & 15) * K + k]);
      } else {
        x[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) x[k] += s[(first + w) * K + k];
      }
    }
  }
}

// A row's mean is a sum in fp32 that was rounded. Where it is larger than the deviations
// its error is one more deviation of all elements (a row of 4099 times 1000.1: 1.2e-4, and
// y 0.04 instead of 0 for eps = 1e-5). There the deviations are summed as well, whose sum
// has an error of their size: their mean is taken off each of them, as a shift of the
// normalised values, and its square off that of their squares. Elsewhere the mean's error
// is no larger than that of the deviations' sum. (Summed in every row: 16384 rows of 1600
// bf16 22.2 us instead of 21.3, 2048 of 16384 28.4 instead of 27.2.) All threads of a row
// decide alike, and not for a NaN or an infinity.
__device__ __forceinline__ bool far_mean(float mean, float rstd) { return fabsf(mean) * rstd > 1.f; }

__device__ __forceinline__ float rstd_of(float var, float eps) { return 1.f / sqrtf(var + eps); }

// TPR threads a row, V vectors each: the row is read once and stays in registers, so
// the squares are taken after the mean, and the weights are on their way with it.
// 8192 rows of 2944 bf16 with the residual 35.8 us, 5.4 TB/s; 16384 of 8192 without mean
// 91 us, 5.9; bound by HBM.
template <typename T, typename W, int E, int TPR, int V>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(const zero_norm_args a) {
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  __shared__ float lds[2 * (TPR < 256 ? 4 : TPR / 64)];
  const int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  if (row >= a.n) return;          // whole rows: with TPR above 64 a block has one
  const int dim = int(a.dim);
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  Span s[V];
  Words<E, T> raw[V];
  Words<E, W> w[V], b[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    s[k] = span_of<E>(t + k * TPR, dim);
    raw[k] = load_row<E>(x, s[k]);
  }
  float v[V][E];
  if (a.residual != nullptr) {
    const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
    T* total = static_cast<T*>(a.total) + row * a.total_stride;
    Words<E, T> more[V];
#pragma unroll
    for (int k = 0; k < V; ++k) more[k] = load_row<E>(res, s[k]);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      w[k] = load_weight<E, W>(a.weight, s[k], 1.f);
      b[k] = load_weight<E, W>(a.bias, s[k], 0.f);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float r[E];
      widen<E, T>(raw[k], v[k]);
      widen<E, T>(more[k], r);
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] += r[e];
      raw[k] = narrow<E, T>(v[k]);
      store_row<E>(total, s[k], raw[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      w[k] = load_weight<E, W>(a.weight, s[k], 1.f);
      b[k] = load_weight<E, W>(a.bias, s[k], 0.f);
    }
  }
  float sum[1] = {0.f};
#pragma unroll
  for (int k = 0; k < V; ++k) {
    widen<E, T>(raw[k], v[k]);
    only_own<E>(s[k], v[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[0] += v[k][e];
  }
  float mean = 0.f;
  if (!a.rms) {
    row_sum<TPR, 1>(sum, lds, 0);
    mean = sum[0] / float(dim);
  }
  sum[0] = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[k][e] -= mean;
    only_own<E>(s[k], v[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[0] = fmaf(v[k][e], v[k][e], sum[0]);
  }
  row_sum<TPR, 1>(sum, lds, 1);
  const float var = sum[0] / float(dim);
  float rstd = rstd_of(var, float(a.eps)), shift = -0.f;
  if (far_mean(mean, rstd)) {
    sum[0] = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[0] += v[k][e];
    row_sum<TPR, 1, true>(sum, lds, 0);
    const float off = sum[0] / float(dim);
    mean += off;
    rstd = rstd_of(fmaxf(var - off * off, 0.f), float(a.eps));
    shift = -off * rstd;
  }
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float wf[E], bf[E];
    widen<E, W>(w[k], wf);
    widen<E, W>(b[k], bf);
#pragma unroll
    for (int e = 0; e < E; ++e) v[k][e] = fmaf(fmaf(v[k][e], rstd, shift), wf[e], bf[e]);
    store_row<E>(y, s[k], narrow<E, T>(v[k]));
  }
}

// A row longer than the registers of a block: three passes over it, the later
// ones from the caches. Element by element, so that y and total may be x. 2048 rows of
// 40000 bf16 91 us, 3.6 TB/s of what has to move; 1024 of 32768, in registers, 30 us, 4.5.
constexpr int kLongThreads = 1024;

template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(const zero_norm_args a) {
  constexpr int E = 16 / int(sizeof(T));
  __shared__ float lds[2 * (kLongThreads / 64)];
  const int64_t row = blockIdx.x;
  const int dim = int(a.dim), vectors = (dim + E - 1) / E;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  T* total = res != nullptr ? static_cast<T*>(a.total) + row * a.total_stride : nullptr;
  float sum[1] = {0.f};
  for (int k = threadIdx.x; k < vectors; k += kLongThreads) {
    const Span s = span_of<E>(k, dim);
    float v[E];
    Words<E, T> raw = load_row<E, false>(x, s);
    widen<E, T>(raw, v);
    if (res != nullptr) {
      float r[E];
      widen<E, T>(load_row<E, false>(res, s), r);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += r[e];
      raw = narrow<E, T>(v);
      store_row<E, false>(total, s, raw);
      widen<E, T>(raw, v);
    }
    only_own<E>(s, v);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[0] += v[e];
  }
  if (res != nullptr) x = total;       // every thread reads back what it wrote
  float mean = 0.f;
  if (!a.rms) {
    row_sum<kLongThreads, 1>(sum, lds, 0);
    mean = sum[0] / float(dim);
  }
  sum[0] = 0.f;
  float dev[1] = {0.f};
  for (int k = threadIdx.x; k < vectors; k += kLongThreads) {
    const Span s = span_of<E>(k, dim);
    float v[E];
    widen<E, T>(load_row<E, false>(x, s), v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] -= mean;
    only_own<E>(s, v);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sum[0] = fmaf(v[e], v[e], sum[0]);
      dev[0] += v[e];
    }
  }
  row_sum<kLongThreads, 1>(sum, lds, 1);
  const float var = sum[0] / float(dim);
  float rstd = rstd_of(var, float(a.eps)), off = 0.f;
  if (far_mean(mean, rstd)) {
    row_sum<kLongThreads, 1>(dev, lds, 0);
    off = dev[0] / float(dim);
    rstd = rstd_of(fmaxf(var - off * off, 0.f), float(a.eps));
  }
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean + off;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
  for (int k = threadIdx.x; k < vectors; k += kLongThreads) {
    const Span s = span_of<E>(k, dim);
    float v[E], w[E], b[E];
    widen<E, T>(load_row<E, false>(x, s), v);
    widen<E, W>(load_weight<E, W>(a.weight, s, 1.f), w);
    widen<E, W>(load_weight<E, W>(a.bias, s, 0.f), b);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf((v[e] - mean - off) * rstd, w[e], b[e]);
    store_row<E, false>(y, s, narrow<E, T>(v));
  }
}

// ---------------------------------------------------------- norm's gradient

// A column's sum, written or added, to a vector of either type.
__device__ __forceinline__ void put_sum(void* out, int32_t type, int col, float sum, int32_t add) {
  if (type == ZERO_BF16) {
    uint16_t* p = static_cast<uint16_t*>(out) + col;
    *p = to_bf16(add ? bf16_lo(*p) + sum : sum);
  } else {
    float* p = static_cast<float*>(out) + col;
    *p = add ? *p + sum : sum;
  }
}

// A block takes every gridDim.x-th group of rows, TPR threads a row, and keeps the
// sums of d_weight and d_bias over its rows in registers; the groups' sums meet in
// LDS and go to the workspace, which norm_grad_join_kernel adds up. One vector a
// thread: with two, or with a wave a row, the sums leave room for too few waves. The
// next rows are read before this one's sums. 16384 rows of 2944 bf16 with the skip path
// 68 us, 5.7 TB/s; bound by HBM. (Blocks of 1024 threads, two rows at a time that
// wait for each other: 87 us.)
template <typename T, typename W, int E, int TPR, int V>
__global__ __launch_bounds__(grad_threads(TPR)) void norm_grad_kernel(const zero_norm_grad_args a, float* ws, int dim4) {
  constexpr int kThreads = grad_threads(TPR), kRows = kThreads / TPR;
  __shared__ float lds[kThreads * V * E];      // row sums, then the groups' column sums
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int dim = int(a.dim);
  const bool skip = a.d_total != nullptr;
  Span s[V];
  Words<E, W> w_raw[V];
  float sum_w[V][E], sum_b[V][E];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    s[k] = span_of<E>(t + k * TPR, dim);
    w_raw[k] = load_weight<E, W>(a.weight, s[k], 1.f);
#pragma unroll
    for (int e = 0; e < E; ++e) sum_w[k][e] = sum_b[k][e] = 0.f;
  }
  struct Row {
    Words<E, T> dy[V], x[V], total[V];
    float mean, rstd;
  };
  const auto read = [&](int64_t row0, Row& r) {
    const int64_t row = row0 + group < a.n ? row0 + group : row0;
    const T* dy = static_cast<const T*>(a.d_y) + row * a.d_y_stride;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      r.dy[k] = load_row<E>(dy, s[k]);
      r.x[k] = load_row<E>(x, s[k]);
    }
    if (skip) {
#pragma unroll
      for (int k = 0; k < V; ++k)
        r.total[k] = load_row<E>(static_cast<const T*>(a.d_total) + row * a.d_total_stride, s[k]);
    }
    r.mean = a.rms ? 0.f : a.mean[row];
    r.rstd = a.rstd[row];
  };
  int turn = 0;
  const int64_t step = int64_t(gridDim.x) * kRows;
  const auto pass = [&](int64_t row0, Row& now) {
    const bool there = row0 + group < a.n;
    const int64_t row = row0 + group;
    const float mean = now.mean, rstd = now.rstd;
    float g[V][E], xh[V][E];
    float c[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float w[E];
      widen<E, T>(now.dy[k], g[k]);
      widen<E, T>(now.x[k], xh[k]);
      widen<E, W>(w_raw[k], w);
      if (kRows == 1 || there) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          xh[k][e] = (xh[k][e] - mean) * rstd;
          sum_w[k][e] = fmaf(g[k][e], xh[k][e], sum_w[k][e]);
          sum_b[k][e] += g[k][e];
          g[k][e] *= w[e];
        }
      }
      if (s[k].lo > 0) {       // the neighbour's: computed, not summed
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e >= s[k].lo) {
            c[0] += g[k][e];
            c[1] = fmaf(g[k][e], xh[k][e], c[1]);
          }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          c[0] += g[k][e];
          c[1] = fmaf(g[k][e], xh[k][e], c[1]);
        }
      }
    }
    if (a.d_x == nullptr) return;
    row_sum<TPR, 2>(c, lds, turn);
    turn ^= 1;
    if (!there) return;
    const float c0 = a.rms ? 0.f : c[0] / float(dim), c1 = c[1] / float(dim);
    T* dx = static_cast<T*>(a.d_x) + row * a.d_x_stride;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float m[E];
#pragma unroll
      for (int e = 0; e < E; ++e) m[e] = 0.f;
      if (skip) widen<E, T>(now.total[k], m);
#pragma unroll
      for (int e = 0; e < E; ++e) g[k][e] = fmaf(fmaf(-xh[k][e], c1, g[k][e] - c0), rstd, m[e]);
      store_row<E>(dx, s[k], narrow<E, T>(g[k]));
    }
  };
  // the next rows are on their way while these are summed
  constexpr int kAhead = V * E > 4 ? 1 : 2;
  Row ring[kAhead + 1];
  int64_t row0 = int64_t(blockIdx.x) * kRows;
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (row0 + k * step < a.n) read(row0 + k * step, ring[k]);
  while (row0 < a.n) {
#pragma unroll
    for (int k = 0; k <= kAhead; ++k) {
      if (row0 >= a.n) break;
      if (row0 + kAhead * step < a.n) read(row0 + kAhead * step, ring[(k + kAhead) % (kAhead + 1)]);
      pass(row0, ring[k]);
      row0 += step;
    }
  }
  if (a.d_weight == nullptr && a.d_bias == nullptr) return;
  float* out = ws + int64_t(blockIdx.x) * 2 * dim4;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (a.d_weight != nullptr) store_row<E, false>(out, s[k], narrow<E, float>(sum_w[k]));
      if (a.d_bias != nullptr) store_row<E, false>(out + dim4, s[k], narrow<E, float>(sum_b[k]));
    }
  } else {
    // [group][V][E][TPR], lanes side by side; a vector's neighbour's elements are left out
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if ((which ? a.d_bias : a.d_weight) == nullptr) continue;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e)
          lds[(group * V * E + k * E + e) * TPR + t] = which ? sum_b[k][e] : sum_w[k][e];
      __syncthreads();
      for (int j = threadIdx.x; j < V * E * TPR; j += kThreads) {
        float x = 0.f;
#pragma unroll
        for (int g = 0; g < kRows; ++g) x += lds[g * V * E * TPR + j];
        const int ke = j / TPR, e = ke % E;
        const Span at = span_of<E>(j % TPR + ke / E * TPR, dim);
        if (e >= at.lo) out[which * dim4 + at.col + e] = x;
      }
    }
  }
}

// Few rows: the columns' sums need the rows' statistics, which are given, but not
// their sums, so blocks of columns and blocks of rows go side by side in one launch,
// and d_y and x are read twice. A block of columns takes a tile of 64 vectors, its 16
// waves every sixteenth row each; a block of rows takes one. 64 rows of 768 bf16 7.2 us
// (a launch and the binding), where two launches with a join of the blocks' sums took
// 10.3; what bounds more rows is the latency of the columns' batches of 128 rows.
constexpr int kFewThreads = 1024, kFewWaves = kFewThreads / 64, kFewBatch = 8;

template <typename T, typename W, int E, int V>
__global__ __launch_bounds__(kFewThreads) void norm_grad_few_kernel(const zero_norm_grad_args a, int col_blocks) {
  __shared__ float lds[kFewWaves * 64 * E];
  const int dim = int(a.dim), n = int(a.n), t = threadIdx.x, lane = t & 63;
  if (int(blockIdx.x) < col_blocks) {
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const Span s = span_of<E>(int(blockIdx.x) * 64 + lane, dim);
    float sum_w[E] = {}, sum_b[E] = {};
    for (int row0 = wave; row0 < n; row0 += kFewWaves * kFewBatch) {
      Words<E, T> dy[kFewBatch], x[kFewBatch];
      float mean[kFewBatch], rstd[kFewBatch];
#pragma unroll
      for (int k = 0; k < kFewBatch; ++k) {
        const int64_t row = min(row0 + k * kFewWaves, n - 1);
        dy[k] = load_row<E, false>(static_cast<const T*>(a.d_y) + row * a.d_y_stride, s);
        x[k] = load_row<E, false>(static_cast<const T*>(a.x) + row * a.x_stride, s);
        mean[k] = a.rms ? 0.f : uniform_load(a.mean + row);
        rstd[k] = uniform_load(a.rstd + row);
      }
#pragma unroll
      for (int k = 0; k < kFewBatch; ++k) {
        if (row0 + k * kFewWaves < n) {
          float g[E], xh[E];
          widen<E, T>(dy[k], g);
          widen<E, T>(x[k], xh);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            sum_w[e] = fmaf(g[e], (xh[e] - mean[k]) * rstd[k], sum_w[e]);
            sum_b[e] += g[e];
          }
        }
      }
    }
    for (int which = 0; which < 2; ++which) {
      void* out = which ? a.d_bias : a.d_weight;
      if (out == nullptr) continue;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) lds[(wave * E + e) * 64 + lane] = which ? sum_b[e] : sum_w[e];
      __syncthreads();
      if (t < 64 * E) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) x += lds[w * E * 64 + t];
        if (t / 64 >= s.lo) put_sum(out, a.grad_type, s.col + t / 64, x, a.accumulate);
      }
    }
    return;
  }
  const int64_t row = int(blockIdx.x) - col_blocks;
  const T* dy = static_cast<const T*>(a.d_y) + row * a.d_y_stride;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* d_total = a.d_total != nullptr ? static_cast<const T*>(a.d_total) + row * a.d_total_stride : nullptr;
  Span s[V];
  Words<E, T> dy_raw[V], x_raw[V], total[V];
  Words<E, W> w_raw[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    s[k] = span_of<E>(t + k * kFewThreads, dim);
    dy_raw[k] = load_row<E, false>(dy, s[k]);
    x_raw[k] = load_row<E, false>(x, s[k]);
    w_raw[k] = load_weight<E, W>(a.weight, s[k], 1.f);
    if (d_total != nullptr) total[k] = load_row<E, false>(d_total, s[k]);
  }
  const float mean = a.rms ? 0.f : uniform_load(a.mean + row), rstd = uniform_load(a.rstd + row);
  float g[V][E], xh[V][E], c[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float w[E];
    widen<E, T>(dy_raw[k], g[k]);
    widen<E, T>(x_raw[k], xh[k]);
    widen<E, W>(w_raw[k], w);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      g[k][e] *= w[e];
      xh[k][e] = (xh[k][e] - mean) * rstd;
      if (e >= s[k].lo) {
        c[0] += g[k][e];
        c[1] = fmaf(g[k][e], xh[k][e], c[1]);
      }
    }
  }
  row_sum<kFewThreads, 2>(c, lds, 0);
  const float c0 = a.rms ? 0.f : c[0] / float(dim), c1 = c[1] / float(dim);
  T* dx = static_cast<T*>(a.d_x) + row * a.d_x_stride;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float m[E];
#pragma unroll
    for (int e = 0; e < E; ++e) m[e] = 0.f;
    if (d_total != nullptr) widen<E, T>(total[k], m);
#pragma unroll
    for (int e = 0; e < E; ++e) g[k][e] = fmaf(fmaf(-xh[k][e], c1, g[k][e] - c0), rstd, m[e]);
    store_row<E>(dx, s[k], narrow<E, T>(g[k]));
  }
}

// Rows of more than 8192 elements, whose sums do not fit the registers: the rows'
// gradient in two passes over each.
template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void norm_grad_long_kernel(const zero_norm_grad_args a) {
  constexpr int E = 16 / int(sizeof(T));
  __shared__ float lds[2 * 2 * (kLongThreads / 64)];
  const int64_t row = blockIdx.x;
  const int dim = int(a.dim), vectors = (dim + E - 1) / E;
  const T* dy = static_cast<const T*>(a.d_y) + row * a.d_y_stride;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* d_total = a.d_total != nullptr ? static_cast<const T*>(a.d_total) + row * a.d_total_stride : nullptr;
  T* dx = static_cast<T*>(a.d_x) + row * a.d_x_stride;
  const float mean = a.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
  float c[2] = {0.f, 0.f};
  for (int k = threadIdx.x; k < vectors; k += kLongThreads) {
    const Span s = span_of<E>(k, dim);
    float g[E], xh[E], w[E];
    widen<E, T>(load_row<E, false>(dy, s), g);
    widen<E, T>(load_row<E, false>(x, s), xh);
    widen<E, W>(load_weight<E, W>(a.weight, s, 1.f), w);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      g[e] *= w[e];
      xh[e] = (xh[e] - mean) * rstd;
    }
    only_own<E>(s, g);
    only_own<E>(s, xh);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      c[0] += g[e];
      c[1] = fmaf(g[e], xh[e], c[1]);
    }
  }
  row_sum<kLongThreads, 2>(c, lds, 0);
  const float c0 = a.rms ? 0.f : c[0] / float(dim), c1 = c[1] / float(dim);
  for (int k = threadIdx.x; k < vectors; k += kLongThreads) {
    const Span s = span_of<E>(k, dim);
    float g[E], xh[E], w[E], m[E];
    widen<E, T>(load_row<E, false>(dy, s), g);
    widen<E, T>(load_row<E, false>(x, s), xh);
    widen<E, W>(load_weight<E, W>(a.weight, s, 1.f), w);
#pragma unroll
    for (int e = 0; e < E; ++e) m[e] = 0.f;
    if (d_total != nullptr) widen<E, T>(load_row<E, false>(d_total, s), m);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      xh[e] = (xh[e] - mean) * rstd;
      g[e] = fmaf(fmaf(-xh[e], c1, g[e] * w[e] - c0), rstd, m[e]);
    }
    store_row<E, false>(dx, s, narrow<E, T>(g));
  }
}

// Their column sums: a thread takes a vector of every gridDim.y-th row. Before
// the rows' gradient, which may overwrite d_y or x.
template <typename T>
__global__ __launch_bounds__(256) void norm_grad_columns_kernel(const zero_norm_grad_args a, float* ws, int dim4) {
  constexpr int E = 16 / int(sizeof(T));
  const int dim = int(a.dim);
  const Span s = span_of<E>(int(blockIdx.x) * 256 + int(threadIdx.x), dim);
  float sum_w[E] = {}, sum_b[E] = {};
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    const float mean = a.rms ? 0.f : uniform_load(a.mean + row), rstd = uniform_load(a.rstd + row);
    float g[E], xh[E];
    widen<E, T>(load_row<E, false>(static_cast<const T*>(a.d_y) + row * a.d_y_stride, s), g);
    widen<E, T>(load_row<E, false>(static_cast<const T*>(a.x) + row * a.x_stride, s), xh);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sum_w[e] = fmaf(g[e], (xh[e] - mean) * rstd, sum_w[e]);
      sum_b[e] += g[e];
    }
  }
  float* out = ws + int64_t(blockIdx.y) * 2 * dim4;
  store_row<E, false>(out, s, narrow<E, float>(sum_w));
  store_row<E, false>(out + dim4, s, narrow<E, float>(sum_b));
}

// The blocks' sums, added up: 64 columns a block, its 16 waves taking every
// 16th row of the workspace. blockIdx.y: d_weight, d_bias.
constexpr int kJoinWaves = 16;

__global__ __launch_bounds__(64 * kJoinWaves) void norm_grad_join_kernel(const float* __restrict__ ws, int blocks, int dim,
                                                                         int dim4, void* d_weight, void* d_bias,
                                                                         int32_t type, int32_t accumulate) {
  void* out = blockIdx.y == 0 ? d_weight : d_bias;
  if (out == nullptr) return;
  __shared__ float part[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = int(blockIdx.x) * 64 + lane;
  float s = 0.f;
  if (col < dim)
#pragma unroll 16
    for (int b = wave; b < blocks; b += kJoinWaves) s += ws[(int64_t(b) * 2 + blockIdx.y) * dim4 + col];
  part[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= dim) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWaves; ++k) s += part[k][lane];
  put_sum(out, type, col, s, accumulate);
}

template <int N>
using Int = std::integral_constant<int, N>;

// A call's launch for its two element types.
template <typename F>
void by_types(int32_t first, int32_t second, const F& go) {
  if (first == ZERO_BF16) second == ZERO_BF16 ? go(uint16_t(), uint16_t()) : go(uint16_t(), float());
  else second == ZERO_BF16 ? go(float(), uint16_t()) : go(float(), float());
}

// With E elements a vector, or 1 where a row has fewer.
template <int E, typename F>
void by_width(int64_t dim, const F& go) {
  if (dim >= E) go(Int<E>());
  else go(Int<1>());
}

}  // namespace

namespace zero {

int launch_embedding(const void* tokens, bool wide, int64_t n, const void* table, int32_t table_type, int64_t rows,
                     int64_t dim, float scale, void* out, int32_t out_type, int64_t out_stride, hipStream_t stream,
                     const char* who) {
  const auto go = [&](auto tv, auto ov) {
    using T = decltype(tv);
    using O = decltype(ov);
    by_width<sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4>(dim, [&](auto ev) {
      constexpr int E = decltype(ev)::value;
      const int64_t tiles = (dim + 64 * E - 1) / (64 * E);
      const int64_t waves = (n + kLookupRows - 1) / kLookupRows * tiles;
      const auto run = [&](auto iv) {
        using I = decltype(iv);
        embedding_kernel<I, T, O, E><<<dim3(uint32_t((waves + 3) / 4)), 256, 0, stream>>>(
            static_cast<const I*>(tokens), int(n), static_cast<const T*>(table), int(rows), int(dim), int(tiles), scale,
            static_cast<O*>(out), out_stride);
      };
      wide ? run(int64_t()) : run(int32_t());
    });
  };
  by_types(table_type, out_type, go);
  return launched(who);
}

int launch_token_order(const void* tokens, bool wide, int64_t n, int64_t rows, int32_t* order, hipStream_t stream,
                       const char* who) {
  const Order o(n);
  // keys are the rows and, behind them, the tokens outside the table
  const int64_t own = (rows + kSplitBlocks) / kSplitBlocks;
  if (n > kSplitFrom && n <= kSplitTokens && own <= kSplitEach) {
    int bits = 0;
    while ((int64_t(1) << bits) < own) ++bits;
    const dim3 grid{uint32_t((rows + own) / own)};
    const auto run = [&](auto iv, auto items) {
      using I = decltype(iv);
      constexpr int N = decltype(items)::value;
      order_split_kernel<I, N><<<grid, kSplitThreads, 0, stream>>>(static_cast<const I*>(tokens), int(n), int(rows),
                                                                   int(own), bits, order + o.row, order + o.pos);
    };
    const auto with = [&](auto iv) {
      if (n <= kSplitThreads * 8) run(iv, Int<8>());
      else run(iv, Int<16>());
    };
    wide ? with(int64_t()) : with(int32_t());
    return launched(who);
  }
  if (n <= kRankTokens) {
    const auto run = [&](auto iv) {
      using I = decltype(iv);
      order_rank_kernel<I><<<dim3(uint32_t((n + kRankEach - 1) / kRankEach)), kRankThreads, 0, stream>>>(
          static_cast<const I*>(tokens), int(n), int(rows), order + o.row, order + o.pos);
    };
    if (n > 0) wide ? run(int64_t()) : run(int32_t());
    return launched(who);
  }
  const int bits = row_bits(rows), passes = (bits + kSortBits - 1) / kSortBits, each = (bits + passes - 1) / passes;
  SortArgs a{};
  a.n = int32_t(n);
  a.rows = int32_t(rows);
  a.blocks = int32_t(o.blocks);
  a.scanned = o.blocks > kScanBlocks;
  a.digits = order + o.digits;
  int32_t *row[2] = {order + o.row, order + o.row2}, *pos[2] = {order + o.pos, order + o.pos2};
  for (int p = 0; p < passes; ++p) {
    const int to = (passes - 1 - p) & 1;       // the last pass ends in the order's own arrays
    const bool first = p == 0;
    a.shift = p * each;
    a.bits = std::min(each, bits - a.shift);
    a.in = first ? tokens : row[to ^ 1];
    a.pos_in = pos[to ^ 1];
    a.row_out = row[to];
    a.pos_out = pos[to];
    const auto run = [&](auto iv, auto fv) {
      using I = decltype(iv);
      constexpr bool FIRST = decltype(fv)::value;
      const dim3 grid{uint32_t(o.blocks)};
      order_count_kernel<I><<<grid, kSortThreads, 0, stream>>>(a);
      if (a.scanned) order_scan_kernel<<<dim3(kSortDigits / 64), 64 * kScanWaves, 0, stream>>>(a.digits, a.blocks);
      order_scatter_kernel<I, FIRST><<<grid, kSortThreads, 0, stream>>>(a);
    };
    if (!first) run(int32_t(), std::false_type());
    else if (wide) run(int64_t(), std::true_type());
    else run(int32_t(), std::true_type());
  }
  return launched(who);
}

int launch_embedding_grad(const int32_t* order, int64_t n, int64_t rows, int64_t dim, const void* d_out,
                          int32_t out_type, int64_t out_stride, float scale, void* grad, int32_t grad_type,
                          int64_t first, int64_t count, bool accumulate, float* ws, hipStream_t stream,
                          const char* who) {
  const Order o(n);
  EmbeddingGradArgs a{};
  a.row = order + o.row;
  a.pos = order + o.pos;
  a.d_out = d_out;
  a.grad = grad;
  a.ws = ws;
  a.stride = out_stride;
  a.first = first;
  a.count = count;
  a.scale = scale;
  a.n = int32_t(n);
  a.dim = int32_t(dim);
  a.dim4 = int32_t((dim + 3) / 4 * 4);
  const bool few = n <= kFewTokens;
  a.piece = few ? int32_t(std::max<int64_t>(1, (n + kWide - 1) / kWide)) : embedding_piece(n);
  a.pieces = int32_t((n + a.piece - 1) / a.piece);
  a.row_lo = int32_t(first / dim);
  a.row_hi = int32_t((first + count + dim - 1) / dim);
  const auto go = [&](auto tv, auto gv) {
    using T = decltype(tv);
    using G = decltype(gv);
    const auto with = [&](auto ev, auto add) {
      constexpr int E = decltype(ev)::value;
      constexpr bool ADD = decltype(add)::value;
      a.tiles = int32_t((dim + 64 * E - 1) / (64 * E));
      const int waves = few ? kWide : 4;
      const int64_t sums = few ? (n > 0 ? a.tiles : 0) : (int64_t(a.pieces) * a.tiles + 3) / 4;
      const int64_t fills = (int64_t(a.row_hi - a.row_lo + kFillRows - 1) / kFillRows * a.tiles + waves - 1) / waves;
      a.sum_blocks = int32_t(sums);
      const dim3 grid(uint32_t(sums + (ADD ? 0 : fills)));
      if (grid.x == 0) return;
      if (few) {
        embedding_grad_few_kernel<T, G, E, ADD><<<grid, 64 * kWide, 0, stream>>>(a);
        return;
      }
      embedding_grad_kernel<T, G, E, ADD><<<grid, 256, 0, stream>>>(a);
      constexpr int J = E == 1 ? 1 : 4;
      a.tiles = int32_t((dim + 64 * J - 1) / (64 * J));
      embedding_join_kernel<G, J, ADD>
          <<<dim3(uint32_t(a.pieces * ((a.tiles + kJoinTiles - 1) / kJoinTiles))), 64 * kJoinTiles, 0, stream>>>(a);
    };
    by_width<sizeof(T) == 2 && sizeof(G) == 2 ? 8 : 4>(dim, [&](auto ev) {
      accumulate ? with(ev, std::true_type()) : with(ev, std::false_type());
    });
  };
  by_types(out_type, grad_type, go);
  return launched(who);
}

static int launch_norm_rows(const zero_norm_args& a, hipStream_t stream, const char* who) {
  const auto go = [&](auto tv, auto wv) {
    using T = decltype(tv);
    using W = decltype(wv);
    constexpr int E = 16 / int(sizeof(T));
    const NormShape s = norm_shape(a.n, (a.dim + E - 1) / E);
    const uint32_t rows = s.threads == 0 || s.threads >= 256 ? 1u : 256u / uint32_t(s.threads);
    const dim3 grid{uint32_t((a.n + rows - 1) / rows)};
    const auto spread = [&](auto threads, auto vectors) {
      constexpr int TPR = decltype(threads)::value, V = decltype(vectors)::value;
      if (s.threads == TPR && s.vectors == V) norm_kernel<T, W, E, TPR, V><<<grid, TPR < 256 ? 256 : TPR, 0, stream>>>(a);
    };
    if (a.dim < E) {
      norm_kernel<T, W, 1, 16, 1><<<grid, 256, 0, stream>>>(a);
      return;
    }
    spread(Int<16>(), Int<1>());
    spread(Int<32>(), Int<1>());
    spread(Int<64>(), Int<1>());
    spread(Int<64>(), Int<2>());
    spread(Int<64>(), Int<4>());
    spread(Int<256>(), Int<1>());
    spread(Int<256>(), Int<2>());
    spread(Int<256>(), Int<4>());
    spread(Int<1024>(), Int<2>());
    spread(Int<1024>(), Int<4>());
    if (s.threads == 0) norm_long_kernel<T, W><<<grid, kLongThreads, 0, stream>>>(a);
  };
  by_types(a.type, a.weight_type, go);
  return launched(who);
}

// Rows of a launch: 2^21 blocks of 1024 threads are 2^31 work-items.
constexpr int64_t kLaunchRows = int64_t(1) << 21;

// p + k elements of the type; NULL stays.
template <typename P>
void advance(P*& p, int32_t type, int64_t k) {
  if (p != nullptr) p = reinterpret_cast<P*>(uintptr_t(p) + uintptr_t(k * (type == ZERO_BF16 ? 2 : 4)));
}

int launch_norm(const zero_norm_args& whole, hipStream_t stream, const char* who) {
  for (int64_t row = 0; row < whole.n; row += kLaunchRows) {
    zero_norm_args a = whole;
    a.n = std::min(kLaunchRows, whole.n - row);
    advance(a.x, a.type, row * a.x_stride);
    advance(a.residual, a.type, row * a.residual_stride);
    advance(a.total, a.type, row * a.total_stride);
    advance(a.y, a.type, row * a.y_stride);
    advance(a.mean, ZERO_F32, row);
    advance(a.rstd, ZERO_F32, row);
    if (int rc = launch_norm_rows(a, stream, who)) return rc;
  }
  return ok();
}

int launch_norm_grad(const zero_norm_grad_args& a, float* ws, hipStream_t stream, const char* who) {
  if (a.n <= few_norm_rows(a.dim)) {
    const auto few = [&](auto tv, auto wv) {
      using T = decltype(tv);
      using W = decltype(wv);
      by_width<16 / int(sizeof(T))>(a.dim, [&](auto ev) {
        constexpr int E = decltype(ev)::value;
        const int cols = a.d_weight != nullptr || a.d_bias != nullptr ? int((a.dim + 64 * E - 1) / (64 * E)) : 0;
        const int rows = a.d_x != nullptr ? int(a.n) : 0;
        const auto run = [&](auto vectors) {
          constexpr int V = decltype(vectors)::value;
          const auto put = [&](int c, int r) {
            if (c + r > 0) norm_grad_few_kernel<T, W, E, V><<<dim3(uint32_t(c + r)), kFewThreads, 0, stream>>>(a, c);
          };
          if (a.d_x == a.d_y || a.d_x == a.x) {      // the columns before the rows write over them
            put(cols, 0);
            put(0, rows);
          } else {
            put(cols, rows);
          }
        };
        if constexpr (E == 4) {
          if (a.dim > kFewThreads * E) {
            run(Int<2>());
            return;
          }
        }
        run(Int<1>());
      });
    };
    by_types(a.type, a.weight_type, few);
    return launched(who);
  }
  const int64_t blocks = norm_grad_blocks(a.n, a.dim);
  const int dim = int(a.dim), dim4 = (dim + 3) / 4 * 4;
  const bool sums = a.d_weight != nullptr || a.d_bias != nullptr;
  const auto go = [&](auto tv, auto wv) {
    using T = decltype(tv);
    using W = decltype(wv);
    constexpr int E = 16 / int(sizeof(T));
    const NormShape s = norm_grad_shape(a.dim, E);
    const auto spread = [&](auto threads, auto vectors) {
      constexpr int TPR = decltype(threads)::value, V = decltype(vectors)::value;
      if (s.threads != TPR || s.vectors != V) return;
      norm_grad_kernel<T, W, E, TPR, V><<<dim3(uint32_t(blocks)), grad_threads(TPR), 0, stream>>>(a, ws, dim4);
    };
    if (a.dim < E) {
      norm_grad_kernel<T, W, 1, 16, 1><<<dim3(uint32_t(blocks)), grad_threads(16), 0, stream>>>(a, ws, dim4);
      return;
    }
    spread(Int<16>(), Int<1>());
    spread(Int<32>(), Int<1>());
    spread(Int<64>(), Int<1>());
    spread(Int<128>(), Int<1>());
    spread(Int<192>(), Int<1>());
    spread(Int<256>(), Int<1>());
    spread(Int<320>(), Int<1>());
    spread(Int<384>(), Int<1>());
    spread(Int<512>(), Int<1>());
    spread(Int<640>(), Int<1>());
    spread(Int<768>(), Int<1>());
    if constexpr (E == 4) {
      spread(Int<512>(), Int<2>());
      spread(Int<640>(), Int<2>());
      spread(Int<768>(), Int<2>());
    }
    spread(Int<1024>(), Int<8 / E>());
    if (s.threads != 0) return;
    if (sums)
      norm_grad_columns_kernel<T><<<dim3(uint32_t((dim + 256 * E - 1) / (256 * E)), uint32_t(blocks)), 256, 0, stream>>>(
          a, ws, dim4);
    if (a.d_x != nullptr && a.n > 0)
      norm_grad_long_kernel<T, W><<<dim3(uint32_t(a.n)), kLongThreads, 0, stream>>>(a);
  };
  by_types(a.type, a.weight_type, go);
  if (sums)
    norm_grad_join_kernel<<<dim3(uint32_t((dim + 63) / 64), 2), 64 * kJoinWaves, 0, stream>>>(
        ws, int(blocks), dim, dim4, a.d_weight, a.d_bias, a.grad_type, a.accumulate);
  return launched(who);
}

}  // namespace zero
