// Kernels of the token-table and norm calls (zero_layers.h) and their launches.
// Part of device.hip, after tensors.hip.
//
//   embedding_kernel         rows of a table, scaled
//   order_rank_kernel        the sort of few tokens, by counting
//   order_count_kernel, order_scatter_kernel
//                            one pass of the sort of many tokens
//   embedding_grad_kernel    sums of pieces of the sorted tokens, and zeros for
//                            the rows without one
//   embedding_join_kernel    the sums of runs that several pieces share
//   norm_kernel, norm_long_kernel
//                            the norm of rows in registers, and of longer ones
//   norm_grad_kernel, norm_grad_long_kernel, norm_grad_columns_kernel,
//   norm_grad_join_kernel    its gradient
#include "layers_internal.h"

namespace {

using zero::kPiece;
using zero::kSortBits;
using zero::kSortBlock;
using zero::kSortDigits;
using zero::kSortItems;
using zero::kSortThreads;
using zero::NormShape;
using zero::Order;

// ------------------------------------------------------- E elements of a row
//
// A lane owns E consecutive elements, of which `cnt` exist (fewer than E at a
// row's end only, none beyond). Rows start at any element, so the accesses are
// declared with their element's alignment: the hardware takes them at any
// address.

template <int E, typename T> struct Words;
template <> struct Words<8, uint16_t> { u32x4 w; };
template <> struct Words<4, uint16_t> { u32x2 w; };
template <> struct Words<4, float> { f32x4 w; };
template <> struct Words<8, float> { f32x4 w, w2; };

template <typename V>
__device__ __forceinline__ V plain_load(const void* p) { return *(const ZERO_GLOBAL V*)p; }

template <int E, bool STREAM = true, typename T>
__device__ __forceinline__ Words<E, T> load_row(const T* p, int cnt) {
  Words<E, T> r;
  if (cnt >= E) {
    if constexpr (sizeof(T) == 2 && E == 8) r.w = STREAM ? stream_load<words4_any>(p) : plain_load<words4_any>(p);
    else if constexpr (sizeof(T) == 2) r.w = STREAM ? stream_load<bf16x4_any>(p) : plain_load<bf16x4_any>(p);
    else r.w = STREAM ? stream_load<f32x4_any>(p) : plain_load<f32x4_any>(p);
    if constexpr (sizeof(T) == 4 && E == 8) r.w2 = STREAM ? stream_load<f32x4_any>(p + 4) : plain_load<f32x4_any>(p + 4);
    return r;
  }
  r = Words<E, T>{};
#pragma unroll
  for (int k = 0; k < E - 1; ++k) {
    if (k >= cnt) continue;
    if constexpr (sizeof(T) == 2) r.w[k >> 1] |= uint32_t(p[k]) << (16 * (k & 1));
    else if constexpr (E == 8) { if (k < 4) r.w[k & 3] = p[k]; else r.w2[k & 3] = p[k]; }
    else r.w[k] = p[k];
  }
  return r;
}

template <int E, typename T>
__device__ __forceinline__ void widen(const Words<E, T>& r, float (&x)[E]) {
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if constexpr (sizeof(T) == 2) x[k] = (k & 1) ? bf16_hi(r.w[k >> 1]) : bf16_lo(r.w[k >> 1]);
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
    if constexpr (sizeof(T) == 2) { if ((k & 1) == 0) r.w[k >> 1] = pack_bf16x2(x[k], x[k + 1]); }
    else if constexpr (E == 8) { if (k < 4) r.w[k & 3] = x[k]; else r.w2[k & 3] = x[k]; }
    else r.w[k] = x[k];
  }
  return r;
}

// The elements [lo, cnt) of the lane's E.
template <int E, typename T>
__device__ __forceinline__ void store_some(T* p, int lo, int cnt, const Words<E, T>& r) {
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if (k < lo || k >= cnt) continue;
    if constexpr (sizeof(T) == 2) p[k] = uint16_t(r.w[k >> 1] >> (16 * (k & 1)));
    else if constexpr (E == 8) p[k] = k < 4 ? r.w[k & 3] : r.w2[k & 3];
    else p[k] = r.w[k];
  }
}

template <int E, bool STREAM = true, typename T>
__device__ __forceinline__ void store_row(T* p, int cnt, const Words<E, T>& r) {
  if (cnt < E) {
    store_some<E, T>(p, 0, cnt, r);
    return;
  }
  if constexpr (STREAM) {
    if constexpr (sizeof(T) == 2 && E == 8) stream_store<words4_any>(p, r.w);
    else if constexpr (sizeof(T) == 2) stream_store<bf16x4_any>(p, r.w);
    else stream_store<f32x4_any>(p, r.w);
    if constexpr (sizeof(T) == 4 && E == 8) stream_store<f32x4_any>(p + 4, r.w2);
  } else {
    if constexpr (sizeof(T) == 2 && E == 8) *(ZERO_GLOBAL words4_any*)p = r.w;
    else if constexpr (sizeof(T) == 2) *(ZERO_GLOBAL bf16x4_any*)p = r.w;
    else *(ZERO_GLOBAL f32x4_any*)p = r.w;
    if constexpr (sizeof(T) == 4 && E == 8) *(ZERO_GLOBAL f32x4_any*)(p + 4) = r.w2;
  }
}

// ------------------------------------------------------------------- lookup

// Token t's row, or `rows` for a token outside the table.
__device__ __forceinline__ int table_row(const void* tokens, bool wide, int64_t t, int rows) {
  const int64_t k = wide ? static_cast<const int64_t*>(tokens)[t] : int64_t(static_cast<const int32_t*>(tokens)[t]);
  return k >= 0 && k < rows ? int(k) : rows;
}
__device__ __forceinline__ int uniform_row(const void* tokens, bool wide, int64_t t, int rows) {
  const int64_t k = wide ? uniform_load(static_cast<const int64_t*>(tokens) + t)
                         : int64_t(uniform_load(static_cast<const int32_t*>(tokens) + t));
  return k >= 0 && k < rows ? int(k) : rows;
}

constexpr int kLookupRows = 4;      // rows of a wave: as many loads in flight

template <typename T, typename O, int E>
__global__ __launch_bounds__(256) void embedding_kernel(const void* __restrict__ tokens, int wide, int n,
                                                        const T* __restrict__ table, int rows, int dim, int tiles,
                                                        float scale, O* __restrict__ out, int64_t stride) {
  const int64_t w = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = w / tiles * kLookupRows;
  if (t0 >= n) return;
  const int col = int(w % tiles) * 64 * E + int(threadIdx.x & 63) * E;
  const int cnt = dim - col;
  Words<E, T> x[kLookupRows];
#pragma unroll
  for (int k = 0; k < kLookupRows; ++k) {
    const int row = t0 + k < n ? uniform_row(tokens, wide, t0 + k, rows) : rows;
    x[k] = load_row<E, false>(table + int64_t(row) * dim + col, row < rows ? cnt : 0);
  }
#pragma unroll
  for (int k = 0; k < kLookupRows; ++k) {
    if (t0 + k >= n) break;
    float v[E];
    widen<E, T>(x[k], v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= scale;
    store_row<E>(out + (t0 + k) * stride + col, cnt, narrow<E, O>(v));
  }
}

// --------------------------------------------------------------------- sort

// Few tokens: a token's place is the number of tokens before it, those of lower
// rows and those of its own row at lower positions. The 64 tokens of a block are
// compared with all of them, its 16 waves taking a part each. The blocks after
// those set the bits of the rows that have a token, 2^18 rows a block.
constexpr int kRankThreads = 1024, kRankWaves = kRankThreads / 64;
constexpr int kBitWords = 8192;

__global__ __launch_bounds__(kRankThreads) void order_rank_kernel(const void* __restrict__ tokens, int wide, int n,
                                                                  int rows, int rank_blocks, int32_t* __restrict__ head,
                                                                  int32_t* __restrict__ row, int32_t* __restrict__ pos,
                                                                  uint32_t* __restrict__ bits) {
  __shared__ int32_t key[zero::kRankTokens + 256];
  __shared__ int32_t part[kRankWaves][64];
  __shared__ uint32_t word[kBitWords];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  if (int(blockIdx.x) >= rank_blocks) {
    const int w0 = (int(blockIdx.x) - rank_blocks) * kBitWords;
    const int words = min(kBitWords, (rows + 31) / 32 - w0);
    for (int k = t; k < words; k += kRankThreads) word[k] = 0;
    __syncthreads();
    for (int k = t; k < n; k += kRankThreads) {
      const int r = table_row(tokens, wide, k, rows);
      const int at = (r >> 5) - w0;
      if (r < rows && at >= 0 && at < words) atomicOr(&word[at], 1u << (r & 31));
    }
    __syncthreads();
    for (int k = t; k < words; k += kRankThreads) bits[w0 + k] = word[k];
    return;
  }
  // a wave's part: whole fours of tokens
  const int each = ((n + kRankWaves - 1) / kRankWaves + 3) / 4 * 4;
  const int padded = each * kRankWaves;         // at most kRankTokens + 60
  for (int k = t; k < padded; k += kRankThreads) key[k] = k < n ? table_row(tokens, wide, k, rows) : 0x7FFFFFFF;
  __syncthreads();
  const int i = int(blockIdx.x) * 64 + lane;
  const int mine = i < n ? key[i] : 0x7FFFFFFF;
  int before = 0;
  for (int j = wave * each; j < (wave + 1) * each; j += 4) {
    const int4 k4 = *reinterpret_cast<const int4*>(&key[j]);
    const int k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) before += (k[e] < mine || (k[e] == mine && j + e < i)) ? 1 : 0;
  }
  part[wave][lane] = before;
  __syncthreads();
  if (wave == 0 && i < n) {
    int at = 0;
#pragma unroll
    for (int k = 0; k < kRankWaves; ++k) at += part[k][lane];
    row[at] = mine;
    pos[at] = i;
  }
  if (blockIdx.x == 0) {       // how many lie in the table
    int live = 0;
    for (int k = t; k < n; k += kRankThreads) live += key[k] < rows ? 1 : 0;
    __syncthreads();
    for (int off = 32; off >= 1; off >>= 1) live += __shfl_xor(live, off, 64);
    if (lane == 0) part[wave][0] = live;
    __syncthreads();
    if (t == 0) {
      int sum = 0;
      for (int k = 0; k < kRankWaves; ++k) sum += part[k][0];
      *head = sum;
    }
  }
}

// Many tokens: passes over the row numbers' digits of up to 9 bits from the
// lowest on, each of which keeps the order of equal digits. A pass counts the
// digits of every block's 2048 tokens, then places every token behind those of
// lower digits, those of earlier blocks and those before it in its block.
struct SortArgs {
  const void* tokens;      // of the first pass; later ones read row_in and pos_in
  int32_t wide, n, rows, shift, bits, blocks;
  const int32_t *row_in, *pos_in;
  int32_t *row_out, *pos_out;
  int32_t *digits, *live, *head;
  uint32_t* present;
};

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void order_count_kernel(SortArgs a) {
  __shared__ int32_t count[kSortDigits];
  const int t = threadIdx.x;
  for (int k = t; k < kSortDigits; k += kSortThreads) count[k] = 0;
  __syncthreads();
  int live = 0;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = int(blockIdx.x) * kSortBlock + k * kSortThreads + t;
    if (i >= a.n) break;
    const int r = FIRST ? table_row(a.tokens, a.wide, i, a.rows) : a.row_in[i];
    atomicAdd(&count[(r >> a.shift) & ((1 << a.bits) - 1)], 1);
    live += r < a.rows ? 1 : 0;
  }
  if (FIRST)        // the bits, cleared for the scatter that follows
    for (int k = int(blockIdx.x) * kSortThreads + t; k < (a.rows + 31) / 32; k += a.blocks * kSortThreads) a.present[k] = 0;
  __syncthreads();
  for (int k = t; k < (1 << a.bits); k += kSortThreads) a.digits[int64_t(blockIdx.x) * kSortDigits + k] = count[k];
  if (FIRST) {
    __shared__ int32_t sum[kSortThreads / 64];
    for (int off = 32; off >= 1; off >>= 1) live += __shfl_xor(live, off, 64);
    if ((t & 63) == 0) sum[t >> 6] = live;
    __syncthreads();
    if (t == 0) a.live[blockIdx.x] = sum[0] + sum[1] + sum[2] + sum[3];
  }
}

template <bool FIRST, bool LAST>
__global__ __launch_bounds__(kSortThreads) void order_scatter_kernel(SortArgs a) {
  constexpr int kWaves = kSortThreads / 64;
  __shared__ int32_t base[kSortDigits];             // where the block's tokens of a digit begin
  __shared__ int32_t seen[kWaves][kSortDigits];     // then: where the wave's do
  __shared__ int32_t wave_sum[kWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int n_digits = 1 << a.bits;
  for (int k = t; k < kWaves * kSortDigits; k += kSortThreads) (&seen[0][0])[k] = 0;
  // two digits a thread: all blocks' tokens of lower digits, and the earlier blocks' of its own
  int total[2] = {0, 0}, before[2] = {0, 0};
  for (int b = 0; b < a.blocks; ++b) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int d = 2 * t + k;
      const int c = d < n_digits ? a.digits[int64_t(b) * kSortDigits + d] : 0;
      total[k] += c;
      before[k] += b < int(blockIdx.x) ? c : 0;
    }
  }
  int up = total[0] + total[1];
  const int own = up;
  for (int off = 1; off < 64; off <<= 1) {
    const int x = __shfl_up(up, off, 64);
    if (lane >= off) up += x;
  }
  if (lane == 63) wave_sum[wave] = up;
  __syncthreads();
  int lower = up - own;
  for (int w = 0; w < wave; ++w) lower += wave_sum[w];
  base[2 * t] = lower + before[0];
  base[2 * t + 1] = lower + total[0] + before[1];
  // a wave's tokens are consecutive: 64 at a time, each one's rank among those of its digit
  const int first = int(blockIdx.x) * kSortBlock + wave * 64 * kSortItems;
  int row[kSortItems], pos[kSortItems], rank[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = first + k * 64 + lane;
    row[k] = i >= a.n ? -1 : FIRST ? table_row(a.tokens, a.wide, i, a.rows) : a.row_in[i];
    pos[k] = i >= a.n ? 0 : FIRST ? i : a.pos_in[i];
  }
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
    if (FIRST && row[k] < a.rows) atomicOr(&a.present[row[k] >> 5], 1u << (row[k] & 31));
  }
  if (LAST && blockIdx.x == 0 && wave == 0) {
    int live = 0;
    for (int b = lane; b < a.blocks; b += 64) live += a.live[b];
    for (int off = 32; off >= 1; off >>= 1) live += __shfl_xor(live, off, 64);
    if (lane == 0) *a.head = live;
  }
}

// ---------------------------------------------------- the table's gradient

struct EmbeddingGradArgs {
  const int32_t *head, *row, *pos;
  const uint32_t* present;
  const void* d_out;
  void* grad;
  float* ws;                 // [pieces][2][dim4]: sums of a run's middle or end, and of its beginning
  int64_t stride, first, count;
  float scale;
  int32_t dim, dim4, tiles, pieces;
  int32_t row_lo, row_hi;    // rows that the part touches
  int32_t sum_blocks, accumulate;
};

// The part's elements of row r at column col, E of them from there: grad's
// element index, and which of the E lie in the part.
struct Place {
  int64_t at;
  int lo, hi;
};
template <int E>
__device__ __forceinline__ Place place_of(const EmbeddingGradArgs& a, int r, int col) {
  Place p;
  p.at = int64_t(r) * a.dim + col - a.first;
  const int64_t end = a.count - p.at;
  p.lo = p.at >= 0 ? 0 : p.at <= -E ? E : int(-p.at);
  p.hi = min(end >= E ? E : end <= 0 ? 0 : int(end), a.dim - col);
  return p;
}

template <int E, typename G>
__device__ __forceinline__ void write_row(const EmbeddingGradArgs& a, const Place& p, const Words<E, G>& old,
                                          const float (&sum)[E]) {
  float v[E];
  if (a.accumulate) {
    widen<E, G>(old, v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(sum[e], a.scale, v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = sum[e] * a.scale;
  }
  G* g = static_cast<G*>(a.grad) + p.at;
  const Words<E, G> w = narrow<E, G>(v);
  if (p.lo == 0 && p.hi >= E) store_row<E>(g, E, w);
  else store_some<E, G>(g, p.lo, p.hi, w);
}

template <int E, typename G>
__device__ __forceinline__ Words<E, G> read_row(const EmbeddingGradArgs& a, const Place& p) {
  const G* g = static_cast<const G*>(a.grad) + p.at;
  if (p.lo == 0 && p.hi >= E) return load_row<E>(g, E);
  Words<E, G> r{};
#pragma unroll
  for (int k = 0; k < E; ++k) {
    if (k < p.lo || k >= p.hi) continue;
    if constexpr (sizeof(G) == 2) r.w[k >> 1] |= uint32_t(g[k]) << (16 * (k & 1));
    else r.w[k] = g[k];
  }
  return r;
}

constexpr int kBatch = 8;      // rows that a wave loads before it adds them

template <typename T, typename G, int E>
__global__ __launch_bounds__(256) void embedding_grad_kernel(const EmbeddingGradArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (int(blockIdx.x) >= a.sum_blocks) {      // zeros, a wave a row
    const int r = a.row_lo + (int(blockIdx.x) - a.sum_blocks) * 4 + wave;
    if (r >= a.row_hi || (uniform_load(a.present + (r >> 5)) >> (r & 31) & 1)) return;
    const Words<E, G> zero{};
    for (int col = lane * E; col < a.dim; col += 64 * E) {
      const Place p = place_of<E>(a, r, col);
      G* g = static_cast<G*>(a.grad) + p.at;
      if (p.lo == 0 && p.hi >= E) store_row<E>(g, E, zero);
      else store_some<E, G>(g, p.lo, p.hi, zero);
    }
    return;
  }
  const int64_t w = int64_t(blockIdx.x) * 4 + wave;
  const int piece = int(w / a.tiles);
  if (piece >= a.pieces) return;
  const int col = int(w % a.tiles) * 64 * E + lane * E;
  const int cnt = a.dim - col;
  const int live = uniform_load(a.head);
  const int i0 = piece * kPiece, i1 = min(i0 + kPiece, live);
  if (i0 >= i1) return;
  const int r_first = uniform_load(a.row + i0), r_last = uniform_load(a.row + i1 - 1);
  if (r_last < a.row_lo || r_first >= a.row_hi) return;
  bool head = i0 > 0 && uniform_load(a.row + i0 - 1) == r_first;     // the run at hand began in an earlier piece
  const int next = i1 < live ? uniform_load(a.row + i1) : -1;
  float sum[E] = {};
  for (int i = i0; i < i1; i += kBatch) {
    int r[kBatch + 1];
    Words<E, T> x[kBatch];
    Words<E, G> old[kBatch];
    Place p[kBatch];
#pragma unroll
    for (int k = 0; k <= kBatch; ++k) r[k] = i + k < i1 ? uniform_load(a.row + i + k) : i + k == i1 ? next : -1;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const bool mine = i + k < i1 && r[k] >= a.row_lo && r[k] < a.row_hi;
      const int64_t at = mine ? int64_t(uniform_load(a.pos + i + k)) * a.stride + col : 0;
      x[k] = load_row<E>(static_cast<const T*>(a.d_out) + at, mine ? cnt : 0);
      p[k] = place_of<E>(a, r[k], col);
      old[k] = Words<E, G>{};
      if (a.accumulate && mine && r[k] != r[k + 1]) old[k] = read_row<E, G>(a, p[k]);
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
        if (head || !end) {
          if (cnt > 0) {
            float* s = a.ws + (int64_t(piece) * 2 + (head ? 0 : 1)) * a.dim4 + col;
            store_row<E, false>(s, cnt, narrow<E, float>(sum));
          }
        } else {
          write_row<E, G>(a, p[k], old[k], sum);
        }
      }
      head = false;
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] = 0.f;
    }
  }
}

template <typename G, int E>
__global__ __launch_bounds__(256) void embedding_join_kernel(const EmbeddingGradArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t w = int64_t(blockIdx.x) * 4 + wave;
  const int piece = int(w / a.tiles);
  if (piece >= a.pieces) return;
  const int col = int(w % a.tiles) * 64 * E + lane * E;
  const int cnt = a.dim - col;
  const int live = uniform_load(a.head);
  const int i0 = piece * kPiece, i1 = i0 + kPiece;
  if (i1 >= live) return;
  const int r = uniform_load(a.row + i1);
  if (uniform_load(a.row + i1 - 1) != r || r < a.row_lo || r >= a.row_hi) return;
  if (i0 > 0 && uniform_load(a.row + i0) == r && uniform_load(a.row + i0 - 1) == r) return;    // began earlier
  const float* s = a.ws + int64_t(piece) * 2 * a.dim4 + col;
  float sum[E];
  widen<E, float>(load_row<E, false>(s + a.dim4, cnt), sum);
  for (int j = piece + 1; j * kPiece < live && uniform_load(a.row + j * kPiece) == r; ++j) {
    s += 2 * a.dim4;
    float v[E];
    widen<E, float>(load_row<E, false>(s, cnt), v);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] += v[e];
  }
  const Place p = place_of<E>(a, r, col);
  Words<E, G> old{};
  if (a.accumulate) old = read_row<E, G>(a, p);
  write_row<E, G>(a, p, old, sum);
}

// --------------------------------------------------------------------- norm

// E elements of a vector of either type, as fp32; ones or zeros where there is none.
template <int E>
__device__ __forceinline__ void load_weight(const void* w, bool bf16, int col, int cnt, float none, float (&x)[E]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = none;
  } else if (bf16) {
    widen<E, uint16_t>(load_row<E, false>(static_cast<const uint16_t*>(w) + col, cnt), x);
  } else {
    widen<E, float>(load_row<E, false>(static_cast<const float*>(w) + col, cnt), x);
  }
}

// The sum of K values over the TPR threads that share a row, in every one of
// them. lds: of a block's waves, for TPR above 64; a block that calls it again
// takes the other half (`turn`), so one barrier a call suffices.
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&x)[K], float* lds, int turn) {
#pragma unroll
  for (int off = (TPR < 64 ? TPR : 64) / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] += __shfl_xor(x[k], off, 64);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    float* s = lds + turn * K * kWaves;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[k * kWaves + (threadIdx.x >> 6)] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) x[k] += s[k * kWaves + w];
    }
  }
}

template <typename T, int TPR, int V>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(const zero_norm_args a) {
  constexpr int E = 16 / int(sizeof(T));
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  __shared__ float lds[2 * (TPR / 64 + 1)];
  const int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  if (row >= a.n) return;          // whole rows: with TPR above 64 a block has one
  const int dim = int(a.dim);
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  Words<E, T> raw[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int col = (t + k * TPR) * E;
    raw[k] = load_row<E>(x + col, dim - col);
  }
  float v[V][E];
  if (a.residual != nullptr) {
    const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
    T* total = static_cast<T*>(a.total) + row * a.total_stride;
    Words<E, T> more[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int col = (t + k * TPR) * E;
      more[k] = load_row<E>(res + col, dim - col);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int col = (t + k * TPR) * E;
      float r[E];
      widen<E, T>(raw[k], v[k]);
      widen<E, T>(more[k], r);
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] += r[e];
      raw[k] = narrow<E, T>(v[k]);
      store_row<E>(total + col, dim - col, raw[k]);
    }
  }
  float s[1] = {0.f};
#pragma unroll
  for (int k = 0; k < V; ++k) {
    widen<E, T>(raw[k], v[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) s[0] += v[k][e];
  }
  float mean = 0.f;
  if (!a.rms) {
    row_sum<TPR, 1>(s, lds, 0);
    mean = s[0] / float(dim);
  }
  s[0] = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int rest = dim - (t + k * TPR) * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float d = e < rest ? v[k][e] - mean : 0.f;
      s[0] = fmaf(d, d, s[0]);
    }
  }
  row_sum<TPR, 1>(s, lds, 1);
  const float rstd = 1.f / sqrtf(s[0] / float(dim) + float(a.eps));
  if (t == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
  const bool bf16 = a.weight_type == ZERO_BF16;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int col = (t + k * TPR) * E;
    float w[E], b[E];
    load_weight<E>(a.weight, bf16, col, dim - col, 1.f, w);
    load_weight<E>(a.bias, bf16, col, dim - col, 0.f, b);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = fmaf((v[k][e] - mean) * rstd, w[e], b[e]);
    store_row<E>(y + col, dim - col, narrow<E, T>(w));
  }
}

// A row longer than the registers of a block: three passes over it, the later
// ones from the caches. Element by element, so that y and total may be x.
constexpr int kLongThreads = 1024;

template <typename T>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(const zero_norm_args a) {
  constexpr int E = 16 / int(sizeof(T));
  __shared__ float lds[2 * (kLongThreads / 64)];
  const int64_t row = blockIdx.x;
  const int dim = int(a.dim);
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + row * a.residual_stride : nullptr;
  T* total = res != nullptr ? static_cast<T*>(a.total) + row * a.total_stride : nullptr;
  float s[1] = {0.f};
  for (int col = threadIdx.x * E; col < dim; col += kLongThreads * E) {
    float v[E];
    Words<E, T> raw = load_row<E, false>(x + col, dim - col);
    widen<E, T>(raw, v);
    if (res != nullptr) {
      float r[E];
      widen<E, T>(load_row<E, false>(res + col, dim - col), r);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += r[e];
      raw = narrow<E, T>(v);
      store_row<E, false>(total + col, dim - col, raw);
      widen<E, T>(raw, v);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s[0] += v[e];
  }
  if (res != nullptr) x = total;       // every thread reads back what it wrote
  float mean = 0.f;
  if (!a.rms) {
    row_sum<kLongThreads, 1>(s, lds, 0);
    mean = s[0] / float(dim);
  }
  s[0] = 0.f;
  for (int col = threadIdx.x * E; col < dim; col += kLongThreads * E) {
    float v[E];
    widen<E, T>(load_row<E, false>(x + col, dim - col), v);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float d = col + e < dim ? v[e] - mean : 0.f;
      s[0] = fmaf(d, d, s[0]);
    }
  }
  row_sum<kLongThreads, 1>(s, lds, 1);
  const float rstd = 1.f / sqrtf(s[0] / float(dim) + float(a.eps));
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
  const bool bf16 = a.weight_type == ZERO_BF16;
  for (int col = threadIdx.x * E; col < dim; col += kLongThreads * E) {
    float v[E], w[E], b[E];
    widen<E, T>(load_row<E, false>(x + col, dim - col), v);
    load_weight<E>(a.weight, bf16, col, dim - col, 1.f, w);
    load_weight<E>(a.bias, bf16, col, dim - col, 0.f, b);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
    store_row<E, false>(y + col, dim - col, narrow<E, T>(w));
  }
}

// ---------------------------------------------------------- norm's gradient

// A block takes every gridDim.x-th row (or group of rows) and keeps the sums of
// d_weight and d_bias over them in registers; its waves' sums meet in LDS and go
// to the workspace, which norm_grad_join_kernel adds up.
template <typename T, int TPR, int V>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_grad_kernel(const zero_norm_grad_args a, float* ws, int dim4) {
  constexpr int E = 16 / int(sizeof(T));
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  __shared__ float lds[4 * (TPR / 64 + 1)];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int dim = int(a.dim);
  float w[V][E], sum_w[V][E], sum_b[V][E];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int col = (t + k * TPR) * E;
    load_weight<E>(a.weight, a.weight_type == ZERO_BF16, col, dim - col, 1.f, w[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) sum_w[k][e] = sum_b[k][e] = 0.f;
  }
  int turn = 0;
  for (int64_t row = int64_t(blockIdx.x) * kRows + group; row < a.n; row += int64_t(gridDim.x) * kRows) {
    const T* dy = static_cast<const T*>(a.d_y) + row * a.d_y_stride;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    Words<E, T> dy_raw[V], x_raw[V], more[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int col = (t + k * TPR) * E;
      dy_raw[k] = load_row<E>(dy + col, dim - col);
      x_raw[k] = load_row<E>(x + col, dim - col);
    }
    const bool with_total = a.d_total != nullptr;
    if (with_total) {
      const T* d_total = static_cast<const T*>(a.d_total) + row * a.d_total_stride;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int col = (t + k * TPR) * E;
        more[k] = load_row<E>(d_total + col, dim - col);
      }
    }
    const float mean = a.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int rest = dim - (t + k * TPR) * E;
      float g[E], xh[E];
      widen<E, T>(dy_raw[k], g);
      widen<E, T>(x_raw[k], xh);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xh[e] = e < rest ? (xh[e] - mean) * rstd : 0.f;
        sum_w[k][e] = fmaf(g[e], xh[e], sum_w[k][e]);
        sum_b[k][e] += g[e];
        const float gw = g[e] * w[k][e];
        s[0] += gw;
        s[1] = fmaf(gw, xh[e], s[1]);
      }
    }
    if (a.d_x == nullptr) continue;
    row_sum<TPR, 2>(s, lds, turn);
    turn ^= 1;
    const float c0 = a.rms ? 0.f : s[0] / float(dim), c1 = s[1] / float(dim);
    T* dx = static_cast<T*>(a.d_x) + row * a.d_x_stride;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int col = (t + k * TPR) * E;
      float g[E], xh[E], m[E];
      widen<E, T>(dy_raw[k], g);
      widen<E, T>(x_raw[k], xh);
#pragma unroll
      for (int e = 0; e < E; ++e) m[e] = 0.f;
      if (with_total) widen<E, T>(more[k], m);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xh[e] = (xh[e] - mean) * rstd;
        g[e] = fmaf(fmaf(-xh[e], c1, g[e] * w[k][e] - c0), rstd, m[e]);
      }
      store_row<E>(dx + col, dim - col, narrow<E, T>(g));
    }
  }
  if (a.d_weight == nullptr && a.d_bias == nullptr) return;
  float* out = ws + int64_t(blockIdx.x) * 2 * dim4;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int col = (t + k * TPR) * E;
      store_row<E, false>(out + col, dim - col, narrow<E, float>(sum_w[k]));
      store_row<E, false>(out + dim4 + col, dim - col, narrow<E, float>(sum_b[k]));
    }
  } else {
    __shared__ float part[256 * V * E];       // [group][V * E][TPR]: lanes next to each other
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e)
          part[(group * V * E + k * E + e) * TPR + t] = which ? sum_b[k][e] : sum_w[k][e];
      __syncthreads();
      for (int j = threadIdx.x; j < V * E * TPR; j += 256) {
        float s = 0.f;
#pragma unroll
        for (int g = 0; g < kRows; ++g) s += part[g * V * E * TPR + j];
        const int ke = j / TPR, col = (j % TPR + ke / E * TPR) * E + ke % E;
        if (col < dim) out[which * dim4 + col] = s;
      }
    }
  }
}

// Rows longer than the registers: the rows' gradient in two passes over each.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void norm_grad_long_kernel(const zero_norm_grad_args a) {
  constexpr int E = 16 / int(sizeof(T));
  __shared__ float lds[2 * (kLongThreads / 64)];
  const int64_t row = blockIdx.x;
  const int dim = int(a.dim);
  const T* dy = static_cast<const T*>(a.d_y) + row * a.d_y_stride;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* d_total = a.d_total != nullptr ? static_cast<const T*>(a.d_total) + row * a.d_total_stride : nullptr;
  T* dx = static_cast<T*>(a.d_x) + row * a.d_x_stride;
  const bool bf16 = a.weight_type == ZERO_BF16;
  const float mean = a.rms ? 0.f : a.mean[row], rstd = a.rstd[row];
  float s[2] = {0.f, 0.f};
  for (int col = threadIdx.x * E; col < dim; col += kLongThreads * E) {
    float g[E], xh[E], w[E];
    widen<E, T>(load_row<E, false>(dy + col, dim - col), g);
    widen<E, T>(load_row<E, false>(x + col, dim - col), xh);
    load_weight<E>(a.weight, bf16, col, dim - col, 1.f, w);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float gw = col + e < dim ? g[e] * w[e] : 0.f;
      s[0] += gw;
      s[1] = fmaf(gw, (xh[e] - mean) * rstd, s[1]);
    }
  }
  row_sum<kLongThreads, 2>(s, lds, 0);
  const float c0 = a.rms ? 0.f : s[0] / float(dim), c1 = s[1] / float(dim);
  for (int col = threadIdx.x * E; col < dim; col += kLongThreads * E) {
    float g[E], xh[E], w[E], m[E];
    widen<E, T>(load_row<E, false>(dy + col, dim - col), g);
    widen<E, T>(load_row<E, false>(x + col, dim - col), xh);
    load_weight<E>(a.weight, bf16, col, dim - col, 1.f, w);
#pragma unroll
    for (int e = 0; e < E; ++e) m[e] = 0.f;
    if (d_total != nullptr) widen<E, T>(load_row<E, false>(d_total + col, dim - col), m);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      xh[e] = (xh[e] - mean) * rstd;
      g[e] = fmaf(fmaf(-xh[e], c1, g[e] * w[e] - c0), rstd, m[e]);
    }
    store_row<E, false>(dx + col, dim - col, narrow<E, T>(g));
  }
}

// Their column sums: a thread takes E columns of every gridDim.y-th row. Before
// the rows' gradient, which may overwrite d_y or x.
template <typename T>
__global__ __launch_bounds__(256) void norm_grad_columns_kernel(const zero_norm_grad_args a, float* ws, int dim4) {
  constexpr int E = 16 / int(sizeof(T));
  const int col = (int(blockIdx.x) * 256 + int(threadIdx.x)) * E, dim = int(a.dim);
  if (col >= dim) return;
  float sum_w[E] = {}, sum_b[E] = {};
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    const float mean = a.rms ? 0.f : uniform_load(a.mean + row), rstd = uniform_load(a.rstd + row);
    float g[E], xh[E];
    widen<E, T>(load_row<E, false>(static_cast<const T*>(a.d_y) + row * a.d_y_stride + col, dim - col), g);
    widen<E, T>(load_row<E, false>(static_cast<const T*>(a.x) + row * a.x_stride + col, dim - col), xh);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sum_w[e] = fmaf(g[e], (xh[e] - mean) * rstd, sum_w[e]);
      sum_b[e] += g[e];
    }
  }
  float* out = ws + int64_t(blockIdx.y) * 2 * dim4 + col;
  store_row<E, false>(out, dim - col, narrow<E, float>(sum_w));
  store_row<E, false>(out + dim4, dim - col, narrow<E, float>(sum_b));
}

// The blocks' sums, added up: 64 columns a block, its 16 waves taking every
// 16th row of the workspace. blockIdx.y: d_weight, d_bias.
constexpr int kJoinWaves = 16;

template <typename G>
__global__ __launch_bounds__(64 * kJoinWaves) void norm_grad_join_kernel(const float* __restrict__ ws, int blocks, int dim,
                                                                         int dim4, G* d_weight, G* d_bias,
                                                                         int accumulate) {
  G* out = blockIdx.y == 0 ? d_weight : d_bias;
  if (out == nullptr) return;
  __shared__ float part[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = int(blockIdx.x) * 64 + lane;
  float s = 0.f;
  if (col < dim)
#pragma unroll 8
    for (int b = wave; b < blocks; b += kJoinWaves) s += ws[(int64_t(b) * 2 + blockIdx.y) * dim4 + col];
  part[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= dim) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWaves; ++k) s += part[k][lane];
  if constexpr (sizeof(G) == 2) {
    out[col] = to_bf16(accumulate ? __uint_as_float(uint32_t(out[col]) << 16) + s : s);
  } else {
    out[col] = accumulate ? out[col] + s : s;
  }
}

// The threads and vectors of a row of `dim` elements, `per` of them a vector.
NormShape norm_shape(int64_t dim, int per, int top) {
  const int64_t vectors = (dim + per - 1) / per;
  static const NormShape shapes[] = {{16, 1}, {64, 1}, {64, 2}, {64, 4}, {256, 2}, {256, 4}, {1024, 2}, {1024, 4}};
  for (const NormShape& s : shapes)
    if (int64_t(s.threads) * s.vectors >= vectors && s.threads * s.vectors <= top) return s;
  return {0, 0};
}

// The longest row of the gradient kernel: its sums take 16 registers twice with 1024 threads.
constexpr int kNormGradDim = 16384;

NormShape norm_grad_shape(int64_t dim, int per) {
  return dim > kNormGradDim ? NormShape{0, 0} : norm_shape(dim, per, 1 << 20);
}

}  // namespace

namespace zero {

int64_t norm_grad_blocks(int64_t n, int64_t dim) {
  const NormShape s = norm_grad_shape(dim, 8);
  const int64_t rows = s.threads == 0 ? 16 : s.threads < 256 ? 256 / s.threads : 1;
  return std::max<int64_t>(1, std::min<int64_t>((n + rows - 1) / rows, 512));
}

int launch_embedding(const void* tokens, bool wide, int64_t n, const void* table, int32_t table_type, int64_t rows,
                     int64_t dim, float scale, void* out, int32_t out_type, int64_t out_stride, hipStream_t stream,
                     const char* who) {
  const auto go = [&](auto tv, auto ov) {
    using T = decltype(tv);
    using O = decltype(ov);
    constexpr int E = sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4;
    const int64_t tiles = (dim + 64 * E - 1) / (64 * E);
    const int64_t waves = (n + kLookupRows - 1) / kLookupRows * tiles;
    embedding_kernel<T, O, E><<<dim3(uint32_t((waves + 3) / 4)), 256, 0, stream>>>(
        tokens, wide, int(n), static_cast<const T*>(table), int(rows), int(dim), int(tiles), scale,
        static_cast<O*>(out), out_stride);
  };
  if (table_type == ZERO_BF16) out_type == ZERO_BF16 ? go(uint16_t(), uint16_t()) : go(uint16_t(), float());
  else out_type == ZERO_BF16 ? go(float(), uint16_t()) : go(float(), float());
  return launched(who);
}

int launch_token_order(const void* tokens, bool wide, int64_t n, int64_t rows, int32_t* order, hipStream_t stream,
                       const char* who) {
  const Order o(n, rows);
  if (n <= kRankTokens) {
    const int rank_blocks = std::max<int>(1, int(n + 63) / 64);
    const int bit_blocks = int((rows + 32 * kBitWords - 1) / (32 * kBitWords));
    order_rank_kernel<<<dim3(uint32_t(rank_blocks + bit_blocks)), kRankThreads, 0, stream>>>(
        tokens, wide, int(n), int(rows), rank_blocks, order, order + o.row, order + o.pos,
        reinterpret_cast<uint32_t*>(order + o.bits));
    return launched(who);
  }
  const int bits = row_bits(rows), passes = (bits + kSortBits - 1) / kSortBits, each = (bits + passes - 1) / passes;
  SortArgs a{};
  a.tokens = tokens;
  a.wide = wide;
  a.n = int32_t(n);
  a.rows = int32_t(rows);
  a.blocks = int32_t(o.blocks);
  a.digits = order + o.digits;
  a.live = order + o.live;
  a.head = order;
  a.present = reinterpret_cast<uint32_t*>(order + o.bits);
  int32_t *row[2] = {order + o.row, order + o.row2}, *pos[2] = {order + o.pos, order + o.pos2};
  for (int p = 0; p < passes; ++p) {
    const int to = (passes - 1 - p) & 1;       // the last pass ends in the order's own arrays
    a.shift = p * each;
    a.bits = std::min(each, bits - a.shift);
    a.row_in = row[to ^ 1];
    a.pos_in = pos[to ^ 1];
    a.row_out = row[to];
    a.pos_out = pos[to];
    const dim3 grid{uint32_t(o.blocks)};
    const bool first = p == 0, last = p == passes - 1;
    if (first) order_count_kernel<true><<<grid, kSortThreads, 0, stream>>>(a);
    else order_count_kernel<false><<<grid, kSortThreads, 0, stream>>>(a);
    if (first && last) order_scatter_kernel<true, true><<<grid, kSortThreads, 0, stream>>>(a);
    else if (first) order_scatter_kernel<true, false><<<grid, kSortThreads, 0, stream>>>(a);
    else if (last) order_scatter_kernel<false, true><<<grid, kSortThreads, 0, stream>>>(a);
    else order_scatter_kernel<false, false><<<grid, kSortThreads, 0, stream>>>(a);
  }
  return launched(who);
}

int launch_embedding_grad(const int32_t* order, int64_t n, int64_t rows, int64_t dim, const void* d_out,
                          int32_t out_type, int64_t out_stride, float scale, void* grad, int32_t grad_type,
                          int64_t first, int64_t count, bool accumulate, float* ws, hipStream_t stream,
                          const char* who) {
  const Order o(n, rows);
  EmbeddingGradArgs a{};
  a.head = order;
  a.row = order + o.row;
  a.pos = order + o.pos;
  a.present = reinterpret_cast<const uint32_t*>(order + o.bits);
  a.d_out = d_out;
  a.grad = grad;
  a.ws = ws;
  a.stride = out_stride;
  a.first = first;
  a.count = count;
  a.scale = scale;
  a.dim = int32_t(dim);
  a.dim4 = int32_t((dim + 3) / 4 * 4);
  a.pieces = int32_t((n + kPiece - 1) / kPiece);
  a.row_lo = int32_t(first / dim);
  a.row_hi = int32_t((first + count + dim - 1) / dim);
  a.accumulate = accumulate;
  const auto go = [&](auto tv, auto gv) {
    using T = decltype(tv);
    using G = decltype(gv);
    constexpr int E = sizeof(T) == 2 && sizeof(G) == 2 ? 8 : 4;
    a.tiles = int32_t((dim + 64 * E - 1) / (64 * E));
    const int64_t sums = (int64_t(a.pieces) * a.tiles + 3) / 4, fills = accumulate ? 0 : (a.row_hi - a.row_lo + 3) / 4;
    a.sum_blocks = int32_t(sums);
    if (sums + fills > 0)
      embedding_grad_kernel<T, G, E><<<dim3(uint32_t(sums + fills)), 256, 0, stream>>>(a);
    if (a.pieces > 1) embedding_join_kernel<G, E><<<dim3(uint32_t(sums)), 256, 0, stream>>>(a);
  };
  if (out_type == ZERO_BF16) grad_type == ZERO_BF16 ? go(uint16_t(), uint16_t()) : go(uint16_t(), float());
  else grad_type == ZERO_BF16 ? go(float(), uint16_t()) : go(float(), float());
  return launched(who);
}

int launch_norm(const zero_norm_args& a, hipStream_t stream, const char* who) {
  const auto go = [&](auto tv) {
    using T = decltype(tv);
    const NormShape s = norm_shape(a.dim, 16 / int(sizeof(T)), 1 << 20);
    const uint32_t rows = s.threads == 0 || s.threads >= 256 ? 1u : 256u / uint32_t(s.threads);
    const dim3 grid{uint32_t((a.n + rows - 1) / rows)};
#define ZERO_NORM(TPR, V) \
  if (s.threads == TPR && s.vectors == V) { \
    norm_kernel<T, TPR, V><<<grid, TPR < 256 ? 256 : TPR, 0, stream>>>(a); \
    return; \
  }
    ZERO_NORM(16, 1)
    ZERO_NORM(64, 1)
    ZERO_NORM(64, 2)
    ZERO_NORM(64, 4)
    ZERO_NORM(256, 2)
    ZERO_NORM(256, 4)
    ZERO_NORM(1024, 2)
    ZERO_NORM(1024, 4)
#undef ZERO_NORM
    norm_long_kernel<T><<<grid, kLongThreads, 0, stream>>>(a);
  };
  a.type == ZERO_BF16 ? go(uint16_t()) : go(float());
  return launched(who);
}

int launch_norm_grad(const zero_norm_grad_args& a, float* ws, hipStream_t stream, const char* who) {
  const int64_t blocks = norm_grad_blocks(a.n, a.dim);
  const int dim = int(a.dim), dim4 = (dim + 3) / 4 * 4;
  const bool sums = a.d_weight != nullptr || a.d_bias != nullptr;
  const auto go = [&](auto tv) {
    using T = decltype(tv);
    constexpr int E = 16 / int(sizeof(T));
    const NormShape s = norm_grad_shape(a.dim, E);
    const dim3 grid{uint32_t(blocks)};
#define ZERO_NORM(TPR, V) \
  if (s.threads == TPR && s.vectors == V) { \
    norm_grad_kernel<T, TPR, V><<<grid, TPR < 256 ? 256 : TPR, 0, stream>>>(a, ws, dim4); \
    return; \
  }
    ZERO_NORM(16, 1)
    ZERO_NORM(64, 1)
    ZERO_NORM(64, 2)
    ZERO_NORM(64, 4)
    ZERO_NORM(256, 2)
    ZERO_NORM(256, 4)
    ZERO_NORM(1024, 2)
    if constexpr (sizeof(T) == 4) ZERO_NORM(1024, 4)
#undef ZERO_NORM
    if (sums)
      norm_grad_columns_kernel<T><<<dim3(uint32_t((dim + 256 * E - 1) / (256 * E)), uint32_t(blocks)), 256, 0, stream>>>(
          a, ws, dim4);
    if (a.d_x != nullptr && a.n > 0) norm_grad_long_kernel<T><<<dim3(uint32_t(a.n)), kLongThreads, 0, stream>>>(a);
  };
  a.type == ZERO_BF16 ? go(uint16_t()) : go(float());
  if (sums) {
    const dim3 grid(uint32_t((dim + 63) / 64), 2);
    if (a.grad_type == ZERO_BF16)
      norm_grad_join_kernel<uint16_t><<<grid, 64 * kJoinWaves, 0, stream>>>(
          ws, int(blocks), dim, dim4, static_cast<uint16_t*>(a.d_weight), static_cast<uint16_t*>(a.d_bias), a.accumulate);
    else
      norm_grad_join_kernel<float><<<grid, 64 * kJoinWaves, 0, stream>>>(
          ws, int(blocks), dim, dim4, static_cast<float*>(a.d_weight), static_cast<float*>(a.d_bias), a.accumulate);
  }
  return launched(who);
}

}  // namespace zero
