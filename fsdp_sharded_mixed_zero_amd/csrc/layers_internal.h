// Internal declarations of the token-table and norm calls (layers.cpp: the
// argument checks and the C ABI on the host; layers.hip: the kernels and their
// launches). Not part of the C ABI.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "zero_internal.h"
#include "zero_layers.h"

namespace zero {

// Sorted tokens that one wave of the table's gradient sums (a multiple of 8), and
// a workspace's rows: two sums for each such piece. Short pieces, so that a few
// tokens are many waves (512 tokens, 1600 wide: 13 us of a call with 8, 17 with 16),
// until the sums cost more than that (32768 tokens, 8192 wide, an eighth of the
// table: 67 us with 8, 59 with 16, 61 with 32).
constexpr int64_t kShortPieces = 4096;
inline int embedding_piece(int64_t n) { return n <= kShortPieces ? 8 : 16; }
inline int64_t embedding_pieces(int64_t n) { return (n + embedding_piece(n) - 1) / embedding_piece(n); }

// Tokens that one block of the sort takes, and the bits of one of its passes.
constexpr int kSortThreads = 512, kSortItems = 4, kSortBlock = kSortThreads * kSortItems;
constexpr int kSortBits = 9, kSortDigits = 1 << kSortBits;

// Up to this many tokens are sorted in one launch whatever the table, and need no scratch.
constexpr int64_t kRankTokens = 12288;

// The parts of an order, in 32-bit words from its start: the sorted tokens' rows,
// `rows` for those outside the table, and positions; then scratch of the sort: rows
// and positions between two passes, and per block its digits' counts, and their
// totals.
struct Order {
  int64_t row, pos, row2, pos2, digits, words;
  int64_t blocks;
  Order(int64_t n) {
    auto up = [](int64_t k) { return (k + 7) / 8 * 8; };
    blocks = (n + kSortBlock - 1) / kSortBlock;
    const int64_t scratch = n > kRankTokens ? 1 : 0;
    row = 0;
    pos = row + up(n) + 8;      // read by eights and one more
    row2 = pos + up(n) + 8;
    pos2 = row2 + scratch * up(n);
    digits = pos2 + scratch * up(n);
    words = digits + scratch * (blocks + 1) * kSortDigits;
  }
};

// Bits of a row number, the one past the end among them.
inline int row_bits(int64_t rows) {
  int b = 1;
  while ((int64_t(1) << b) <= rows) ++b;
  return b;
}

// How a norm's row of 16-byte vectors is spread: the threads that share it, and
// the vectors that each takes; threads 0: a row too long for the registers. A wave
// a row needs no barrier: up to two vectors a lane, from 1024 rows on up to four (16384
// rows of 1600 bf16: 21 us, 26 with 256 threads a row; rows of 2944: 38 us with six, 36
// with 256 threads); fewer rows take more threads each, for the latency (8 rows of 1600:
// 3.6 us instead of 6.0).
struct NormShape {
  int threads, vectors;
};

inline NormShape norm_shape(int64_t n, int64_t vectors) {
  if (n >= 1024 && vectors > 128 && vectors <= 256) return {64, 4};
  static const NormShape shapes[] = {{16, 1}, {32, 1}, {64, 1}, {64, 2}, {256, 1}, {256, 2}, {256, 4}, {1024, 2}, {1024, 4}};
  for (const NormShape& s : shapes)
    if (int64_t(s.threads) * s.vectors >= vectors) return s;
  return {0, 0};
}

// The same for the gradient, rows of `dim` elements, `per` of them a vector. Its two
// sums a column take 16 registers for a vector of bf16, so a thread takes one, or
// one of fp32 (5003 rows of 1111: 20 us of a call, 21.4 with two) while 768 threads
// suffice and two beyond. The fewest threads of one list for both types: idle ones cost
// a wave's share of the registers (16384 rows of 2560 bf16 with 320 threads 64.0 us, with
// 384 65.2; of 2100 62.6 and 66.2; 8192 of 5120 with 640 71.0, with 768 72.0; 5003 of
// 1111 fp32 with 320 23.3, with 384 23.8; 8192 of 2560 fp32 with 640 65.0, with 768 66.0).
// With 1024 threads of 128 registers 4 spill for bf16 (20 bytes a lane) and 13 for fp32
// (56): 8192 rows of 8192 bf16 112 us, 4.8 TB/s. Twice as many sums spill more: rows of
// more than 8192 elements take two kernels (4096 rows of 12000 bf16: 259 us in registers).
inline NormShape norm_grad_shape(int64_t dim, int per) {
  const int64_t vectors = (dim + per - 1) / per;
  if (vectors <= 32) return {vectors <= 16 ? 16 : 32, 1};
  for (int v = 1; v <= 8 / per; ++v)
    for (int t : {64, 128, 192, 256, 320, 384, 512, 640, 768, 1024}) {
      if (t == 1024 && v < 8 / per) break;
      if (int64_t(t) * v >= vectors) return {t, v};       // two of fp32: from 512 threads on
    }
  return {0, 0};
}

// Up to this many rows the gradient takes one launch, in which the columns read every
// row again. Against two launches, us: 256 rows of 768 bf16 8.2 and 10.4, 384 10.4 and
// 10.3, 512 13.4 and 9.9; 384 rows of 8192 bf16 13.9 and 17.0, 512 16.9 and 19.3, 1024
// 30.5 and 30.8. Rows of more than 8192 elements have kernels of their own.
inline int64_t few_norm_rows(int64_t dim) { return dim > 8192 ? -1 : dim > 4096 ? 512 : 256; }

// Threads of a block of the gradient: as many rows at a time as 512 threads take.
constexpr int grad_threads(int per_row) { return per_row >= 512 ? per_row : 512 / per_row * per_row; }

// Blocks of the norm's gradient, each of which leaves one row of partial sums of
// d_weight and one of d_bias: two a CU where there are rows enough (16384 rows of
// 2944 bf16: 74 us of a call with 512, 84 with 384 and 768, 95 with 256), and two
// rows a block, or group of its threads, where they are few.
inline int64_t norm_grad_blocks(int64_t n, int64_t dim) {
  const NormShape s = norm_grad_shape(dim, 8);
  const int64_t rows = s.threads == 0 ? 16 : grad_threads(s.threads) / s.threads;
  const int64_t groups = (n + rows - 1) / rows;
  return std::max<int64_t>(1, std::min<int64_t>(groups, std::min<int64_t>(512, std::max<int64_t>(256, groups / 2))));
}

// The launches of calls whose arguments have been checked.
int launch_embedding(const void* tokens, bool wide, int64_t n, const void* table, int32_t table_type, int64_t rows,
                     int64_t dim, float scale, void* out, int32_t out_type, int64_t out_stride, hipStream_t stream,
                     const char* who);
int launch_token_order(const void* tokens, bool wide, int64_t n, int64_t rows, int32_t* order, hipStream_t stream,
                       const char* who);
int launch_embedding_grad(const int32_t* order, int64_t n, int64_t rows, int64_t dim, const void* d_out,
                          int32_t out_type, int64_t out_stride, float scale, void* grad, int32_t grad_type,
                          int64_t first, int64_t count, bool accumulate, float* ws, hipStream_t stream,
                          const char* who);
int launch_norm(const zero_norm_args& a, hipStream_t stream, const char* who);
int launch_norm_grad(const zero_norm_grad_args& a, float* ws, hipStream_t stream, const char* who);

}  // namespace zero
