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
// a workspace's rows: two sums for each such piece.
inline int embedding_piece(int64_t n) { return n <= 4096 ? 8 : 16; }
inline int64_t embedding_pieces(int64_t n) { return (n + embedding_piece(n) - 1) / embedding_piece(n); }

// Tokens that one block of the sort takes, and the bits of one of its passes.
constexpr int kSortThreads = 512, kSortItems = 4, kSortBlock = kSortThreads * kSortItems;
constexpr int kSortBits = 9, kSortDigits = 1 << kSortBits;

// Up to this many tokens are sorted by counting, in one launch.
constexpr int64_t kRankTokens = 12288;

// The parts of an order, in 32-bit words from its start: the sorted tokens' rows,
// `rows` for those outside the table, and positions; then scratch of the sort: rows
// and positions between two passes, and per block its digits' counts.
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
    words = digits + scratch * blocks * kSortDigits;
  }
};

// Bits of a row number, the one past the end among them.
inline int row_bits(int64_t rows) {
  int b = 1;
  while ((int64_t(1) << b) <= rows) ++b;
  return b;
}

// How a norm's row is spread: threads that share it, and the 16-byte vectors
// that each takes; vectors 0: a row too long for the registers.
struct NormShape {
  int threads, vectors;
};

// Blocks of the norm's gradient, each of which leaves one row of partial sums of
// d_weight and one of d_bias.
int64_t norm_grad_blocks(int64_t n, int64_t dim);

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
