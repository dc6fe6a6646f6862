// Internal declarations of the tensor-list calls (tensors.cpp: the list, the
// argument checks and the C ABI on the host; tensors.hip: the kernels and
// their launches). Not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>
#include <vector>

#include "zero_internal.h"
#include "zero_tensors.h"

namespace zero {

// Elements of one unit of work: four 8-bit blocks. A unit lies in one tensor.
constexpr int kUnitBlocks = 4;
constexpr int kUnitElems = kUnitBlocks * ZERO_STATE8_BLOCK;

// Elements that one wave of the norm takes.
constexpr int kSqChunk = 4096;

// The device table: first[n + 1], the running count of units (first[t] is the
// first unit of tensor t, first[n] the total), padded to 16 bytes; the same of
// the norm's chunks; then the n records, as the caller described them.
inline size_t table_chunks_at(int32_t n) { return (size_t(n) + 1 + 3) / 4 * 16; }
inline size_t table_records_at(int32_t n) { return 2 * table_chunks_at(n); }
inline size_t table_bytes(int32_t n) { return table_records_at(n) + size_t(n) * sizeof(zero_tensor); }

}  // namespace zero

struct zero_tensors_s {
  std::vector<zero_tensor> t;
  std::vector<int32_t> first, chunk;   // running counts of units and of chunks
  std::vector<std::pair<uintptr_t, uintptr_t>> owned;   // byte ranges of the list's buffers, sorted, disjoint
  int32_t param_type = 0, grad_type = 0, state_bits = 0;
  int32_t top_group = 0;      // the largest group in use
  void* table = nullptr;      // set by the upload
  int device = -1;
};

namespace zero {

// The hyperparameters of a step as the kernels take them.
struct GroupConst {
  float beta1, omb1, beta2, omb2, lr_wd, step_size, inv_sqrt_bc2, eps;
};

struct StepConst {
  const double* rank_sq;
  int32_t n_ranks;
  int32_t clip_on;
  double max_norm, clip_eps;
  GroupConst g[ZERO_TENSOR_GROUPS];
  AdamWExact x[ZERO_TENSOR_GROUPS];
};

// The current device in *dev; ZERO_OK or an error.
int current_device(int* dev, const char* who);
// The launches of a call whose arguments have been checked.
int launch_upload(const zero_tensors_s* h, void* table, hipStream_t stream, const char* who);
int launch_sqnorm(const zero_tensors_s* h, const void* const* grads, double* out, int32_t accumulate, double* ws,
                  hipStream_t stream, const char* who);
int launch_adamw(const zero_tensors_s* h, const void* const* grads, const StepConst& c, hipStream_t stream,
                 const char* who);
int launch_state8(const zero_tensors_s* h, bool import, const float* const* m, const float* const* v,
                  hipStream_t stream, const char* who);

}  // namespace zero
