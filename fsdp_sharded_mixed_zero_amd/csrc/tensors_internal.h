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

// With a 32-bit state the units of a tensor begin up to 31 elements before it, so
// that its fp32 masters fall into units (and waves) by whole 128-byte lines:
// the elements between such a line's start and the first master.
constexpr int kLineElems = 32;
constexpr int line_phase(uintptr_t master) { return int((master >> 2) & (kLineElems - 1)); }

// Elements that one wave of the norm takes.
constexpr int kSqChunk = 4096;

// Slots of a running count: runs of 2^shift units, as many as kSlots of them;
// slot[s] is the tensor that holds unit s << shift, where a search begins.
constexpr int kSlots = 2048;

// The device table: first[n + 1], the running count of units (first[t] is the
// first unit of tensor t, first[n] the total), and its slots; the same two of
// the norm's chunks; then the n records, as the caller described them. Each
// part starts at a multiple of 16 bytes.
struct Table {
  size_t first[2], slot[2], records, bytes;   // byte offsets; [0] units, [1] chunks
  explicit Table(int32_t n) {
    size_t at = 0;
    for (int k = 0; k < 2; ++k) {
      first[k] = at;
      at += (size_t(n) + 1 + 3) / 4 * 16;
      slot[k] = at;
      at += size_t(kSlots) * sizeof(int32_t);
    }
    records = at;
    bytes = at + size_t(n) * sizeof(zero_tensor);
  }
};

}  // namespace zero

struct zero_tensors_s {
  std::vector<zero_tensor> t;
  std::vector<int32_t> first[2];   // running counts of units and of chunks
  int32_t shift[2] = {0, 0};       // of their slots
  std::vector<int32_t> partial;    // running count of tensors that end inside a unit
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
