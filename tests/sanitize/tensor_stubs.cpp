// Stand-ins for the tensor-list launches in a host-only build of the library
// (beside device_stubs.cpp); the host tests that run there never call them.
#include "tensors_internal.h"
namespace zero {
int current_device(int* dev, const char*) { *dev = 0; return ZERO_OK; }
int launch_upload(const zero_tensors_s*, void*, hipStream_t, const char*) { return -1; }
int launch_sqnorm(const zero_tensors_s*, const void* const*, double*, int32_t, double*, hipStream_t, const char*) { return -1; }
int launch_adamw(const zero_tensors_s*, const void* const*, const StepConst&, hipStream_t, const char*) { return -1; }
int launch_state8(const zero_tensors_s*, bool, const float* const*, const float* const*, hipStream_t, const char*) { return -1; }
}
