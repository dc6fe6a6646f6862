// Stand-ins for the token-table and norm launches in a host-only build of the
// library (beside device_stubs.cpp); the host tests that run there never call them.
#include "layers_internal.h"
namespace zero {
int launch_embedding(const void*, bool, int64_t, const void*, int32_t, int64_t, int64_t, float, void*, int32_t, int64_t,
                     hipStream_t, const char*) { return -1; }
int launch_token_order(const void*, bool, int64_t, int64_t, int32_t*, hipStream_t, const char*) { return -1; }
int launch_embedding_grad(const int32_t*, int64_t, int64_t, int64_t, const void*, int32_t, int64_t, float, void*, int32_t,
                          int64_t, int64_t, bool, float*, hipStream_t, const char*) { return -1; }
int launch_norm(const zero_norm_args&, hipStream_t, const char*) { return -1; }
int launch_norm_grad(const zero_norm_grad_args&, float*, hipStream_t, const char*) { return -1; }
}
