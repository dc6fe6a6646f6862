// The library's device code as one translation unit: the tensor-list kernels
// use the conversions, sums, clip coefficient and update of the flat ones.
#include "kernels.hip"
#include "tensors.hip"
