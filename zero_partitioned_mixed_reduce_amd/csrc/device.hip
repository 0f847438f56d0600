// The library's device code as one translation unit: the sharded step's kernels, and the
// gradient lists' kernels, which use their 16-bit formats and device-scope stores.
#include "kernels.hip"
#include "grads.hip"
