// The recurrence's gradient kernels for bf16 inputs.
#include "kla_recurrence_backward.cuh"

namespace kla {
template cudaError_t launch_recurrence_backward_io<__nv_bfloat16>(const RecGradArgs&, int*, cudaStream_t);
}  // namespace kla
