// The recurrence's gradient kernels for f32 inputs.
#include "kla_recurrence_backward.cuh"

namespace kla {
template cudaError_t launch_recurrence_backward_io<float>(const RecGradArgs&, int*, cudaStream_t);
}  // namespace kla
