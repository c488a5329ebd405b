// The recurrence's forward kernels for f32 inputs.
#include "kla_recurrence_kernels.cuh"

namespace kla {
template cudaError_t launch_recurrence_io<float>(const RecArgs&, cudaStream_t);
template cudaError_t launch_recurrence_step_io<float>(const RecArgs&, cudaStream_t);
}  // namespace kla
