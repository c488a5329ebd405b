// The recurrence's forward kernels for bf16 inputs.
#include "kla_recurrence_kernels.cuh"

namespace kla {
template cudaError_t launch_recurrence_io<__nv_bfloat16>(const RecArgs&, cudaStream_t);
template cudaError_t launch_recurrence_step_io<__nv_bfloat16>(const RecArgs&, cudaStream_t);
}  // namespace kla
