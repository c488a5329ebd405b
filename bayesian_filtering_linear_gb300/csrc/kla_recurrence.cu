// Host side of the gated linear recurrence: the kernels by type.
#include <cuda_bf16.h>

#include "kla_launch.h"

namespace kla {

template <typename IO>
cudaError_t launch_recurrence_io(const RecArgs& a, cudaStream_t s);
template <typename IO>
cudaError_t launch_recurrence_step_io(const RecArgs& a, cudaStream_t s);
template <typename IO>
cudaError_t launch_recurrence_backward_io(const RecGradArgs& a, int* parts, cudaStream_t s);

namespace {

// grate[h, d]: the blocks' sums over the cluster's ranks and the batch, in a fixed
// order: 32 channels a block, its eight rows of threads over the sums.
__global__ void __launch_bounds__(256) kla_recurrence_rate_kernel(const float* part, float* grate, int parts, int B, int HD) {
  __shared__ float sums[8][32];
  const int row = threadIdx.x / 32, col = threadIdx.x % 32, i = blockIdx.x * 32 + col;
  float x = 0.f;
  if (i < HD)
#pragma unroll 4
    for (long long n = row; n < (long long)parts * B; n += 8) x += part[n * HD + i];
  sums[row][col] = x;
  __syncthreads();
  if (row > 0 || i >= HD) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) x += sums[r][col];
  grate[i] = -x;
}

}  // namespace

cudaError_t launch_recurrence(const RecArgs& a, cudaStream_t s) {
  return a.io == IO_BF16 ? launch_recurrence_io<__nv_bfloat16>(a, s) : launch_recurrence_io<float>(a, s);
}

cudaError_t launch_recurrence_step(const RecArgs& a, cudaStream_t s) {
  return a.io == IO_BF16 ? launch_recurrence_step_io<__nv_bfloat16>(a, s) : launch_recurrence_step_io<float>(a, s);
}

cudaError_t launch_recurrence_backward(const RecGradArgs& a, cudaStream_t s) {
  int parts = 0;
  const cudaError_t e = a.f.io == IO_BF16 ? launch_recurrence_backward_io<__nv_bfloat16>(a, &parts, s)
                                          : launch_recurrence_backward_io<float>(a, &parts, s);
  if (e != cudaSuccess || !a.part) return e;
  const int HD = a.f.H * a.f.D;
  kla_recurrence_rate_kernel<<<(HD + 31) / 32, 256, 0, s>>>(a.part, a.grate, parts, a.f.B, HD);
  return cudaGetLastError();
}

}  // namespace kla
