// The delta rule's chunked kernels in a build of the test's own, in which every
// wait ends as ever but counts as run out for the threads [first, last) of one
// stage: 0 prepare, 1 chain, 2 output or gradients.
struct Chosen {
  int first, last;
};
__device__ Chosen chosen;
#define KLA_RAN_OUT ((int)threadIdx.x >= chosen.first && (int)threadIdx.x < chosen.last)
#include "kla_delta.cu"
#include "kla_delta_backward.cu"
#include "kla_delta_chunk.cu"

using namespace kla;

extern "C" size_t delta_waits_bytes(int B, int Hk, int H, int T, int dk, int dv) {
  return delta_backward_bytes(B, Hk, H, T, dk, dv);
}

// bf16, d_k ≤ 64. Forward where go is null.
extern "C" int delta_waits(const void* q, const void* k, const void* v, const void* g, const void* beta,
                           const float* state0, void* o, float* stateT, const void* go, void* gq, void* gk, void* gv,
                           void* gg, void* gbeta, float* gstate0, int B, int Hk, int H, int T, int dk, int dv,
                           void* space, int sms, int stage, int first, int last) {
  const DeltaArgs a{q, k, v, g, beta, state0, o, stateT, B, Hk, H, T, dk, dv, IO_BF16, 1.f};
  const DeltaGradArgs d{go, nullptr, gq, gk, gv, gg, gbeta, gstate0};
  size_t bytes = 0;
  const delta::Workspace w = delta::workspace(space, B, Hk, H, T, dk, dv, go != nullptr, &bytes);
  const DeltaGradArgs* grad = go ? &d : nullptr;
  for (int i = 0; i < 3; ++i) {
    const Chosen now = i == stage ? Chosen{first, last} : Chosen{0, 0};
    cudaError_t e = cudaMemcpyToSymbol(chosen, &now, sizeof now);
    if (e == cudaSuccess) {
      if (i == 0) e = delta::prepare_dk<__nv_bfloat16, 64>(a, grad, w, 0);
      else if (i == 1) e = delta::chain_dk<__nv_bfloat16, 64>(a, grad, w, sms, 0);
      else if (go) e = delta::grad_dk<__nv_bfloat16, 64>(a, d, w, sms, 0);
      else e = delta::output_dk<__nv_bfloat16, 64>(a, w, sms, 0);
    }
    if (e == cudaSuccess && i == 2 && w.part) {
      delta::kla_delta_share_kernel<__nv_bfloat16><<<64, 256>>>(a, d, w.part);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return (int)e;
  }
  return 0;
}
