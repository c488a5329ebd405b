// One decode token of the gated delta rule (sm_103a), the state in place:
//
//   u = β (v − a Sᵀk),   S ← a S + k uᵀ,   o = scale · Sᵀq,   a = e^g
//
// Work layout: a warp owns 16 columns of one head's state, eight lanes down
// the rows and four across (one 16-byte load each, so a row's segment is two
// whole sectors). A lane loads its rows once and keeps them in registers from
// the dot product with k to the store, so the state crosses HBM once each
// way, 8 bytes per element, which bounds the step; the sums over rows are
// three lane exchanges, and no warp waits for another. The state decays by a in
// two floats (decay_of), so that thousands of weak decays do not add up their
// roundings.
#include "kla_device.cuh"
#include "kla_launch.h"

namespace kla {

namespace {

template <typename IO, int DK>
__global__ void __launch_bounds__(256) kla_delta_step_kernel(const DeltaArgs a) {
  constexpr int R = DK / 8;  // rows of a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long bh = blockIdx.x;
  const int h = (int)(bh % a.H);
  const long long key = (bh / a.H) * a.Hk + h / (a.H / a.Hk);
  const int j0 = warp * 16 + (lane & 3) * 4, r0 = lane >> 2;

  const IO* qv = reinterpret_cast<const IO*>(a.q) + key * DK;
  const IO* kv = reinterpret_cast<const IO*>(a.k) + key * DK;
  const IO* vv = reinterpret_cast<const IO*>(a.v) + bh * a.dv;
  const float* src = a.state0 + (size_t)bh * DK * a.dv + j0;
  float* dst = a.stateT + (size_t)bh * DK * a.dv + j0;

  float4 S[R];
  float k[R], q[R];
#pragma unroll
  for (int r = 0; r < R; ++r) S[r] = *reinterpret_cast<const float4*>(src + (size_t)(r0 + 8 * r) * a.dv);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    k[r] = to_f32<IO>(kv[r0 + 8 * r]);
    q[r] = to_f32<IO>(qv[r0 + 8 * r]);
  }
  float low;
  const float decay = decay_of(to_f32<IO>(reinterpret_cast<const IO*>(a.g)[bh]), low);
  const float beta = to_f32<IO>(reinterpret_cast<const IO*>(a.beta)[bh]);

  float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < R; ++r) {
    p[0] = fmaf(k[r], S[r].x, p[0]);
    p[1] = fmaf(k[r], S[r].y, p[1]);
    p[2] = fmaf(k[r], S[r].z, p[2]);
    p[3] = fmaf(k[r], S[r].w, p[3]);
  }
  float u[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int m = 4; m < 32; m <<= 1) p[c] += __shfl_xor_sync(~0u, p[c], m);
    u[c] = beta * (to_f32<IO>(vv[j0 + c]) - decay * p[c]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    S[r].x = fmaf(decay, S[r].x, fmaf(k[r], u[0], low * S[r].x));
    S[r].y = fmaf(decay, S[r].y, fmaf(k[r], u[1], low * S[r].y));
    S[r].z = fmaf(decay, S[r].z, fmaf(k[r], u[2], low * S[r].z));
    S[r].w = fmaf(decay, S[r].w, fmaf(k[r], u[3], low * S[r].w));
    o[0] = fmaf(q[r], S[r].x, o[0]);
    o[1] = fmaf(q[r], S[r].y, o[1]);
    o[2] = fmaf(q[r], S[r].z, o[2]);
    o[3] = fmaf(q[r], S[r].w, o[3]);
    *reinterpret_cast<float4*>(dst + (size_t)(r0 + 8 * r) * a.dv) = S[r];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int m = 4; m < 32; m <<= 1) o[c] += __shfl_xor_sync(~0u, o[c], m);
  if (lane < 4) {
    IO* out = reinterpret_cast<IO*>(a.o) + bh * a.dv + j0;
#pragma unroll
    for (int c = 0; c < 4; ++c) out[c] = from_f32<IO>(a.scale * o[c]);
  }
}

template <typename IO>
void launch_io(const DeltaArgs& a, cudaStream_t s) {
  const unsigned blocks = (unsigned)((long long)a.B * a.H), threads = 2 * a.dv;  // a warp per 16 columns
  switch (a.dk) {
    case 16: kla_delta_step_kernel<IO, 16><<<blocks, threads, 0, s>>>(a); break;
    case 32: kla_delta_step_kernel<IO, 32><<<blocks, threads, 0, s>>>(a); break;
    case 64: kla_delta_step_kernel<IO, 64><<<blocks, threads, 0, s>>>(a); break;
    default: kla_delta_step_kernel<IO, 128><<<blocks, threads, 0, s>>>(a); break;
  }
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs& a, cudaStream_t s) {
  if (a.io == IO_BF16) launch_io<__nv_bfloat16>(a, s);
  else launch_io<float>(a, s);
  return cudaGetLastError();
}

}  // namespace kla
