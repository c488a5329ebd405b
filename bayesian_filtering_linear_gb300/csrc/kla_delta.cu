// The gated delta rule over a sequence, token by token (sm_103a):
//
//   u_t = β_t (v_t − a_t S_{t−1}ᵀ k_t),   S_t = a_t S_{t−1} + k_t u_tᵀ,   o_t = scale · S_tᵀ q_t
//
// The columns of a state are independent recurrences that share k, q, a, β.
// A lane keeps RL rows of one column in registers, as fp32 pairs for the
// packed arithmetic, and G = DK / RL neighbouring lanes hold a column; the
// two dot products end in log2(G) lane exchanges. Tokens come through shared
// memory sixteen at a time, the next sixteen on their way in registers
// meanwhile. Per state element a token costs five multiply-adds (k·S, q·S and
// a S + k u, a in two floats); the chain from one token to the next is a dot
// product, its exchanges and the update, which is what bounds a call with few
// heads. The decay's second float keeps weak decays: a factor next to 1 is off
// by up to 2^-25, and where it is the same for hundreds of tokens all of them
// add up (1024 heads of 16 × 16, 512 tokens, g = -1e-5: 2.4e-5 of the state).
#include "kla_device.cuh"
#include "kla_launch.h"

namespace kla {

namespace {

constexpr int kTile = 16, kThreads = 128;  // tokens staged at a time

template <typename IO>
__device__ __forceinline__ float4 load_four(const IO* p);
template <>
__device__ __forceinline__ float4 load_four<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load_four<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}

template <typename IO, int DK>
__global__ void __launch_bounds__(kThreads) kla_delta_recurrent_kernel(const DeltaArgs a) {
  constexpr int RL = DK >= 64 ? 16 : DK / 4, G = DK / RL, NC = kThreads / G, Q4 = RL / 4;
  constexpr int NK = (kTile * DK / 4 + kThreads - 1) / kThreads;  // fours of k and of q a thread brings
  static_assert(kTile * NC / 4 <= kThreads, "");
  __shared__ __align__(16) float ks[2][kTile][DK], qs[2][kTile][DK], vs[2][kTile][NC], os[2][kTile][NC];
  __shared__ float4 gates[2][kTile];  // decay in two floats, β
  const int tid = threadIdx.x, r = tid % G, c = tid / G;
  const int col_blocks = (a.dv + NC - 1) / NC;
  const long long bh = blockIdx.x / col_blocks;
  const int c0 = (int)(blockIdx.x % col_blocks) * NC, j = c0 + c;
  const bool mine = j < a.dv;  // heads narrower than a block leave lanes idle
  const int h = (int)(bh % a.H);
  const long long key = (bh / a.H) * a.Hk + h / (a.H / a.Hk);
  const int T = a.T;
  const IO* q = reinterpret_cast<const IO*>(a.q) + key * T * DK;
  const IO* k = reinterpret_cast<const IO*>(a.k) + key * T * DK;
  const IO* v = reinterpret_cast<const IO*>(a.v) + bh * T * a.dv + c0;
  const IO* g = reinterpret_cast<const IO*>(a.g) + bh * T;
  const IO* beta = reinterpret_cast<const IO*>(a.beta) + bh * T;
  IO* o = reinterpret_cast<IO*>(a.o) + bh * T * a.dv + c0;
  const int vt = tid / (NC / 4), vc = tid % (NC / 4) * 4;  // the thread's four of a tile of v and o
  const bool vin = tid < kTile * NC / 4 && c0 + vc < a.dv;

  // rows of the lane: float4 groups r, r + G, ... so that G lanes read one
  // stretch of k and q
  f2 S[2 * Q4];
#pragma unroll
  for (int i = 0; i < Q4; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = 0.f, y = 0.f;
      if (a.state0 && mine) {
        const float* p = a.state0 + ((size_t)bh * DK + (i * G + r) * 4 + 2 * e) * a.dv + j;
        x = p[0];
        y = p[a.dv];
      }
      S[2 * i + e] = f2_make(x, y);
    }

  float4 kx[NK], qx[NK], vx;
  float gx = 0.f, bx = 0.f;
  auto fetch = [&](int t0) {  // a tile's inputs into registers (zeros past the end)
    const int len = T - t0;
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int e = (tid + i * kThreads) * 4;
      kx[i] = qx[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e < kTile * DK && e / DK < len) {
        kx[i] = load_four<IO>(k + (size_t)t0 * DK + e);
        qx[i] = load_four<IO>(q + (size_t)t0 * DK + e);
      }
    }
    vx = make_float4(0.f, 0.f, 0.f, 0.f);
    if (vin && vt < len) vx = load_four<IO>(v + (size_t)(t0 + vt) * a.dv + vc);
    if (tid < kTile) {
      gx = tid < len ? to_f32<IO>(g[t0 + tid]) : 0.f;
      bx = tid < len ? to_f32<IO>(beta[t0 + tid]) : 0.f;
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int e = (tid + i * kThreads) * 4;
      if (e < kTile * DK) {
        *reinterpret_cast<float4*>(&ks[b][0][0] + e) = kx[i];
        *reinterpret_cast<float4*>(&qs[b][0][0] + e) = qx[i];
      }
    }
    if (tid < kTile * NC / 4) *reinterpret_cast<float4*>(&vs[b][vt][vc]) = vx;
    if (tid < kTile) {
      float low;
      const float a = decay_of(gx, low);
      gates[b][tid] = make_float4(a, low, bx, 0.f);
    }
  };
  if (T > 0) fetch(0);
  const int tiles = (T + kTile - 1) / kTile;
  for (int n = 0; n < tiles; ++n) {
    const int t0 = n * kTile, len = min(kTile, T - t0), b = n & 1;
    put(b);
    __syncthreads();  // (and the tile before the last is read)
    if (n + 1 < tiles) fetch(t0 + kTile);
    auto token = [&](int t) {
      f2 kk[2 * Q4], p0 = 0, p1 = 0;
#pragma unroll
      for (int i = 0; i < Q4; ++i) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&ks[b][t][(i * G + r) * 4]);
        kk[2 * i] = x.x;
        kk[2 * i + 1] = x.y;
        p0 = f2_fma(x.x, S[2 * i], p0);
        p1 = f2_fma(x.y, S[2 * i + 1], p1);
      }
      p0 = f2_add(p0, p1);
      float p = f2_lo(p0) + f2_hi(p0);
#pragma unroll
      for (int m = 1; m < G; m <<= 1) p += __shfl_xor_sync(~0u, p, m);
      const float4 ab = gates[b][t];
      const float u = ab.z * (vs[b][t][c] - ab.x * p);
      const f2 u2 = f2_make(u, u), a2 = f2_make(ab.x, ab.x), low2 = f2_make(ab.y, ab.y);
      f2 o0 = 0, o1 = 0;
#pragma unroll
      for (int i = 0; i < Q4; ++i) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&qs[b][t][(i * G + r) * 4]);
        S[2 * i] = f2_fma(a2, S[2 * i], f2_fma(kk[2 * i], u2, f2_mul(low2, S[2 * i])));
        S[2 * i + 1] = f2_fma(a2, S[2 * i + 1], f2_fma(kk[2 * i + 1], u2, f2_mul(low2, S[2 * i + 1])));
        o0 = f2_fma(x.x, S[2 * i], o0);
        o1 = f2_fma(x.y, S[2 * i + 1], o1);
      }
      o0 = f2_add(o0, o1);
      float y = f2_lo(o0) + f2_hi(o0);
#pragma unroll
      for (int m = 1; m < G; m <<= 1) y += __shfl_xor_sync(~0u, y, m);
      if (r == 0) os[b][t][c] = y;
    };
    if (len == kTile) {  // unrolled, so that one token's output overlaps the next one's chain
#pragma unroll 8
      for (int t = 0; t < kTile; ++t) token(t);
    } else {
      for (int t = 0; t < len; ++t) token(t);
    }
    __syncthreads();
    if (vin && vt < len) {
      const float4 y = *reinterpret_cast<const float4*>(&os[b][vt][vc]);
      IO* p = o + (size_t)(t0 + vt) * a.dv + vc;
      p[0] = from_f32<IO>(a.scale * y.x), p[1] = from_f32<IO>(a.scale * y.y);
      p[2] = from_f32<IO>(a.scale * y.z), p[3] = from_f32<IO>(a.scale * y.w);
    }
  }
  if (a.stateT && mine) {
#pragma unroll
    for (int i = 0; i < 2 * Q4; ++i) {
      float* p = a.stateT + ((size_t)bh * DK + ((i >> 1) * G + r) * 4 + 2 * (i & 1)) * a.dv + j;
      p[0] = f2_lo(S[i]);
      p[a.dv] = f2_hi(S[i]);
    }
  }
}

template <typename IO, int DK>
void launch_dk(const DeltaArgs& a, cudaStream_t s) {
  constexpr int NC = kThreads / (DK >= 64 ? DK / 16 : 4);
  const unsigned blocks = (unsigned)((long long)a.B * a.H * ((a.dv + NC - 1) / NC));
  kla_delta_recurrent_kernel<IO, DK><<<blocks, kThreads, 0, s>>>(a);
}

template <typename IO>
void launch_io(const DeltaArgs& a, cudaStream_t s) {
  switch (a.dk) {
    case 16: launch_dk<IO, 16>(a, s); break;
    case 32: launch_dk<IO, 32>(a, s); break;
    case 64: launch_dk<IO, 64>(a, s); break;
    default: launch_dk<IO, 128>(a, s); break;
  }
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs& a, cudaStream_t s) {
  if (a.io == IO_BF16) launch_io<__nv_bfloat16>(a, s);
  else launch_io<float>(a, s);
  return cudaGetLastError();
}

}  // namespace kla
