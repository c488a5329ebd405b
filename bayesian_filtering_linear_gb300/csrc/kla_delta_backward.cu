// Gradients of the gated delta rule (sm_103a), chunk by chunk from the end.
//
// With D_ts the decay from token s to token t of a chunk, G_t the decay from
// its start and E_t the decay to its end, the chunk's states follow from the
// state S before it by
//   A = tril(β_t D_ts k_t·k_s, −1),  M = (I + A)^-1,  U = M β(V − G K S),
//   P = tril(D_ts q_t·k_s),          O = scale (G Q S + P U),  S' = G_end S + Kᵀ(E U),
// and with O' = scale dL/dO, Z = dL/dS' their gradients by
//   dU = Pᵀ O' + E K Z,  dR = Mᵀ dU,  dA = −tril(dR Uᵀ, −1),  dP = tril(O' Uᵀ)
//   dV = β dR,  dS = G_end Z + Qᵀ(G O') − Kᵀ(β G dR)
//   dQ = G O' Sᵀ + (dP D) K
//   X = (dA D) K − G dR Sᵀ,  Y = E U Zᵀ + (dP D)ᵀ Q + (β dA D)ᵀ K
//   dK = β X + Y,  dβ = dR·V + k·X
//   dg_t = G_end <Z, S> + Σ_{s≥t} G_s (q·O' Sᵀ − β k·dR Sᵀ)_s + Σ_{s<t} E_s k_s·(U Zᵀ)_s
//          + Σ_{s'≥t} Σ_{s<t} (dP P + dA A)_s's
// (X holds the terms in which k_t multiplies the state before it, Y those in
// which it is written to the state.) The decay's gradient could also be had
// from q·dQ, k·X and k·Y alone, as a running sum of their differences; but
// behind a strong decay those cancel to nothing and leave their roundings,
// while every product above carries the decay it is the gradient of.
//
// One block walks a head's chunks of 16 tokens; the states before them come
// from a forward pass. Gradients of q and k that several value heads share
// are summed from per-head fp32 parts in a fixed order.
#include "kla_device.cuh"
#include "kla_launch.h"

namespace kla {

namespace {

constexpr int C = kDeltaCkpt, kThreads = 256;

// out[m][n] = Σ_k a(m,k) b(k,n) by all threads, one element each at a time
template <typename FA, typename FB, typename FO>
__device__ __forceinline__ void matmul(int M, int N, int K, FA a, FB b, FO out) {
  for (int i = threadIdx.x; i < M * N; i += kThreads) {
    const int m = i / N, n = i % N;
    float s = 0.f;
    for (int k = 0; k < K; ++k) s = fmaf(a(m, k), b(k, n), s);
    out(m, n, s);
  }
}

template <typename IO>
__global__ void __launch_bounds__(kThreads) kla_delta_backward_kernel(const DeltaArgs a, const DeltaGradArgs d,
                                                                     const float* ckpt, float* part) {
  extern __shared__ __align__(16) float sm[];
  const int dk = a.dk, dv = a.dv, T = a.T, tid = threadIdx.x;
  const long long bh = blockIdx.x;
  const int h = (int)(bh % a.H);
  const long long key = (bh / a.H) * a.Hk + h / (a.H / a.Hk);
  const int chunks = (T + C - 1) / C;
  float* S = sm;                // [dk][dv]
  float* Z = S + dk * dv;       // [dk][dv]
  float* K = Z + dk * dv;       // [C][dk]
  float* Q = K + C * dk;
  float* V = Q + C * dk;        // [C][dv]
  float* O = V + C * dv;
  float* U = O + C * dv;
  float* R = U + C * dv;
  float* X = R + C * dv;        // [C][dk]
  float* Y = X + C * dk;
  float* M = Y + C * dk;        // [C][C]
  float* P = M + C * C;
  float* A = P + C * C;
  float* dP = A + C * C;
  float* D = dP + C * C;
  float* W = D + C * C;         // (dP P + dA A), then its sums along s
  __shared__ float gc[C], be[C], red[kThreads / 32], line[C];
  __shared__ double cum[C];
  const size_t sz = (size_t)dk * dv;
  for (int i = tid; i < dk * dv; i += kThreads) Z[i] = d.gstateT ? d.gstateT[bh * sz + i] : 0.f;
  for (int n = chunks - 1; n >= 0; --n) {
    const int t0 = n * C, len = min(C, T - t0);
    for (int i = tid; i < dk * dv; i += kThreads) S[i] = ckpt[((size_t)bh * chunks + n) * sz + i];
    for (int i = tid; i < C * dk; i += kThreads) {
      const bool in = i < len * dk;
      const size_t at = ((size_t)key * T + t0) * dk + i;
      K[i] = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.k)[at]) : 0.f;
      Q[i] = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.q)[at]) : 0.f;
    }
    for (int i = tid; i < C * dv; i += kThreads) {
      const bool in = i < len * dv;
      const size_t at = ((size_t)bh * T + t0) * dv + i;
      V[i] = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.v)[at]) : 0.f;
      O[i] = in && d.go ? a.scale * to_f32<IO>(reinterpret_cast<const IO*>(d.go)[at]) : 0.f;
    }
    if (tid < C) {
      const bool in = tid < len;
      const float x = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.g)[(size_t)bh * T + t0 + tid]) : 0.f;
      gc[tid] = x < -104.f ? -104.f : x;  // e^-104 is 0 in fp32, and sums stay finite
      be[tid] = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.beta)[(size_t)bh * T + t0 + tid]) : 0.f;
    }
    __syncthreads();
    if (tid == 0) {
      double x = 0;
      for (int t = 0; t < C; ++t) cum[t] = x += gc[t];
    }
    __syncthreads();
    if (tid < C * C) D[tid] = tid % C <= tid / C ? expf((float)(cum[tid / C] - cum[tid % C])) : 0.f;
    __syncthreads();
    matmul(C, C, dk, [&](int t, int i) { return K[t * dk + i]; }, [&](int i, int s) { return K[s * dk + i]; },
           [&](int t, int s, float x) { A[t * C + s] = s < t ? be[t] * D[t * C + s] * x : 0.f; });
    matmul(C, C, dk, [&](int t, int i) { return Q[t * dk + i]; }, [&](int i, int s) { return K[s * dk + i]; },
           [&](int t, int s, float x) { P[t * C + s] = D[t * C + s] * x; });
    matmul(C, dv, dk, [&](int t, int i) { return K[t * dk + i]; }, [&](int i, int j) { return S[i * dv + j]; },
           [&](int t, int j, float x) { R[t * dv + j] = be[t] * (V[t * dv + j] - expf((float)cum[t]) * x); });
    __syncthreads();
    if (tid < C) {  // column tid of M by forward substitution
      for (int t = 0; t < C; ++t) {
        float x = t == tid ? 1.f : 0.f;
        for (int s = tid; s < t; ++s) x = fmaf(-A[t * C + s], M[s * C + tid], x);
        M[t * C + tid] = x;
      }
    }
    __syncthreads();
    auto G = [&](int t) { return expf((float)cum[t]); };
    auto E = [&](int t) { return expf((float)(cum[C - 1] - cum[t])); };
    matmul(C, dv, C, [&](int t, int s) { return M[t * C + s]; }, [&](int s, int j) { return R[s * dv + j]; },
           [&](int t, int j, float x) { U[t * dv + j] = x; });
    __syncthreads();
    matmul(C, dv, C + dk, [&](int s, int i) { return i < C ? P[i * C + s] : E(s) * K[s * dk + i - C]; },
           [&](int i, int j) { return i < C ? O[i * dv + j] : Z[(i - C) * dv + j]; },
           [&](int s, int j, float x) { R[s * dv + j] = x; });
    __syncthreads();
    // dR = Mᵀ dU, column by column in registers
    for (int j = tid; j < dv; j += kThreads) {
      float x[C];
      for (int s = 0; s < C; ++s) {
        x[s] = 0.f;
        for (int t = s; t < C; ++t) x[s] = fmaf(M[t * C + s], R[t * dv + j], x[s]);
      }
      for (int s = 0; s < C; ++s) R[s * dv + j] = x[s];
    }
    __syncthreads();
    matmul(C, C, dv, [&](int t, int j) { return R[t * dv + j]; }, [&](int j, int s) { return U[s * dv + j]; },
           [&](int t, int s, float x) {
             W[t * C + s] = s < t ? -x * A[t * C + s] : 0.f;
             A[t * C + s] = s < t ? -D[t * C + s] * x : 0.f;
           });
    __syncthreads();
    matmul(C, C, dv, [&](int t, int j) { return O[t * dv + j]; }, [&](int j, int s) { return U[s * dv + j]; },
           [&](int t, int s, float x) {
             if (s < t) W[t * C + s] = fmaf(x, P[t * C + s], W[t * C + s]);
             dP[t * C + s] = D[t * C + s] * x;
           });
    float zs = 0.f;
    for (int i = tid; i < dk * dv; i += kThreads) zs = fmaf(Z[i], S[i], zs);
    zs *= G(C - 1);
    __syncthreads();
    float* uz = M;  // [C]: (E U Zᵀ)_t · k_t
    matmul(C, dk, dv, [&](int t, int j) { return U[t * dv + j]; }, [&](int j, int i) { return Z[i * dv + j]; },
           [&](int t, int i, float x) { Y[t * dk + i] = E(t) * x; });
    __syncthreads();
    if (tid < C) {
      float x = 0.f;
      for (int i = 0; i < dk; ++i) x = fmaf(Y[tid * dk + i], K[tid * dk + i], x);
      uz[tid] = x;
    }
    __syncthreads();
    matmul(C, dk, dv, [&](int t, int j) { return R[t * dv + j]; }, [&](int j, int i) { return S[i * dv + j]; },
           [&](int t, int i, float x) { X[t * dk + i] = -G(t) * x; });
    __syncthreads();
    if (tid < C) {
      float x = 0.f;
      for (int i = 0; i < dk; ++i) x = fmaf(X[tid * dk + i], K[tid * dk + i], x);
      line[tid] = be[tid] * x;
      float sum = 0.f;  // W's row tid: W[tid][t] becomes the sum over s < t
      for (int t = 0; t < C; ++t) {
        const float w = W[tid * C + t];
        W[tid * C + t] = sum;
        sum += w;
      }
    }
    __syncthreads();
    matmul(C, dk, C, [&](int t, int s) { return A[t * C + s]; }, [&](int s, int i) { return K[s * dk + i]; },
           [&](int t, int i, float x) { X[t * dk + i] += x; });
    matmul(C, dk, 2 * C, [&](int s, int t) { return t < C ? dP[t * C + s] : be[t - C] * A[(t - C) * C + s]; },
           [&](int t, int i) { return t < C ? Q[t * dk + i] : K[(t - C) * dk + i]; },
           [&](int s, int i, float x) { Y[s * dk + i] += x; });
    for (int m = 16; m; m >>= 1) zs += __shfl_xor_sync(~0u, zs, m);
    if ((tid & 31) == 0) red[tid >> 5] = zs;
    __syncthreads();
    const bool shared_keys = a.Hk != a.H;
    const int w = tid >> 5, l = tid & 31;
    for (int t = w; t < C; t += kThreads / 32) {
      float acc = 0.f, kx = 0.f;
      for (int i = l; i < dk; i += 32) {
        float dq = 0.f;
        for (int j = 0; j < dv; ++j) dq = fmaf(O[t * dv + j], S[i * dv + j], dq);
        dq *= G(t);
        acc = fmaf(Q[t * dk + i], dq, acc);
        for (int s = 0; s <= t; ++s) dq = fmaf(dP[t * C + s], K[s * dk + i], dq);
        const float x = X[t * dk + i], y = Y[t * dk + i];
        kx = fmaf(K[t * dk + i], x, kx);
        if (t < len) {
          const float gk = fmaf(be[t], x, y);
          if (shared_keys) {
            float* p = part + ((size_t)bh * T + t0 + t) * 2 * dk;
            p[i] = dq;
            p[dk + i] = gk;
          } else {
            const size_t at = ((size_t)key * T + t0 + t) * dk + i;
            reinterpret_cast<IO*>(d.gq)[at] = from_f32<IO>(dq);
            reinterpret_cast<IO*>(d.gk)[at] = from_f32<IO>(gk);
          }
        }
      }
      float rv = 0.f;
      for (int j = l; j < dv; j += 32) {
        rv = fmaf(R[t * dv + j], V[t * dv + j], rv);
        if (t < len) reinterpret_cast<IO*>(d.gv)[((size_t)bh * T + t0 + t) * dv + j] = from_f32<IO>(be[t] * R[t * dv + j]);
      }
      for (int m = 16; m; m >>= 1) {
        acc += __shfl_xor_sync(~0u, acc, m);
        kx += __shfl_xor_sync(~0u, kx, m);
        rv += __shfl_xor_sync(~0u, rv, m);
      }
      if (l == 0) {
        line[t] += acc;
        if (t < len) reinterpret_cast<IO*>(d.gbeta)[(size_t)bh * T + t0 + t] = from_f32<IO>(rv + kx);
      }
    }
    __syncthreads();
    if (tid < len) {
      float y = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) y += red[i];
      for (int s = C - 1; s >= tid; --s) y += line[s] + W[s * C + tid];
      for (int s = 0; s < tid; ++s) y += uz[s];
      reinterpret_cast<IO*>(d.gg)[(size_t)bh * T + t0 + tid] = from_f32<IO>(y);
    }
    __syncthreads();
    const float ge = G(C - 1);
    matmul(dk, dv, 2 * C, [&](int i, int t) { return t < C ? G(t) * Q[t * dk + i] : -be[t - C] * G(t - C) * K[(t - C) * dk + i]; },
           [&](int t, int j) { return t < C ? O[t * dv + j] : R[(t - C) * dv + j]; },
           [&](int i, int j, float x) { Z[i * dv + j] = fmaf(ge, Z[i * dv + j], x); });
    __syncthreads();
  }
  if (d.gstate0)
    for (int i = tid; i < dk * dv; i += kThreads) d.gstate0[bh * sz + i] = Z[i];
}

// gq, gk of a key head: the sum over its value heads, in order.
template <typename IO>
__global__ void __launch_bounds__(256) kla_delta_share_kernel(const DeltaArgs a, const DeltaGradArgs d,
                                                             const float* part) {
  const long long n = (long long)a.B * a.Hk * a.T * 2 * a.dk;
  const int rep = a.H / a.Hk, w = 2 * a.dk;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int e = (int)(i % w);
    const long long t = i / w % a.T, key = i / w / a.T;
    float x = 0.f;
    for (int r = 0; r < rep; ++r) x += part[((key * rep + r) * a.T + t) * w + e];
    IO* out = reinterpret_cast<IO*>(e < a.dk ? d.gq : d.gk);
    out[(key * a.T + t) * a.dk + e % a.dk] = from_f32<IO>(x);
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t delta_backward_bytes(int B, int Hk, int H, int T, int dk, int dv) {
  const size_t bh = (size_t)B * H, chunks = ((size_t)T + C - 1) / C;
  return align256(bh * chunks * dk * dv * sizeof(float)) + (Hk != H ? bh * T * 2 * dk * sizeof(float) : 0);
}

cudaError_t launch_delta_backward(const DeltaArgs& a, const DeltaGradArgs& g, void* workspace, cudaStream_t s) {
  float* ckpt = reinterpret_cast<float*>(workspace);
  const size_t chunks = ((size_t)a.T + C - 1) / C;
  float* part = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                         align256((size_t)a.B * a.H * chunks * a.dk * a.dv * sizeof(float)));
  DeltaArgs f = a;
  f.o = nullptr;
  f.stateT = nullptr;
  cudaError_t e = launch_delta_recurrent(f, ckpt, s);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)(2 * a.dk * a.dv + C * (4 * a.dk + 4 * a.dv) + 6 * C * C) * sizeof(float);
  auto run = [&](auto kernel) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return;
    kernel<<<(unsigned)((long long)a.B * a.H), kThreads, smem, s>>>(a, g, ckpt, part);
    e = cudaGetLastError();
  };
  if (a.io == IO_BF16) run(kla_delta_backward_kernel<__nv_bfloat16>);
  else run(kla_delta_backward_kernel<float>);
  if (e != cudaSuccess || a.Hk == a.H) return e;
  const long long blocks = ((long long)a.B * a.Hk * a.T * 2 * a.dk + 255) / 256;
  const unsigned grid = (unsigned)(blocks < (1LL << 30) ? blocks : 1LL << 30);
  if (a.io == IO_BF16) kla_delta_share_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, g, part);
  else kla_delta_share_kernel<float><<<grid, 256, 0, s>>>(a, g, part);
  return cudaGetLastError();
}

}  // namespace kla
