// The gated delta rule over a sequence in chunks of 64 tokens, on the tensor
// cores (sm_103a). With c_t the cumulative log decay inside a chunk, G_t = e^c_t,
// E_t = e^(c_end − c_t), D_ts = e^(c_t − c_s) and S the state before the chunk:
//
//   A = tril(β_t D_ts k_t·k_s, −1),  M = (I + A)^-1
//   U = M β(V − G K S),   S' = G_end S + Kᵀ(E U)
//   O = scale (G Q S + tril(D_ts q_t·k_s) U)
//
// Three kernels. `prepare` (a block per chunk and head) makes M. `chain` (a
// block per head and 64 columns, in order over the chunks) carries S in
// registers: three products and three round trips between TMEM, registers and
// shared memory per chunk, whose latency bounds it. `output` (a block per
// chunk, head and 64 columns) makes O. The backward pass runs the same chain
// from the end with Mᵀ (see kla_delta_backward.cu).
//
// Operands are bf16 parts (kla_umma.cuh): bf16 inputs are exact in one, states
// and everything that flows into them are kept in three, so that a state is as
// exact as in fp32; the outputs of bf16 calls are made from two parts (2^-16,
// against the 2^-8 of their rounding). Log decays are summed in 64 bits and
// kept as two floats, so that D of late tokens is exact behind a strong decay.
#include "kla_delta_chunk.cuh"

namespace kla {
namespace delta {

namespace {

// dst[n×n] = ± a·b for n = 16 or 32, all with row length 68; four columns a task.
__device__ __forceinline__ void small_matmul(float* dst, const float* a, const float* b, int n, bool neg, int task) {
  const int i = task / (n / 4), j = task % (n / 4) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float x = a[i * 68 + k];
    const float4 y = *reinterpret_cast<const float4*>(b + k * 68 + j);
    s.x = fmaf(x, y.x, s.x);
    s.y = fmaf(x, y.y, s.y);
    s.z = fmaf(x, y.z, s.z);
    s.w = fmaf(x, y.w, s.w);
  }
  if (neg) s = make_float4(-s.x, -s.y, -s.z, -s.w);
  *reinterpret_cast<float4*>(dst + i * 68 + j) = s;
}

// M = (I + A)^-1 for A strictly lower, 64 × 64 with row length 68: substitution in the 16 × 16 blocks on the diagonal,
// then [[X, 0], [L, Y]]^-1 = [[X', 0], [−Y' L X', Y']] for 32 and 64. L X' goes where A's upper blocks would be.
__device__ void invert(float* A, float* M, int tid) {
  if (tid < 64) {
    const int b = tid & 48, c = tid & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = i == c ? 1.f : 0.f;
#pragma unroll
      for (int s = 0; s < i; ++s) x[i] = fmaf(-A[(b + i) * 68 + b + s], x[s], x[i]);
      M[(b + i) * 68 + b + c] = x[i];
    }
  } else {
    for (int i = tid - 64; i < 64 * 64; i += kThreads - 64)
      if ((i >> 10) != ((i & 63) >> 4)) M[(i >> 6) * 68 + (i & 63)] = 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int n = 16; n <= 32; n *= 2) {
    const int tasks = n * n / 4, p = tid / tasks, o = p * 2 * n * 68 + p * 2 * n;  // pair p of blocks
    const bool mine = p < 32 / n;
    if (mine) small_matmul(A + o + n, A + o + n * 68, M + o, n, false, tid % tasks);
    __syncthreads();
    if (mine) small_matmul(M + o + n * 68, M + o + n * 68 + n, A + o + n, n, true, tid % tasks);
    __syncthreads();
  }
}

template <typename IO, int DK, bool BWD>
struct PrepareSmem {
  static constexpr int PARTS = kParts<IO>, IN = PARTS * DK / 64 * kTileBytes;
  static constexpr int K = 0, Q = IN, P = Q + (BWD ? IN : 0), O = P + (BWD ? 3 * kTileBytes : 0),
                       GO = O + PARTS * kTileBytes, A = O, M = A + 64 * 68 * 4;  // A and M are done with before O and GO
  static constexpr int kEnd = BWD && GO + 3 * kTileBytes > M + 64 * 68 * 4 ? GO + 3 * kTileBytes : M + 64 * 68 * 4;
  static constexpr int kBytes = kEnd + 1024;
};

template <typename IO, int DK, bool BWD>
__global__ void __launch_bounds__(kThreads) kla_delta_prepare_kernel(const DeltaArgs a, const DeltaGradArgs d,
                                                                    const Workspace w) {
  using L = PrepareSmem<IO, DK, BWD>;
  constexpr int PARTS = L::PARTS, COLS = BWD ? 256 : 64;
  extern __shared__ char raw[];
  char* sm = align1024(raw);
  __shared__ float hi[C], lo[C], G[C], be[C];
  __shared__ uint64_t bar;
  __shared__ uint32_t slot;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const Where at = where(a, blockIdx.x);
  const IO* k = reinterpret_cast<const IO*>(a.k) + ((size_t)at.key * a.T + at.t0) * a.dk;
  TileLoad<IO, DK, kThreads> kl, ql;
  kl.fetch(k, at.len, a.dk, 0, tid);
  if (BWD) ql.fetch(reinterpret_cast<const IO*>(a.q) + ((size_t)at.key * a.T + at.t0) * a.dk, at.len, a.dk, 0, tid);
  if (warp == 0) tmem_alloc(&slot, COLS);
  if (tid == 32) mbar_init(&bar, 1);
  if (warp == 2) {  // the gates: two tokens a lane
    double x[2];
    float b[2];
    const size_t row = (size_t)at.bh * a.T + at.t0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const bool in = t < at.len;
      const float g = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.g)[row + t]) : 0.f;
      x[i] = g < kMinLog ? kMinLog : g;
      b[i] = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.beta)[row + t]) : 0.f;
    }
    x[1] += x[0];
    double sum = x[1];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const double y = __shfl_up_sync(~0u, sum, m);
      if (lane >= m) sum += y;
    }
    const double before = __shfl_up_sync(~0u, sum, 1), total = __shfl_sync(~0u, sum, 31);
    float* out = w.gates + at.chunk * kGates;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const double c = lane ? before + x[i] : x[i];
      const float h = (float)c, l = (float)(c - h), g = expf(h) * (1.f + l);
      hi[t] = h, lo[t] = l, G[t] = g, be[t] = b[i];
      out[t] = h, out[C + t] = l, out[2 * C + t] = g, out[3 * C + t] = expf((float)(total - c)), out[4 * C + t] = b[i];
    }
  }
  kl.put(sm + L::K, tid);
  if (BWD) ql.put(sm + L::Q, tid);
  fence_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(slot), base = uniform(smem_addr(sm));
  const Operand<PARTS, false> Kr{base + L::K, DK / 64 * kTileBytes, kTileBytes}, Qr{base + L::Q, DK / 64 * kTileBytes, kTileBytes};
  bool ok = true;
  if (warp == 0 && elect()) {
    mma<64, 64, DK>(tm, Kr, Kr);
    if (BWD) mma<64, 64, DK>(tm + 64, Qr, Kr);
    commit(&bar);
  }
  float* A = reinterpret_cast<float*>(sm + L::A);
  float* M = reinterpret_cast<float*>(sm + L::M);
  const int quad = warp & 3, half = warp >> 2, r0 = 16 * quad + (lane >> 2), c0 = 32 * half + 2 * (lane & 3);
  const uint32_t rows = (uint32_t)(32 * quad) << 16;
  mbar_wait(&bar, 0, ok);
  fence_after();
  float v[16];
  tmem_load(tm + rows + 32 * half, v);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int t = r0 + (i & 2) * 4, s = c0 + (i >> 2) * 8 + (i & 1);
    A[t * 68 + s] = s < t ? be[t] * decay(hi, lo, t, s) * v[i] : 0.f;
  }
  if (BWD) {  // P, scaled
    tmem_load(tm + 64 + rows + 32 * half, v);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const int t = r0 + (i & 2) * 4, s = c0 + (i >> 2) * 8;
      const float x = s <= t ? a.scale * decay(hi, lo, t, s) * v[i] : 0.f;
      const float y = s + 1 <= t ? a.scale * decay(hi, lo, t, s + 1) * v[i + 1] : 0.f;
      store_pair<3>(sm + L::P, kTileBytes, t, s, x, y);
    }
  }
  __syncthreads();
  invert(A, M, tid);
  float* out = w.M + at.chunk * C * C;
  for (int i = tid; i < C * C / 4; i += kThreads) {
    float4 x = *reinterpret_cast<const float4*>(M + (i >> 4) * 68 + (i & 15) * 4);
    if (!ok) x.x = x.y = x.z = x.w = __int_as_float(0x7fc00000);  // a wait ran out
    reinterpret_cast<float4*>(out)[i] = x;
  }
  if (BWD) {
    const int DV = pad64(a.dv);
    __syncthreads();
    for (int sl = 0; sl < DV / 64; ++sl) {
      const IO* go = reinterpret_cast<const IO*>(d.go);
      TileLoad<IO, 64, kThreads> ol;
      ol.fetch(go + (go ? ((size_t)at.bh * a.T + at.t0) * a.dv : 0), go ? at.len : 0, a.dv, sl * 64, tid);
      ol.put(sm + L::O, tid);
#pragma unroll
      for (int j = 0; j < ol.N; ++j) {
        const int i = tid + j * kThreads, r = i >> 3;
        float x[8];
        ol.eight(j, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= a.scale * G[r];
        store_eight<3>(sm + L::GO, kTileBytes, r, (i & 7) * 8, x);
      }
      fence_async();
      fence_before();
      __syncthreads();
      fence_after();
      if (warp == 0 && elect()) {
        const Operand<3, true> Pt{base + L::P, kTileBytes, kTileBytes}, GO{base + L::GO, kTileBytes, kTileBytes};
        const Operand<PARTS, true> O{base + L::O, kTileBytes, kTileBytes}, Qt{base + L::Q, DK / 64 * kTileBytes, kTileBytes};
        mma<64, 64, 64>(tm + 128, Pt, O);
        mma<DK, 64, 64>(tm + 192, Qt, GO);
        commit(&bar);
      }
      mbar_wait(&bar, (sl + 1) & 1, ok);
      fence_after();
      const float bad = ok ? 0.f : __int_as_float(0x7fc00000);
      tmem_load(tm + 128 + rows + 32 * half, v);
      float* R = w.R + at.chunk * C * DV + sl * 64;
#pragma unroll
      for (int i = 0; i < 16; i += 2)
        store_two(R + (r0 + (i & 2) * 4) * DV + c0 + (i >> 2) * 8, v[i] + bad, v[i + 1] + bad);
      float* Z = w.Z + at.chunk * DK * DV + sl * 64;
#pragma unroll
      for (int rb = 0; rb < DK / 64; ++rb) {
        tmem_load(tm + 192 + rows + ((uint32_t)(16 * rb) << 16) + 32 * half, v);
        const int r = (DK == 64 ? 16 * quad : 32 * quad + 16 * rb) + (lane >> 2);
#pragma unroll
        for (int i = 0; i < 16; i += 2) store_two(Z + (r + (i & 2) * 4) * DV + c0 + (i >> 2) * 8, v[i], v[i + 1]);
      }
      fence_before();
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 0) tmem_free(tm, COLS);
}

// ---- the chain ----------------------------------------------------------------------
// X: the state (rev: its gradient). Per chunk, with Y = K X:
//   forward:  W = β(V − G Y),       U = M W,   X = G_end X + Kᵀ(E U)
//   reverse:  W = Pᵀ O' + E Y,     dR = Mᵀ W,  X = G_end X + Qᵀ(G O') − Kᵀ(β G dR)
// Eight warps walk the chunks; four more bring K and M of the next chunk as
// parts, two chunks deep.
constexpr int kChainThreads = 256, kFeedThreads = 128;

template <typename IO, int DK>
struct ChainSmem {
  static constexpr int KB = kParts<IO> * DK / 64 * kTileBytes, MB = 3 * kTileBytes;
  static constexpr int K = 0, M = 2 * KB, X = M + 2 * MB, W = X + 3 * DK * 128, kBytes = W + MB + 1024;
};

template <typename IO, int DK, bool REV>
__global__ void __launch_bounds__(kChainThreads + kFeedThreads) kla_delta_chain_kernel(const DeltaArgs a,
                                                                                      const DeltaGradArgs d,
                                                                                      const Workspace w) {
  using L = ChainSmem<IO, DK>;
  constexpr int PARTS = kParts<IO>, RB = DK / 64;
  extern __shared__ char raw[];
  char* sm = align1024(raw);
  __shared__ uint64_t full[2], empty[2], done[3];
  __shared__ uint32_t slot;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int DV = pad64(a.dv), N = (a.T + C - 1) / C;
  const long long bh = blockIdx.x / (DV / 64);
  const int col = (int)(blockIdx.x % (DV / 64)) * 64;
  const long long key = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&full[i], kFeedThreads), mbar_init(&empty[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&done[i], 1);
  }
  if (warp == 0) tmem_alloc(&slot, 256);
  fence_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(slot), base = uniform(smem_addr(sm));
  bool ok = true;
  if (tid >= kChainThreads) {
    const int ft = tid - kChainThreads;
    const IO* k = reinterpret_cast<const IO*>(a.k) + (size_t)key * a.T * a.dk;
    for (int i = 0; i < N; ++i) {
      const int n = REV ? N - 1 - i : i, b = i & 1;
      const float4* src = reinterpret_cast<const float4*>(w.M + ((size_t)bh * N + n) * C * C);
      float4 m[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[2 * j] = src[(ft + j * kFeedThreads) * 2];
        m[2 * j + 1] = src[(ft + j * kFeedThreads) * 2 + 1];
      }
      TileLoad<IO, DK, kFeedThreads> kl;
      if (PARTS == 1) kl.fetch(k + (size_t)n * C * a.dk, min(C, a.T - n * C), a.dk, 0, ft);
      if (i >= 2) mbar_wait(&empty[b], ((i >> 1) - 1) & 1, ok);
      if (PARTS > 1) kl.fetch(k + (size_t)n * C * a.dk, min(C, a.T - n * C), a.dk, 0, ft);  // too many to hold while waiting
      kl.put(sm + L::K + b * L::KB, ft);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = ft + j * kFeedThreads;
        float x[8] = {m[2 * j].x, m[2 * j].y, m[2 * j].z, m[2 * j].w,
                      m[2 * j + 1].x, m[2 * j + 1].y, m[2 * j + 1].z, m[2 * j + 1].w};
        store_eight<3>(sm + L::M + b * L::MB, kTileBytes, e >> 3, (e & 7) * 8, x);
      }
      fence_async();
      mbar_arrive(&full[b]);
    }
  } else {
    const int quad = warp & 3, half = warp >> 2;
    const int r0 = 16 * quad + (lane >> 2), c0 = 32 * half + 2 * (lane & 3);
    const uint32_t rows = (uint32_t)(32 * quad) << 16;
    int xr[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) xr[rb] = (DK == 64 ? 16 * quad : 32 * quad + 16 * rb) + (lane >> 2);
    float X[RB][16];
    const float* first = REV ? d.gstateT : a.state0;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int r = xr[rb] + (i & 2) * 4, c = col + c0 + (i >> 2) * 8;
        float2 x = make_float2(0.f, 0.f);
        if (first && r < a.dk && c < a.dv) x = load_two(first + ((size_t)bh * a.dk + r) * a.dv + c);
        X[rb][i] = x.x, X[rb][i + 1] = x.y;
      }
    // this chunk's rows of V (rev: Pᵀ O') and gates, loaded a chunk ahead
    float ga[2], gb[2], gend = 0.f, B[16];
    float2 raw_b[8];
    float raw_g[2][3];
    auto fetch = [&](int i) {
      const int n = REV ? N - 1 - i : i, len = min(C, a.T - n * C);
      const size_t chunk = (size_t)bh * N + n;
      const float* gates = w.gates + chunk * kGates;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = r0 + 8 * e;
#pragma unroll
        for (int m = 0; m < 3; ++m) raw_g[e][m] = gates[(2 + m) * C + t];
        const IO* v = reinterpret_cast<const IO*>(a.v) + ((size_t)bh * a.T + n * C + t) * a.dv + col + c0;
        const float* p = w.R + (chunk * C + t) * DV + col + c0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (REV) raw_b[2 * j + e] = load_two(p + 8 * j);
          else raw_b[2 * j + e] = t < len && col + c0 + 8 * j < a.dv ? load_two(v + 8 * j) : make_float2(0.f, 0.f);
        }
      }
      return gates[2 * C + C - 1];
    };
    float next_end = fetch(0);
    for (int i = 0; i < N; ++i) {
      const int n = REV ? N - 1 - i : i, b = i & 1;
      const uint32_t parity = i & 1;
      const size_t chunk = (size_t)bh * N + n;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          store_pair<3>(sm + L::X, DK * 128, xr[rb] + (e & 2) * 4, c0 + (e >> 2) * 8, X[rb][e], X[rb][e + 1]);
      fence_async();
      fence_before();
      bar_sync(1, kChainThreads);
      const Operand<PARTS, false> Kr{base + L::K + b * L::KB, RB * kTileBytes, kTileBytes};
      const Operand<PARTS, true> Kt{base + L::K + b * L::KB, RB * kTileBytes, kTileBytes};
      const Operand<3, REV> Mx{base + L::M + b * L::MB, kTileBytes, kTileBytes};
      const Operand<3, true> Xs{base + L::X, DK * 128, DK * 128}, Ws{base + L::W, kTileBytes, kTileBytes};
      if (warp == 0) {
        mbar_wait(&full[b], (i >> 1) & 1, ok);
        fence_after();
        if (elect()) {
          mma<64, 64, DK>(tm, Kr, Xs);
          commit(&done[0]);
        }
      }
      // while that runs: the state goes out; in reverse its slot first gives up Qᵀ(G O')
      float F[REV ? RB : 1][16];
      float* Xout = (REV ? w.Z : w.S) + chunk * DK * DV + col + c0;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          float* p = Xout + (xr[rb] + (e & 2) * 4) * DV + (e >> 2) * 8;
          if (REV) {
            const float2 x = load_two(p);
            F[rb][e] = x.x, F[rb][e + 1] = x.y;
          } else {
            store_two(p, X[rb][e], X[rb][e + 1]);
          }
        }
      gend = next_end;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float G = raw_g[e][0], E = raw_g[e][1], be = raw_g[e][2];
        ga[e] = REV ? E : -be * G;  // Y's factor in W
        gb[e] = REV ? -be * G : E;  // U's (dR's) on its way into X
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = raw_b[2 * j + e];
          B[4 * j + 2 * e] = REV ? x.x : be * x.x, B[4 * j + 2 * e + 1] = REV ? x.y : be * x.y;
        }
      }
      if (i + 1 < N) next_end = fetch(i + 1);
      float v[16];
      mbar_wait(&done[0], parity, ok);
      fence_after();
      tmem_load(tm + rows + 32 * half, v);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const int o = (e & 2) >> 1;
        store_pair<3>(sm + L::W, kTileBytes, r0 + 8 * o, c0 + (e >> 2) * 8, fmaf(ga[o], v[e], B[e]),
                      fmaf(ga[o], v[e + 1], B[e + 1]));
      }
      fence_async();
      fence_before();
      bar_sync(1, kChainThreads);
      if (warp == 0 && elect()) {
        fence_after();
        mma<64, 64, 64>(tm + 64, Mx, Ws);
        commit(&done[1]);
      }
      mbar_wait(&done[1], parity, ok);
      fence_after();
      tmem_load(tm + 64 + rows + 32 * half, v);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const int o = (e & 2) >> 1;
        store_pair<3>(sm + L::W, kTileBytes, r0 + 8 * o, c0 + (e >> 2) * 8, gb[o] * v[e], gb[o] * v[e + 1]);
      }
      fence_async();
      fence_before();
      bar_sync(1, kChainThreads);
      if (warp == 0 && elect()) {
        fence_after();
        mma<DK, 64, 64>(tm + 128, Kt, Ws);
        commit(&done[2]);
        commit(&empty[b]);
      }
      float* Uout = (REV ? w.R : w.U) + (chunk * C + r0) * DV + col + c0;
#pragma unroll
      for (int e = 0; e < 16; e += 2) store_two(Uout + (e & 2) * 4 * DV + (e >> 2) * 8, v[e], v[e + 1]);
      if (REV) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            store_two(Xout + (xr[rb] + (e & 2) * 4) * DV + (e >> 2) * 8, X[rb][e], X[rb][e + 1]);
      }
      mbar_wait(&done[2], parity, ok);
      fence_after();
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        tmem_load(tm + 128 + rows + ((uint32_t)(16 * rb) << 16) + 32 * half, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) X[rb][e] = fmaf(gend, X[rb][e], REV ? v[e] + F[REV ? rb : 0][e] : v[e]);
      }
    }
    float* last = REV ? d.gstate0 : a.stateT;
    if (last) {
      const float bad = ok ? 0.f : __int_as_float(0x7fc00000);  // a wait ran out
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int r = xr[rb] + (i & 2) * 4, c = col + c0 + (i >> 2) * 8;
          if (r < a.dk && c < a.dv)
            store_two(last + ((size_t)bh * a.dk + r) * a.dv + c, X[rb][i] + bad, X[rb][i + 1] + bad);
        }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 0) tmem_free(tm, 256);
}

// ---- the output ----------------------------------------------------------------------
template <typename IO, int DK>
struct OutputSmem {
  static constexpr int IN = kParts<IO> * DK / 64 * kTileBytes, PN = sizeof(IO) == 2 ? 2 : 3;
  static constexpr int K = 0, Q = IN, S = 2 * IN, U = S + PN * DK * 128, P = U + PN * kTileBytes,
                       kBytes = P + PN * kTileBytes + 1024;
};

template <typename IO, int DK>
__global__ void __launch_bounds__(kThreads) kla_delta_output_kernel(const DeltaArgs a, const Workspace w) {
  using L = OutputSmem<IO, DK>;
  constexpr int PARTS = kParts<IO>, PN = L::PN;
  extern __shared__ char raw[];
  char* sm = align1024(raw);
  __shared__ float hi[C], lo[C], G[C];
  __shared__ uint64_t bar;
  __shared__ uint32_t slot;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int DV = pad64(a.dv);
  const Where at = where(a, blockIdx.x / (DV / 64));
  const int col = (int)(blockIdx.x % (DV / 64)) * 64;
  if (warp == 0) tmem_alloc(&slot, 128);
  if (tid == 32) mbar_init(&bar, 1);
  const size_t row = (size_t)at.key * a.T + at.t0;
  TileLoad<IO, DK, kThreads> kl, ql;
  PartsLoad<PN, DK, kThreads> xl;
  PartsLoad<PN, C, kThreads> ul;
  kl.fetch(reinterpret_cast<const IO*>(a.k) + row * a.dk, at.len, a.dk, 0, tid);
  ql.fetch(reinterpret_cast<const IO*>(a.q) + row * a.dk, at.len, a.dk, 0, tid);
  xl.fetch(w.S + at.chunk * DK * DV + col, DV, tid);
  ul.fetch(w.U + at.chunk * C * DV + col, DV, tid);
  if (tid < C) {
    const float* g = w.gates + at.chunk * kGates + tid;
    hi[tid] = g[0], lo[tid] = g[C], G[tid] = g[2 * C];
  }
  kl.put(sm + L::K, tid);
  ql.put(sm + L::Q, tid);
  xl.put(sm + L::S, tid);
  ul.put(sm + L::U, tid);
  fence_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(slot), base = uniform(smem_addr(sm));
  bool ok = true;
  if (warp == 0 && elect()) {
    const Operand<PARTS, false> Kr{base + L::K, DK / 64 * kTileBytes, kTileBytes}, Qr{base + L::Q, DK / 64 * kTileBytes, kTileBytes};
    mma<64, 64, DK>(tm, Qr, Kr);
    mma<64, 64, DK>(tm + 64, Qr, Operand<PN, true>{base + L::S, DK * 128, DK * 128});
    commit(&bar);
  }
  const int quad = warp & 3, half = warp >> 2, r0 = 16 * quad + (lane >> 2), c0 = 32 * half + 2 * (lane & 3);
  const uint32_t rows = (uint32_t)(32 * quad) << 16;
  mbar_wait(&bar, 0, ok);
  fence_after();
  float v[16], y[16];
  tmem_load(tm + rows + 32 * half, v);
  tmem_load(tm + 64 + rows + 32 * half, y);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const int t = r0 + (i & 2) * 4, s = c0 + (i >> 2) * 8;
    store_pair<PN>(sm + L::P, kTileBytes, t, s, s <= t ? decay(hi, lo, t, s) * v[i] : 0.f,
                   s + 1 <= t ? decay(hi, lo, t, s + 1) * v[i + 1] : 0.f);
  }
  fence_async();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 0 && elect()) {
    mma<64, 64, 64>(tm, Operand<PN, false>{base + L::P, kTileBytes, kTileBytes},
                    Operand<PN, true>{base + L::U, kTileBytes, kTileBytes});
    commit(&bar);
  }
  mbar_wait(&bar, 1, ok);
  fence_after();
  tmem_load(tm + rows + 32 * half, v);
  IO* o = reinterpret_cast<IO*>(a.o) + ((size_t)at.bh * a.T + at.t0) * a.dv + col;
  const float scale = ok ? a.scale : __int_as_float(0x7fc00000);  // a wait ran out
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const int t = r0 + (i & 2) * 4, c = c0 + (i >> 2) * 8;
    if (t < at.len && col + c < a.dv)
      store_two(o + (size_t)t * a.dv + c, scale * fmaf(G[t], y[i], v[i]), scale * fmaf(G[t], y[i + 1], v[i + 1]));
  }
  fence_before();
  __syncthreads();
  if (warp == 0) tmem_free(tm, 128);
}

template <typename F, typename... Args>
cudaError_t run(F kernel, int smem, unsigned blocks, int threads, cudaStream_t s, const Args&... args) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, threads, smem, s>>>(args...);
  return cudaGetLastError();
}

unsigned chunks(const DeltaArgs& a) { return (unsigned)((long long)a.B * a.H * ((a.T + C - 1) / C)); }

template <typename IO, int DK>
cudaError_t prepare_dk(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, cudaStream_t s) {
  if (d)
    return run(kla_delta_prepare_kernel<IO, DK, true>, PrepareSmem<IO, DK, true>::kBytes, chunks(a), kThreads, s, a, *d, w);
  return run(kla_delta_prepare_kernel<IO, DK, false>, PrepareSmem<IO, DK, false>::kBytes, chunks(a), kThreads, s, a,
             DeltaGradArgs{}, w);
}
template <typename IO, int DK>
cudaError_t chain_dk(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, bool rev, cudaStream_t s) {
  const unsigned blocks = (unsigned)((long long)a.B * a.H * (pad64(a.dv) / 64));
  const int threads = kChainThreads + kFeedThreads, smem = ChainSmem<IO, DK>::kBytes;
  if (rev) return run(kla_delta_chain_kernel<IO, DK, true>, smem, blocks, threads, s, a, *d, w);
  return run(kla_delta_chain_kernel<IO, DK, false>, smem, blocks, threads, s, a, DeltaGradArgs{}, w);
}
template <typename IO, int DK>
cudaError_t output_dk(const DeltaArgs& a, const Workspace& w, cudaStream_t s) {
  return run(kla_delta_output_kernel<IO, DK>, OutputSmem<IO, DK>::kBytes, chunks(a) * (pad64(a.dv) / 64), kThreads, s, a, w);
}

}  // namespace

Workspace workspace(void* base, int B, int Hk, int H, int T, int dk, int dv, bool backward, size_t* bytes) {
  const size_t n = (size_t)B * H * (((size_t)T + C - 1) / C), DK = pad64(dk), DV = pad64(dv);
  size_t at = 0;
  auto take = [&](size_t floats) {
    float* p = reinterpret_cast<float*>(reinterpret_cast<char*>(base) + at);
    at += (floats * sizeof(float) + 255) / 256 * 256;
    return p;
  };
  Workspace w{};
  w.M = take(n * C * C);
  w.gates = take(n * kGates);
  w.S = take(n * DK * DV);
  w.U = take(n * C * DV);
  if (backward) {
    w.Z = take(n * DK * DV);
    w.R = take(n * C * DV);
    if (Hk != H) w.part = take((size_t)B * H * T * 2 * dk);
  }
  *bytes = at;
  return w;
}

cudaError_t launch_prepare(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, cudaStream_t s) {
  const bool wide = pad64(a.dk) == 128;
  if (a.io == IO_BF16) return wide ? prepare_dk<__nv_bfloat16, 128>(a, d, w, s) : prepare_dk<__nv_bfloat16, 64>(a, d, w, s);
  return wide ? prepare_dk<float, 128>(a, d, w, s) : prepare_dk<float, 64>(a, d, w, s);
}

cudaError_t launch_chain(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, bool rev, cudaStream_t s) {
  const bool wide = pad64(a.dk) == 128;
  if (a.io == IO_BF16)
    return wide ? chain_dk<__nv_bfloat16, 128>(a, d, w, rev, s) : chain_dk<__nv_bfloat16, 64>(a, d, w, rev, s);
  return wide ? chain_dk<float, 128>(a, d, w, rev, s) : chain_dk<float, 64>(a, d, w, rev, s);
}

}  // namespace delta

// Few tokens are faster one by one (see kla_delta.cu); the choice depends on the length alone.
bool delta_chunked(int T) { return T > 64; }

size_t delta_forward_bytes(int B, int Hk, int H, int T, int dk, int dv) {
  size_t n = 0;
  if (delta_chunked(T)) delta::workspace(nullptr, B, Hk, H, T, dk, dv, false, &n);
  return n;
}

cudaError_t launch_delta_forward(const DeltaArgs& a, void* workspace, cudaStream_t s) {
  if (!delta_chunked(a.T)) return launch_delta_recurrent(a, s);
  size_t n = 0;
  const delta::Workspace w = delta::workspace(workspace, a.B, a.Hk, a.H, a.T, a.dk, a.dv, false, &n);
  cudaError_t e = delta::launch_prepare(a, nullptr, w, s);
  if (e == cudaSuccess) e = delta::launch_chain(a, nullptr, w, false, s);
  if (e != cudaSuccess) return e;
  const bool wide = delta::pad64(a.dk) == 128;
  if (a.io == IO_BF16)
    return wide ? delta::output_dk<__nv_bfloat16, 128>(a, w, s) : delta::output_dk<__nv_bfloat16, 64>(a, w, s);
  return wide ? delta::output_dk<float, 128>(a, w, s) : delta::output_dk<float, 64>(a, w, s);
}

}  // namespace kla
