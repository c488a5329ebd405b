// The gated delta rule over a sequence in chunks of 64 tokens, on the tensor
// cores (sm_103a). With c_t the cumulative log decay inside a chunk, G_t = e^c_t,
// E_t = e^(c_end − c_t), D_ts = e^(c_t − c_s) and S the state before the chunk:
//
//   A = tril(β_t D_ts k_t·k_s, −1),  M = (I + A)^-1
//   U = M β(V − G K S),   S' = G_end S + Kᵀ(E U)
//   O = scale (G Q S + tril(D_ts q_t·k_s) U)
//
// Three kernels. `prepare` (a block per chunk and head) makes M and with it
// W = −M (β G K) and M (β V). `chain` (a block per head and 64 or 32 columns, in
// order over the chunks) carries S in registers: U = M (β V) + W S and the
// update, two products and two round trips between TMEM, registers and shared
// memory per chunk; its latency (1.3 to 1.5 us a chunk) or, with a block on most
// SMs, DRAM bounds it. `output` (a block per chunk, head and 64 columns) makes
// O. The backward pass runs the same chain from the end with Mᵀ, beside the
// other (see kla_delta_backward.cu). At 8 × 16 heads of 64 × 64 and 4096 tokens in
// bf16: prepare 179 us (shared memory's data pipe, 82% busy with four blocks an
// SM), chain 110 (640 MB, 5.8 TB/s), output 107 (460 MB, 4.3 TB/s).
//
// Operands are bf16 parts (kla_umma.cuh): bf16 inputs are exact in one, states
// and everything else that is made of them are kept in three, so that states and
// outputs are as exact as in fp32 and a bf16 output is rounded once (two parts,
// 2^-16, would turn some 1 in 2000 outputs to the next step and save 2 to 5% of
// a call: output 97 for 106 us, gradients 358 for 405). Cumulative log decays are kept as sums
// of two floats, in powers of two, so that D of late tokens is exact behind a
// strong decay.
#include <algorithm>
#include <cmath>

#include "kla_delta_chunk.cuh"

namespace kla {
namespace delta {

namespace {

// Four columns j of row i of ± a·b, over k in [k0, k1): matrices of row length 68, k0 and k1 multiples of four.
__device__ __forceinline__ void four_columns(float* dst, const float* a, const float* b, int i, int j, int k0, int k1,
                                             float sign) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = k0; k < k1; k += 4) {
    const float4 x = *reinterpret_cast<const float4*>(a + i * 68 + k);
    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 y = *reinterpret_cast<const float4*>(b + (k + e) * 68 + j);
      s.x = fmaf(f[e], y.x, s.x);
      s.y = fmaf(f[e], y.y, s.y);
      s.z = fmaf(f[e], y.z, s.z);
      s.w = fmaf(f[e], y.w, s.w);
    }
  }
  *reinterpret_cast<float4*>(dst + i * 68 + j) = make_float4(sign * s.x, sign * s.y, sign * s.z, sign * s.w);
}

// M = (I + A)^-1 for A strictly lower, 64 × 64 with row length 68: substitution in the 16 × 16 blocks on the diagonal (a
// lane per column; each entry as it is found goes into all later ones, from D, the blocks' columns), then
// [[X, 0], [L, Y]]^-1 = [[X', 0], [−Y' L X', Y']] for 32 and 64 (X', Y' lower triangular, so the sums start at the column
// or end at the row). L X' goes where A's upper blocks would be. Powers of A are not used: they grow like binomials where
// keys repeat.
constexpr int kDiagRow = 20, kDiagFloats = 4 * 16 * kDiagRow;
__device__ void invert(float* A, float* M, const float* D, int warp, int lane) {
  if (warp < 2) {
    const int b = warp * 32 + (lane & 16), c = lane & 15;
    const float* col = D + (b >> 4) * 16 * kDiagRow;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.f : 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      M[(b + s) * 68 + b + c] = x[s];
#pragma unroll
      for (int i = (s + 1) & ~3; i < 16; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(col + s * kDiagRow + i);
        if (i > s) x[i] = fmaf(-f.x, x[s], x[i]);
        if (i + 1 > s) x[i + 1] = fmaf(-f.y, x[s], x[i + 1]);
        if (i + 2 > s) x[i + 2] = fmaf(-f.z, x[s], x[i + 2]);
        x[i + 3] = fmaf(-f.w, x[s], x[i + 3]);
      }
    }
  } else {
    for (int i = (warp - 2) * 32 + lane; i < 64 * 16; i += kThreads - 64) {
      const int r = i >> 4, c = (i & 15) * 4;
      if ((r >> 4) != (c >> 4)) *reinterpret_cast<float4*>(M + r * 68 + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __syncthreads();
  const int o = (warp >> 1) * (32 * 68 + 32), i16 = lane & 15, j16 = ((warp & 1) * 2 + (lane >> 4)) * 4;  // two pairs of 16
  if (warp < 4) four_columns(A + o + 16, A + o + 16 * 68, M + o, i16, j16, 0, 16, 1.f);
  __syncthreads();
  if (warp < 4) four_columns(M + o + 16 * 68, M + o + 16 * 68 + 16, A + o + 16, i16, j16, 0, 16, -1.f);
  __syncthreads();
  four_columns(A + 32, A + 32 * 68, M, lane, warp * 4, warp * 4, 32, 1.f);
  __syncthreads();
  four_columns(M + 32 * 68, M + 32 * 68 + 32, A + 32, warp * 4 + (lane >> 3), (lane & 7) * 4, 0, warp * 4 + 4, -1.f);
  __syncthreads();
}

template <typename IO, int DK, bool BWD>
struct PrepareSmem {
  static constexpr int PARTS = kParts<IO>, IN = PARTS * DK / 64 * kTileBytes, ROWS = PARTS * kTileBytes;
  static constexpr int M3 = 3 * kTileBytes;
  // T1 first holds A (with the cumulative logs and the diagonal blocks' columns behind it), T2 the inverse in fp32.
  // Forward, the two products of M follow one another with T1 as their operand, and V lies where the inverse was:
  // four blocks fit on an SM (8 × 16 heads of 64, 4096 tokens: 191 -> 180 us; 16 heads of 128, 65536 tokens, three
  // blocks that two places in TMEM held back before: 505 -> 485).
  static constexpr int MB = 64 * 68 * 4 > ROWS ? 64 * 68 * 4 : ROWS;
  static constexpr int K = 0, Q = IN, V0 = Q + (BWD ? IN : 0), P = V0 + (BWD ? ROWS : 0), T1 = P + (BWD ? M3 : 0),
                       M = T1 + M3, A = T1, T2 = BWD ? M : T1, V = BWD ? V0 : M;
  static_assert((64 * 68 + 2 * C + kDiagFloats) * 4 <= M3, "");
  static constexpr int kBytes = M + (BWD ? M3 : MB);
  static_assert(kBytes <= kMaxBytes && V % 1024 == 0, "");
  static constexpr int kFit = 228 * 1024 / (kBytes + 2048);
  static constexpr int kBlocks = BWD ? (kBytes <= 110 * 1024 ? 2 : 1) : kFit < 4 ? kFit : 4;  // of an SM
};

// (h + l) += (yh + yl), the sum again as two floats
__device__ __forceinline__ void add_two(float& h, float& l, float yh, float yl) {
  const float s = h + yh, t = s - h;
  const float e = ((h - (s - t)) + (yh - t)) + (l + yl);
  h = s + e;
  l = e - (h - s);
}

// Blocks of a product from TMEM: `BLOCKS` of them across columns (ROWS = 64) or down 128 rows
template <int ROWS, int BLOCKS>
__device__ __forceinline__ void drain(uint32_t tm, float* out, const Lanes& l, int tid) {
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    Fragment f;
    tmem_load(tm + ((uint32_t)(32 * l.quad + (ROWS == 64 ? 0 : 16 * b)) << 16) + (ROWS == 64 ? 64 * b : 0) + 32 * l.half, f.v);
    f.store(out + b * kBlock, tid);
  }
}

// 64 × 64 BLOCKS of a product as the chain's operand (see Workspace). A lane's four words of a row turn into one eight.
template <int BLOCKS>
__device__ __forceinline__ void drain_parts(uint32_t tm, char* out, const Lanes& l) {
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    Fragment f;
    tmem_load(tm + ((uint32_t)(32 * l.quad) << 16) + 64 * b + 32 * l.half, f.v);
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int r = l.r + 8 * o, c = 4 * l.half + (l.lane & 3);
      char* to = out + (((c ^ r) & 7) << 4);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float &x = f.v[4 * j + 2 * o], &y = f.v[4 * j + 2 * o + 1];
          u[j] = bf16_pair(x, y);
          x -= __uint_as_float(u[j] << 16);
          y -= __uint_as_float(u[j] & 0xffff0000u);
        }
        turn_four(u, l.lane);
        const int row = p < 2 ? b * 128 + r + 16 * (l.quad + p) : BLOCKS * 128 + b * 64 + r;
        *reinterpret_cast<uint4*>(to + row * 128) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
}

template <typename IO, int DK, bool BWD>
__global__ void __launch_bounds__(kThreads, PrepareSmem<IO, DK, BWD>::kBlocks) kla_delta_prepare_kernel(const DeltaArgs a, const DeltaGradArgs d,
                                                                    const Workspace w) {
  using L = PrepareSmem<IO, DK, BWD>;
  // TMEM holds two blocks of 256 columns: forward, U's product takes W's place where both would need more than 128
  constexpr bool AFTER = !BWD && DK == 128;
  constexpr int PARTS = L::PARTS, COLS = BWD && DK == 128 ? 256 : 128, NB = DK / 64, UC = AFTER ? 0 : DK;
  extern __shared__ __align__(1024) char sm[];  // the swizzle counts rows from 1024-byte boundaries
  __shared__ __align__(16) float G[C], E[C], be[C], nbG[C];  // decays from the start and to the end, β, −β G
  __shared__ uint64_t bar;
  __shared__ uint32_t slot;
  float2* logs = reinterpret_cast<float2*>(sm + L::A + 64 * 68 * 4);  // behind A, until T1 comes
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const Where at = where(a, blockIdx.x);
  const int DV = pad64(a.dv);
  const size_t krow = ((size_t)at.key * a.T + at.t0) * a.dk, vrow = ((size_t)at.bh * a.T + at.t0) * a.dv;
  TileLoad<IO, DK, kThreads> kl, ql;
  kl.fetch(reinterpret_cast<const IO*>(a.k) + krow, at.len, a.dk, 0, tid);
  if (BWD) ql.fetch(reinterpret_cast<const IO*>(a.q) + krow, at.len, a.dk, 0, tid);
  if (warp == 0) tmem_alloc(&slot, COLS);
  if (tid == 32) mbar_init(&bar, 1);
  if (warp == 2) {  // the gates: two tokens a lane, cumulative logs as sums of two floats
    float gh[2], gl[2], b[2];
    const size_t row = (size_t)at.bh * a.T + at.t0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const bool in = t < at.len;
      const float g = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.g)[row + t]) : 0.f;
      const float c = g < kMinLog ? kMinLog : g;
      gh[i] = c * kLog2e;  // in powers of two from here on
      gl[i] = fmaf(c, kLog2e, -gh[i]) + c * kLog2eLow;
      b[i] = in ? to_f32<IO>(reinterpret_cast<const IO*>(a.beta)[row + t]) : 0.f;
    }
    add_two(gh[1], gl[1], gh[0], gl[0]);
    float sh = gh[1], sl = gl[1];  // sums over the lanes up to this one
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const float yh = __shfl_up_sync(~0u, sh, m), yl = __shfl_up_sync(~0u, sl, m);
      if (lane >= m) add_two(sh, sl, yh, yl);
    }
    const float th = __shfl_sync(~0u, sh, 31), tl = __shfl_sync(~0u, sl, 31);
    float ph = __shfl_up_sync(~0u, sh, 1), pl = __shfl_up_sync(~0u, sl, 1);
    if (lane == 0) ph = pl = 0.f;
    float* out = w.gates + at.chunk * kGates;
    float low;
    const float whole = whole_decay(th, tl, low);
    if (lane == 31) out[5 * C] = low;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      float h = ph, l = pl;
      add_two(h, l, gh[i], gl[i]);
      const float g = t == C - 1 ? whole : exp2_of(h + l), e = exp2_of((th - h) + (tl - l));
      logs[t] = make_float2(h, l), G[t] = g, E[t] = e, be[t] = b[i], nbG[t] = -b[i] * g;
      out[t] = h, out[C + t] = l, out[2 * C + t] = g, out[3 * C + t] = e, out[4 * C + t] = b[i];
    }
  }
  kl.put(sm + L::K, tid);
  if (BWD) ql.put(sm + L::Q, tid);
  bool ok = true;
  uint32_t phase = 0;
  auto finish = [&] {  // the products issued so far
    mbar_wait(&bar, phase, ok);
    phase ^= 1;
    fence_after();
  };
  auto publish = [&] {  // this block's shared-memory writes and TMEM reads, before the next products
    fence_async();
    fence_before();
    __syncthreads();
    fence_after();
  };
  publish();
  const uint32_t tm = uniform(slot), base = uniform(smem_addr(sm));
  const Operand<PARTS, false> Kr{base + L::K, NB * kTileBytes, kTileBytes}, Qr{base + L::Q, NB * kTileBytes, kTileBytes};
  const Operand<PARTS, true> Kt{base + L::K, NB * kTileBytes, kTileBytes}, Qt{base + L::Q, NB * kTileBytes, kTileBytes};
  const Operand<PARTS, true> Vt{base + L::V, kTileBytes, kTileBytes};
  const Operand<3, false> T1r{base + L::T1, kTileBytes, kTileBytes}, T2r{base + L::T2, kTileBytes, kTileBytes};
  const Operand<3, false> Pr{base + L::P, kTileBytes, kTileBytes};
  const Operand<3, true> T1t{base + L::T1, kTileBytes, kTileBytes}, T2t{base + L::T2, kTileBytes, kTileBytes};
  if (warp == 0 && elect()) {
    mma<64, 64, DK>(tm, Kr, Kr);
    if (BWD) mma<64, 64, DK>(tm + 64, Qr, Kr);
    commit(&bar);
  }
  float* A = reinterpret_cast<float*>(sm + L::A);
  float* M = reinterpret_cast<float*>(sm + L::M);
  float* diag = reinterpret_cast<float*>(logs + C);
  const Lanes l(tid);
  const int quad = warp & 3, half = warp >> 2, r0 = l.r, c0 = l.c;
  const uint32_t rows = (uint32_t)(32 * quad) << 16;
  TileLoad<IO, 64, kThreads> vl;
  vl.fetch(reinterpret_cast<const IO*>(a.v) + vrow, at.len, a.dv, 0, tid);
  finish();
  float v[16];
  tmem_load(tm + rows + 32 * half, v);
  float D[16];
  decays(logs, l, D);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const int t = r0 + (i & 2) * 4, s = c0 + (i >> 2) * 8;
    const float x = s < t ? be[t] * D[i] * v[i] : 0.f, y = s + 1 < t ? be[t] * D[i + 1] * v[i + 1] : 0.f;
    store_two(A + t * 68 + s, x, y);
    if (half == quad >> 1 && i >> 3 == (quad & 1)) {  // of the 16 × 16 blocks on the diagonal, the columns too
      float* p = diag + (quad * 16 + (s & 15)) * kDiagRow + (t & 15);
      p[0] = x;
      p[kDiagRow] = y;
    }
  }
  if (BWD) {  // P, scaled
    Fragment p;
    tmem_load(tm + 64 + rows + 32 * half, p.v);
#pragma unroll
    for (int i = 0; i < 16; ++i) p.v[i] *= a.scale * D[i];
    p.put<3>(sm + L::P, kTileBytes, r0, c0);
  }
  __syncthreads();
  invert(A, M, diag, warp, lane);
  float m[2][8];  // two eights of M a thread
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = tid + j * kThreads;
    const float4* p = reinterpret_cast<const float4*>(M + (i >> 3) * 68 + (i & 7) * 8);
    const float4 x = p[0], y = p[1];
    m[j][0] = x.x, m[j][1] = x.y, m[j][2] = x.z, m[j][3] = x.w, m[j][4] = y.x, m[j][5] = y.y, m[j][6] = y.z, m[j][7] = y.w;
  }
  __syncthreads();
  // M times factors of its rows or columns, as parts: inputs are then operands as they are, exact in one part
  auto put_m = [&](int to, const float* by_column, const float* by_row) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = tid + j * kThreads, r = i >> 3, c = (i & 7) * 8;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = m[j][e];
      if (by_column) {
        const float4 f = *reinterpret_cast<const float4*>(by_column + c), g = *reinterpret_cast<const float4*>(by_column + c + 4);
        x[0] *= f.x, x[1] *= f.y, x[2] *= f.z, x[3] *= f.w, x[4] *= g.x, x[5] *= g.y, x[6] *= g.z, x[7] *= g.w;
      }
      if (by_row) {
        const float f = by_row[r];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= f;
      }
      store_eight<3>(sm + to, kTileBytes, r, c, x);
    }
  };
  put_m(L::T1, nbG, nullptr);
  if (BWD) put_m(L::T2, be, nullptr);
  vl.put(sm + L::V, tid);
  publish();
  if (warp == 0 && elect()) {
    mma<64, DK, 64>(tm, T1r, Kt);
    if (BWD) mma<64, 64, 64>(tm + DK, T2r, Vt);
    commit(&bar);
  }
  const int slices = DV / 64;
  if (slices > 1) vl.fetch(reinterpret_cast<const IO*>(a.v) + vrow, at.len, a.dv, 64, tid);
  finish();
  if (!BWD) {
    put_m(L::T2, be, nullptr);
    if (AFTER) drain_parts<NB>(tm, w.W + at.chunk * 3 * NB * kTileBytes, l);
    publish();
    if (warp == 0 && elect()) {
      mma<64, 64, 64>(tm + UC, T2r, Vt);
      commit(&bar);
    }
  }
  if (!AFTER) drain_parts<NB>(tm, w.W + at.chunk * 3 * NB * kTileBytes, l);
  if (!BWD) finish();
  drain<64, 1>(tm + UC, w.U + at.chunk * C * DV, l, tid);
  if (slices > 1) {
    vl.put(sm + L::V, tid);
    publish();
    if (warp == 0 && elect()) {
      mma<64, 64, 64>(tm + UC, T2r, Vt);
      commit(&bar);
    }
    finish();
    drain<64, 1>(tm + UC, w.U + at.chunk * C * DV + kBlock, l, tid);
  }
  if (BWD) {  // Mᵀ (E K) = (E M)ᵀ K, and Mᵀ Pᵀ O' = (P M)ᵀ O'
    const IO* go = reinterpret_cast<const IO*>(d.go);
    vl.fetch(go + (go ? vrow : 0), go ? at.len : 0, a.dv, 0, tid);
    put_m(L::T1, nullptr, E);
    put_m(L::T2, nullptr, nullptr);
    publish();
    if (warp == 0 && elect()) {
      mma<64, DK, 64>(tm, T1t, Kt);
      mma<64, 64, 64>(tm + DK, Pr, T2t);
      commit(&bar);
    }
    finish();
    drain_parts<NB>(tm, w.Wr + at.chunk * 3 * NB * kTileBytes, l);
    Fragment pm;
    tmem_load(tm + DK + rows + 32 * half, pm.v);
    pm.put<3>(sm + L::T1, kTileBytes, r0, c0);
    for (int sl = 0; sl < slices; ++sl) {
      if (sl) vl.fetch(go + (go ? vrow : 0), go ? at.len : 0, a.dv, sl * 64, tid);
      vl.put(sm + L::V, tid);
#pragma unroll
      for (int j = 0; j < vl.N; ++j) {  // G O'
        const int i = tid + j * kThreads, r = i >> 3;
        float x[8];
        vl.eight(j, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= a.scale * G[r];
        store_eight<3>(sm + L::T2, kTileBytes, r, (i & 7) * 8, x);
      }
      publish();
      if (warp == 0 && elect()) {
        mma<64, 64, 64>(tm, T1t, Vt);
        mma<DK, 64, 64>(tm + 64, Qt, T2t);
        commit(&bar);
      }
      finish();
      drain<64, 1>(tm, w.R + at.chunk * C * DV + sl * kBlock, l, tid);
      drain<DK, NB>(tm + 64, w.Z + at.chunk * DK * DV + sl * NB * kBlock, l, tid);
    }
  }
  fence_before();
  if (__syncthreads_or(!ok)) {  // a wait ran out: M (β V) and Mᵀ Pᵀ O' carry it into everything that comes of the chunk
    bool in = true;
    mbar_wait(&bar, phase ^ 1, in);
    const int dv = pad64(a.dv);
    const size_t block = (size_t)block_again() * C * dv;
    fill_nan(w.U + block, C, dv, dv, thread_again(), kThreads);
    if (BWD) fill_nan(w.R + block, C, dv, dv, thread_again(), kThreads);
  }
  if (warp == 0) tmem_free(tm, COLS);
}

// ---- the chain ----------------------------------------------------------------------
// X: the state (rev: its gradient), W: −M (β G K) (rev: Mᵀ (E K)). Per chunk:
//   forward:  U = M (β V) + W X,       X = G_end X + Kᵀ(E U)
//   reverse:  dR = Mᵀ Pᵀ O' + W X,     X = G_end X + Qᵀ(G O') − Kᵀ(β G dR)
// Eight warps walk the chunks, each with a quarter of the rows and half of the
// columns; others bring K (fp32: as parts, twice the warps) of the next chunk and
// start the copy of W, two chunks deep where shared memory holds them; one issues
// the products and the copies of M (β V) and the gates. The eight warps read no
// global memory on the way forward: loads ahead in registers cost them a stall
// of 700 of 5000 cycles a chunk, and W as fp32 to be made into parts here another
// 800 (d_k 128). Instructions are bound by their reads of shared memory (64 × 16
// by 16 × 32 takes 26 to 30 cycles): W's largest and middle parts are one operand
// of 128 rows, and with 32 columns X's and U's three parts lie side by side (65536 tokens, 16 heads of 128: 1900 -> 1730 us; with 64
// columns side by side took more, 125 us against 111 of the headline shape).
constexpr int kChainThreads = 256;
template <typename IO>
constexpr int kFeedThreads = 128 * (sizeof(IO) / 2);
template <typename IO>
constexpr int kChainBlock = kChainThreads + kFeedThreads<IO> + 32;

template <typename IO, int DK, int NV>
struct ChainSmem {
  static constexpr int KB = kParts<IO> * DK / 64 * kTileBytes, WB = 3 * DK / 64 * kTileBytes;
  static constexpr int STAGES = sizeof(IO) == 4 && DK == 128 ? 1 : 2;
  static constexpr int IN = NV * C * 4, GATES = (kGates - 2 * C) * 4;  // a chunk's M (β V), gates
  static constexpr int TILES = (3 * NV + 63) / 64;  // of X's and U's parts side by side
  static constexpr int K = 0, W = STAGES * KB, X = W + STAGES * WB, U = X + TILES * DK * 128, B = U + TILES * kTileBytes,
                       AHEAD = B + 2 * (IN + GATES) <= kMaxBytes ? 2 : 1, kBytes = B + AHEAD * (IN + GATES);
  static_assert(kBytes <= kMaxBytes, "");
};

// A wait of any warp ran out: U (rev: dR) of the block's columns and its last state say so. (Within the kernel it cost the
// long case 2%.)
template <typename IO, bool REV, int NV>
__device__ __noinline__ void mark_chain(const DeltaArgs& a, const DeltaGradArgs& d, const Workspace& w) {
  const int dv = pad64(a.dv), n = (a.T + C - 1) / C, c0 = (int)(block_again() % (dv / NV)) * NV;
  const size_t head = block_again() / (dv / NV);
  float* u = (REV ? w.R : w.U) + head * n * C * dv + c0 / 64 * kBlock + c0 % 64 * 16;  // (a half: threads 128 to 255 of 256)
  for (int i = 0; i < n; ++i, u += C * dv) fill_nan(u, 4, NV * 16, 1024, thread_again(), kChainBlock<IO>);
  float* const last = REV ? d.gstate0 : a.stateT;
  if (last && c0 < a.dv)
    fill_nan(last + head * a.dk * a.dv + c0, a.dk, min(NV, a.dv - c0), a.dv, thread_again(), kChainBlock<IO>);
}

// NV: columns of a block, 64 or 32.
template <typename IO, int DK, bool REV, int NV>
__device__ __forceinline__ void chain(const DeltaArgs& a, const DeltaGradArgs& d, const Workspace& w) {
  using L = ChainSmem<IO, DK, NV>;
  constexpr int PARTS = kParts<IO>, RB = DK / 64, STAGES = L::STAGES, FEED = kFeedThreads<IO>, J = NV / 16;
  extern __shared__ __align__(1024) char sm[];  // the swizzle counts rows from 1024-byte boundaries
  __shared__ uint64_t full[STAGES], empty[STAGES], done[2], loaded[L::AHEAD];
  __shared__ uint32_t slot;
  const int tid = threadIdx.x, warp = uniform(tid >> 5);
  const int DV = pad64(a.dv), N = (a.T + C - 1) / C;
  const long long bh = blockIdx.x / (DV / NV);
  const int part = (int)(blockIdx.x % (DV / NV)), col = part * NV / 64 * 64;  // the 64 columns it is in
  const long long key = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], FEED + 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&done[i], 1);
    for (int i = 0; i < L::AHEAD; ++i) mbar_init(&loaded[i], 1);
  }
  constexpr int COLS = 128;  // NV, or three times 32: X's product, then U's
  if (warp == 0) tmem_alloc(&slot, COLS);
  fence_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(slot), base = uniform(smem_addr(sm));
  bool ok = true;
  float* const blocks_u = (REV ? w.R : w.U) + (size_t)bh * N * C * DV + col * 64;
  if (warp == kChainBlock<IO> / 32 - 1) {  // the products, and a chunk's M (β V) (rev: Mᵀ Pᵀ O') and gates one or two chunks ahead
    auto bring = [&](int i) {
      if (i >= N) return;
      const int n = REV ? N - 1 - i : i, b = i % L::AHEAD;
      const float *u = blocks_u + (size_t)n * C * DV, *g = w.gates + ((size_t)bh * N + n) * kGates + 2 * C;
      const uint32_t to = base + L::B + b * (L::IN + L::GATES);
      mbar_expect(&loaded[b], L::IN + L::GATES);
      bulk_copy(to + L::IN, g, L::GATES, &loaded[b]);
      if (NV == 64) {
        bulk_copy(to, u, L::IN, &loaded[b]);
      } else {  // the half's threads of each eight of columns
        for (int j = 0; j < 4; ++j) bulk_copy(to + j * 2048, u + j * 1024 + (part & 1) * 512, 2048, &loaded[b]);
      }
    };
    if (elect())
      for (int i = 0; i < L::AHEAD; ++i) bring(i);
    __syncwarp();
    for (int i = 0; i < N; ++i) {
      const int b = STAGES == 2 ? i & 1 : 0;
      const uint32_t Wb = base + L::W + b * L::WB;
      const Operand<1, false> Whm{Wb, 0, 2 * kTileBytes}, Wl{Wb + RB * 2 * kTileBytes, 0, kTileBytes};
      const Operand<PARTS, true> Kt{base + L::K + b * L::KB, RB * kTileBytes, kTileBytes};
      auto Xp = [&](int p) { return Operand<1, true>{base + L::X + p * DK * 128, 0, DK * 128}; };
      mbar_wait(&full[b], STAGES == 2 ? (i >> 1) & 1 : i & 1, ok);
      bar_sync(1, kChainThreads + 32);
      fence_after();
      if (elect()) {
        if (NV == 32) {
          mma<128, 3 * NV, DK>(tm, Whm, Xp(0));
          mma<64, NV, DK>(tm + 2 * NV, Wl, Xp(0), true);
        } else {
          mma<128, NV, DK>(tm, Whm, Xp(2));
          mma<64, NV, DK>(tm, Wl, Xp(0), true);
          mma<128, NV, DK>(tm, Whm, Xp(1), true);
          mma<128, NV, DK>(tm, Whm, Xp(0), true);
        }
        commit(&done[0]);
      }
      __syncwarp();
      bar_sync(2, kChainThreads + 32);
      fence_after();
      if (elect()) {
        if (NV == 32) {
          const Operand<1, true> Us{base + L::U, 0, kTileBytes};
          auto Kp = [&](int p) { return Operand<1, true>{Kt.addr + p * Kt.part, 0, Kt.block}; };
          if (PARTS == 3) {
            mma<DK, 3 * NV, 64>(tm, Kp(1), Us);
            mma<DK, NV, 64>(tm, Kp(2), Us, true);
          }
          mma<DK, 3 * NV, 64>(tm, Kp(0), Us, PARTS == 3);
        } else {
          mma<DK, NV, 64>(tm, Kt, Operand<3, true>{base + L::U, kTileBytes, kTileBytes});
        }
        commit(&done[1]);
        commit(&empty[b]);
        bring(i + L::AHEAD);
      }
      __syncwarp();
    }
    bool in = true;  // no copy and no product's arrival is under way when the block ends, also where a wait ran out
    for (int i = max(N - STAGES, 0); i < N; ++i) {
      mbar_wait(&full[i % STAGES], i / STAGES & 1, in);
      mbar_wait(&empty[i % STAGES], i / STAGES & 1, in);
    }
    for (int i = max(N - L::AHEAD, 0); i < N; ++i) mbar_wait(&loaded[i % L::AHEAD], i / L::AHEAD & 1, in);
    ok &= in;
  } else if (warp >= kChainThreads / 32) {
    const int ft = tid - kChainThreads;
    const IO* k = reinterpret_cast<const IO*>(a.k) + (size_t)key * a.T * a.dk;
    const char* W = (REV ? w.Wr : w.W) + (size_t)bh * N * L::WB;
    for (int i = 0; i < N; ++i) {
      const int n = REV ? N - 1 - i : i, b = STAGES == 2 ? i & 1 : 0;
      const uint32_t before = STAGES == 2 ? ((i >> 1) - 1) & 1 : (i - 1) & 1;
      TileLoad<IO, DK, FEED> kl;  // comes in ahead of the wait for its place
      kl.fetch(k + (size_t)n * C * a.dk, min(C, a.T - n * C), a.dk, 0, ft);
      if (i >= STAGES) mbar_wait(&empty[b], before, ok);
      if (ft == 0) {
        mbar_expect(&full[b], L::WB);
        bulk_copy(base + L::W + b * L::WB, W + (size_t)n * L::WB, L::WB, &full[b]);
      }
      kl.put(sm + L::K + b * L::KB, ft);
      fence_async();
      mbar_arrive(&full[b]);
    }
  } else {
    // the warp's eights of columns: of the 64, the 32 of `half` from the j0-th on; in the block's tiles, from column lc on
    const int sub = warp >> 2, half = NV == 64 ? sub : part & 1, j0 = NV == 64 ? 0 : 2 * sub;
    const int vt = half * 128 + (tid & 127);  // the thread of 256 whose fragments these are
    const Lanes l(vt);
    const int lc = NV / 2 * sub + 2 * (l.lane & 3), gc = col + 32 * half + 8 * j0 + 2 * (l.lane & 3);
    const uint32_t rows = ((uint32_t)(32 * l.quad) << 16) + NV / 2 * sub;
    Columns<J> X[RB];
    const float* first = REV ? d.gstateT : a.state0;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int e = 0; e < 4 * J; e += 2) {
        const int r = block_row<DK>(l, rb) + (e & 2) * 4, c = gc + (e >> 2) * 8;
        float2 x = make_float2(0.f, 0.f);
        if (first && r < a.dk && c < a.dv) x = load_two(first + ((size_t)bh * a.dk + r) * a.dv + c);
        X[rb].v[e] = x.x, X[rb].v[e + 1] = x.y;
      }
    float* const blocks_x = (REV ? w.Z : w.S) + (size_t)bh * N * DK * DV + col * DK;
    auto load_product = [&](uint32_t from, float (&v)[4 * J]) {
      if constexpr (NV == 32) tmem_load_sum(from, NV, v);
      else tmem_load(from, v);
    };
    auto load_both = [&](uint32_t from, float (&x)[4 * J], float (&y)[4 * J]) {
      if constexpr (NV == 32) tmem_load_both_sum(from, NV, x, y);
      else tmem_load_both(from, x, y);
    };
    // three parts, NV columns each
    auto put = [&](const Columns<J>& f, int to, int tile, int r0) {
#pragma unroll
      for (int e = 0; e < 4 * J; e += 2) {
        const int r = r0 + (e & 2) * 4, c = lc + (e >> 2) * 8;
        char* p = sm + to + r * 128 + ((((c >> 3) ^ r) & 7) << 4) + (c & 7) * 2;
        float x = f.v[e], y = f.v[e + 1];
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          const uint32_t v = bf16_pair(x, y);
          if (NV == 64) *reinterpret_cast<uint32_t*>(p + m * tile) = v;
          else *reinterpret_cast<uint32_t*>(m == 1 ? reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(p) ^ 64) : p + (m >> 1) * tile) = v;
          x -= __uint_as_float(v << 16);
          y -= __uint_as_float(v & 0xffff0000u);
        }
      }
    };
    for (int i = 0; i < N; ++i) {
      const int n = REV ? N - 1 - i : i;
      const uint32_t parity = i & 1;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) put(X[rb], L::X, DK * 128, block_row<DK>(l, rb));
      fence_async();
      fence_before();
      bar_arrive(1, kChainThreads + 32);
      // while the product runs: the state goes out; in reverse its slot first gives up Qᵀ(G O')
      Columns<J> F[REV ? RB : 1];
      float* Xout = blocks_x + (size_t)n * DK * DV;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        if (REV) F[rb].load(Xout + rb * kBlock, vt, j0);
        else X[rb].store(Xout + rb * kBlock, vt, j0);
      }
      const char* const brought = sm + L::B + i % L::AHEAD * (L::IN + L::GATES);
      const float* const gates = reinterpret_cast<const float*>(brought + L::IN);
      Columns<J> B, u, s;
      mbar_wait(&loaded[i % L::AHEAD], i / L::AHEAD & 1, ok);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float4 x = reinterpret_cast<const float4*>(brought)[(j0 + j) * (NV * 4) + (NV == 64 ? vt : vt & 127)];
        B.v[4 * j] = x.x, B.v[4 * j + 1] = x.y, B.v[4 * j + 2] = x.z, B.v[4 * j + 3] = x.w;
      }
      const float gend = gates[C - 1], glow = gates[3 * C];
      float g[2];  // −β G, or E
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const float* q = gates + l.r + 8 * o;
        g[o] = REV ? -q[2 * C] * q[0] : q[C];
      }
      mbar_wait(&done[0], parity, ok);
      fence_after();
      load_both(tm + rows, u.v, s.v);
#pragma unroll
      for (int e = 0; e < 4 * J; ++e) u.v[e] += s.v[e] + B.v[e];
#pragma unroll
      for (int e = 0; e < 4 * J; ++e) s.v[e] = g[(e & 2) >> 1] * u.v[e];
      put(s, L::U, kTileBytes, l.r);
      fence_async();
      fence_before();
      bar_arrive(2, kChainThreads + 32);
      u.store(blocks_u + (size_t)n * C * DV, vt, j0);
      if (REV) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) X[rb].store(Xout + rb * kBlock, vt, j0);
      }
      mbar_wait(&done[1], parity, ok);
      fence_after();
      Columns<J> more[RB];
      if constexpr (RB == 2) load_both(tm + rows, more[0].v, more[1].v);
      else load_product(tm + rows, more[0].v);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int e = 0; e < 4 * J; ++e)
          X[rb].v[e] = fmaf(gend, X[rb].v[e], fmaf(glow, X[rb].v[e], REV ? more[rb].v[e] + F[REV ? rb : 0].v[e] : more[rb].v[e]));
    }
    float* const last = REV ? d.gstate0 : a.stateT;
    if (last) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int e = 0; e < 4 * J; e += 2) {
          const int r = block_row<DK>(l, rb) + (e & 2) * 4, c = gc + (e >> 2) * 8;
          if (r < a.dk && c < a.dv)
            store_two(last + ((size_t)bh * a.dk + r) * a.dv + c, X[rb].v[e], X[rb].v[e + 1]);
        }
    }
  }
  fence_before();
  if (__syncthreads_or(!ok)) mark_chain<IO, REV, NV>(a, d, w);
  if (warp == 0) tmem_free(tm, COLS);
}

// BOTH: a second row of blocks walks the reverse chain, which needs nothing of the forward one.
template <typename IO, int DK, bool BOTH, int NV>
__global__ void __launch_bounds__(kChainBlock<IO>)
    kla_delta_chain_kernel(const DeltaArgs a, const DeltaGradArgs d, const Workspace w) {
  if (BOTH && blockIdx.y == 1) chain<IO, DK, true, NV>(a, d, w);
  else chain<IO, DK, false, NV>(a, d, w);
}

// ---- the output ----------------------------------------------------------------------
template <typename IO, int DK>
struct OutputSmem {
  static constexpr int IN = kParts<IO> * DK / 64 * kTileBytes, PN = 3;  // parts of what is not an input
  // U and P come when the products with K, Q and S are done, in their places
  static constexpr int K = 0, Q = IN, S = 2 * IN > PN * kTileBytes ? 2 * IN : PN * kTileBytes, U = K, P = S,
                       kBytes = S + PN * DK * 128, kFit = 228 * 1024 / (kBytes + 2048), kBlocks = kFit < 4 ? kFit : 4;  // of an SM
  static_assert(kBytes <= kMaxBytes, "");
};

template <typename IO, int DK>
__global__ void __launch_bounds__(kThreads, OutputSmem<IO, DK>::kBlocks)
    kla_delta_output_kernel(const DeltaArgs a, const Workspace w, unsigned ahead) {
  using L = OutputSmem<IO, DK>;
  constexpr int PARTS = kParts<IO>, PN = L::PN;
  extern __shared__ __align__(1024) char sm[];  // the swizzle counts rows from 1024-byte boundaries
  __shared__ __align__(16) float2 logs[C];
  __shared__ float G[C];
  __shared__ uint64_t bar;
  __shared__ uint32_t slot;
  const int tid = threadIdx.x, warp = uniform(tid >> 5);
  const int DV = pad64(a.dv);
  const Where at = where(a, blockIdx.x / (DV / 64));
  const int col = (int)(blockIdx.x % (DV / 64)) * 64;
  if (warp == 0) tmem_alloc(&slot, 128);
  if (tid == 32) mbar_init(&bar, 1);
  const size_t row = (size_t)at.key * a.T + at.t0;
  TileLoad<IO, DK, kThreads> kl, ql;
  const Lanes l(tid);
  Fragment xl[DK / 64], ul;
  kl.fetch(reinterpret_cast<const IO*>(a.k) + row * a.dk, at.len, a.dk, 0, tid);
  ql.fetch(reinterpret_cast<const IO*>(a.q) + row * a.dk, at.len, a.dk, 0, tid);
#pragma unroll
  for (int rb = 0; rb < DK / 64; ++rb) xl[rb].load(w.S + at.chunk * DK * DV + col * DK + rb * kBlock, tid);
  ul.load(w.U + at.chunk * C * DV + col * 64, tid);
  // For the block that follows on this SM, into L2, where fewer than four blocks cover for each other (65536 tokens,
  // 16 heads of 128, with three blocks an SM: 562 -> 527 us, with the two of now 636; d_k 64 in bf16, whose inputs are
  // half as many bytes: 116 -> 120).
  const unsigned after = blockIdx.x + ahead;
  if (L::kBlocks < 4 && tid == 128 && col == 0 && after < gridDim.x) {
    const Where next = where(a, after / (DV / 64));
    prefetch_rows<IO>(a.k, next.key, next, a.T, a.dk);
    prefetch_rows<IO>(a.q, next.key, next, a.T, a.dk);
    prefetch(w.U + next.chunk * C * DV, C * DV * 4);
    prefetch(w.S + next.chunk * DK * DV, DK * DV * 4);
  }
  if (tid < C) {
    const float* g = w.gates + at.chunk * kGates + tid;
    logs[tid] = make_float2(g[0], g[C]), G[tid] = g[2 * C];
  }
  kl.put(sm + L::K, tid);
  ql.put(sm + L::Q, tid);
#pragma unroll
  for (int rb = 0; rb < DK / 64; ++rb) xl[rb].put<PN>(sm + L::S, DK * 128, block_row<DK>(l, rb), l.c);
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
  const int half = l.half;
  const uint32_t rows = (uint32_t)(32 * l.quad) << 16;
  mbar_wait(&bar, 0, ok);
  fence_after();
  ul.put<PN>(sm + L::U, kTileBytes, l.r, l.c);
  float v[16], y[16];
  tmem_load(tm + rows + 32 * half, v);
  {
    Fragment p;
    decays(logs, l, p.v);
#pragma unroll
    for (int i = 0; i < 16; ++i) p.v[i] *= v[i];
    p.put<PN>(sm + L::P, kTileBytes, l.r, l.c);
  }
  tmem_load(tm + 64 + rows + 32 * half, y);
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
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = a.scale * fmaf(G[l.r + (i & 2) * 4], y[i], v[i]);
  store_rows(reinterpret_cast<IO*>(a.o) + ((size_t)at.bh * a.T + at.t0) * a.dv, l, col, at.len, a.dv, v);
  fence_before();
  if (__syncthreads_or(!ok)) {  // a wait ran out
    bool in = true;
    mbar_wait(&bar, 1, in);
    const int slices = pad64(a.dv) / 64, c0 = (int)(block_again() % slices) * 64;
    const Where rows = where(a, block_again() / slices);
    fill_nan(reinterpret_cast<IO*>(a.o) + ((size_t)rows.bh * a.T + rows.t0) * a.dv + c0, rows.len, min(64, a.dv - c0), a.dv,
             thread_again(), kThreads);
  }
  if (warp == 0) tmem_free(tm, 128);
}

unsigned chunks(const DeltaArgs& a) { return (unsigned)((long long)a.B * a.H * ((a.T + C - 1) / C)); }

template <typename IO, int DK>
cudaError_t prepare_dk(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, cudaStream_t s) {
  if (d)
    return run(kla_delta_prepare_kernel<IO, DK, true>, PrepareSmem<IO, DK, true>::kBytes, chunks(a), kThreads, s, a, *d, w);
  return run(kla_delta_prepare_kernel<IO, DK, false>, PrepareSmem<IO, DK, false>::kBytes, chunks(a), kThreads, s, a,
             DeltaGradArgs{}, w);
}
template <typename IO, int DK, int NV>
cudaError_t chain_nv(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, cudaStream_t s) {
  const unsigned blocks = (unsigned)((long long)a.B * a.H * (pad64(a.dv) / NV));
  const int smem = ChainSmem<IO, DK, NV>::kBytes;
  if (d) return run(kla_delta_chain_kernel<IO, DK, true, NV>, smem, dim3(blocks, 2), kChainBlock<IO>, s, a, *d, w);
  return run(kla_delta_chain_kernel<IO, DK, false, NV>, smem, blocks, kChainBlock<IO>, s, a, DeltaGradArgs{}, w);
}
template <typename IO, int DK>
cudaError_t chain_dk(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, int num_sms, cudaStream_t s) {
  // A chunk's latency bounds the chain, and blocks of 32 columns take less of it (64 tokens, d 128: 1.5 us against
  // 2.5; d 64: 1.3 against 1.7), as long as every block has an SM; with more heads than that W and K would be brought
  // in twice (128 heads, d 64, 4096 tokens: 162 us against 114; 64 heads, d 128: 196 against 167).
  if ((long long)a.B * a.H * (pad64(a.dv) / 32) * (d ? 2 : 1) <= num_sms) return chain_nv<IO, DK, 32>(a, d, w, s);
  return chain_nv<IO, DK, 64>(a, d, w, s);
}
template <typename IO, int DK>
cudaError_t output_dk(const DeltaArgs& a, const Workspace& w, int num_sms, cudaStream_t s) {
  using L = OutputSmem<IO, DK>;
  const unsigned slices = pad64(a.dv) / 64;
  return run(kla_delta_output_kernel<IO, DK>, L::kBytes, chunks(a) * slices, kThreads, s, a, w,
             (num_sms * L::kBlocks + slices - 1) / slices * slices);
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
  w.gates = take(n * kGates);
  const size_t tiles = n * C * DK * 3 / 2;  // floats of three parts
  w.W = reinterpret_cast<char*>(take(tiles));
  w.S = take(n * DK * DV);
  w.U = take(n * C * DV);
  if (backward) {
    w.Wr = reinterpret_cast<char*>(take(tiles));
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

cudaError_t launch_chain(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, int num_sms, cudaStream_t s) {
  const bool wide = pad64(a.dk) == 128;
  if (a.io == IO_BF16)
    return wide ? chain_dk<__nv_bfloat16, 128>(a, d, w, num_sms, s) : chain_dk<__nv_bfloat16, 64>(a, d, w, num_sms, s);
  return wide ? chain_dk<float, 128>(a, d, w, num_sms, s) : chain_dk<float, 64>(a, d, w, num_sms, s);
}

}  // namespace delta

// Chunks, or token by token (kla_delta.cu)? The estimated times of both, in
// microseconds, fitted to bf16 calls, launches included, on a GB300. Token by
// token: 0.19 us a token (d_k 64; 0.16 and 0.23 for 16 and 128), or 3.3e6 elements
// a microsecond where heads are many (heads of few rows count as 40 rows). Chunks:
// 20 us of launches and first waits and, by latency, 1.7 us a chunk (23 and 2.1 for
// d_k 128), or by work, 0.052 us a chunk and head (0.116). Measured in a captured
// graph, one by one / chunks, in bf16 and in fp32, whose chunks take longer: 8
// heads of 64 × 64, 64 tokens 14 / 15 and 13 / 18 us, 128 tokens 26 / 17 and
// 24 / 19; 128 such heads, 64 tokens 18 / 17 and 17 / 19, 128 tokens 33 / 23 and
// 31 / 27; 1024, 32 tokens 49 / 74 and 49 / 90, 64 tokens 91 / 77 and 92 / 100 (where
// chunks are taken); 1024 heads of 16 × 16, 512 tokens 136 / 387 and 137 / 480; 128
// heads of 128 × 128, 64 tokens 54 / 28 and 54 / 40. Past 512 tokens always chunks:
// one by one, a rounding per token adds up (1e-6 of the state after a thousand).
bool delta_chunked(int B, int H, int T, int dk, int dv) {
  if (T > 512) return true;
  const double heads = (double)B * H, chunks = (T + delta::C - 1) / delta::C;
  const bool wide = delta::pad64(dk) == 128;
  const double tokens = 4.5 + T * std::hypot(0.145 + 0.0007 * dk, heads * dv * std::max(dk, 40) / 3.3e6);
  const double work = (wide ? 0.116 : 0.052) * heads * chunks * (delta::pad64(dv) / (wide ? 128.0 : 64.0));
  return std::max((wide ? 23.0 : 20.0) + (wide ? 2.1 : 1.7) * chunks, 15.0 + work) < tokens;
}

size_t delta_forward_bytes(int B, int Hk, int H, int T, int dk, int dv) {
  size_t n = 0;
  if (delta_chunked(B, H, T, dk, dv)) delta::workspace(nullptr, B, Hk, H, T, dk, dv, false, &n);
  return n;
}

cudaError_t launch_delta_forward(const DeltaArgs& a, int num_sms, void* workspace, cudaStream_t s) {
  if (!delta_chunked(a.B, a.H, a.T, a.dk, a.dv)) return launch_delta_recurrent(a, s);
  size_t n = 0;
  const delta::Workspace w = delta::workspace(workspace, a.B, a.Hk, a.H, a.T, a.dk, a.dv, false, &n);
  cudaError_t e = delta::launch_prepare(a, nullptr, w, s);
  if (e == cudaSuccess) e = delta::launch_chain(a, nullptr, w, num_sms, s);
  if (e != cudaSuccess) return e;
  const bool wide = delta::pad64(a.dk) == 128;
  if (a.io == IO_BF16)
    return wide ? delta::output_dk<__nv_bfloat16, 128>(a, w, num_sms, s) : delta::output_dk<__nv_bfloat16, 64>(a, w, num_sms, s);
  return wide ? delta::output_dk<float, 128>(a, w, num_sms, s) : delta::output_dk<float, 64>(a, w, num_sms, s);
}

}  // namespace kla
