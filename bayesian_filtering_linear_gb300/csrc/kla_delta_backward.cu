// Gradients of the gated delta rule (sm_103a), in chunks of 64 tokens on the
// tensor cores. With the notation of kla_delta_chunk.cu, P = tril(D_ts q_t·k_s),
// O' = scale dL/dO and Z = dL/dS' for the state after the chunk:
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
// Four steps: `prepare` makes, ahead of the chain, Mᵀ (E K), Mᵀ Pᵀ O' and Qᵀ(G O');
// the chain runs forward for S and U, and beside it from the end for Z and dR;
// then a block per chunk and head makes everything else here. Gradients of q and
// k that several value heads share are summed from per-head fp32 parts in a
// fixed order. At 8 × 16 heads of 64 × 64 and 4096 tokens in bf16: prepare 350 us,
// the chains 234 (1.45 GB, 6.2 TB/s), gradients 378: two blocks an SM, bound by
// their steps' latencies, so that a block's loads start together at its start, and
// the inputs of the block that follows on the SM are sent into L2 (425 -> 358 with
// operands of two parts, 402 with three, 378 with the number of slices a constant).
// Sixteen warps instead of eight leave 64 registers a thread: 473 us.
#include "kla_delta_chunk.cuh"

namespace kla {
namespace delta {

namespace {

template <typename IO, int DK>
struct GradSmem {
  static constexpr int PN = 3;  // parts of what is not an input
  static constexpr int IN = kParts<IO> * DK / 64 * kTileBytes, ROWS = PN * kTileBytes;
  static constexpr int K = 0, Q = IN, O = 2 * IN, U = O + kParts<IO> * kTileBytes, R = U + ROWS, S = R + ROWS,
                       kStage = S + PN * DK * 128;
  // once the products with S and Z are done: (dP P + dA A), then the masked dP, dA and β dA
  static constexpr int W = O, dP = O, dA = dP + ROWS, bA = dA + ROWS, kEnd = bA + ROWS;
  static constexpr int kBytes = kStage > kEnd ? kStage : kEnd;
  static constexpr int kBlocks = DK == 64 && kBytes <= 108 * 1024 ? 2 : 1;  // of an SM
  // Two slices of 64 columns of V add to the same sums. Where TMEM has room each has accumulators of its own, added in
  // registers: what a slice's small products add to the other's whole sums is cut off too often (24 times).
  static constexpr int kSet = kBlocks == 1 && DK == 64 ? 256 : 0;
  // fp32 with d_k 128 has no room: the first slice's sums wait in registers (440 -> 533 us at 2 × 16 heads of 128 × 128
  // and 4096 tokens, for errors of 2e-7 to 3e-7 instead of 7e-7). bf16 outputs are rounded by far more.
  static constexpr bool kKeep = sizeof(IO) == 4 && DK == 128;
  static_assert(W + 64 * 65 * 4 <= kBytes && kBytes <= kMaxBytes, "");
};

// Per row of a fragment: the sum over its four lanes; lane 0 of the four keeps it.
__device__ __forceinline__ float row4(float x) {
  x += __shfl_xor_sync(~0u, x, 1);
  return x + __shfl_xor_sync(~0u, x, 2);
}

// Columns c and c + 1 of row r of a tile of parts.
template <int PARTS>
__device__ __forceinline__ float2 tile_two(const char* tile, int part, int r, int c) {
  const char* p = tile + (c >> 6) * kTileBytes + r * 128 + ((((c >> 3) ^ r) & 7) << 4) + (c & 7) * 2;
  float2 x = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = PARTS - 1; i >= 0; --i) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p + i * part);
    x.x += __uint_as_float(u << 16);
    x.y += __uint_as_float(u & 0xffff0000u);
  }
  return x;
}

// SLICES: of 64 columns of V (padded).
template <typename IO, int DK, int SLICES>
__global__ void __launch_bounds__(kThreads, GradSmem<IO, DK>::kBlocks) kla_delta_grad_kernel(const DeltaArgs a, const DeltaGradArgs d,
                                                                 const Workspace w, unsigned ahead) {
  using L = GradSmem<IO, DK>;
  constexpr int PARTS = kParts<IO>, PN = L::PN, NB = DK / 64;  // NB: 32-column blocks of a thread in DK columns
  constexpr bool KEEP = L::kKeep && SLICES == 2;
  constexpr int SET = L::kSet, COLS = DK == 64 && !SET ? 256 : 512, SH = 3 * DK;  // TMEM: dQ, X, Y of DK columns, then 64 shared
  extern __shared__ __align__(1024) char sm[];  // the swizzle counts rows from 1024-byte boundaries
  __shared__ __align__(16) float2 logs[C];
  __shared__ float G[C], E[C], be[C], rv[2][C], before[C], from[2][C], to[2][C], kx[2][C], zs[8];
  __shared__ uint64_t bar;
  __shared__ uint32_t slot;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  constexpr int DV = 64 * SLICES, slices = SLICES;
  const Where at = where(a, blockIdx.x);
  const size_t krow = (size_t)at.key * a.T + at.t0, vrow = (size_t)at.bh * a.T + at.t0;
  const IO* k = reinterpret_cast<const IO*>(a.k) + krow * a.dk;
  const IO* q = reinterpret_cast<const IO*>(a.q) + krow * a.dk;
  const IO* v_in = reinterpret_cast<const IO*>(a.v) + vrow * a.dv;
  const IO* go = d.go ? reinterpret_cast<const IO*>(d.go) + vrow * a.dv : nullptr;
  const float* Sw = w.S + at.chunk * DK * DV;
  const float* Zw = w.Z + at.chunk * DK * DV;
  const float* Uw = w.U + at.chunk * C * DV;
  const float* Rw = w.R + at.chunk * C * DV;
  if (warp == 0) tmem_alloc(&slot, COLS);
  if (tid == 32) mbar_init(&bar, 1);
  if (tid < C) {
    const float* g = w.gates + at.chunk * kGates + tid;
    logs[tid] = make_float2(g[0], g[C]), G[tid] = g[2 * C], E[tid] = g[3 * C], be[tid] = g[4 * C];
  }
  const Lanes l(tid);
  // a slice's inputs, whose loads run ahead of the waits for the products before them
  TileLoad<IO, 64, kThreads> ol;
  Fragment ul, rl, xl[NB], zl[NB], vl;
  auto bring = [&](int sl) {
    rl.load(Rw + sl * kBlock, tid);
    ol.fetch(go ? go : v_in, go ? at.len : 0, a.dv, sl * 64, tid);
    ul.load(Uw + sl * kBlock, tid);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) xl[nb].load(Sw + (sl * NB + nb) * kBlock, tid);
    load_rows(v_in, l, sl * 64, at.len, a.dv, vl.v);
  };
  auto bring_z = [&](int sl) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) zl[nb].load(Zw + (sl * NB + nb) * kBlock, tid);
  };
  {
    TileLoad<IO, DK, kThreads> kl, ql;
    kl.fetch(k, at.len, a.dk, 0, tid);
    ql.fetch(q, at.len, a.dk, 0, tid);
    bring(0);
    if (tid == 128 && blockIdx.x + ahead < gridDim.x) {  // for the block that follows on this SM, into L2 (383 -> 358 us)
      const Where next = where(a, blockIdx.x + ahead);
      const int in = C * DV * 4, state = DK * DV * 4;
      prefetch_rows<IO>(a.k, next.key, next, a.T, a.dk);
      prefetch_rows<IO>(a.q, next.key, next, a.T, a.dk);
      prefetch_rows<IO>(a.v, next.bh, next, a.T, a.dv);
      if (d.go) prefetch_rows<IO>(d.go, next.bh, next, a.T, a.dv);
      prefetch(w.U + next.chunk * C * DV, in);
      prefetch(w.R + next.chunk * C * DV, in);
      prefetch(w.S + next.chunk * DK * DV, state);
      prefetch(w.Z + next.chunk * DK * DV, state);
    }
    kl.put(sm + L::K, tid);
    ql.put(sm + L::Q, tid);
  }
  fence_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(slot), base = uniform(smem_addr(sm));
  const Operand<PARTS, false> Kr{base + L::K, NB * kTileBytes, kTileBytes}, Qr{base + L::Q, NB * kTileBytes, kTileBytes};
  const Operand<PARTS, true> Kt{base + L::K, NB * kTileBytes, kTileBytes}, Qt{base + L::Q, NB * kTileBytes, kTileBytes};
  const Operand<PARTS, false> Or{base + L::O, kTileBytes, kTileBytes};
  const Operand<PN, false> Ur{base + L::U, kTileBytes, kTileBytes}, Rr{base + L::R, kTileBytes, kTileBytes};
  const Operand<PN, false> Sr{base + L::S, DK * 128, DK * 128};
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
  const int quad = warp & 3, half = warp >> 2, r0 = l.r, c0 = l.c;
  const uint32_t rows = (uint32_t)(32 * quad) << 16;
  // entries (t, s), (t, s + 1) of a 64 × 64 fragment at index e of 16
  auto row_of = [&](int e) { return r0 + (e & 2) * 4; };
  auto col_of = [&](int e) { return c0 + (e >> 2) * 8; };

  if (warp == 0 && elect()) {  // A and P before their decays, where dQ and X come later
    mma<64, 64, DK>(tm, Kr, Kr);
    mma<64, 64, DK>(tm + 64, Qr, Kr);
    commit(&bar);
  }
  float kk[16], qk[16], v[16], rdot[2] = {};
  finish();
  tmem_load(tm + rows + 32 * half, kk);
  tmem_load(tm + 64 + rows + 32 * half, qk);
  // products with U, S: dP, dA before masks, dQ = O' Sᵀ, X = dR Sᵀ (dP and dA wait in the shared columns and in Y's)
  float kept[KEEP ? 2 + 2 * NB : 1][16] = {};
  for (int sl = 0; sl < slices; ++sl) {
    if (sl) finish();
    if (KEEP && sl) {
      tmem_load(tm + SH + rows + 32 * half, kept[0]);
      tmem_load(tm + 2 * DK + rows + 32 * half, kept[KEEP ? 1 : 0]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          tmem_load(tm + m * DK + rows + NB * 32 * half + 32 * nb, kept[KEEP ? 2 + 2 * nb + m : 0]);
    }
    ol.put(sm + L::O, tid);
    ul.put<PN>(sm + L::U, kTileBytes, l.r, l.c);
    rl.put<PN>(sm + L::R, kTileBytes, l.r, l.c);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) xl[nb].put<PN>(sm + L::S, DK * 128, block_row<DK>(l, nb), l.c);
    publish();
    if (warp == 0 && elect()) {
      const uint32_t to = tm + sl * SET;
      const bool more = !SET && !KEEP && sl > 0;
      mma<64, 64, 64>(to + SH, Or, Ur, more);
      mma<64, 64, 64>(to + 2 * DK, Rr, Ur, more);
      mma<64, DK, 64>(to, Or, Sr, more);
      mma<64, DK, 64>(to + DK, Rr, Sr, more);
      commit(&bar);
    }
    // while that runs, what comes of dR alone
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int o = (e & 2) >> 1;
      rdot[o] = fmaf(rl.v[e], vl.v[e], rdot[o]);
      rl.v[e] *= be[r0 + 8 * o];
    }
    store_rows(reinterpret_cast<IO*>(d.gv) + vrow * a.dv, l, sl * 64, at.len, a.dv, rl.v);
    if (sl + 1 < slices) bring(sl + 1);
    else bring_z(sl);
  }
  auto load_sum = [&](uint32_t from, float (&x)[16]) {  // of both slices
    tmem_load(from, x);
    if (SET && slices > 1) {
      float y[16];
      tmem_load(from + SET, y);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] += y[e];
    }
  };
  float gp[16], ga[16];
  finish();
  load_sum(tm + SH + rows + 32 * half, gp);
  load_sum(tm + 2 * DK + rows + 32 * half, ga);
  if (KEEP)
#pragma unroll
    for (int e = 0; e < 16; ++e) gp[e] += kept[0][e], ga[e] += kept[KEEP ? 1 : 0][e];
  fence_before();
  // Y = U Zᵀ, and <Z, S>, from the last slice on, whose U and S are at hand
  float z = 0.f, kept_y[KEEP ? NB : 1][16] = {};
  for (int sl = slices - 1; sl >= 0; --sl) {
    if (sl + 1 < slices) {
      finish();
      if (KEEP)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) tmem_load(tm + 2 * DK + rows + NB * 32 * half + 32 * nb, kept_y[KEEP ? nb : 0]);
      ul.put<PN>(sm + L::U, kTileBytes, l.r, l.c);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      zl[nb].put<PN>(sm + L::S, DK * 128, block_row<DK>(l, nb), l.c);
#pragma unroll
      for (int e = 0; e < 16; ++e) z = fmaf(xl[nb].v[e], zl[nb].v[e], z);
    }
    publish();
    if (warp == 0 && elect()) {
      mma<64, DK, 64>(tm + sl * SET + 2 * DK, Ur, Sr, !SET && !KEEP && sl + 1 < slices);
      commit(&bar);
    }
    if (sl) {
      ul.load(Uw + (sl - 1) * kBlock, tid);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) xl[nb].load(Sw + ((sl - 1) * NB + nb) * kBlock, tid);
      bring_z(sl - 1);
    }
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) z += __shfl_xor_sync(~0u, z, m);
  if (lane == 0) zs[warp] = z;
  // masks and decays while that runs; (dP P + dA A) goes through registers until the tiles are free
  float ww[16];
  decays(logs, l, ww);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int t = row_of(e), s = col_of(e) + (e & 1);
    const float p = a.scale * ww[e] * gp[e], x = s < t ? -ww[e] * ga[e] : 0.f;
    ww[e] = s < t ? fmaf(p, qk[e], be[t] * x * kk[e]) : 0.f;
    gp[e] = p, ga[e] = x;
  }
  finish();
  // dQ, X, Y so far into registers, with their decays and their products with q and k
  float acc[3][NB][16], aq[2] = {}, ax[2] = {}, ay[2] = {};
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int cb = NB * 32 * half + 32 * nb;
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      load_sum(tm + m * DK + rows + cb, acc[m][nb]);
      if (KEEP)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[m][nb][e] += m < 2 ? kept[KEEP ? 2 + 2 * nb + m : 0][e] : kept_y[KEEP ? nb : 0][e];
    }
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const int t = row_of(e), o = (e & 2) >> 1, c = cb + 2 * (lane & 3) + (e >> 2) * 8;
      const float2 kv = tile_two<PARTS>(sm + L::K, NB * kTileBytes, t, c), qv = tile_two<PARTS>(sm + L::Q, NB * kTileBytes, t, c);
      const float f[3] = {a.scale * G[t], -G[t], E[t]};
#pragma unroll
      for (int m = 0; m < 3; ++m) acc[m][nb][e] *= f[m], acc[m][nb][e + 1] *= f[m];
      aq[o] += acc[0][nb][e] * qv.x + acc[0][nb][e + 1] * qv.y;
      ax[o] += acc[1][nb][e] * kv.x + acc[1][nb][e + 1] * kv.y;
      ay[o] += acc[2][nb][e] * kv.x + acc[2][nb][e + 1] * kv.y;
    }
  }
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int t = r0 + 8 * o;
    const float f = row4(fmaf(be[t], ax[o], aq[o])), x = row4(ay[o]);
    const float y = row4(rdot[o]);
    if ((lane & 3) == 0) from[half][t] = f, to[half][t] = x, rv[half][t] = y;
  }
  float* W = reinterpret_cast<float*>(sm + L::W);
#pragma unroll
  for (int e = 0; e < 16; ++e) W[row_of(e) * 65 + col_of(e) + (e & 1)] = ww[e];
  fence_before();
  __syncthreads();
  {  // W[t][s] becomes the sum of its row before s, four lanes a row; then before[s] the sum of column s from row s on
    const int r = tid >> 2, seg = tid & 3, s0 = seg * 16;
    float x[16], sum = 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      x[s] = W[r * 65 + s0 + s];
      sum += x[s];
    }
    float run = 0.f;
#pragma unroll
    for (int m = 1; m < 4; ++m) {
      const float y = __shfl_up_sync(~0u, sum, m);
      if (seg >= m) run += y;
    }
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      W[r * 65 + s0 + s] = run;
      run += x[s];
    }
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int t = s0; t < s0 + 16; ++t)
      if (t >= r) sum += W[t * 65 + r];
    sum = row4(sum);
    if (seg == 0) before[r] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const int t = row_of(e), s = col_of(e);
    store_pair<PN>(sm + L::dP, kTileBytes, t, s, gp[e], gp[e + 1]);
    store_pair<PN>(sm + L::dA, kTileBytes, t, s, ga[e], ga[e + 1]);
    store_pair<PN>(sm + L::bA, kTileBytes, t, s, be[t] * ga[e], be[t] * ga[e + 1]);
  }
  publish();
  if (warp == 0 && elect()) {
    const Operand<PN, false> P{base + L::dP, kTileBytes, kTileBytes}, A{base + L::dA, kTileBytes, kTileBytes};
    const Operand<PN, true> Pt{base + L::dP, kTileBytes, kTileBytes}, At{base + L::bA, kTileBytes, kTileBytes};
    mma<64, DK, 64>(tm, P, Kt);
    mma<64, DK, 64>(tm + DK, A, Kt);
    mma_sum<64, DK, 64>(tm + 2 * DK, Pt, Qt, At, Kt);
    commit(&bar);
  }
  finish();
  if (!ok) {  // the last of an even number of products may still run
    bool in = true;
    mbar_wait(&bar, 1, in);
  }
  // a wait of any thread ran out: everything from here on is no number (gv comes of no product)
  const float bad = __syncthreads_or(!ok) ? __int_as_float(0x7fc00000) : 0.f;
  if (warp == 1) {  // the decay's gradient: sums of `from` from a token on, of `to` before it; two a lane
    float x = 0.f;
    for (int i = 0; i < 8; ++i) x += zs[i];
    x *= G[C - 1];
    const int t = 2 * lane;
    const float f0 = from[0][t] + from[1][t], f1 = from[0][t + 1] + from[1][t + 1];
    const float t0 = to[0][t] + to[1][t], t1 = to[0][t + 1] + to[1][t + 1];
    float after = f0 + f1, ahead = t0 + t1;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const float f = __shfl_down_sync(~0u, after, m), y = __shfl_up_sync(~0u, ahead, m);
      if (lane + m < 32) after += f;
      if (lane >= m) ahead += y;
    }
    const float f2 = __shfl_down_sync(~0u, after, 1), y = __shfl_up_sync(~0u, ahead, 1);
    const float from1 = f1 + (lane < 31 ? f2 : 0.f), to0 = lane ? y : 0.f;
    IO* gg = reinterpret_cast<IO*>(d.gg) + vrow + t;
    if (t < at.len) gg[0] = from_f32<IO>((x + before[t]) + (f0 + from1) + to0 + bad);
    if (t + 1 < at.len) gg[1] = from_f32<IO>((x + before[t + 1]) + from1 + (to0 + t0) + bad);
  }
  ax[0] = ax[1] = 0.f;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int cb = NB * 32 * half + 32 * nb;
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      tmem_load(tm + m * DK + rows + cb, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[m][nb][e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const int t = row_of(e), o = (e & 2) >> 1, c = cb + 2 * (lane & 3) + (e >> 2) * 8;
      const float2 kv = tile_two<PARTS>(sm + L::K, NB * kTileBytes, t, c);
      float *x = acc[1][nb] + e, *y = acc[2][nb] + e;
      ax[o] += x[0] * kv.x + x[1] * kv.y;
      y[0] = fmaf(be[t], x[0], y[0]) + bad;
      y[1] = fmaf(be[t], x[1], y[1]) + bad;
      acc[0][nb][e] += bad;
      acc[0][nb][e + 1] += bad;
    }
    const int cs = cb - 32 * half;  // store_rows counts the half's 32 columns itself
    if (w.part) {
      float* p = w.part + vrow * 2 * a.dk;
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const int t = row_of(e), c = cb + 2 * (lane & 3) + (e >> 2) * 8;
        if (t >= at.len || c >= a.dk) continue;
        store_two(p + (size_t)t * 2 * a.dk + c, acc[0][nb][e], acc[0][nb][e + 1]);
        store_two(p + (size_t)t * 2 * a.dk + a.dk + c, acc[2][nb][e], acc[2][nb][e + 1]);
      }
    } else {
      store_rows(reinterpret_cast<IO*>(d.gq) + krow * a.dk, l, cs, at.len, a.dk, acc[0][nb]);
      store_rows(reinterpret_cast<IO*>(d.gk) + krow * a.dk, l, cs, at.len, a.dk, acc[2][nb]);
    }
  }
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const float x = row4(ax[o]);
    if ((lane & 3) == 0) kx[half][r0 + 8 * o] = x;
  }
  fence_before();
  __syncthreads();
  if (tid < at.len) reinterpret_cast<IO*>(d.gbeta)[vrow + tid] = from_f32<IO>(rv[0][tid] + rv[1][tid] + kx[0][tid] + kx[1][tid] + bad);
  if (warp == 0) tmem_free(tm, COLS);
}

// gq, gk of a key head: the sum over its value heads, in order; four elements a thread.
template <typename IO>
__global__ void __launch_bounds__(256) kla_delta_share_kernel(const DeltaArgs a, const DeltaGradArgs d,
                                                             const float* part) {
  const int rep = a.H / a.Hk, w = a.dk / 2;  // fours in a row of both
  const long long row = (long long)a.T * w, n = (long long)a.B * a.Hk * row;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long key = i / row, in = i - key * row, t = in / w;
    const int e = (int)(in - t * w) * 4;
    const float4* p = reinterpret_cast<const float4*>(part) + key * rep * row + in;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < rep; ++r) {
      const float4 y = p[r * row];
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    IO* out = reinterpret_cast<IO*>(e < a.dk ? d.gq : d.gk) + (key * a.T + t) * a.dk + (e < a.dk ? e : e - a.dk);
    store_two(out, x.x, x.y);
    store_two(out + 2, x.z, x.w);
  }
}

template <typename IO, int DK>
cudaError_t grad_dk(const DeltaArgs& a, const DeltaGradArgs& g, const Workspace& w, int num_sms, cudaStream_t s) {
  const unsigned blocks = (unsigned)((long long)a.B * a.H * ((a.T + C - 1) / C));
  using L = GradSmem<IO, DK>;
  const unsigned ahead = num_sms * L::kBlocks;
  if (pad64(a.dv) == 64) return run(kla_delta_grad_kernel<IO, DK, 1>, L::kBytes, blocks, kThreads, s, a, g, w, ahead);
  return run(kla_delta_grad_kernel<IO, DK, 2>, L::kBytes, blocks, kThreads, s, a, g, w, ahead);
}

}  // namespace
}  // namespace delta

size_t delta_backward_bytes(int B, int Hk, int H, int T, int dk, int dv) {
  size_t n = 0;
  delta::workspace(nullptr, B, Hk, H, T, dk, dv, true, &n);
  return n;
}

cudaError_t launch_delta_backward(const DeltaArgs& a, const DeltaGradArgs& g, int num_sms, void* workspace,
                                  cudaStream_t s) {
  size_t n = 0;
  const delta::Workspace w = delta::workspace(workspace, a.B, a.Hk, a.H, a.T, a.dk, a.dv, true, &n);
  cudaError_t e = delta::launch_prepare(a, &g, w, s);
  if (e == cudaSuccess) e = delta::launch_chain(a, &g, w, num_sms, s);
  if (e != cudaSuccess) return e;
  const bool wide = delta::pad64(a.dk) == 128;
  if (a.io == IO_BF16)
    e = wide ? delta::grad_dk<__nv_bfloat16, 128>(a, g, w, num_sms, s) : delta::grad_dk<__nv_bfloat16, 64>(a, g, w, num_sms, s);
  else
    e = wide ? delta::grad_dk<float, 128>(a, g, w, num_sms, s) : delta::grad_dk<float, 64>(a, g, w, num_sms, s);
  if (e != cudaSuccess || a.Hk == a.H) return e;
  const long long blocks = ((long long)a.B * a.Hk * a.T * (a.dk / 2) + 255) / 256;
  const unsigned grid = (unsigned)(blocks < (1LL << 30) ? blocks : 1LL << 30);
  if (a.io == IO_BF16) delta::kla_delta_share_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, g, w.part);
  else delta::kla_delta_share_kernel<float><<<grid, 256, 0, s>>>(a, g, w.part);
  return cudaGetLastError();
}

}  // namespace kla
