// Gradients of the gated linear recurrence (sm_103a), instantiated by type in
// kla_recurrence_backward_f32.cu and kla_recurrence_backward_bf16.cu. With
// G_t = dL/dh_t in all:
//
//   G_t = gy_t + a_{t+1} G_{t+1}
//   gx = G s σ(i),  gi = G s σ(i) σ(-i) x
//   dL/dlog a = G u,  u = a h_{t-1} + s' σ(i) x,  s' = ds/dlog a = 0, -a²/s or -a
//   gg = dL/dlog a · (1, σ(-g) or -rate σ(g) σ(-g));  grate = -Σ dL/dlog a · σ(g)
//
// (where s = 0, at a = 1, s' has no value and its term is left out). Inputs and
// gy are read once and the gradients written once; HBM and the issue of
// instructions (73 an element with both gates) bound it. The kernel
// goes from the last tile to the first as the forward's goes from the first to
// the last: the state before a tile comes from the checkpoints that the forward
// pass stored (in fp32: outputs in bf16 would put their rounding into every
// gradient), and a warp's eight tokens need the maps of the warps before them
// for h and of those behind them for G, which are exchanged together. Forward
// through its tokens a warp makes P and V, u = P h + V with h the state before
// the warp, and both maps (G's is Σ P gy, with the same A); then, back through
// them, G and the gradients. What the last loop needs and registers have no room
// for stays in shared memory at the thread's own place: e^-g where g was (and i),
// s σ(i) and the gate's term beside. The gradients leave over the tile's own rows,
// in pieces of 16 bytes.
//
// Measured, bf16 with both gates: 304 tiles of 64 channels and 1024 tokens, one
// block each, 70 us (4.0 TB/s), issue slots 55% busy at sixteen warps an SM (128
// registers); B8 H16 T4096 D64, 128 tiles in clusters of two, 152 us. Three blocks
// of 80 registers an SM and one stage of tiles: 136 us for 456 tiles, no better a
// tile; blocks of four warps and 32 tokens, four an SM: 5% slower.
#pragma once

#include "kla_recurrence_kernels.cuh"

namespace kla {
namespace rec {

constexpr int kBackWarps = 8, kBackThreads = 32 * kBackWarps, kBackTok = kRecTile / kBackWarps;
// Stages of the ring of tiles: two, or for fp32, whose tiles are twice as large, one that two blocks take turns by.
template <typename IO>
constexpr int kBackStages = sizeof(IO) == 2 ? 2 : 1;

// A pair of floats at the thread's own place of a tile: where a pair of one (fp32) or of two streams was (bf16).
__device__ __forceinline__ void keep(float* a, float*, f2 v) { *reinterpret_cast<f2*>(a) = v; }
__device__ __forceinline__ f2 kept(const float* a, const float*) { return *reinterpret_cast<const f2*>(a); }
__device__ __forceinline__ void keep(__nv_bfloat16* a, __nv_bfloat16* b, f2 v) {
  *reinterpret_cast<float*>(a) = f2_lo(v);
  *reinterpret_cast<float*>(b) = f2_hi(v);
}
__device__ __forceinline__ f2 kept(const __nv_bfloat16* a, const __nv_bfloat16* b) {
  return f2_make(*reinterpret_cast<const float*>(a), *reinterpret_cast<const float*>(b));
}
// s σ(i) of a token's pair and, with a gate, the gate's term: in an array of the
// thread's own, the gate's term in fp32 where i was.
template <typename IO, bool GATE>
struct Own {
  static constexpr bool BOTH = GATE && sizeof(IO) == 2;
  static constexpr size_t BYTES = (BOTH ? 2 : 1) * (size_t)kBackTok * kBackThreads * sizeof(f2);
  f2* at;
  __device__ __forceinline__ explicit Own(void* p) : at(reinterpret_cast<f2*>(p) + (BOTH ? 2 : 1) * threadIdx.x) {}
  __device__ __forceinline__ void put(int j, IO* i, f2 b, f2 term) const {
    if (BOTH) {
      *reinterpret_cast<ulonglong2*>(at + 2 * j * kBackThreads) = make_ulonglong2(b, term);
    } else {
      at[j * kBackThreads] = b;
      if (GATE) *reinterpret_cast<f2*>(i) = term;
    }
  }
  __device__ __forceinline__ ulonglong2 get(int j, const IO* i) const {
    if (BOTH) return *reinterpret_cast<const ulonglong2*>(at + 2 * j * kBackThreads);
    return make_ulonglong2(at[j * kBackThreads], GATE ? *reinterpret_cast<const f2*>(i) : 0);
  }
};

// What a warp's tokens do to h and to G.
struct WarpMaps {
  ulonglong2 A[32];  // and Al
  f2 S[32], R[32];
  __device__ __forceinline__ f2 h(int lane, f2 v) const { return apply<false>(A[lane].x, A[lane].y, S[lane], v); }
  __device__ __forceinline__ f2 g(int lane, f2 v) const { return apply<false>(A[lane].x, A[lane].y, R[lane], v); }
};

// Forward through a warp's tokens: its maps of h and (in r) of G, and for each token the decay, P and V.
template <typename IO, int DECAY, int SCALE, bool GATE, bool NEAR>
__device__ __forceinline__ Map forth(IO* tile, const Own<IO, GATE>& own, f2 rate, f2 (&hi)[kBackTok], f2 (&P)[kBackTok], f2 (&V)[kBackTok], f2& r) {
  constexpr int S = kRecTile * kChans;
  const f2 one = f2_both(1.f), minus = f2_both(-1.f);
  Map m{0, 0, 0};
  Product<DECAY, NEAR> prod;
  r = 0;
#pragma unroll
  for (int j = 0; j < kBackTok; ++j) {
    IO* const at = tile + j * kChans;
    const f2 x = pair_at<IO>(at);
    f2 open = one, shut = 0;
    if (GATE) {
      const f2 e = f2_exp_neg_held(pair_at<IO>(at + 2 * S));
      open = f2_rcp(f2_add(one, e));
      shut = f2_mul(e, open);
    }
    Decay a;
    f2 y = 0;  // -log a, but for a sigmoid
    if (DECAY == kRecLog) {
      a = decay_of_log<NEAR>(y = minus_pair_at(at + S));
    } else {
      const f2 e = f2_exp_neg_held(pair_at<IO>(at + S));
      keep(at + S, at + 2 * S, e);
      if (DECAY == kRecSigmoid) a = decay_of_sigmoid(e);
      else a = decay_of_log<NEAR>(y = f2_mul(rate, f2_rcp(f2_add(one, e))));
    }
    const f2 xo = GATE ? f2_mul(x, open) : x;
    f2 w = 0, bx = xo, b = open;  // s' σ(i) x, s σ(i) x and s σ(i)
    if (SCALE == kRecSqrt) {
      const f2 v = spread(a.less), rs = spread_rsqrt(v), s = f2_mul(v, rs);
      b = GATE ? f2_mul(s, open) : s;
      bx = f2_mul(s, xo);
      // -a²/s, near 1 as s - 1/s (no digits are lost while a² is not small)
      if (NEAR) w = f2_mul(f2_fma(rs, minus, s), xo);
      else w = f2_mul(f2_mul(f2_mul(a.hi, a.hi), f2_mul(rs, minus)), xo);
    } else if (SCALE == kRecComplement) {
      b = GATE ? f2_mul(a.less, open) : a.less;
      bx = f2_mul(a.less, xo);
      w = f2_mul(f2_mul(a.hi, minus), xo);
    }
    if (SCALE != kRecPlain || GATE) own.put(j, at + 2 * S, b, GATE ? f2_mul(bx, shut) : 0);
    hi[j] = NEAR ? a.hi : a.nearest();
    const f2 ah = f2_fma(a.hi, m.S, f2_mul(a.lo, m.S));
    V[j] = SCALE == kRecPlain ? ah : f2_add(ah, w);
    m.S = f2_add(ah, bx);
    prod.times(a, y);
    P[j] = prod.value();
    r = f2_fma(P[j], pair_at<IO>(at + 3 * S), r);
  }
  prod.end(m);
  return m;
}

// For two channels in which a state that the thread's tokens meet (`odd`) or a G is not finite: as one_by_one of the
// forward pass, from the last token back, storing what is not finite among the gradients of the thread's tokens. `sum`,
// `z`: the rates' sum and what reaches the state before the first token, put right where they are not finite. (The
// headline with an infinite state takes 1.4 ms, with NaN alone 0.2.)
template <typename IO, int DECAY, int SCALE, bool GATE>
__device__ __forceinline__ void one_by_one_back(const RecGradArgs& q, int c, int rank, int k, int w, f2 rate, bool odd, const Own<IO, GATE>& own,
                                                f2& sum, f2& z) {
  const RecArgs& p = q.f;
  const Place at(c, p.H, p.D);
  const int tiles = (int)(((long long)p.T + kRecTile - 1) / kRecTile);
  const auto before = [&](int tile) { return *reinterpret_cast<const f2*>(p.ckpt + (long long)tile * p.C + c); };
  const auto inf = [](f2 s) { return isinf(f2_lo(s)) || isinf(f2_hi(s)); };
  if (odd) {  // is one infinite, or are all others NaN? (a tile between two finite states has none, one behind NaN only those)
    odd = false;
#pragma unroll 1
    for (int tile = rank; tile < tiles && !odd; tile += k) {
      f2 h = before(tile);
      const f2 next = tile + 1 < tiles ? before(tile + 1) : f2_both(__int_as_float(0x7fc00000));
      if ((isnan(f2_lo(h)) || isfinite(f2_lo(next))) && (isnan(f2_hi(h)) || isfinite(f2_hi(next)))) continue;
      odd = inf(h);
#pragma unroll 1
      for (long long t = (long long)tile * kRecTile; t < p.T && t < (tile + 1LL) * kRecTile && !odd; t += kFew)
        h = few_states<IO, DECAY, SCALE, GATE>(p, at, (int)t, rate, h, [&](int, f2 s) { return !(odd |= inf(s)); });
    }
  }
  const bool lo = !odd && isfinite(f2_lo(z)), hi = !odd && isfinite(f2_hi(z));
  const f2 one = f2_both(1.f), minus = f2_both(-1.f);
  f2 behind = q.ghT ? *reinterpret_cast<const f2*>(q.ghT + c) : 0, rates = 0;
  const auto done = [&](f2 s) { return (lo || isnan(f2_lo(s))) && (hi || isnan(f2_hi(s))); };
  if (lo && hi) return;
  static_assert(kFew == kBackTok, "a warp's tokens");
  int few_at = (p.T - 1) / kFew;
#pragma unroll 1
  for (; few_at >= 0 && !done(behind); --few_at) {
    const int t0 = few_at * kFew;
    Two<IO> g[kFew], gy[kFew];
    few<IO>(g, p.g, at.of(p.g), t0, p.T);
    if (q.gy.p) few<IO>(gy, q.gy, at.of(q.gy), t0, p.T);
    bool here = odd;
#pragma unroll
    for (int j = kFew - 1; j >= 0; --j) {
      if (j >= p.T - t0) continue;
      f2 y;
      const Decay a = decay_of<IO, DECAY, false>(g[j].v, rate, y);
      const f2 G = q.gy.p ? f2_add(behind, pair_at<IO>(gy[j].v)) : behind;
      here |= !finite(G);
      behind = apply<true>(a.hi, a.lo, 0, G);
      own.at[j * kBackThreads * (own.BOTH ? 2 : 1)] = G;
    }
    if (!here || t0 / kRecTile % k != rank || t0 / kBackTok % kBackWarps != w) continue;
    f2 h = before(t0 / kRecTile);
#pragma unroll 1
    for (int t = t0 / kRecTile * kRecTile; t < t0; t += kFew)
      h = few_states<IO, DECAY, SCALE, GATE>(p, at, t, rate, h, [](int, f2) { return true; });
    const auto of = [&](const auto& t, int j) {
      return reinterpret_cast<IO*>(const_cast<void*>(t.p)) + at.of(t) + (long long)(t0 + j) * t.st;
    };
#pragma unroll 1
    for (int j = 0; j < min(kFew, p.T - t0); ++j) {
      const IO *const x = of(p.x, j), *const g = of(p.g, j), *const i = GATE ? of(p.i, j) : nullptr;
      const f2 G = own.at[j * kBackThreads * (own.BOTH ? 2 : 1)];
      f2 open = one, shut = 0, b = one, slope = 0, y;  // b: s; slope: s'
      const Decay a = decay_of<IO, DECAY, false>(g, rate, y);
      if (GATE) {
        const f2 e = f2_exp_neg_held(pair_at<IO>(i));
        open = f2_rcp(f2_add(one, e));
        shut = f2_mul(e, open);
      }
      const f2 xo = f2_mul(pair_at<IO>(x), open);
      if (SCALE == kRecSqrt) {
        const f2 v = spread(a.less), rs = spread_rsqrt(v);
        b = f2_mul(v, rs);
        slope = f2_mul(f2_mul(a.hi, a.hi), f2_mul(rs, minus));
      } else if (SCALE == kRecComplement) {
        b = a.less;
        slope = f2_mul(a.hi, minus);
      }
      put_odd(of(q.gx, j), f2_mul(G, f2_mul(b, open)));
      if (GATE) put_odd(of(q.gi, j), f2_mul(G, f2_mul(f2_mul(b, xo), shut)));
      f2 by_log = f2_mul(G, apply<true>(a.hi, a.lo, SCALE == kRecPlain ? 0 : f2_mul(slope, xo), h));
      if (DECAY != kRecLog) {
        const f2 e = f2_exp_neg_held(pair_at<IO>(g)), sg = f2_rcp(f2_add(one, e));
        if (DECAY == kRecRate) {
          by_log = f2_mul(by_log, sg);
          rates = f2_add(rates, by_log);
          by_log = f2_mul(by_log, f2_mul(rate, minus));
        }
        by_log = f2_mul(by_log, f2_mul(e, sg));
      }
      put_odd(of(q.gg, j), by_log);
      h = token<IO, DECAY, SCALE, GATE>(x, g, i, rate, h);
    }
  }
  if (few_at >= 0) rates = f2_add(rates, f2_make(isnan(f2_lo(behind)) ? f2_lo(behind) : 0.f, isnan(f2_hi(behind)) ? f2_hi(behind) : 0.f));
  // (tokens that were passed over add finite values)
  sum = finite_or(sum, f2_make(isfinite(f2_lo(rates)) ? f2_lo(sum) : f2_lo(rates), isfinite(f2_hi(rates)) ? f2_hi(sum) : f2_hi(rates)));
  z = finite_or(z, behind);
}

template <typename IO, int DECAY, int SCALE, bool GATE>
__global__ void __launch_bounds__(kBackThreads, 2) kla_recurrence_grad_kernel(const RecGradArgs q, int k) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ WarpMaps maps[kBackWarps];
  __shared__ const IO* places[Copier<IO, kBackThreads, kRecTile>::GROUPS][7];
  constexpr int S = kRecTile * kChans, STAGE = 4 * S;
  BlockMap* const blocks = reinterpret_cast<BlockMap*>(smem);  // [2][k]
  IO* const ring = reinterpret_cast<IO*>(smem + block_maps_bytes(k));
  const Own<IO, GATE> own(ring + kBackStages<IO> * STAGE);
  const RecArgs& p = q.f;
  const int rank = blockIdx.x % k, c0 = blockIdx.x / k * kChans, w = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (k > 1) cluster_arrive();  // every block of the cluster has started before another stores to it

  // this thread's copies
  using Copy = Copier<IO, kBackThreads, kRecTile>;
  const int cc = c0 + Copy::group();
  const bool copies = cc < p.C;
  const Place at(copies ? cc : 0, p.H, p.D);
  // (kept in shared memory: the registers are needed)
  const IO** const from = places[threadIdx.x % Copy::GROUPS];
  if (threadIdx.x < Copy::GROUPS) {
    from[0] = reinterpret_cast<const IO*>(p.x.p) + at.of(p.x);
    from[1] = reinterpret_cast<const IO*>(p.g.p) + at.of(p.g);
    if (GATE) from[2] = reinterpret_cast<const IO*>(p.i.p) + at.of(p.i);
    if (q.gy.p) from[3] = reinterpret_cast<const IO*>(q.gy.p) + at.of(q.gy);
    from[4] = reinterpret_cast<const IO*>(q.gx.p) + at.of(q.gx);
    from[5] = reinterpret_cast<const IO*>(q.gg.p) + at.of(q.gg);
    if (GATE) from[6] = reinterpret_cast<const IO*>(q.gi.p) + at.of(q.gi);
  }
  __syncthreads();
  auto fetch = [&](int step) {
    if (copies && step >= 0) {
      const long long first = ((long long)step * k + rank) * kRecTile;
      const int t0 = (int)(first < p.T ? first : p.T);
      IO* const d = ring + (kBackStages<IO> == 2 ? (step & 1) * STAGE : 0);
      Copy::tile(d, from[0], p.x.st, t0, p.T, 0);
      Copy::tile(d + S, from[1], p.g.st, t0, p.T, still<IO, DECAY>());
      if (GATE) Copy::tile(d + 2 * S, from[2], p.i.st, t0, p.T, 0);
      if (q.gy.p) Copy::tile(d + 3 * S, from[3], q.gy.st, t0, p.T, 0);
    }
    cp_async_commit();
  };

  // this lane's channels
  const int c = c0 + 2 * lane;
  const bool live = c < p.C;
  const Place my(live ? c : 0, p.H, p.D);
  f2 rate = 0, z = 0, sum = 0;  // z: what reaches the step's last token from behind it
  if (DECAY == kRecRate && live)
    rate = rates_at(p.rate + (long long)my.h * p.D + my.d);
  if (q.ghT && live) z = *reinterpret_cast<const f2*>(q.ghT + c);
  const bool near = DECAY == kRecRate && near_rates(rate);

  if (!q.gy.p)  // no copies: zeros
    for (int i = threadIdx.x; i < kBackStages<IO> * S * (int)sizeof(IO) / 16; i += kBackThreads)
      reinterpret_cast<uint4*>(ring + (i / (S * (int)sizeof(IO) / 16)) * STAGE + 3 * S)[i % (S * (int)sizeof(IO) / 16)] = make_uint4(0, 0, 0, 0);
  const f2 one = f2_both(1.f), minus_rate = f2_mul(rate, f2_both(-1.f));
  const int steps = (int)(((long long)p.T + kRecTile * k - 1) / (kRecTile * k));
  bool odd = false;  // a state that the thread's tokens meet is not finite
  fetch(steps - 1);
  for (int step = steps - 1; step >= 0; --step) {
    const long long first = ((long long)step * k + rank) * kRecTile, t0 = first + w * kBackTok;
    f2 h = 0;
    if (live && first < p.T) h = *reinterpret_cast<const f2*>(p.ckpt + first / kRecTile * p.C + c);
    cp_async_wait<0>();
    __syncthreads();
    if (kBackStages<IO> == 2) fetch(step - 1);  // (the last loop of the step before has read that stage)
    IO* const tile = ring + (kBackStages<IO> == 2 ? (step & 1) * STAGE : 0) + w * kBackTok * kChans + 2 * lane;
    f2 hi[kBackTok], P[kBackTok], V[kBackTok], r;
    Map m;
    if (near) m = forth<IO, DECAY, SCALE, GATE, DECAY == kRecRate>(tile, own, rate, hi, P, V, r);
    else m = forth<IO, DECAY, SCALE, GATE, false>(tile, own, rate, hi, P, V, r);
    maps[w].A[lane] = make_ulonglong2(m.A, m.Al), maps[w].S[lane] = m.S, maps[w].R[lane] = r;
    __syncthreads();
    f2 next = z;
    if (k > 1) {  // the block's map of G to every block of the cluster
      BlockMap* const half = blocks + (step & 1) * k;
      if (step == steps - 1) cluster_wait();
      if (w == kBackWarps - 1) {
        Map t{m.A, m.Al, r};
#pragma unroll
        for (int v = kBackWarps - 2; v >= 0; --v) {
          t.S = maps[v].g(lane, t.S);
          lengthen(t.A, t.Al, maps[v].A[lane].x, maps[v].A[lane].y);
        }
        for (int o = 0; o < k; ++o) half[rank].put(lane, o, t);
      }
      cluster_arrive();  // (by all: with the others' arrivals not held up by their stores, the headline took 213 us for 163)
      cluster_wait();
      for (int o = k - 1; o >= 0; --o) {
        if (o == rank) z = next;
        next = half[o].of(lane, next);
      }
    }
#pragma unroll
    for (int v = 0; v < kBackWarps - 1; ++v)
      if (v < w) h = maps[v].h(lane, h);
    f2 behind = z;
#pragma unroll
    for (int v = kBackWarps - 1; v >= 0; --v) {
      if (v == w) behind = z;
      if (k == 1 || v > w) z = maps[v].g(lane, z);
    }
    if (k > 1) z = next;
    if (t0 < p.T) {
      odd |= !finite(f2_add(h, m.S));
      const int n = (int)min((long long)kBackTok, p.T - t0);
#pragma unroll
      for (int j = kBackTok - 1; j >= 0; --j) {  // G in the decays' place, dL/dlog a in V's
        const f2 G = f2_add(behind, pair_at<IO>(tile + 3 * S + j * kChans));
        behind = f2_mul(hi[j], G);
        hi[j] = G;
        V[j] = f2_mul(G, f2_fma(P[j], h, V[j]));
      }
#pragma unroll
      for (int j = 0; j < kBackTok; ++j) {
        IO* const o = tile + j * kChans;
        const f2 G = hi[j];
        f2 by_log = V[j];
        if (DECAY != kRecLog) {
          const f2 e = kept(o + S, o + 2 * S), open = f2_rcp(f2_add(one, e)), shut = f2_mul(e, open);
          if (DECAY == kRecRate) {
            by_log = f2_mul(by_log, open);
            sum = f2_add(sum, by_log);  // (behind the last token σ(g) is 2^-126)
            by_log = f2_mul(by_log, f2_mul(minus_rate, shut));
          } else {
            by_log = f2_mul(by_log, shut);
          }
        }
        if (SCALE == kRecPlain && !GATE) {
          put_pair(o, G);
        } else {
          const ulonglong2 b = own.get(j, o + 2 * S);
          put_pair(o, f2_mul(G, b.x));
          if (GATE) put_pair(o + 2 * S, f2_mul(G, b.y));
        }
        put_pair(o + S, by_log);
      }
      __syncwarp();
      // the warp's rows leave in pieces of 16 bytes
      if (copies) {
        constexpr int ROWS = 32 / Copy::GROUPS;
        const int row = lane / Copy::GROUPS;
        const IO* const rows = ring + (kBackStages<IO> == 2 ? (step & 1) * STAGE : 0) + (w * kBackTok + row) * kChans + Copy::group();
        const auto leave = [&](int stream, long long st) {
          IO* out = const_cast<IO*>(from[4 + stream]) + (t0 + row) * st;
#pragma unroll
          for (int r = 0; r < kBackTok; r += ROWS, out += ROWS * st)
            if (row + r < n) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(rows + r * kChans + stream * S);
        };
        leave(0, q.gx.st);
        leave(1, q.gg.st);
        if (GATE) leave(2, q.gi.st);
      }
    }
    if (kBackStages<IO> == 1) {
      __syncthreads();
      fetch(step - 1);
    }
  }
  __syncwarp();  // (other lanes have stored gradients of this one's channels)
  if (live && (odd || !finite(z)))
    one_by_one_back<IO, DECAY, SCALE, GATE>(q, c, rank, k, w, rate, odd, own, sum, z);
  if (q.gh0 && live && rank == 0 && w == 0) *reinterpret_cast<f2*>(q.gh0 + c) = z;
  if (DECAY == kRecRate && q.part) {  // the block's sums of the rates' gradients, in a fixed order
    __syncthreads();
    maps[w].S[lane] = sum;
    __syncthreads();
    if (w == 0 && live) {
#pragma unroll
      for (int v = 1; v < kBackWarps; ++v) sum = f2_add(sum, maps[v].S[lane]);
      *reinterpret_cast<f2*>(q.part + (long long)rank * p.C + c) = sum;
    }
  }
}

}  // namespace rec

template <typename IO>
cudaError_t launch_recurrence_backward_io(const RecGradArgs& a, int* parts, cudaStream_t s) {
  return rec::by_kind(a.f, [&](auto d, auto sc, auto gate) {
    constexpr size_t ring = rec::kBackStages<IO> * 4 * (size_t)kRecTile * rec::kChans * sizeof(IO);
    constexpr size_t own = rec::Own<IO, decltype(gate)::value>::BYTES;
    return rec::launch_clusters<rec::kla_recurrence_grad_kernel<IO, decltype(d)::value, decltype(sc)::value, decltype(gate)::value>,
                                rec::kBackThreads, ring + own>(a, (a.f.C + rec::kChans - 1) / rec::kChans,
                                                               (int)(((long long)a.f.T + kRecTile - 1) / kRecTile), parts, s);
  });
}

}  // namespace kla
