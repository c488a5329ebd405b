// The forward kernels of the gated linear recurrence (sm_103a), instantiated by
// type in kla_recurrence_f32.cu and kla_recurrence_bf16.cu:
//
//   h_t = a_t h_{t-1} + s(a_t) σ(i_t) x_t,  y_t = h_t
//   a = e^g, σ(g) or exp(-rate σ(g));  s = 1, sqrt(1 - a²) or 1 - a
//
// Every input is read once and every output written once, so HBM bounds it;
// next comes the issue of instructions (37 an element with both gates, five of
// them special functions). A cluster of blocks goes along the sequence, a tile of
// 64 or 128 tokens a block at a time. A warp runs through its sixteen tokens from a state
// of zero, keeping for each the outcome Y and the product P of the decays so far,
// and leaves its map (A, S), while the next tile is on its way. The maps of the
// block's warps meet in shared memory, those of the cluster's blocks are stored in
// each other's, and from them every warp knows the state h that it starts from:
// y_t = P_t h + Y_t. Nothing waits but barriers and nothing goes through memory.
// (No block may end before the others' stores into its shared memory have come:
// the last step's barrier is behind the last of them.)
//
// Measured: 608 tiles of 64 channels, one block each, 4096 tokens in bf16, 6.15
// TB/s (91% of a copy); B8 H16 T4096 D64 bf16, 128 tiles in clusters of four, 67 us
// (4.0 TB/s): 512 blocks leave a sixth of the 608 places empty, and the cluster's
// exchange takes the rest. Eight tokens a warp took 90 us: the composition of the
// maps costs as much for half the tokens.
#pragma once

#include "kla_recurrence.cuh"

namespace kla {
namespace rec {

constexpr int kTok = 16;  // tokens a warp
// Warps of a block: four, or where channels are few (so few that clusters of
// sixteen fit) and sequences longer than those reach in a step, eight, which halve
// the exchanges. Measured, bf16, four and eight: 65536 tokens of 16 heads of 128 258
// and 243 us, of one head of 64 158 and 114, 16384 of four heads of 64 45 and 33;
// the headline, whose channels are many, 67 and 73.
constexpr int kNarrow = 4, kWide = 8;
// Stages of the ring of tiles and blocks an SM. In bf16 a second stage and a fourth block are better than a fifth block
// (headline 70 us with one stage; five blocks of 96 registers 90) or three blocks (76); fp32 tiles are twice as large.
template <typename IO>
constexpr int kStages = sizeof(IO) == 2 ? 2 : 1;
template <typename IO, int WARPS>
constexpr int kBlocks = (sizeof(IO) == 2 ? 16 : WARPS == kNarrow ? 12 : 8) / WARPS;

// A decay (y: -log a, but for a sigmoid) and the factor s σ(i) x of a pair, from what is read.
template <typename IO, int DECAY, bool NEAR>
__device__ __forceinline__ Decay decay_of(const IO* g, f2 rate, f2& y) {
  y = 0;
  if (DECAY == kRecSigmoid) return decay_of_sigmoid(f2_exp_neg_held(pair_at<IO>(g)));
  if (DECAY == kRecRate) y = f2_mul(rate, f2_rcp(f2_add(f2_exp_neg(pair_at<IO>(g)), f2_both(1.f))));
  else y = minus_pair_at(g);
  return decay_of_log<NEAR>(y);
}
// All of a warp's rates are too small for a decay far from 1.
__device__ __forceinline__ bool near_rates(f2 rate) {
  return __all_sync(~0u, fminf(f2_lo(rate), f2_hi(rate)) >= 0.f && fmaxf(f2_lo(rate), f2_hi(rate)) <= kNear);
}
template <int SCALE>
__device__ __forceinline__ f2 scaled(f2 x, f2 less) {
  if (SCALE == kRecSqrt) return f2_mul(x, spread_sqrt(spread(less)));
  if (SCALE == kRecComplement) return f2_mul(x, less);
  return x;
}

// The state behind one token, from the state before it.
template <typename IO, int DECAY, int SCALE, bool GATE>
__device__ __forceinline__ f2 token(const IO* x_at, const IO* g_at, const IO* i_at, f2 rate, f2 h) {
  f2 x = pair_at<IO>(x_at), y;
  const Decay a = decay_of<IO, DECAY, false>(g_at, rate, y);
  x = scaled<SCALE>(x, a.less);
  if (GATE) x = f2_mul(x, f2_rcp(f2_add(f2_exp_neg(pair_at<IO>(i_at)), f2_both(1.f))));
  return apply<true>(a.hi, a.lo, x, h);
}
// x, or `other` where it is not finite
__device__ __forceinline__ f2 finite_or(f2 x, f2 other) {
  return f2_make(isfinite(f2_lo(x)) ? f2_lo(x) : f2_lo(other), isfinite(f2_hi(x)) ? f2_hi(x) : f2_hi(other));
}
// Eight tokens of two channels, all on their way at the same time; behind the last token, the last one again.
constexpr int kFew = 8;
template <typename IO>
struct alignas(2 * sizeof(IO)) Two {
  IO v[2];
};
template <typename IO, typename Tensor>
__device__ __forceinline__ void few(Two<IO> (&r)[kFew], const Tensor& x, long long at, int t, int T) {
#pragma unroll
  for (int j = 0; j < kFew; ++j)
    r[j] = *reinterpret_cast<const Two<IO>*>(reinterpret_cast<const IO*>(x.p) + at + min((long long)t + j, (long long)T - 1) * x.st);
}
// The states behind tokens t to t + 7 (as many as there are), given to `f` with their number one after the other until
// it says no; returns the last one.
template <typename IO, int DECAY, int SCALE, bool GATE, typename F>
__device__ __forceinline__ f2 few_states(const RecArgs& p, const Place& at, int t, f2 rate, f2 h, F f) {
  Two<IO> x[kFew], g[kFew], i[kFew];
  few<IO>(x, p.x, at.of(p.x), t, p.T);
  few<IO>(g, p.g, at.of(p.g), t, p.T);
  if (GATE) few<IO>(i, p.i, at.of(p.i), t, p.T);
#pragma unroll
  for (int j = 0; j < kFew; ++j) {
    if (j >= p.T - t) return h;
    h = token<IO, DECAY, SCALE, GATE>(x[j].v, g[j].v, i[j].v, rate, h);
    if (!f(j, h)) return h;
  }
  return h;
}
// For two channels whose last state is not finite, as none is behind the first such one. From that one on the kernel's
// own values are NaN, where they should be infinite until a token makes NaN of them: this goes from the first state `h`
// through the tokens one by one, until what is left is NaN or, by `last`, finite, and a thread stores what is not finite
// where it has stored before. (Every thread of a channel goes through all of its tokens: the headline with an infinite
// state takes 0.9 ms, and 0.07 with NaN alone.)
template <typename IO, int DECAY, int SCALE, bool GATE, int kWarps>
__device__ __forceinline__ void one_by_one(const RecArgs& p, int c, int rank, int k, int w, f2 rate, f2 h, f2 last) {
  const Place at(c, p.H, p.D);
  const long long y_at = at.of(p.y);
  const bool lo = isfinite(f2_lo(last)), hi = isfinite(f2_hi(last));
  const auto done = [&](f2 s) { return (lo || isnan(f2_lo(s))) && (hi || isnan(f2_hi(s))); };
#pragma unroll 1
  for (long long t = 0; t < p.T; t += kFew) {
    const bool mine = t / (kWarps * kTok) % k == rank && t / kTok % kWarps == w;
    if (mine && p.ckpt && t % kRecTile == 0) put_odd(p.ckpt + t / kRecTile * p.C + c, h);
    h = few_states<IO, DECAY, SCALE, GATE>(p, at, (int)t, rate, h, [&](int j, f2 s) {
      if (mine && p.y.p) put_odd(reinterpret_cast<IO*>(p.y.p) + y_at + (t + j) * p.y.st, s);
      return true;
    });
    if (done(h)) return;
  }
  if (p.hT && rank == 0 && w == 0) put_odd(p.hT + c, h);
}

template <typename IO, int DECAY, int SCALE, bool GATE, bool NEAR, int S>  // S: elements a stream
__device__ __forceinline__ Map segment(const IO* tile, f2 rate, f2 (&P)[kTok], f2 (&Y)[kTok]) {
  Map m{0, 0, 0};
  Product<DECAY, NEAR> prod;
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    f2 x = pair_at<IO>(tile + j * kChans), y;
    const Decay a = decay_of<IO, DECAY, NEAR>(tile + S + j * kChans, rate, y);
    x = scaled<SCALE>(x, a.less);
    if (GATE) x = f2_mul(x, f2_rcp(f2_add(f2_exp_neg(pair_at<IO>(tile + 2 * S + j * kChans)), f2_both(1.f))));
    m.S = apply<false>(a.hi, a.lo, x, m.S);
    prod.times(a, y);
    P[j] = prod.value();
    Y[j] = m.S;
  }
  prod.end(m);
  return m;
}

template <typename IO, int DECAY, int SCALE, bool GATE, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kBlocks<IO, kWarps>) kla_recurrence_kernel(const RecArgs p, int k) {
  constexpr int kThreads = 32 * kWarps, kTile = kWarps * kTok;
  __shared__ f2 start[32];  // the first states (hT may lie where h0 does)
  extern __shared__ __align__(16) unsigned char smem[];
  BlockMap* const blocks = reinterpret_cast<BlockMap*>(smem);  // [2][k]
  IO* const tile = reinterpret_cast<IO*>(smem + block_maps_bytes(k));
  constexpr int S = kTile * kChans, STAGE = (GATE ? 3 : 2) * S;
  const int rank = blockIdx.x % k, c0 = blockIdx.x / k * kChans, w = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (k > 1) cluster_arrive();  // every block of the cluster has started before another stores to it

  // this thread's copies
  using Copy = Copier<IO, kThreads, kTile>;
  const int cc = c0 + Copy::group();
  const bool copies = cc < p.C;
  const Place at(copies ? cc : 0, p.H, p.D);
  const IO* const sx = reinterpret_cast<const IO*>(p.x.p) + at.of(p.x);
  const IO* const sg = reinterpret_cast<const IO*>(p.g.p) + at.of(p.g);
  const IO* const si = reinterpret_cast<const IO*>(p.i.p) + (GATE ? at.of(p.i) : 0);
  auto fetch = [&](long long step) {
    const long long first = (step * k + rank) * kTile;
    const int t0 = (int)(first < p.T ? first : p.T);
    IO* const d = tile + (kStages<IO> == 2 ? (step & 1) * STAGE : 0);
    if (copies) {
      Copy::tile(d, sx, p.x.st, t0, p.T, 0);
      Copy::tile(d + S, sg, p.g.st, t0, p.T, still<IO, DECAY>());
      if (GATE) Copy::tile(d + 2 * S, si, p.i.st, t0, p.T, 0);
    }
    cp_async_commit();
  };

  // this lane's channels
  const int c = c0 + 2 * lane;
  const bool live = c < p.C;
  const Place my(live ? c : 0, p.H, p.D);
  IO* const y = p.y.p ? reinterpret_cast<IO*>(p.y.p) + my.of(p.y) : nullptr;
  f2 rate = 0, h = 0;  // h: the state before the step's tokens
  if (DECAY == kRecRate && live)
    rate = rates_at(p.rate + (long long)my.h * p.D + my.d);
  if (p.h0 && live) h = *reinterpret_cast<const f2*>(p.h0 + c);
  if (w == 0) start[lane] = h;
  const bool near = DECAY == kRecRate && near_rates(rate);

  const long long steps = ((long long)p.T + kTile * k - 1) / (kTile * k);
  fetch(0);
  for (long long step = 0; step < steps; ++step) {
    cp_async_wait<0>();
    __syncthreads();
    f2 P[kTok], Y[kTok];
    if (kStages<IO> == 2 && step + 1 < steps) fetch(step + 1);
    IO* const now = tile + (kStages<IO> == 2 ? (step & 1) * STAGE : 0);
    const IO* const mine = now + w * kTok * kChans + 2 * lane;
    // the warps' maps: over their own rows of x, which no one needs any more, or, where the next tile comes there, behind the ring
    const auto map_of = [&](int v) {
      return reinterpret_cast<f2*>(kStages<IO> == 2 ? now + v * kTok * kChans : tile + STAGE) + (kStages<IO> == 2 ? 0 : 96 * v) + lane;
    };
    Map m;
    if (near) m = segment<IO, DECAY, SCALE, GATE, DECAY == kRecRate, S>(mine, rate, P, Y);
    else m = segment<IO, DECAY, SCALE, GATE, false, S>(mine, rate, P, Y);
    __syncwarp();
    map_of(w)[0] = m.A, map_of(w)[32] = m.Al, map_of(w)[64] = m.S;
    __syncthreads();
    if (kStages<IO> == 1 && step + 1 < steps) fetch(step + 1);
    f2 next = h;
    if (k > 1) {  // the block's map to every block of the cluster
      BlockMap* const half = blocks + (step & 1) * k;
      if (step == 0) cluster_wait();
      if (w == 0) {
#pragma unroll
        for (int v = 1; v < kWarps; ++v) {
          const f2 A = map_of(v)[0], Al = map_of(v)[32];
          m.S = apply<false>(A, Al, map_of(v)[64], m.S);
          lengthen(m.A, m.Al, A, Al);
        }
        for (int r = 0; r < k; ++r) half[rank].put(lane, r, m);
      }
      if (w == 0) cluster_arrive();
      else cluster_arrive_only();
      cluster_wait();
      for (int r = 0; r < k; ++r) {
        if (r == rank) h = next;
        next = half[r].of(lane, next);
      }
    }
    const long long first = (step * k + rank) * kTile;
    f2 mystart = h;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      if (v == w) mystart = h;
      if (k == 1 || v < w) h = apply<false>(map_of(v)[0], map_of(v)[32], map_of(v)[64], h);
    }
    if (k > 1) h = next;
    const long long t0 = first + w * kTok;
    if (p.ckpt && live && t0 < p.T && t0 % kRecTile == 0) *reinterpret_cast<f2*>(p.ckpt + t0 / kRecTile * p.C + c) = mystart;
    if (live && y) {
      IO* out = y + t0 * p.y.st;
      if (t0 + kTok <= p.T) {
#pragma unroll
        for (int j = 0; j < kTok; ++j, out += p.y.st) put_pair(out, f2_fma(P[j], mystart, Y[j]));
      } else {
#pragma unroll
        for (int j = 0; j < kTok; ++j, out += p.y.st)
          if (t0 + j < p.T) put_pair(out, f2_fma(P[j], mystart, Y[j]));
      }
    }
  }
  if (!live) return;
  if (p.hT && rank == 0 && w == 0) *reinterpret_cast<f2*>(p.hT + c) = h;
  if (!finite(h)) one_by_one<IO, DECAY, SCALE, GATE, kWarps>(p, c, rank, k, w, rate, start[lane], h);
}

// One token: a thread takes two channels.
template <typename IO, int DECAY, int SCALE, bool GATE>
__global__ void __launch_bounds__(128) kla_recurrence_step_kernel(const RecArgs p) {
  const int c = 2 * (blockIdx.x * 128 + threadIdx.x);
  if (c >= p.C) return;
  const f2 h = *reinterpret_cast<const f2*>(p.h0 + c);
  f2 rate = 0;
  if (DECAY == kRecRate) rate = rates_at(p.rate + c % (p.H * p.D));
  const f2 next = token<IO, DECAY, SCALE, GATE>(reinterpret_cast<const IO*>(p.x.p) + c, reinterpret_cast<const IO*>(p.g.p) + c,
                                                reinterpret_cast<const IO*>(p.i.p) + (GATE ? c : 0), rate, h);
  *reinterpret_cast<f2*>(p.hT + c) = next;
  put_pair(reinterpret_cast<IO*>(p.y.p) + c, next);
}

// Calls f with the compile-time kinds of a call.
template <typename F>
inline cudaError_t by_kind(const RecArgs& a, F f) {
  using std::integral_constant;
  auto gate = [&](auto d, auto s) { return a.i.p ? f(d, s, std::true_type()) : f(d, s, std::false_type()); };
  auto scale = [&](auto d) {
    if (a.scale == kRecSqrt) return gate(d, integral_constant<int, kRecSqrt>());
    if (a.scale == kRecComplement) return gate(d, integral_constant<int, kRecComplement>());
    return gate(d, integral_constant<int, kRecPlain>());
  };
  if (a.decay == kRecSigmoid) return scale(integral_constant<int, kRecSigmoid>());
  if (a.decay == kRecRate) return scale(integral_constant<int, kRecRate>());
  return scale(integral_constant<int, kRecLog>());
}

// Shared memory of a block, but for the cluster's maps: the ring of tiles and, where the warps' maps have no place in it, those.
template <typename IO>
constexpr size_t forward_bytes(int warps, bool gate) {
  return kStages<IO> * (gate ? 3 : 2) * (size_t)warps * kTok * kChans * sizeof(IO) +
         (kStages<IO> == 2 ? 0 : warps * 96 * sizeof(f2));
}

}  // namespace rec

template <typename IO>
cudaError_t launch_recurrence_io(const RecArgs& a, cudaStream_t s) {
  const int tiles = (a.C + rec::kChans - 1) / rec::kChans;
  return rec::by_kind(a, [&](auto d, auto sc, auto gate) {
    const auto along = [&](int warps) { return (int)(((long long)a.T + warps * rec::kTok - 1) / (warps * rec::kTok)); };
    const auto go = [&](auto warps) {
      constexpr int W = decltype(warps)::value;
      return rec::launch_clusters<
          rec::kla_recurrence_kernel<IO, decltype(d)::value, decltype(sc)::value, decltype(gate)::value, W>, 32 * W,
          rec::forward_bytes<IO>(W, decltype(gate)::value)>(a, tiles, along(W), nullptr, s);
    };
    if (along(rec::kNarrow) > kRecMaxCluster) {
      int device = 0;
      const cudaError_t e = cudaGetDevice(&device);
      if (e != cudaSuccess) return e;
      constexpr auto narrow =
          rec::kla_recurrence_kernel<IO, decltype(d)::value, decltype(sc)::value, decltype(gate)::value, rec::kNarrow>;
      const int most = rec::clusters_at_once<narrow, 32 * rec::kNarrow, rec::forward_bytes<IO>(rec::kNarrow, decltype(gate)::value)>(
          device, kRecMaxCluster);
      if (most < 0) return cudaGetLastError();
      if (tiles <= most) return go(std::integral_constant<int, rec::kWide>());
    }
    return go(std::integral_constant<int, rec::kNarrow>());
  });
}

template <typename IO>
cudaError_t launch_recurrence_step_io(const RecArgs& a, cudaStream_t s) {
  const unsigned blocks = (unsigned)((a.C + 255) / 256);
  return rec::by_kind(a, [&](auto d, auto sc, auto gate) {
    rec::kla_recurrence_step_kernel<IO, decltype(d)::value, decltype(sc)::value, decltype(gate)::value><<<blocks, 128, 0, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace kla
