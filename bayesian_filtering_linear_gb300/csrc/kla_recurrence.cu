// The gated linear recurrence over whole sequences, and one decode token
// (sm_103a):
//
//   h_t = a_t h_{t-1} + s(a_t) σ(i_t) x_t,  y_t = h_t
//   a = e^g, σ(g) or exp(-rate σ(g));  s = 1, sqrt(1 - a²) or 1 - a
//
// Every input is read once and every output written once, so HBM bounds it;
// next come the special functions (five an element with both gates). A cluster
// of blocks goes along the sequence, a tile of 64 tokens a block at a time;
// the next tile is on its way by asynchronous copies meanwhile. A warp runs
// through its eight tokens from a state of zero and leaves its map (A, S); the
// maps of the block's warps meet in shared memory, those of the cluster's
// blocks are stored in each other's, and from them every warp knows the state
// that it starts from. Nothing waits but barriers, nothing goes through
// memory, and results do not depend on the cluster's size beyond rounding.
#include <algorithm>

#include "kla_recurrence.cuh"

namespace kla {

namespace {

using namespace rec;

// The decays and factors of a warp's tokens.
template <typename IO>
__device__ __forceinline__ void tokens_of(const RecArgs& p, const IO* tile, int off, f2 rate, Decay (&a)[kTok], f2 (&bx)[kTok]) {
  constexpr int S = kTile * kChans;  // elements a stream
  f2 less[kTok];
  if (p.decay == kRecSigmoid) {
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const f2 g = pair_at<IO>(tile + S + off + j * kChans);
      float h[2], l[2], m[2];
      decay_of_sigmoid(exp_neg(f2_lo(g)), h[0], l[0], m[0]);
      decay_of_sigmoid(exp_neg(f2_hi(g)), h[1], l[1], m[1]);
      a[j].hi = f2_make(h[0], h[1]), a[j].lo = f2_make(l[0], l[1]), less[j] = f2_make(m[0], m[1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      f2 la = pair_at<IO>(tile + S + off + j * kChans);
      if (p.decay == kRecRate)
        la = f2_mul(rate, f2_make(rcp_approx(1.f + exp_neg(f2_lo(la))), rcp_approx(1.f + exp_neg(f2_hi(la)))));
      decay_of_log(la, a[j], less[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    bx[j] = pair_at<IO>(tile + off + j * kChans);
    if (p.scale == kRecSqrt) {  // 1 - a² = -(a - 1)(2 + (a - 1))
      const f2 v = f2_mul(f2_neg(less[j]), f2_add(f2_both(2.f), less[j]));
      bx[j] = f2_mul(bx[j], f2_make(sqrtf(fmaxf(f2_lo(v), 0.f)), sqrtf(fmaxf(f2_hi(v), 0.f))));
    } else if (p.scale == kRecComplement) {
      bx[j] = f2_mul(bx[j], f2_neg(less[j]));
    }
    if (p.i.p) {
      const f2 i = pair_at<IO>(tile + 2 * S + off + j * kChans);
      bx[j] = f2_mul(bx[j], f2_make(rcp_approx(1.f + exp_neg(f2_lo(i))), rcp_approx(1.f + exp_neg(f2_hi(i)))));
    }
  }
}

template <typename IO>
__global__ void __launch_bounds__(kThreads, sizeof(IO) == 2 ? 3 : 2) kla_recurrence_kernel(const RecArgs p, int k) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  IO* const ring = reinterpret_cast<IO*>(smem + sizeof(Shared));
  constexpr int S = kTile * kChans, STAGE = 3 * S;
  const int rank = blockIdx.x % k, c0 = blockIdx.x / k * kChans, w = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (k > 1) cluster_arrive();  // every block of the cluster has started before another stores to it

  // this thread's copies
  using Copy = Copier<IO>;
  const int cc = c0 + Copy::group();
  const bool copies = cc < p.C;
  const Place at(copies ? cc : 0, p.H, p.D);
  const IO* const sx = reinterpret_cast<const IO*>(p.x.p) + at.of(p.x);
  const IO* const sg = reinterpret_cast<const IO*>(p.g.p) + at.of(p.g);
  const IO* const si = reinterpret_cast<const IO*>(p.i.p) + (p.i.p ? at.of(p.i) : 0);
  auto fetch = [&](long long step, int stage) {
    const long long first = (step * k + rank) * kTile;
    if (copies && first < p.T) {
      IO* const d = ring + stage * STAGE;
      Copy::tile(d, sx, p.x.st, (int)first, p.T);
      Copy::tile(d + S, sg, p.g.st, (int)first, p.T);
      if (p.i.p) Copy::tile(d + 2 * S, si, p.i.st, (int)first, p.T);
    }
    cp_async_commit();
  };

  // this lane's channels
  const int c = c0 + 2 * lane;
  const bool live = c < p.C;
  const Place my(live ? c : 0, p.H, p.D);
  IO* const y = p.y.p ? reinterpret_cast<IO*>(p.y.p) + my.of(p.y) : nullptr;
  f2 rate = 0, h = 0;  // h: the state before the step's tokens
  if (p.rate && live) rate = f2_neg(*reinterpret_cast<const f2*>(p.rate + (long long)my.h * p.D + my.d));
  if (p.h0 && live) h = *reinterpret_cast<const f2*>(p.h0 + c);

  const long long steps = ((long long)p.T + kTile * k - 1) / (kTile * k);
  fetch(0, 0);
  for (long long step = 0; step < steps; ++step) {
    const int stage = (int)(step & 1);
    fetch(step + 1, stage ^ 1);
    cp_async_wait<1>();
    __syncthreads();
    const long long first = (step * k + rank) * kTile, t0 = first + w * kTok;
    const int n = (int)(t0 >= p.T ? 0 : min((long long)kTok, p.T - t0));  // this warp's tokens
    Decay a[kTok];
    f2 bx[kTok];
    Map m{f2_both(1.f), 0, 0};
    if (n > 0) {
      tokens_of<IO>(p, ring + stage * STAGE, w * kTok * kChans + 2 * lane, rate, a, bx);
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (j < n) {
          m.S = apply(a[j].hi, a[j].lo, bx[j], m.S);
          lengthen(m.A, m.Al, a[j].hi, a[j].lo);
        }
      }
    }
    sh.warp[w][0][lane] = m.A, sh.warp[w][1][lane] = m.Al, sh.warp[w][2][lane] = m.S;
    __syncthreads();
    f2 next = h;
    if (k > 1) {  // the block's map to every block of the cluster
      Map b{f2_both(1.f), 0, 0};
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const f2 A = sh.warp[v][0][lane], Al = sh.warp[v][1][lane];
        b.S = apply(A, Al, sh.warp[v][2][lane], b.S);
        lengthen(b.A, b.Al, A, Al);
      }
      if (step == 0) cluster_wait();
      for (int r = w; r < k; r += kWarps) {
        put_remote(&sh.block[stage][rank][0][lane], r, b.A);
        put_remote(&sh.block[stage][rank][1][lane], r, b.Al);
        put_remote(&sh.block[stage][rank][2][lane], r, b.S);
      }
      cluster_arrive();
      cluster_wait();
      for (int r = 0; r < k; ++r) {
        if (r == rank) h = next;
        next = apply(sh.block[stage][r][0][lane], sh.block[stage][r][1][lane], sh.block[stage][r][2][lane], next);
      }
    }
    if (p.ckpt && w == 0 && live && first < p.T)
      *reinterpret_cast<f2*>(p.ckpt + first / kTile * p.C + c) = h;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      if (k > 1 && v >= w) break;
      if (v == w) next = h;
      h = apply(sh.warp[v][0][lane], sh.warp[v][1][lane], sh.warp[v][2][lane], h);
    }
    if (k == 1) {  // here `next` is the warp's start and h the next step's
      const f2 s = next;
      next = h, h = s;
    }
    if (live && y) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (j < n) {
          h = apply(a[j].hi, a[j].lo, bx[j], h);
          put_pair(y + (t0 + j) * p.y.st, h);
        }
      }
    }
    h = next;
  }
  if (k > 1 && steps == 0) cluster_wait();
  if (p.hT && live && rank == 0 && w == 0) *reinterpret_cast<f2*>(p.hT + c) = h;
}

// One token: a thread takes two channels.
template <typename IO>
__global__ void __launch_bounds__(128) kla_recurrence_step_kernel(const RecArgs p) {
  const int c = 2 * (blockIdx.x * 128 + threadIdx.x);
  if (c >= p.C) return;
  const Place my(c, p.H, p.D);
  f2 x = pair_at<IO>(reinterpret_cast<const IO*>(p.x.p) + my.of(p.x));
  f2 g = pair_at<IO>(reinterpret_cast<const IO*>(p.g.p) + my.of(p.g));
  const f2 h = *reinterpret_cast<const f2*>(p.h0 + c);
  if (p.i.p) {
    const f2 i = pair_at<IO>(reinterpret_cast<const IO*>(p.i.p) + my.of(p.i));
    x = f2_mul(x, f2_make(rcp_approx(1.f + exp_neg(f2_lo(i))), rcp_approx(1.f + exp_neg(f2_hi(i)))));
  }
  Decay a;
  f2 less;
  if (p.decay == kRecSigmoid) {
    float u[2], l[2], m[2];
    decay_of_sigmoid(exp_neg(f2_lo(g)), u[0], l[0], m[0]);
    decay_of_sigmoid(exp_neg(f2_hi(g)), u[1], l[1], m[1]);
    a.hi = f2_make(u[0], u[1]), a.lo = f2_make(l[0], l[1]), less = f2_make(m[0], m[1]);
  } else {
    if (p.decay == kRecRate)
      g = f2_mul(f2_neg(*reinterpret_cast<const f2*>(p.rate + (long long)my.h * p.D + my.d)),
                 f2_make(rcp_approx(1.f + exp_neg(f2_lo(g))), rcp_approx(1.f + exp_neg(f2_hi(g)))));
    decay_of_log(g, a, less);
  }
  if (p.scale == kRecSqrt) {
    const f2 v = f2_mul(f2_neg(less), f2_add(f2_both(2.f), less));
    x = f2_mul(x, f2_make(sqrtf(fmaxf(f2_lo(v), 0.f)), sqrtf(fmaxf(f2_hi(v), 0.f))));
  } else if (p.scale == kRecComplement) {
    x = f2_mul(x, f2_neg(less));
  }
  const f2 next = apply(a.hi, a.lo, x, h);
  *reinterpret_cast<f2*>(p.hT + c) = next;
  put_pair(reinterpret_cast<IO*>(p.y.p) + my.of(p.y), next);
}

template <typename IO>
cudaError_t launch_io(const RecArgs& a, int num_sms, cudaStream_t s) {
  const size_t smem = sizeof(Shared) + 2 * 3 * (size_t)kTile * kChans * sizeof(IO);
  const int tiles = (a.C + kChans - 1) / kChans;
  return launch_rec_cluster(kla_recurrence_kernel<IO>, a, tiles, rec_cluster(tiles, a.T, num_sms * (sizeof(IO) == 2 ? 3 : 2)),
                            smem, s);
}

}  // namespace

int rec_cluster(int tiles, int T, int resident) {
  const int along = (T + kTile - 1) / kTile;
  return std::max(1, std::min({resident / std::max(tiles, 1), along, kRecMaxCluster}));
}

cudaError_t launch_recurrence(const RecArgs& a, int num_sms, cudaStream_t s) {
  return a.io == IO_BF16 ? launch_io<__nv_bfloat16>(a, num_sms, s) : launch_io<float>(a, num_sms, s);
}

cudaError_t launch_recurrence_step(const RecArgs& a, cudaStream_t s) {
  const unsigned blocks = (unsigned)((a.C + 255) / 256);
  if (a.io == IO_BF16) kla_recurrence_step_kernel<__nv_bfloat16><<<blocks, 128, 0, s>>>(a);
  else kla_recurrence_step_kernel<float><<<blocks, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kla
