// Gradients of the gated linear recurrence (sm_103a). With G_t = dL/dh_t in all:
//
//   G_t = gy_t + a_{t+1} G_{t+1}
//   gx = G s σ(i),  gi = G s σ(i) σ(-i) x
//   dL/dlog a = G (a h_{t-1} + s' σ(i) x),  s' = ds/dlog a = 0, -a²/s or -a
//   gg = dL/dlog a · (1, σ(-g) or -rate σ(g) σ(-g));  grate = -Σ dL/dlog a · σ(g)
//
// (where s = 0, at a = 1, s' has no value and its term is left out). Inputs and
// gy are read once and the gradients written once, and HBM bounds it; next come
// the special functions (seven an element with both gates). The kernel is the
// forward's run from the last tile to the first: the state before a tile comes
// from the checkpoints that the forward pass stored (in fp32: outputs in bf16
// would put their rounding into every gradient), a warp's tokens need the maps
// of the warps before them for h and of those behind them for G, which are
// exchanged together, and G goes from tile to tile as the state does forward.
// What the last loop needs and registers have no room for stays in shared
// memory at the thread's own place: e^-g where g was, the gate's term beside.
#include "kla_recurrence.cuh"

namespace kla {

namespace {

using namespace rec;

// e^-g of a pair into the thread's own place of the tile, and back: in g's (fp32), or half in g's and half in i's (bf16).
__device__ __forceinline__ void keep_exp(float* g, float*, f2 e) { *reinterpret_cast<f2*>(g) = e; }
__device__ __forceinline__ f2 kept_exp(const float* g, const float*) { return *reinterpret_cast<const f2*>(g); }
__device__ __forceinline__ void keep_exp(__nv_bfloat16* g, __nv_bfloat16* i, f2 e) {
  *reinterpret_cast<float*>(g) = f2_lo(e);
  *reinterpret_cast<float*>(i) = f2_hi(e);
}
__device__ __forceinline__ f2 kept_exp(const __nv_bfloat16* g, const __nv_bfloat16* i) {
  return f2_make(*reinterpret_cast<const float*>(g), *reinterpret_cast<const float*>(i));
}

template <typename IO>
__global__ void __launch_bounds__(kThreads, sizeof(IO) == 2 ? 2 : 1) kla_recurrence_grad_kernel(const RecGradArgs q, int k) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  f2* const gate_term = reinterpret_cast<f2*>(smem + sizeof(Shared)) + threadIdx.x;  // [kTok][kThreads]
  IO* const ring = reinterpret_cast<IO*>(smem + sizeof(Shared) + kTok * kThreads * sizeof(f2));
  constexpr int S = kTile * kChans, STAGE = 4 * S;
  const RecArgs& p = q.f;
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
  const IO* const sy = reinterpret_cast<const IO*>(q.gy.p) + (q.gy.p ? at.of(q.gy) : 0);
  auto fetch = [&](long long step, int stage) {
    const long long first = (step * k + rank) * kTile;
    if (copies && step >= 0 && first < p.T) {
      IO* const d = ring + stage * STAGE;
      Copy::tile(d, sx, p.x.st, (int)first, p.T);
      Copy::tile(d + S, sg, p.g.st, (int)first, p.T);
      if (p.i.p) Copy::tile(d + 2 * S, si, p.i.st, (int)first, p.T);
      if (q.gy.p) Copy::tile(d + 3 * S, sy, q.gy.st, (int)first, p.T);
    }
    cp_async_commit();
  };

  // this lane's channels
  const int c = c0 + 2 * lane;
  const bool live = c < p.C;
  const Place my(live ? c : 0, p.H, p.D);
  IO* const gx = reinterpret_cast<IO*>(q.gx.p) + my.of(q.gx);
  IO* const gg = reinterpret_cast<IO*>(q.gg.p) + my.of(q.gg);
  IO* const gi = reinterpret_cast<IO*>(q.gi.p) + (q.gi.p ? my.of(q.gi) : 0);
  f2 rate = 0, z = 0, sum = 0;  // z: what reaches the step's last token from behind it
  if (p.rate && live) rate = f2_neg(*reinterpret_cast<const f2*>(p.rate + (long long)my.h * p.D + my.d));
  if (q.ghT && live) z = *reinterpret_cast<const f2*>(q.ghT + c);

  const f2 one = f2_both(1.f);
  const long long steps = ((long long)p.T + kTile * k - 1) / (kTile * k);
  fetch(steps - 1, (int)((steps - 1) & 1));
  for (long long step = steps - 1; step >= 0; --step) {
    const int stage = (int)(step & 1);
    const long long first = (step * k + rank) * kTile, t0 = first + w * kTok;
    const int n = (int)(t0 >= p.T ? 0 : min((long long)kTok, p.T - t0));  // this warp's tokens
    f2 h = 0;
    if (live && first < p.T) h = *reinterpret_cast<const f2*>(p.ckpt + first / kTile * p.C + c);
    cp_async_wait<0>();
    __syncthreads();
    fetch(step - 1, stage ^ 1);  // (the last loop of the step before has read that stage)
    IO* const tile = ring + stage * STAGE + w * kTok * kChans + 2 * lane;
    f2 hi[kTok], lo[kTok], b[kTok], bx[kTok], u[kTok];
    Map m{one, 0, 0};
    f2 r = 0;
    if (n > 0) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        const f2 x = pair_at<IO>(tile + j * kChans), g = pair_at<IO>(tile + S + j * kChans);
        f2 open = one, shut = 0;
        if (p.i.p) {
          const f2 i = pair_at<IO>(tile + 2 * S + j * kChans);
          const f2 e = f2_make(exp_neg(f2_lo(i)), exp_neg(f2_hi(i)));
          open = f2_rcp(f2_add(one, e));
          shut = f2_mul(e, open);
        }
        f2 less, la = g;
        if (p.decay != kRecLog) {
          const f2 e = f2_make(exp_neg(f2_lo(g)), exp_neg(f2_hi(g)));
          keep_exp(tile + S + j * kChans, tile + 2 * S + j * kChans, e);
          if (p.decay == kRecRate) {
            la = f2_mul(rate, f2_rcp(f2_add(one, e)));
          } else {
            float v[2], l[2], d[2];
            decay_of_sigmoid(f2_lo(e), v[0], l[0], d[0]);
            decay_of_sigmoid(f2_hi(e), v[1], l[1], d[1]);
            hi[j] = f2_make(v[0], v[1]), lo[j] = f2_make(l[0], l[1]), less = f2_make(d[0], d[1]);
          }
        }
        if (p.decay != kRecSigmoid) {
          Decay a;
          decay_of_log(la, a, less);
          hi[j] = a.hi, lo[j] = a.lo;
        }
        const f2 xo = f2_mul(x, open);
        if (p.scale == kRecSqrt) {
          const f2 v = f2_mul(f2_neg(less), f2_add(f2_both(2.f), less));
          const float v0 = f2_lo(v), v1 = f2_hi(v);
          const f2 rs = f2_make(v0 > 0.f ? rsqrtf(v0) : 0.f, v1 > 0.f ? rsqrtf(v1) : 0.f);
          b[j] = f2_mul(f2_mul(v, rs), open);
          u[j] = f2_neg(f2_mul(f2_mul(f2_mul(hi[j], hi[j]), rs), xo));
        } else if (p.scale == kRecComplement) {
          b[j] = f2_mul(f2_neg(less), open);
          u[j] = f2_neg(f2_mul(hi[j], xo));
        } else {
          b[j] = open;
          u[j] = 0;
        }
        bx[j] = f2_mul(b[j], x);
        if (p.i.p) gate_term[j * kThreads] = f2_mul(bx[j], shut);
      }
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (j < n) {
          m.S = apply(hi[j], lo[j], bx[j], m.S);
          lengthen(m.A, m.Al, hi[j], lo[j]);
        }
      }
#pragma unroll
      for (int j = kTok - 1; j >= 0; --j) {
        if (j < n) {
          if (q.gy.p) r = f2_add(r, pair_at<IO>(tile + 3 * S + j * kChans));
          r = f2_fma(hi[j], r, f2_mul(lo[j], r));
        }
      }
    }
    sh.warp[w][0][lane] = m.A, sh.warp[w][1][lane] = m.Al, sh.warp[w][2][lane] = m.S, sh.warp[w][3][lane] = r;
    __syncthreads();
    f2 next = z;
    if (k > 1) {  // the block's map of G to every block of the cluster
      Map t{one, 0, 0};
#pragma unroll
      for (int v = kWarps - 1; v >= 0; --v) {
        const f2 A = sh.warp[v][0][lane], Al = sh.warp[v][1][lane];
        t.S = apply(A, Al, sh.warp[v][3][lane], t.S);
        lengthen(t.A, t.Al, A, Al);
      }
      if (step == steps - 1) cluster_wait();
      for (int o = w; o < k; o += kWarps) {
        put_remote(&sh.block[stage][rank][0][lane], o, t.A);
        put_remote(&sh.block[stage][rank][1][lane], o, t.Al);
        put_remote(&sh.block[stage][rank][2][lane], o, t.S);
      }
      cluster_arrive();
      cluster_wait();
      for (int o = k - 1; o >= 0; --o) {
        if (o == rank) z = next;
        next = apply(sh.block[stage][o][0][lane], sh.block[stage][o][1][lane], sh.block[stage][o][2][lane], next);
      }
    }
#pragma unroll
    for (int v = 0; v < kWarps; ++v)
      if (v < w) h = apply(sh.warp[v][0][lane], sh.warp[v][1][lane], sh.warp[v][2][lane], h);
#pragma unroll
    for (int v = kWarps - 1; v >= 0; --v) {
      if (k > 1 && v <= w) break;
      if (v == w) next = z;
      z = apply(sh.warp[v][0][lane], sh.warp[v][1][lane], sh.warp[v][3][lane], z);
    }
    if (k == 1) {  // here `next` is what reaches the warp and z what reaches the step before
      const f2 s = next;
      next = z, z = s;
    }
    if (n > 0) {
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (j < n) {
          const f2 ah = f2_fma(hi[j], h, f2_mul(lo[j], h));
          u[j] = f2_add(ah, u[j]);
          h = f2_add(ah, bx[j]);
        }
      }
#pragma unroll
      for (int j = kTok - 1; j >= 0; --j) {
        if (j < n) {
          f2 G = z;
          if (q.gy.p) G = f2_add(G, pair_at<IO>(tile + 3 * S + j * kChans));
          z = f2_fma(hi[j], G, f2_mul(lo[j], G));
          f2 by_log = f2_mul(G, u[j]);
          if (p.decay != kRecLog) {
            const f2 e = kept_exp(tile + S + j * kChans, tile + 2 * S + j * kChans);
            const f2 open = f2_rcp(f2_add(one, e)), shut = f2_mul(e, open);
            if (p.decay == kRecRate) {
              by_log = f2_mul(by_log, open);
              sum = f2_add(sum, by_log);
              by_log = f2_mul(by_log, f2_mul(rate, shut));
            } else {
              by_log = f2_mul(by_log, shut);
            }
          }
          if (live) {
            const long long t = t0 + j;
            put_pair(gx + t * q.gx.st, f2_mul(G, b[j]));
            put_pair(gg + t * q.gg.st, by_log);
            if (p.i.p) put_pair(gi + t * q.gi.st, f2_mul(G, gate_term[j * kThreads]));
          }
        }
      }
    }
    z = next;
  }
  if (q.gh0 && live && rank == 0 && w == 0) *reinterpret_cast<f2*>(q.gh0 + c) = z;
  if (q.part) {  // the block's sums of the rates' gradients, in a fixed order
    __syncthreads();
    sh.warp[w][0][lane] = sum;
    __syncthreads();
    if (w == 0 && live) {
#pragma unroll
      for (int v = 1; v < kWarps; ++v) sum = f2_add(sum, sh.warp[v][0][lane]);
      *reinterpret_cast<f2*>(q.part + (long long)rank * p.C + c) = sum;
    }
  }
}

// grate[h, d]: the blocks' sums over the cluster's ranks and the batch.
__global__ void __launch_bounds__(128) kla_recurrence_rate_kernel(const float* part, float* grate, int parts, int B, int HD) {
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i >= HD) return;
  float x = 0.f;
  for (long long n = 0; n < (long long)parts * B; ++n) x += part[n * HD + i];
  grate[i] = -x;
}

template <typename IO>
cudaError_t launch_io(const RecGradArgs& a, int num_sms, cudaStream_t s) {
  const size_t smem = sizeof(Shared) + kTok * kThreads * sizeof(f2) + 2 * 4 * (size_t)kTile * kChans * sizeof(IO);
  const int tiles = (a.f.C + kChans - 1) / kChans, k = rec_cluster(tiles, a.f.T, num_sms * (sizeof(IO) == 2 ? 2 : 1));
  const cudaError_t e = launch_rec_cluster(kla_recurrence_grad_kernel<IO>, a, tiles, k, smem, s);
  if (e != cudaSuccess || !a.part) return e;
  const int HD = a.f.H * a.f.D;
  kla_recurrence_rate_kernel<<<(HD + 127) / 128, 128, 0, s>>>(a.part, a.grate, k, a.f.B, HD);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_recurrence_backward(const RecGradArgs& a, int num_sms, cudaStream_t s) {
  return a.f.io == IO_BF16 ? launch_io<__nv_bfloat16>(a, num_sms, s) : launch_io<float>(a, num_sms, s);
}

}  // namespace kla
