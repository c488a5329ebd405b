// Pieces shared by the kernels of the gated linear recurrence: the decays and
// scales from their inputs, segments' maps, tiles of inputs and the exchange
// between the blocks of a cluster.
//
// Every channel (b, h, d) is a recurrence of its own, h <- a h + b x, so a
// tile is 64 channels (in the flat order b, h, d) by 64 tokens: a warp takes
// eight of the tokens and a lane two of the channels, in packed arithmetic.
// A segment of tokens acts on the state before it as h -> A h + S.
//
// Decays near 1 multiply by the thousand, and one float of a decay is off by
// up to 2^-25, always the same way where a is the same. So a decay is a float
// and the rest that it leaves (1 - a is known to a few 2^-24 of itself), and
// so are the products of decays.
#pragma once

#include "kla_device.cuh"
#include "kla_launch.h"

namespace kla {
namespace rec {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kTok = 8;  // tokens a warp
constexpr int kTile = kRecTile, kChans = 64;                 // tokens and channels a tile
static_assert(kTile == kWarps * kTok, "a tile is the warps' tokens");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ f2 f2_both(float x) { return f2_make(x, x); }
__device__ __forceinline__ f2 f2_neg(f2 x) { return x ^ 0x8000000080000000ull; }

// e^-x, held at 2^126 or below, whose reciprocal is still a normal number
__device__ __forceinline__ float exp_neg(float x) { return fminf(ex2(x * -1.4426950408889634f), 0x1p126f); }

// A decay as the float nearest to it and the rest.
struct Decay {
  f2 hi, lo;
};

// a - 1 and a of one decay given its logarithm: a polynomial near 1 (Taylor's,
// the first term left out is 3e-8 of the value), else the exponential.
__device__ __forceinline__ void decay_of_log(f2 la, Decay& a, f2& less) {
  constexpr float kNear = 0.375f;
  f2 p = f2_both(1.f / 5040.f);
  p = f2_fma(p, la, f2_both(1.f / 720.f));
  p = f2_fma(p, la, f2_both(1.f / 120.f));
  p = f2_fma(p, la, f2_both(1.f / 24.f));
  p = f2_fma(p, la, f2_both(1.f / 6.f));
  p = f2_fma(p, la, f2_both(0.5f));
  p = f2_fma(f2_mul(p, la), la, la);
  const f2 one = f2_both(1.f), hi = f2_add(one, p);
  const f2 lo = f2_add(p, f2_neg(f2_add(hi, f2_neg(one))));
  float h[2] = {f2_lo(hi), f2_hi(hi)}, l[2] = {f2_lo(lo), f2_hi(lo)}, m[2] = {f2_lo(p), f2_hi(p)};
  const float x[2] = {f2_lo(la), f2_hi(la)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float e = ex2(x[i] * 1.4426950408889634f);
    const bool near = fabsf(x[i]) < kNear;
    h[i] = near ? h[i] : e;
    l[i] = near ? l[i] : 0.f;
    m[i] = near ? m[i] : e - 1.f;
  }
  a.hi = f2_make(h[0], h[1]);
  a.lo = f2_make(l[0], l[1]);
  less = f2_make(m[0], m[1]);
}

// The same of a sigmoid: e = e^-g, a = 1 / (1 + e).
__device__ __forceinline__ void decay_of_sigmoid(float e, float& hi, float& lo, float& less) {
  const float s = rcp_approx(1.f + e);
  less = -e * s;
  hi = 1.f + less;
  lo = less - (hi - 1.f);
  if (e > 1.f) hi = s, lo = 0.f, less = s - 1.f;
}

// The map of a segment, h -> A h + S: A in two floats.
struct Map {
  f2 A, Al, S;
};
__device__ __forceinline__ f2 apply(f2 A, f2 Al, f2 S, f2 h) { return f2_fma(A, h, f2_fma(Al, h, S)); }
// A <- a A
__device__ __forceinline__ void lengthen(f2& A, f2& Al, f2 hi, f2 lo) {
  const f2 p = f2_mul(hi, A), rest = f2_fma(hi, A, f2_neg(p));
  Al = f2_fma(hi, Al, f2_fma(lo, A, rest));
  A = p;
}

// ---- a token's pair of channels from a tile in shared memory ------------------
template <typename IO>
__device__ __forceinline__ f2 pair_at(const IO* p);
template <>
__device__ __forceinline__ f2 pair_at<float>(const float* p) {
  return *reinterpret_cast<const f2*>(p);
}
template <>
__device__ __forceinline__ f2 pair_at<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return f2_make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void put_pair(float* p, f2 v) { *reinterpret_cast<f2*>(p) = v; }
__device__ __forceinline__ void put_pair(__nv_bfloat16* p, f2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f2_lo(v), f2_hi(v));
}

// Where a flat channel lies.
struct Place {
  int b, h, d;
  __device__ __forceinline__ Place(int c, int H, int D) {
    d = c % D;
    const int bh = c / D;
    h = bh % H;
    b = bh / H;
  }
  template <typename Tensor>
  __device__ __forceinline__ long long of(const Tensor& t) const { return b * t.sb + h * t.sh + d; }
};

// One stream's share of a tile's copies, 16 bytes a copy: a thread keeps its
// channels and goes through the tokens.
template <typename IO>
struct Copier {
  static constexpr int VE = 16 / sizeof(IO), GROUPS = kChans / VE, ROWS = kThreads / GROUPS;
  __device__ __forceinline__ static int group() { return threadIdx.x % GROUPS * VE; }
  // tokens [t0, min(t0 + kTile, T)) of the stream at `src` (its thread's channels) into `dst`
  __device__ __forceinline__ static void tile(IO* dst, const IO* src, long long st, int t0, int T) {
#pragma unroll
    for (int r = 0; r < kTile; r += ROWS) {
      const int row = r + threadIdx.x / GROUPS;
      if (t0 + row < T) cp_async16(dst + row * kChans + group(), src + (long long)(t0 + row) * st);
    }
  }
};

// ---- clusters ------------------------------------------------------------------
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores a pair at the place of `p` (this block's shared memory) in the block of rank `rank`.
__device__ __forceinline__ void put_remote(const void* p, int rank, f2 v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// The segments' maps of a block's warps, and of a cluster's blocks (in two
// halves, used in turn, so that one barrier a step is enough).
struct Shared {
  f2 warp[kWarps][4][32];
  f2 block[2][kRecMaxCluster][3][32];
};

// Launches `tiles` clusters of k blocks.
template <typename Args>
inline cudaError_t launch_rec_cluster(void (*kernel)(Args, int), const Args& a, int tiles, int k, size_t smem,
                                      cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)k;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)tiles * (unsigned)k);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = k > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, a, k);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rec
}  // namespace kla
