// Pieces shared by the kernels of the gated linear recurrence: the decays and
// scales from their inputs, segments' maps, tiles of inputs and the exchange
// between the blocks of a cluster.
//
// Every channel (b, h, d) is a recurrence of its own, h <- a h + b x, so a
// tile is 64 channels (in the flat order b, h, d) by 64 tokens: the block's
// warps share the tokens and a lane takes two of the channels, in packed
// arithmetic. A segment of tokens acts on the state before it as h -> A h + S.
//
// Decays near 1 multiply by the thousand, and one float of a decay is off by
// up to 2^-25, always the same way where a is the same. So a decay is a float
// and the rest that it leaves (1 - a is known to a few 2^-24 of itself), and
// so are the products of decays that the state is carried by.
#pragma once

#include <atomic>

#include "kla_device.cuh"
#include "kla_launch.h"

namespace kla {
namespace rec {

constexpr int kChans = 64;  // channels a tile

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The smaller and the larger of two; NaN where one is (fminf and fmaxf give the other).
__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(max_nan(x, 0.f)));
  return y;
}
__device__ __forceinline__ f2 f2_both(float x) { return f2_make(x, x); }
__device__ __forceinline__ f2 f2_ex2(f2 x) { return f2_make(ex2(f2_lo(x)), ex2(f2_hi(x))); }
// e^-x
__device__ __forceinline__ f2 f2_exp_neg(f2 x) { return f2_ex2(f2_mul(x, f2_both(-1.4426950408889634f))); }
// The same, held at 2^126 or below, whose reciprocal is still a normal number.
__device__ __forceinline__ f2 f2_exp_neg_held(f2 x) {
  const f2 e = f2_exp_neg(x);
  return f2_make(min_nan(f2_lo(e), 0x1p126f), min_nan(f2_hi(e), 0x1p126f));
}
// Two channels' rates, held at 2^80 or below (infinite ones: a = 0): times the σ(g) behind the last token, 0 or, of
// the held exponential, 2^-126, that is no decay.
__device__ __forceinline__ f2 rates_at(const float* p) {
  const float2 r = *reinterpret_cast<const float2*>(p);
  return f2_make(min_nan(r.x, 0x1p80f), min_nan(r.y, 0x1p80f));
}

// A decay: a float, the rest that it leaves, and 1 - a.
struct Decay {
  f2 hi, lo, less;
  __device__ __forceinline__ f2 nearest() const { return f2_add(hi, lo); }
};
__device__ __forceinline__ f2 one_minus(f2 x) { return f2_fma(x, f2_both(-1.f), f2_both(1.f)); }
// What `hi`, at least a half, leaves of 1 - less (1 - hi is exact), where wanted.
__device__ __forceinline__ f2 rest_of(f2 hi, f2 less, bool n0, bool n1) {
  const f2 r = f2_fma(less, f2_both(-1.f), one_minus(hi));
  return f2_make(n0 ? f2_lo(r) : 0.f, n1 ? f2_hi(r) : 0.f);
}

// Of y = -log a: near a = 1 (y in [0, 0.375]) a polynomial for 1 - a, which
// corrects the exponential, elsewhere that alone. NEAR: all are, and hi is the
// float nearest to a. The polynomial is y (1 - c1 y + ...), (1 - e^-y) / y
// interpolated at the five Chebyshev points of the interval, off by 4.3e-8 of the
// value at most; Taylor's needs two terms more for that.
constexpr float kNear = 0.375f;
template <bool NEAR>
__device__ __forceinline__ Decay decay_of_log(f2 y) {
  f2 p = f2_fma(y, f2_both(0x1.d3c856p-8f), f2_both(-0x1.523554p-5f));
  p = f2_fma(p, y, f2_both(0x1.553ae2p-3f));
  p = f2_fma(p, y, f2_both(-0x1.ffff62p-2f));
  p = f2_fma(f2_mul(p, y), y, y);
  Decay a;
  if (NEAR) {
    a.less = p;
    a.hi = one_minus(p);
    a.lo = f2_fma(p, f2_both(-1.f), one_minus(a.hi));
  } else {
    const bool n0 = fabsf(f2_lo(y) - 0.5f * kNear) <= 0.5f * kNear, n1 = fabsf(f2_hi(y) - 0.5f * kNear) <= 0.5f * kNear;
    a.hi = f2_exp_neg(y);
    a.lo = rest_of(a.hi, p, n0, n1);
    const f2 far = one_minus(a.hi);
    a.less = f2_make(n0 ? f2_lo(p) : f2_lo(far), n1 ? f2_hi(p) : f2_hi(far));
  }
  return a;
}

// Of a sigmoid: e = e^-g (held), a = 1 / (1 + e).
__device__ __forceinline__ Decay decay_of_sigmoid(f2 e) {
  Decay a;
  a.hi = f2_rcp(f2_add(e, f2_both(1.f)));
  a.less = f2_mul(e, a.hi);
  a.lo = rest_of(a.hi, a.less, f2_lo(e) <= 1.f, f2_hi(e) <= 1.f);
  return a;
}

// 1 - a², its square root and one over that: where it is below the normal
// numbers, or a above 1, both count as zero.
__device__ __forceinline__ f2 spread(f2 less) { return f2_mul(less, f2_fma(less, f2_both(-1.f), f2_both(2.f))); }
__device__ __forceinline__ f2 spread_sqrt(f2 v) { return f2_make(sqrt_fast(f2_lo(v)), sqrt_fast(f2_hi(v))); }
__device__ __forceinline__ f2 spread_rsqrt(f2 v) {
  const float a = f2_lo(v), b = f2_hi(v);
  return f2_make(a >= 0x1p-126f ? rsqrt_fast(a) : 0.f, b >= 0x1p-126f ? rsqrt_fast(b) : 0.f);
}

// The map of a segment, h -> A h + S: A in two floats.
struct Map {
  f2 A, Al, S;
};
// Infinite values held at the largest float (and NaN, which the product with the upper part keeps).
__device__ __forceinline__ f2 held(f2 x) {
  float a, b;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(a) : "f"(f2_lo(x)), "f"(0x1.fffffep127f));
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(b) : "f"(f2_hi(x)), "f"(0x1.fffffep127f));
  return f2_make(a, b);
}
__device__ __forceinline__ bool finite(f2 x) { return isfinite(f2_lo(x)) && isfinite(f2_hi(x)); }
// A h + S. The rest of A is zero or below zero as often as above, and its product with an infinite h would make NaN of
// what stays infinite: it meets the h that is held. Along the sequence the maps go without (the two instructions more
// took the headline from 67 to 70 us) and leave NaN, by which the kernels' ends find the channels to go through again.
template <bool HELD>
__device__ __forceinline__ f2 apply(f2 A, f2 Al, f2 S, f2 h) { return f2_fma(A, h, f2_fma(Al, HELD ? held(h) : h, S)); }
// A <- a A
__device__ __forceinline__ void lengthen(f2& A, f2& Al, f2 hi, f2 lo) {
  const f2 p = f2_mul(hi, A);
  const f2 rest = f2_fma(hi, A, f2_mul(p, f2_both(-1.f)));
  Al = f2_fma(hi, Al, f2_fma(lo, A, rest));
  A = p;
}

// The product of a segment's decays so far: by logarithms, where those are known,
// its value for the tokens' outcomes and the sum, of which the segment's own
// A comes in the end; else in two floats all along.
template <int DECAY, bool NEAR>
struct Product {
  f2 A = f2_both(1.f), rest = 0;  // rest: the sum of -log a, or what A leaves
  __device__ __forceinline__ void times(const Decay& a, f2 y) {
    if (DECAY == kRecSigmoid) {
      lengthen(A, rest, a.hi, a.lo);
    } else {
      A = NEAR ? f2_mul(a.hi, A) : f2_fma(a.hi, A, f2_mul(a.lo, A));
      rest = f2_add(rest, y);
    }
  }
  __device__ __forceinline__ f2 value() const { return DECAY == kRecSigmoid ? f2_add(A, rest) : A; }
  __device__ __forceinline__ void end(Map& m) const {
    if (DECAY == kRecSigmoid) {
      m.A = A, m.Al = rest;
    } else {
      const Decay a = decay_of_log<false>(rest);
      m.A = a.hi, m.Al = a.lo;
    }
  }
};

// ---- a token's pair of channels -------------------------------------------------
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
__device__ __forceinline__ f2 minus_pair_at(const float* p) { return f2_mul(pair_at<float>(p), f2_both(-1.f)); }
__device__ __forceinline__ f2 minus_pair_at(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p) ^ 0x80008000u;
  return f2_make(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void put_pair(float* p, f2 v) { *reinterpret_cast<f2*>(p) = v; }
__device__ __forceinline__ void put_pair(__nv_bfloat16* p, f2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f2_lo(v), f2_hi(v));
}
// Stores those of a pair that are not finite.
template <typename T>
__device__ __forceinline__ void put_odd(T* p, f2 v) {
  if (!isfinite(f2_lo(v))) p[0] = from_f32<T>(f2_lo(v));
  if (!isfinite(f2_hi(v))) p[1] = from_f32<T>(f2_hi(v));
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
template <typename IO, int THREADS, int TILE>
struct Copier {
  static constexpr int VE = 16 / sizeof(IO), GROUPS = kChans / VE, ROWS = THREADS / GROUPS;
  __device__ __forceinline__ static int group() { return threadIdx.x % GROUPS * VE; }
  __device__ __forceinline__ static int row() { return threadIdx.x / GROUPS; }
  // tokens [t0, t0 + TILE) of the stream, `src` its thread's channels of token 0, into `dst`; behind T, `fill`s
  __device__ __forceinline__ static void tile(IO* dst, const IO* src, long long st, int t0, int T, uint32_t fill) {
    dst += row() * kChans + group();
    src += (long long)(t0 + row()) * st;
    const long long down = ROWS * st;
    if (T - t0 >= TILE) {
#pragma unroll
      for (int r = 0; r < TILE; r += ROWS, src += down) cp_async16(dst + r * kChans, src);
    } else {
#pragma unroll
      for (int r = 0; r < TILE; r += ROWS, src += down) {
        if (row() + r < T - t0) cp_async16(dst + r * kChans, src);
        else *reinterpret_cast<uint4*>(dst + r * kChans) = make_uint4(fill, fill, fill, fill);
      }
    }
  }
};

// What stands for g behind the last token: a decay of one.
template <typename IO, int DECAY>
__device__ __forceinline__ uint32_t still() {
  if (DECAY == kRecLog) return 0;
  if (sizeof(IO) == 2) return DECAY == kRecSigmoid ? 0x7f807f80u : 0xff80ff80u;  // ±∞
  return DECAY == kRecSigmoid ? 0x7f800000u : 0xff800000u;
}

// ---- clusters ------------------------------------------------------------------
// (`arrive` for a block that has stored in the others' shared memory before it, `arrive_only` for one that has not)
__device__ __forceinline__ void cluster_arrive_only() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores a pair at the place of `p` (this block's shared memory) in the block of rank `rank`.
__device__ __forceinline__ void put_remote(const void* p, int rank, f2 v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

__device__ __forceinline__ void put_remote(const void* p, int rank, uint32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// The maps of a cluster's blocks, [2][k], in two halves, used in turn, so that one barrier a step is enough.
// Al, which is 2^-24 of A at most, in bf16: eight bits of it are enough, and more blocks fit an SM.
struct BlockMap {
  f2 A[32], S[32];
  uint32_t Al[32];
  __device__ __forceinline__ f2 of(int lane, f2 h) const {
    const uint32_t l = Al[lane];
    return apply<false>(A[lane], f2_make(__uint_as_float(l << 16), __uint_as_float(l & 0xffff0000u)), S[lane], h);
  }
  // into the same place of the block of rank `rank`
  __device__ __forceinline__ void put(int lane, int rank, const Map& m) {
    const __nv_bfloat162 l = __floats2bfloat162_rn(f2_lo(m.Al), f2_hi(m.Al));
    put_remote(&A[lane], rank, m.A);
    put_remote(&S[lane], rank, m.S);
    put_remote(&Al[lane], rank, *reinterpret_cast<const uint32_t*>(&l));
  }
};
__host__ __device__ constexpr size_t block_maps_bytes(int k) { return k > 1 ? 2 * (size_t)k * sizeof(BlockMap) : 0; }

inline cudaLaunchConfig_t cluster_config(unsigned blocks, int k, int threads, size_t smem, cudaLaunchAttribute* attr,
                                         cudaStream_t s) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = (unsigned)k;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem + block_maps_bytes(k);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of k blocks that the current device holds at once, asked for once a kernel, size and device.
template <auto KERNEL, int THREADS, size_t SMEM>
int clusters_at_once(int device, int k) {
  static std::atomic<int> known[64][kRecMaxCluster + 1];  // count + 1
  const bool keep = device >= 0 && device < 64;
  int n = keep ? known[device][k].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n - 1;
  if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(SMEM + block_maps_bytes(kRecMaxCluster))) !=
          cudaSuccess ||
      cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return -1;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = cluster_config(k, k, THREADS, SMEM, attr, nullptr);
  if (cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg) != cudaSuccess) return -1;
  if (keep) known[device][k].store(n + 1, std::memory_order_relaxed);
  return n;
}

// Launches `tiles` clusters of as many blocks as there are tiles `along` the
// sequence, as far as the device holds all clusters at once: a second wave
// would take as long as the first. `used`: the blocks of a cluster.
template <auto KERNEL, int THREADS, size_t SMEM, typename Args>
cudaError_t launch_clusters(const Args& a, int tiles, int along, int* used, cudaStream_t s) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  constexpr int sizes[] = {16, 12, 8, 7, 6, 5, 4, 3, 2, 1};  // above eight, 12 and 16: of 12 the device holds 432 bf16 blocks of the
                                                            // forward kernel in all, of 9 to 15 else 364 to 430; 16 goes the furthest
  static_assert(sizes[0] == kRecMaxCluster, "the largest");
  int k = 1;
  for (int n : sizes) {
    if (n > along && n > 1) continue;
    const int most = clusters_at_once<KERNEL, THREADS, SMEM>(device, n);
    if (most < 0) return cudaGetLastError();
    if (tiles <= most) {
      k = n;
      break;
    }
  }
  if (used) *used = k;
  if (k == 1) {
    KERNEL<<<(unsigned)tiles, THREADS, SMEM, s>>>(a, 1);
    return cudaGetLastError();
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = cluster_config((unsigned)tiles * (unsigned)k, k, THREADS, SMEM, attr, s);
  e = cudaLaunchKernelEx(&cfg, KERNEL, a, k);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rec
}  // namespace kla
