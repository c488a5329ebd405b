// Layer norm with the residual sum before it, and its gradients (sm_103a):
//
//   total = x + residual (rounded as it is stored),  n = (total - mean) r,  y = n w + b,  r = 1 / sqrt(var + ε)
//   gx = gtotal + r (g w - mean(g w) - n mean(g w n)),   gw = Σ g n,  gb = Σ g
//
// Every element is read once and written once, so HBM bounds it. A row stays in
// the registers of its lanes (eight to all of a block's, by its width), so the
// variance is the mean square of differences from the mean, as exact as the
// mean, at no further reads; the gradients make both again from the row rather
// than read them. Backward a group of lanes goes through rows, the next ones on
// their way by asynchronous copies meanwhile, and adds up the weight's and the
// bias's gradients of its columns in registers; blocks leave partial sums, and a
// second kernel adds those, both in a fixed order.
//
// Measured, 32768 rows of 1024 in bf16: with the residual 45.6 us (5.9 TB/s), the
// gradients 47 us and 5 for the sums (before: 86 with the next row in registers and
// a warp a row, where 254 registers left eight warps an SM; 56 with sums of one
// thread a block; three blocks of two rows at a time, 164 registers, are faster
// than four of 128, which spill). Rows that do not all begin on 16 bytes are read in
// pairs where they are bf16 and all begin on four (38972 of 446 with the residual: 26
// us, by elements 34; gradients of 20000: 20, by elements 24, by copies of four bytes
// 21), else an element at a time (8188 of 517 in fp32, gradients 14 us and 5).
#include <algorithm>

#include "kla_device.cuh"
#include "kla_launch.h"
#include "kla_prepare.cuh"

namespace kla {

namespace {

// VEC elements of a row as they lie in memory.
template <typename IO, int VEC>
struct Raw;
template <>
struct Raw<float, 4> {
  float4 v;
  __device__ __forceinline__ void to(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
  __device__ __forceinline__ void from(const float (&x)[4]) { v = make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void to(float (&x)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  __device__ __forceinline__ void from(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    v = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void to(float (&x)[2]) const { x[0] = __uint_as_float(v << 16), x[1] = __uint_as_float(v & 0xffff0000u); }
  __device__ __forceinline__ void from(const float (&x)[2]) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(x[0], x[1]);
    v = *reinterpret_cast<const uint32_t*>(&y);
  }
};
template <typename IO>
struct Raw<IO, 1> {
  IO v;
  __device__ __forceinline__ void to(float (&x)[1]) const { x[0] = to_f32<IO>(v); }
  __device__ __forceinline__ void from(const float (&x)[1]) { v = from_f32<IO>(x[0]); }
};

// VEC floats of the weight or the bias.
template <int VEC>
__device__ __forceinline__ void params(const float* p, float (&w)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (VEC == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *p;
  }
}

// A row over LANES lanes: lane l holds the NV pieces of VEC elements that begin
// at (l + LANES j) VEC. LANES is 8 or 32 (lanes of a warp), or some warps of the
// block, its part `grp`. Sums N values over a row; `space`: N floats for
// each of the row's warps, others at the next call.
template <int LANES, int THREADS, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float* space, int grp) {
  static_assert(N == 1 || N == 2, "one sum or two");
  constexpr int W = LANES < 32 ? LANES : 32;
  if constexpr (N == 2) {  // even lanes go on with one sum, odd lanes with the other
    const bool odd = threadIdx.x & 1;
    const float other = __shfl_xor_sync(~0u, odd ? x[0] : x[1], 1);
    float s = (odd ? x[1] : x[0]) + other;
#pragma unroll
    for (int m = 2; m < W; m <<= 1) s += __shfl_xor_sync(~0u, s, m);
    if constexpr (LANES > 32) {
      if (threadIdx.x % 32 < 2) space[threadIdx.x % LANES / 32 * 2 + threadIdx.x % 32] = s;
    } else {
      const float t = __shfl_xor_sync(~0u, s, 1);
      x[0] = odd ? t : s, x[1] = odd ? s : t;
    }
  } else {
#pragma unroll
    for (int m = 1; m < W; m <<= 1) x[0] += __shfl_xor_sync(~0u, x[0], m);
    if constexpr (LANES > 32)
      if (threadIdx.x % 32 == 0) space[threadIdx.x % LANES / 32] = x[0];
  }
  if constexpr (LANES > 32) {
    if (LANES == THREADS) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "n"(LANES) : "memory");
#pragma unroll
    for (int n = 0; n < N; ++n) {
      x[n] = space[n];
#pragma unroll
      for (int i = 1; i < LANES / 32; ++i) x[n] += space[i * N + n];
    }
  }
}

template <typename IO, int VEC, int NV>
__device__ __forceinline__ void fetch(Raw<IO, VEC> (&r)[NV], const IO* row, int l, int lanes, int D) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = (l + lanes * j) * VEC;
    if (e < D) r[j] = *reinterpret_cast<const Raw<IO, VEC>*>(row + e);
  }
}

template <typename IO, int VEC, int NV, int LANES, int THREADS>
__global__ void __launch_bounds__(THREADS) kla_layer_norm_kernel(const LayerNormArgs p) {
  using R = Raw<IO, VEC>;
  __shared__ float space[2][THREADS / 32];
  const int l = threadIdx.x % LANES;
  const long long row = (long long)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const bool on = row < p.rows;
  R a[NV], b[NV];
  float x[NV][VEC], s[1] = {0.f}, v[1] = {0.f};
  if (on) fetch<IO, VEC, NV>(a, reinterpret_cast<const IO*>(p.x) + row * p.x_stride, l, LANES, p.D);
  if (on && p.residual)
    fetch<IO, VEC, NV>(b, reinterpret_cast<const IO*>(p.residual) + row * p.residual_stride, l, LANES, p.D);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = (l + LANES * j) * VEC;
    const bool in = on && e < p.D;
    if (in && p.residual) {
      float u[VEC], w[VEC];
      a[j].to(u);
      b[j].to(w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) u[i] += w[i];
      a[j].from(u);
      *reinterpret_cast<R*>(reinterpret_cast<IO*>(p.total) + row * p.D + e) = a[j];
    }
    if (in) a[j].to(x[j]);
    else
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j][i] = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[0] += x[j][i];
  }
  row_sums<LANES, THREADS>(s, space[0], 0);
  const float mean = s[0] * p.inv_d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = (l + LANES * j) * VEC < p.D;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      x[j][i] -= mean;
      if (in) v[0] = fmaf(x[j][i], x[j][i], v[0]);
    }
  }
  row_sums<LANES, THREADS>(v, space[1], 0);
  const float r = 1.f / sqrtf(fmaf(v[0], p.inv_d, p.eps));
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = (l + LANES * j) * VEC;
    if (!on || e >= p.D) continue;
    float w[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[j][i] *= r;
    if (p.weight) {
      params<VEC>(p.weight + e, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j][i] *= w[i];
    }
    if (p.bias) {
      params<VEC>(p.bias + e, w);
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j][i] += w[i];
    }
    R y;
    y.from(x[j]);
    *reinterpret_cast<R*>(reinterpret_cast<IO*>(p.y) + row * p.D + e) = y;
  }
}

// A thread's pieces of the rows ahead, S - 1 of them on their way by asynchronous
// copies into places that no other thread reads (so nothing waits but the
// copies); two-byte elements and their pairs come through registers, one row
// ahead. What no copy reaches (behind a row's end, a gradient
// that is not there) stays zero.
template <typename IO, int VEC, int NV, int LANES, int THREADS, int S>
struct Ahead {
  using R = Raw<IO, VEC>;
  static constexpr bool ASYNC = sizeof(R) == 16 || sizeof(IO) == 4;
  static constexpr int P = (NV * VEC + 1) / 2;  // pairs of elements a thread
  static constexpr size_t BYTES = ASYNC ? (size_t)S * 3 * NV * THREADS * sizeof(R) : 0;
  R* ring;  // [S][3][NV][THREADS]
  R next[ASYNC ? 1 : 3][ASYNC ? 1 : NV];
  const IO* at[3];
  long long down[3], left;
  int step;
  bool in[NV];  // pieces that the row has
  __device__ __forceinline__ Ahead(unsigned char* smem, const LayerNormGradArgs& p, long long row, int rows_a_step, int l)
      : ring(reinterpret_cast<R*>(smem)), left(p.rows - row), step(rows_a_step) {
    const void* const from[3] = {p.x, p.gy, p.gtotal};
    const long long stride[3] = {p.x_stride, p.gy_stride, p.gtotal_stride};
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      at[s] = from[s] ? reinterpret_cast<const IO*>(from[s]) + row * stride[s] + l * VEC : nullptr;
      down[s] = step * stride[s];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) in[j] = (l + LANES * j) * VEC < p.D;
    float zero[VEC] = {};
    R r;
    r.from(zero);
    if constexpr (ASYNC) {
      for (int i = threadIdx.x; i < S * 3 * NV * THREADS; i += THREADS) ring[i] = r;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) next[0][j] = next[1][j] = next[2][j] = r;
    }
  }
  __device__ __forceinline__ R* place(int stage, int stream, int j) const {
    return ring + ((stage * 3 + stream) * NV + j) * THREADS + threadIdx.x;
  }
  // the next row of the thread's group, `step` rows after the one before
  __device__ __forceinline__ void fetch(int stage) {
    if (left > 0) {
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        if (!at[s]) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (!in[j]) continue;
          const IO* const from = at[s] + LANES * j * VEC;
          if constexpr (sizeof(R) == 16) cp_async16(place(stage, s, j), from);
          else if constexpr (ASYNC)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(place(stage, s, j))), "l"(from) : "memory");
          else next[s][j] = *reinterpret_cast<const R*>(from);
        }
        at[s] += down[s];
      }
    }
    left -= step;
    if (ASYNC) cp_async_commit();
  }
  __device__ __forceinline__ void pairs(int stage, int stream, f2 (&x)[P]) const {
    float v[2 * P];
    if constexpr (NV * VEC % 2) v[2 * P - 1] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float u[VEC];
      if constexpr (ASYNC) place(stage, stream, j)->to(u);
      else next[stream][j].to(u);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j * VEC + i] = u[i];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = f2_make(v[2 * i], v[2 * i + 1]);
  }
};

// Two rounds of sums a row: Σx and Σ g w, then with d = x - mean Σ d² and Σ g w d.
template <typename IO, int VEC, int NV, int LANES, int THREADS, int S, int MIN>
__global__ void __launch_bounds__(THREADS, MIN) kla_layer_norm_grad_kernel(const LayerNormGradArgs p) {
  using R = Raw<IO, VEC>;
  using Rows = Ahead<IO, VEC, NV, LANES, THREADS, S>;
  constexpr int GROUPS = THREADS / LANES, P = Rows::P, E = NV * VEC;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float space[2][THREADS / 32 * 2];
  const int l = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  float* const room = space[0] + grp * (LANES / 32 * 2);
  const int step = gridDim.x * GROUPS;
  const long long first = (long long)blockIdx.x * GROUPS;
  f2 gw[P] = {}, gb[P] = {}, w[P];
  {
    float v[2 * P];
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) {
      const int e = (l + LANES * (i / VEC)) * VEC + i % VEC;
      v[i] = !p.weight || e >= p.D || i >= E ? 1.f : p.weight[e];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = f2_make(v[2 * i], v[2 * i + 1]);
  }
  Rows rows(smem, p, first + grp, step, l);
  if (Rows::ASYNC) __syncthreads();
#pragma unroll
  for (int i = 0; i < (Rows::ASYNC ? S - 1 : 1); ++i) rows.fetch(i);
  int stage = 0;
  for (long long at = first; at < p.rows; at += step) {
    const long long row = at + grp;
    f2 x[P], g[P], t[P], s2 = 0, v2 = 0;
    if (Rows::ASYNC) {
      rows.fetch(stage == 0 ? S - 1 : stage - 1);
      cp_async_wait<S - 1>();
    }
    rows.pairs(stage, 0, x);
    rows.pairs(stage, 1, g);
    if (!Rows::ASYNC) {
      rows.pairs(stage, 2, t);
      rows.fetch(0);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      s2 = f2_add(s2, x[i]);
      v2 = f2_fma(g[i], w[i], v2);
    }
    float s[2] = {f2_lo(s2) + f2_hi(s2), f2_lo(v2) + f2_hi(v2)};
    row_sums<LANES, THREADS>(s, room, grp);
    const float mean = s[0] * p.inv_d;
    s2 = v2 = 0;
    float away[NV];  // zeros behind the row's end stay
#pragma unroll
    for (int j = 0; j < NV; ++j) away[j] = rows.in[j] ? -mean : 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = f2_add(x[i], f2_make(away[2 * i / VEC], 2 * i + 1 < E ? away[(2 * i + 1) / VEC < NV ? (2 * i + 1) / VEC : 0] : 0.f));
      s2 = f2_fma(x[i], x[i], s2);
      v2 = f2_fma(f2_mul(g[i], w[i]), x[i], v2);
    }
    float v[2] = {f2_lo(s2) + f2_hi(s2), f2_lo(v2) + f2_hi(v2)};
    row_sums<LANES, THREADS>(v, room + THREADS / 32 * 2, grp);
    if (row < p.rows) {
      IO* const out = reinterpret_cast<IO*>(p.gx) + row * p.D + l * VEC;
      const float r = 1.f / sqrtf(fmaf(v[0], p.inv_d, p.eps));
      const float rest = -r * (s[1] * p.inv_d), by_n = -r * (v[1] * p.inv_d * r);
      if (Rows::ASYNC && p.gtotal) rows.pairs(stage, 2, t);
      float o[2 * P];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const f2 n = f2_mul(x[i], f2_make(r, r));
        gw[i] = f2_fma(g[i], n, gw[i]);
        gb[i] = f2_add(gb[i], g[i]);
        f2 y = f2_fma(f2_mul(g[i], w[i]), f2_make(r, r), f2_fma(n, f2_make(by_n, by_n), f2_make(rest, rest)));
        if (p.gtotal) y = f2_add(y, t[i]);
        o[2 * i] = f2_lo(y), o[2 * i + 1] = f2_hi(y);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!rows.in[j]) continue;
        float u[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) u[i] = o[j * VEC + i];
        R y;
        y.from(u);
        *reinterpret_cast<R*>(out + LANES * j * VEC) = y;
      }
    }
    if (Rows::ASYNC) stage = stage + 1 == S ? 0 : stage + 1;
  }
  if (!p.part) return;
  // the block's sums of its groups, a group after the other
  float* const part = p.part + (long long)blockIdx.x * 2 * p.D;
  float* const sums = reinterpret_cast<float*>(smem + Rows::BYTES);  // [2][D], where there are groups
  for (int n = 0; n < GROUPS; ++n) {
    if (n == grp) {
      float* const out = n == GROUPS - 1 ? part : sums;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int e = (l + LANES * (i / VEC)) * VEC + i % VEC;
        const float a = i % 2 ? f2_hi(gw[i / 2]) : f2_lo(gw[i / 2]), b = i % 2 ? f2_hi(gb[i / 2]) : f2_lo(gb[i / 2]);
        if (e < p.D) {
          out[e] = n ? sums[e] + a : a;
          out[p.D + e] = n ? sums[p.D + e] + b : b;
        }
      }
    }
    if (GROUPS > 1) __syncthreads();
  }
}

// Sums the blocks' partials: eight columns a block (32 bytes of a partial), its
// 128 rows of threads over the blocks, four loads of a thread on their way at a time.
__global__ void __launch_bounds__(1024) kla_layer_norm_sum_kernel(const LayerNormGradArgs p, int blocks) {
  __shared__ float sums[128][9];
  const int row = threadIdx.x / 8, col = threadIdx.x % 8, c = blockIdx.x * 8 + col, n = 2 * p.D;
  float x = 0.f;
  if (c < n) {
    const float* const part = p.part + c;
    for (int b = row; b < blocks; b += 4 * 128) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = b + 128 * i < blocks ? part[(long long)(b + 128 * i) * n] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) x += v[i];
    }
  }
  sums[row][col] = x;
  __syncthreads();
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32, mine = blockIdx.x * 8 + w;  // a warp adds up one column
  if (w >= 8) return;
  x = (sums[lane][w] + sums[lane + 32][w]) + (sums[lane + 64][w] + sums[lane + 96][w]);
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(~0u, x, m);
  if (lane == 0 && mine < n) {
    float* const out = mine < p.D ? p.gweight : p.gbias;
    if (out) out[mine < p.D ? mine : mine - p.D] = x;
  }
}

// Pieces a lane, lanes a row and threads a block, and backward stages and blocks an SM.
template <int NV_, int LANES_, int THREADS_>
struct Shape {
  static constexpr int NV = NV_, LANES = LANES_, THREADS = THREADS_;
};
template <int NV, int LANES, int THREADS, int S_, int MIN_>
struct BackShape : Shape<NV, LANES, THREADS> {
  static constexpr int S = S_, MIN = MIN_;
};

// Forward, by the row's width in pieces (of 16 bytes; else pairs or single elements): the smallest shape that holds the
// row, as the next one costs more at every step (210 MB of rows of 1024 in pieces of 16 bytes: bf16 37 us with 32 lanes, 39
// with 128; of 2048 with 128 lanes and four pieces 39, with two 35; fp32 rows of 50 elements 40 with eight lanes, 57 with
// 32). Up to 512 pieces, fp32 rows of 501 take 36 us with 128 lanes and 38 with 64, bf16 rows of 411 take 63 and 47.
template <typename IO, int VEC, typename F>
void by_width(int pieces, F f) {
  if constexpr (VEC >= 4) {
    if (pieces <= 8) return f(Shape<1, 8, 256>());
    if (pieces <= 32) return f(Shape<1, 32, 256>());
    if (pieces <= 64) return f(Shape<2, 32, 256>());
    if (pieces <= 128) return f(Shape<4, 32, 256>());
    if (pieces <= 256) return f(Shape<2, 128, 128>());
    if (pieces <= 512) return f(Shape<4, 128, 128>());
    if (pieces <= 1024) return f(Shape<4, 256, 256>());
    return f(Shape<4, 512, 512>());
  } else {
    if (pieces <= 64) return f(Shape<8, 8, 256>());
    if (pieces <= 128) return f(Shape<4, 32, 256>());
    if (pieces <= 256) return f(Shape<8, 32, 256>());
    if (pieces <= 512 && sizeof(IO) == 4) return f(Shape<4, 128, 128>());
    if (pieces <= 512) return f(Shape<8, 64, 64>());
    if (pieces <= 1024) return f(Shape<8, 128, 128>());
    if (pieces <= 2048) return f(Shape<8, 256, 256>());
    if (pieces <= 4096) return f(Shape<8, 512, 512>());
    return f(Shape<16, 512, 512>());
  }
}

// Backward, where a lane also keeps the sums of its columns: more lanes with fewer pieces, but few warps a row, which
// wait for each other twice (5000 rows of 3001 with 16 and 8 warps: 99 and 70 us in fp32, 115 and 46 in bf16; 4000 of
// 4090 in bf16: 59 and 39). The smallest shape that holds the row again (210 MB of bf16 rows of 1024: 41 us, with the next
// shape 65; of 4096: 46 and 69; fp32 rows of 255 elements: 45 and 51, of 1023: 45 and 53; fp32 rows of 1024
// in pieces of 16 bytes would take 38 with the next one, and take 43).
template <int VEC, typename F>
void by_width_back(int pieces, F f) {
  if constexpr (VEC == 8) {
    if (pieces <= 8) return f(BackShape<1, 8, 128, 3, 4>());
    if (pieces <= 32) return f(BackShape<1, 32, 128, 3, 4>());
    if (pieces <= 64) return f(BackShape<2, 32, 128, 3, 3>());
    if (pieces <= 128) return f(BackShape<2, 64, 128, 3, 3>());
    if (pieces <= 256) return f(BackShape<2, 128, 128, 3, 3>());
    if (pieces <= 512) return f(BackShape<4, 128, 128, 2, 2>());
    return f(BackShape<4, 256, 256, 3, 1>());
  } else if constexpr (VEC == 4) {
    if (pieces <= 8) return f(BackShape<1, 8, 128, 3, 4>());
    if (pieces <= 32) return f(BackShape<1, 32, 128, 3, 4>());
    if (pieces <= 64) return f(BackShape<2, 32, 128, 3, 5>());
    if (pieces <= 128) return f(BackShape<4, 32, 128, 3, 3>());
    if (pieces <= 256) return f(BackShape<4, 64, 128, 3, 3>());
    if (pieces <= 512) return f(BackShape<4, 128, 128, 3, 3>());
    if (pieces <= 1024) return f(BackShape<4, 256, 256, 3, 2>());
    return f(BackShape<4, 512, 512, 2, 1>());
  } else if constexpr (VEC == 2) {
    if (pieces <= 128) return f(BackShape<4, 32, 128, 3, 5>());
    if (pieces <= 256) return f(BackShape<4, 64, 128, 3, 4>());
    if (pieces <= 512) return f(BackShape<4, 128, 128, 3, 4>());
    if (pieces <= 1024) return f(BackShape<8, 128, 128, 3, 3>());
    if (pieces <= 2048) return f(BackShape<8, 256, 256, 3, 1>());
    return f(BackShape<8, 512, 512, 2, 1>());
  } else {
    if (pieces <= 128) return f(BackShape<4, 32, 128, 4, 5>());
    if (pieces <= 256) return f(BackShape<8, 32, 128, 3, 4>());
    if (pieces <= 512) return f(BackShape<8, 64, 128, 3, 4>());
    if (pieces <= 640) return f(BackShape<5, 128, 128, 4, 4>());
    if (pieces <= 768) return f(BackShape<6, 128, 128, 4, 4>());
    if (pieces <= 1024) return f(BackShape<8, 128, 128, 3, 4>());
    if (pieces <= 2048) return f(BackShape<16, 128, 128, 3, 2>());
    if (pieces <= 4096) return f(BackShape<16, 256, 256, 2, 1>());
    return f(BackShape<16, 512, 512, 2, 1>());
  }
}

// Blocks of the gradients' kernel: MIN an SM, for each leaves partial sums. That is about as many as the device holds at
// once; with sums, the rings of fp32 rows of 372 to 1024 let an SM hold two for MIN = 3, and of 2052 to 4096 one for two.
template <typename Sh>
int grad_blocks(long long rows, int num_sms) {
  constexpr int groups = Sh::THREADS / Sh::LANES;
  return (int)std::max(1LL, std::min((rows + groups - 1) / groups, (long long)num_sms * Sh::MIN));
}

// Calls f with the elements of a piece: 16 bytes where all rows begin on them, else of two-byte elements pairs where
// all rows begin on four bytes, else one.
struct Rows {
  const void* p;
  long long stride;
};
template <typename IO, typename F>
void by_piece(int D, std::initializer_list<Rows> all, F f) {
  auto fits = [&](int elements) {
    if (D % elements) return false;
    for (const Rows& r : all)
      if (r.p && (r.stride % elements || reinterpret_cast<uintptr_t>(r.p) % (elements * sizeof(IO)))) return false;
    return true;
  };
  constexpr int VE = 16 / sizeof(IO);
  if (fits(VE)) return f(std::integral_constant<int, VE>());
  if constexpr (sizeof(IO) == 2)
    if (fits(2)) return f(std::integral_constant<int, 2>());
  f(std::integral_constant<int, 1>());
}

template <typename IO>
cudaError_t launch_io(const LayerNormArgs& a, cudaStream_t s) {
  auto go = [&](auto ve, auto shape) {
    using Sh = decltype(shape);
    constexpr int G = Sh::THREADS / Sh::LANES;
    const unsigned blocks = (unsigned)((a.rows + G - 1) / G);
    kla_layer_norm_kernel<IO, decltype(ve)::value, Sh::NV, Sh::LANES, Sh::THREADS><<<blocks, Sh::THREADS, 0, s>>>(a);
  };
  by_piece<IO>(a.D, {{a.x, a.x_stride}, {a.residual, a.residual_stride}, {a.y, a.D}, {a.total, a.D}}, [&](auto ve) {
    by_width<IO, decltype(ve)::value>(a.D / ve, [&](auto shape) { go(ve, shape); });
  });
  return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_io(const LayerNormGradArgs& a, int num_sms, cudaStream_t s) {
  int blocks = 0;
  cudaError_t e = cudaSuccess;
  auto go = [&](auto ve, auto shape) {
    using Sh = decltype(shape);
    constexpr int V = decltype(ve)::value;
    constexpr auto kernel = kla_layer_norm_grad_kernel<IO, V, Sh::NV, Sh::LANES, Sh::THREADS, Sh::S, Sh::MIN>;
    constexpr size_t ring = Ahead<IO, V, Sh::NV, Sh::LANES, Sh::THREADS, Sh::S>::BYTES;
    constexpr bool groups = Sh::LANES < Sh::THREADS;  // which add up their sums in shared memory
    constexpr size_t most = ring + (groups ? 2 * Sh::LANES * Sh::NV * V * sizeof(float) : 0);
    const size_t smem = ring + (a.part && groups ? 2 * (size_t)a.D * sizeof(float) : 0);
    blocks = grad_blocks<Sh>(a.rows, num_sms);
    if constexpr (most > 40 * 1024) e = prepare_kernel<kernel>(most);
    if (e == cudaSuccess) kernel<<<blocks, Sh::THREADS, smem, s>>>(a);
  };
  by_piece<IO>(a.D, {{a.x, a.x_stride}, {a.gy, a.gy_stride}, {a.gtotal, a.gtotal_stride}, {a.gx, a.D}}, [&](auto ve) {
    by_width_back<decltype(ve)::value>(a.D / ve, [&](auto shape) { go(ve, shape); });
  });
  if (e != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess || !a.part) return e;
  kla_layer_norm_sum_kernel<<<(2 * a.D + 7) / 8, 1024, 0, s>>>(a, blocks);
  return cudaGetLastError();
}

}  // namespace

size_t layer_norm_partial_bytes(long long rows, int D, int num_sms) {
  int most = 0;  // of rows in pieces of any kind
  auto count = [&](auto shape) { most = std::max(most, grad_blocks<decltype(shape)>(rows, num_sms)); };
  by_width_back<1>(D, count);
  if (D % 2 == 0) by_width_back<2>(D / 2, count);
  if (D % 4 == 0) by_width_back<4>(D / 4, count);
  if (D % 8 == 0) by_width_back<8>(D / 8, count);
  return (size_t)most * 2 * (size_t)D * sizeof(float);
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
  return a.io == IO_BF16 ? launch_io<__nv_bfloat16>(a, s) : launch_io<float>(a, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, int num_sms, cudaStream_t s) {
  return a.io == IO_BF16 ? launch_io<__nv_bfloat16>(a, num_sms, s) : launch_io<float>(a, num_sms, s);
}

}  // namespace kla
