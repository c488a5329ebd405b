// Layer norm with the residual sum before it, and its gradients (sm_103a):
//
//   total = x + residual (rounded as it is stored),  n = (total - mean) r,  y = n w + b,  r = 1 / sqrt(var + ε)
//   gx = gtotal + r (g w - mean(g w) - n mean(g w n)),   gw = Σ g n,  gb = Σ g
//
// Every element is read once and written once, so HBM bounds it. A row stays in
// the registers of its lanes (eight, a warp or a block, by its width), so the
// variance is the mean square of differences from the mean, as exact as the
// mean, at no further reads; the gradients make both again from the row rather
// than read them. Backward a group of lanes goes through rows, the next one on
// its way while one is worked on, and adds up the weight's and the bias's
// gradients of its columns in registers; blocks leave partial sums, and a
// second kernel adds those, both in a fixed order.
#include <algorithm>

#include "kla_device.cuh"
#include "kla_launch.h"

namespace kla {

namespace {

constexpr int kThreads = 256;

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
template <typename IO>
struct Raw<IO, 1> {
  IO v;
  __device__ __forceinline__ void to(float (&x)[1]) const { x[0] = to_f32<IO>(v); }
  __device__ __forceinline__ void from(const float (&x)[1]) { v = from_f32<IO>(x[0]); }
};

// A row over LANES lanes: lane l holds the NV pieces of VEC elements that begin
// at (l + LANES j) VEC. LANES is 8 or 32 (lanes of a warp) or 256 (the block).
template <int LANES>
__device__ __forceinline__ float row_sum(float x, float* space) {
#pragma unroll
  for (int m = 1; m < (LANES < 32 ? LANES : 32); m <<= 1) x += __shfl_xor_sync(~0u, x, m);
  if (LANES > 32) {
    if (threadIdx.x % 32 == 0) space[threadIdx.x / 32] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 32; ++i) x += space[i];
  }
  return x;
}

template <typename IO, int VEC, int NV>
__device__ __forceinline__ void fetch(Raw<IO, VEC> (&r)[NV], const IO* row, int l, int lanes, int D) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = (l + lanes * j) * VEC;
    if (e < D) r[j] = *reinterpret_cast<const Raw<IO, VEC>*>(row + e);
  }
}

// x becomes the normalised row (zero behind its end); returns r. `space`: 16 floats a call.
template <int VEC, int NV, int LANES>
__device__ __forceinline__ float standardise(float (&x)[NV][VEC], int l, int D, float inv_d, float eps, float* space) {
  float s = 0.f, v = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += x[j][i];
  const float mean = row_sum<LANES>(s, space) * inv_d;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = (l + LANES * j) * VEC < D;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      x[j][i] = in ? x[j][i] - mean : 0.f;
      v = fmaf(x[j][i], x[j][i], v);
    }
  }
  const float r = 1.f / sqrtf(fmaf(row_sum<LANES>(v, space + 8), inv_d, eps));
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[j][i] *= r;
  return r;
}

template <typename IO, int VEC, int NV, int LANES>
__global__ void __launch_bounds__(kThreads) kla_layer_norm_kernel(const LayerNormArgs p) {
  using R = Raw<IO, VEC>;
  __shared__ float space[16];
  const int l = threadIdx.x % LANES;
  const long long row = (long long)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const bool on = row < p.rows;
  R a[NV], b[NV];
  float x[NV][VEC];
  if (on) fetch<IO, VEC, NV>(a, reinterpret_cast<const IO*>(p.x) + row * p.x_stride, l, LANES, p.D);
  if (on && p.residual)
    fetch<IO, VEC, NV>(b, reinterpret_cast<const IO*>(p.residual) + row * p.residual_stride, l, LANES, p.D);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = (l + LANES * j) * VEC;
    const bool in = on && e < p.D;
    if (in && p.residual) {
      float u[VEC], v[VEC];
      a[j].to(u);
      b[j].to(v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) u[i] += v[i];
      a[j].from(u);
      *reinterpret_cast<R*>(reinterpret_cast<IO*>(p.total) + row * p.D + e) = a[j];
    }
    if (in) a[j].to(x[j]);
    else
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[j][i] = 0.f;
  }
  standardise<VEC, NV, LANES>(x, l, p.D, p.inv_d, p.eps, space);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = (l + LANES * j) * VEC;
    if (!on || e >= p.D) continue;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float w = p.weight ? p.weight[e + i] : 1.f;
      x[j][i] = p.bias ? fmaf(x[j][i], w, p.bias[e + i]) : x[j][i] * w;
    }
    R y;
    y.from(x[j]);
    *reinterpret_cast<R*>(reinterpret_cast<IO*>(p.y) + row * p.D + e) = y;
  }
}

template <typename IO, int VEC, int NV, int LANES, int THREADS>
__global__ void __launch_bounds__(THREADS) kla_layer_norm_grad_kernel(const LayerNormGradArgs p) {
  using R = Raw<IO, VEC>;
  constexpr int GROUPS = THREADS / LANES;
  __shared__ float space[32];
  const int l = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const long long step = (long long)gridDim.x * GROUPS;
  float gw[NV][VEC] = {}, gb[NV][VEC] = {};
  R nx[NV], ng[NV], nt[NV];
  auto ahead = [&](long long row) {
    if (row >= p.rows) return;
    fetch<IO, VEC, NV>(nx, reinterpret_cast<const IO*>(p.x) + row * p.x_stride, l, LANES, p.D);
    if (p.gy) fetch<IO, VEC, NV>(ng, reinterpret_cast<const IO*>(p.gy) + row * p.gy_stride, l, LANES, p.D);
    if (p.gtotal) fetch<IO, VEC, NV>(nt, reinterpret_cast<const IO*>(p.gtotal) + row * p.gtotal_stride, l, LANES, p.D);
  };
  ahead((long long)blockIdx.x * GROUPS + grp);
  for (long long first = (long long)blockIdx.x * GROUPS; first < p.rows; first += step) {
    const long long row = first + grp;
    const bool on = row < p.rows;
    float x[NV][VEC], g[NV][VEC];
    R t[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = on && (l + LANES * j) * VEC < p.D;
      if (in) nx[j].to(x[j]);
      else
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[j][i] = 0.f;
      if (in && p.gy) ng[j].to(g[j]);
      else
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[j][i] = 0.f;
      t[j] = nt[j];
    }
    ahead(row + step);
    const float r = standardise<VEC, NV, LANES>(x, l, p.D, p.inv_d, p.eps, space);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = (l + LANES * j) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        gw[j][i] = fmaf(g[j][i], on ? x[j][i] : 0.f, gw[j][i]);
        gb[j][i] += g[j][i];
        if (p.weight && e < p.D) g[j][i] *= p.weight[e + i];
        s1 += g[j][i];
        s2 = fmaf(g[j][i], x[j][i], s2);
      }
    }
    s1 = row_sum<LANES>(s1, space + 16) * p.inv_d;
    s2 = row_sum<LANES>(s2, space + 24) * p.inv_d;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = (l + LANES * j) * VEC;
      if (!on || e >= p.D) continue;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = r * (g[j][i] - fmaf(x[j][i], s2, s1));
      if (p.gtotal) {
        float u[VEC];
        t[j].to(u);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] += u[i];
      }
      R y;
      y.from(o);
      *reinterpret_cast<R*>(reinterpret_cast<IO*>(p.gx) + row * p.D + e) = y;
    }
  }
  if (!p.part) return;
  // the block's sums of its groups, a group after the other
  extern __shared__ float sums[];  // [2][D]
  for (int n = 0; n < GROUPS; ++n) {
    if (n == grp) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int e = (l + LANES * j) * VEC + i;
          if (e < p.D) {
            sums[e] = n ? sums[e] + gw[j][i] : gw[j][i];
            sums[p.D + e] = n ? sums[p.D + e] + gb[j][i] : gb[j][i];
          }
        }
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < 2 * p.D; e += THREADS) p.part[(long long)blockIdx.x * 2 * p.D + e] = sums[e];
}

// Sums the blocks' partials: 32 columns a block, its warps over the blocks.
__global__ void __launch_bounds__(kThreads) kla_layer_norm_sum_kernel(const LayerNormGradArgs p, int blocks) {
  __shared__ float sums[kThreads / 32][33];
  const int w = threadIdx.x / 32, c = blockIdx.x * 32 + threadIdx.x % 32;
  float x = 0.f;
  if (c < 2 * p.D)
    for (int b = w; b < blocks; b += kThreads / 32) x += p.part[(long long)b * 2 * p.D + c];
  sums[w][threadIdx.x % 32] = x;
  __syncthreads();
  if (w == 0 && c < 2 * p.D) {
    for (int i = 1; i < kThreads / 32; ++i) x += sums[i][threadIdx.x];
    float* out = c < p.D ? p.gweight : p.gbias;
    if (out) out[c < p.D ? c : c - p.D] = x;
  }
}

// Lanes a row and pieces a lane, by the row's width in pieces of VEC.
template <typename F>
void by_width(int pieces, bool vec, F f) {
  using std::integral_constant;
#define KLA_LN(NV, LANES) return f(integral_constant<int, NV>(), integral_constant<int, LANES>())
  if (vec) {
    if (pieces <= 8) KLA_LN(1, 8);
    if (pieces <= 32) KLA_LN(1, 32);
    if (pieces <= 64) KLA_LN(2, 32);
    if (pieces <= 128) KLA_LN(4, 32);
    if (pieces <= 256) KLA_LN(1, 256);
    if (pieces <= 512) KLA_LN(2, 256);
    if (pieces <= 1024) KLA_LN(4, 256);
    KLA_LN(8, 256);
  }
  if (pieces <= 128) KLA_LN(4, 32);
  if (pieces <= 1024) KLA_LN(32, 32);
  KLA_LN(32, 256);
#undef KLA_LN
}

constexpr int kGradThreads = 128;
template <int LANES>
constexpr int grad_threads() { return LANES > 32 ? LANES : kGradThreads; }

// Blocks of the gradients' kernel: as many as the device holds at once, for each leaves partial sums.
int grad_blocks(long long rows, int lanes, int num_sms) {
  const int groups = (lanes > 32 ? lanes : kGradThreads) / lanes;
  return (int)std::max(1LL, std::min((rows + groups - 1) / groups, (long long)num_sms * (lanes > 32 ? 2 : 4)));
}

// Rows that all begin on 16 bytes.
struct Rows {
  const void* p;
  long long stride;
};
template <typename IO>
bool vector_rows(int D, std::initializer_list<Rows> all) {
  constexpr int VE = 16 / sizeof(IO);
  if (D % VE) return false;
  for (const Rows& r : all)
    if (r.p && (r.stride % VE || reinterpret_cast<uintptr_t>(r.p) % 16)) return false;
  return true;
}

template <typename IO>
cudaError_t launch_io(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(IO);
  const bool vec = vector_rows<IO>(a.D, {{a.x, a.x_stride}, {a.residual, a.residual_stride}, {a.y, a.D},
                                         {a.total, a.D}});
  by_width(vec ? a.D / VE : a.D, vec, [&](auto nv, auto lanes) {
    constexpr int NV = decltype(nv)::value, LANES = decltype(lanes)::value, G = kThreads / LANES;
    const unsigned blocks = (unsigned)((a.rows + G - 1) / G);
    if constexpr (NV <= 8)
      if (vec) return (void)(kla_layer_norm_kernel<IO, VE, NV, LANES><<<blocks, kThreads, 0, s>>>(a));
    if constexpr (NV == 32 || (NV == 4 && LANES == 32))
      kla_layer_norm_kernel<IO, 1, NV, LANES><<<blocks, kThreads, 0, s>>>(a);
  });
  return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_io(const LayerNormGradArgs& a, int num_sms, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(IO);
  const bool vec = vector_rows<IO>(a.D, {{a.x, a.x_stride}, {a.gy, a.gy_stride}, {a.gtotal, a.gtotal_stride},
                                         {a.gx, a.D}});
  int blocks = 0;
  cudaError_t e = cudaSuccess;
  by_width(vec ? a.D / VE : a.D, vec, [&](auto nv, auto lanes) {
    constexpr int NV = decltype(nv)::value, LANES = decltype(lanes)::value, THREADS = grad_threads<LANES>();
    blocks = grad_blocks(a.rows, LANES, num_sms);
    const size_t smem = a.part ? 2 * (size_t)a.D * sizeof(float) : 0;
    auto go = [&](auto kernel) {
      if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e == cudaSuccess) kernel<<<blocks, THREADS, smem, s>>>(a);
    };
    if constexpr (NV <= 8)
      if (vec) return go(kla_layer_norm_grad_kernel<IO, VE, NV, LANES, THREADS>);
    if constexpr (NV == 32 || (NV == 4 && LANES == 32)) go(kla_layer_norm_grad_kernel<IO, 1, NV, LANES, THREADS>);
  });
  if (e != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess || !a.part) return e;
  kla_layer_norm_sum_kernel<<<(2 * a.D + 31) / 32, kThreads, 0, s>>>(a, blocks);
  return cudaGetLastError();
}

}  // namespace

size_t layer_norm_partial_bytes(long long rows, int D, int num_sms) {
  // the most that any choice of lanes asks for: groups of eight lanes do not for wide rows, but share a block's bound
  return (size_t)std::max(grad_blocks(rows, 256, num_sms), grad_blocks(rows, 32, num_sms)) * 2 * (size_t)D * sizeof(float);
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t s) {
  return a.io == IO_BF16 ? launch_io<__nv_bfloat16>(a, s) : launch_io<float>(a, s);
}

cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, int num_sms, cudaStream_t s) {
  return a.io == IO_BF16 ? launch_io<__nv_bfloat16>(a, num_sms, s) : launch_io<float>(a, num_sms, s);
}

}  // namespace kla
