// Norm of queries and keys for each head, with the position rotation in the
// same pass, and its gradients (sm_103a):
//
//   n = x r w,  r = 1 / sqrt(mean(x²) + ε)  (RMS)  or  1 / sqrt(Σx² + ε)  (L2)  or 1
//   y = n with its first 2R entries turned pairwise by the angle pos · f_i
//       (and scaled by rot_scale): pairs (i, i + R) or (2i, 2i + 1)
//
// backward, with gn the rotation's transpose applied to gy and gw = gn w:
//   gx = r (gw − x r² (gw·x) / n_eff),   dL/dw = Σ gn x r    (n_eff = D for RMS, 1 for L2)
//
// Every element is read once and written once, so HBM bounds it. A row of a
// head is held by a group of lanes, 16 bytes a lane; the sum of squares is a
// few lane exchanges, and the other member of a pair is in the lane itself
// (neighbouring pairs) or one exchange away (halves). A group keeps one token
// and goes through heads, so that the angles, which cost more than the rest
// of a row, are computed once for all heads of the group. Input strides are
// free: a projection's [B,T,H,D] is read in place and leaves as [B,H,T,D].
//
// Angles: pos·f / 2π is formed from f/2π as an unevaluated sum of floats, each
// term's whole turns taken off exactly, and the rest given to sincospif, so
// that a position of billions is as exact as the first.
#include <algorithm>

#include "kla_device.cuh"
#include "kla_launch.h"

namespace kla {

namespace {

constexpr int kThreads = 256;
constexpr int kNormNone = 0, kNormRms = 1;  // else L2

// 16 bytes of a row as fp32
template <typename IO>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const float* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* x) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};

__device__ __forceinline__ float fraction(float x) { return x - rintf(x); }

// The part of a turn that pos·f leaves: in [-0.5, 0.5] turns, for |pos| < 2^44.
__device__ __forceinline__ float turn_of(long long pos, float f) {
  // 1/2π = k0 + k1 + k2 (to 2^-78), and f/2π = h + l + m
  constexpr float k0 = 0x1.45f306p-3f, k1 = 0x1.b9391p-28f, k2 = 0x1.529fc2p-54f;
  const float h = f * k0, e = fmaf(f, k0, -h);
  const float h1 = f * k1, e1 = fmaf(f, k1, -h1);
  const float l = e + h1, m = ((e - (l - h1)) + (h1 - (l - (l - h1)))) + e1 + f * k2;
  // pos = p1·2^20 + p0, both exact in fp32
  const float part[2] = {(float)(pos & 0xfffff), (float)(pos >> 20) * 1048576.f};
  float turn = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float p = part[i];
    const float x = p * h, xe = fmaf(p, h, -x);  // p·h = x + xe exactly, and the same for l
    const float y = p * l, ye = fmaf(p, l, -y);
    turn += (fraction(x) + fraction(xe)) + (fraction(y) + fmaf(p, m, ye));
  }
  return fraction(turn);
}

// The angles of a lane's elements, as y = x·c + other·s with the sign of the
// element's place in its pair in s.
template <int VE>
__device__ __forceinline__ void angles(const NormRopeArgs& a, long long pos, int e0, float* c, float* s) {
  const int R = a.rot / 2;
#pragma unroll
  for (int j = 0; j < VE; ++j) {
    const int e = e0 + j;
    c[j] = 1.f;
    s[j] = 0.f;
    if (e < a.rot) {
      const int i = a.layout ? e / 2 : (e < R ? e : e - R);
      const bool first = a.layout ? !(e & 1) : e < R;
      float sn, cs;
      sincospif(2.f * turn_of(pos, a.inv_freq[i]), &sn, &cs);
      c[j] = cs * a.rot_scale;
      s[j] = (first ? -sn : sn) * a.rot_scale;
    }
  }
}

// The other members of a lane's pairs. `aligned`: R is a multiple of the lane's elements (halves).
template <int VE>
__device__ __forceinline__ void others(const NormRopeArgs& a, int lane_in_row, bool aligned, float* row, const float* x,
                                       float* o) {
  const int R = a.rot / 2, e0 = lane_in_row * VE;
  if (a.layout) {
#pragma unroll
    for (int j = 0; j < VE; ++j) o[j] = x[j ^ 1];
  } else if (aligned) {
    const int d = R / VE;
    const int lane = threadIdx.x & 31;
    const int from = e0 < R ? lane + d : (e0 < a.rot ? lane - d : lane);
#pragma unroll
    for (int j = 0; j < VE; ++j) o[j] = __shfl_sync(~0u, x[j], from);
  } else {  // through the group's row in shared memory
#pragma unroll
    for (int j = 0; j < VE; ++j) row[e0 + j] = x[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const int e = e0 + j;
      o[j] = e < R ? row[e + R] : (e < a.rot ? row[e - R] : 0.f);
    }
    __syncwarp();
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) x += __shfl_xor_sync(~0u, x, m);
  return x;
}

__device__ __forceinline__ float inv_size(const NormRopeArgs& a, float sum) {
  if (a.norm == kNormNone) return 1.f;
  return 1.0f / sqrtf((a.norm == kNormRms ? sum / (float)a.D : sum) + a.eps);
}

// A group of LPR lanes: one token, a range of the heads of q followed by those
// of k. BWD also sums the weight gradients of the block.
template <typename IO, int D, bool BWD>
__global__ void __launch_bounds__(kThreads) kla_norm_rope_kernel(const NormRopeArgs a, int splits) {
  constexpr int VE = Vec<IO>::N, LPR = D / VE, GROUPS = kThreads / LPR;
  __shared__ float rows[GROUPS][D];
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR, e0 = l * VE;
  const bool aligned = (a.rot / 2) % VE == 0;
  const int heads = a.q.H + a.k.H, per = (heads + splits - 1) / splits;
  const long long tokens = (long long)a.B * a.T;
  float accq[BWD ? VE : 1] = {}, acck[BWD ? VE : 1] = {};
  // whole blocks step together, so that every lane of a warp takes part in its exchanges
  const long long total = tokens * splits, stride = (long long)gridDim.x * GROUPS;
  for (long long base = (long long)blockIdx.x * GROUPS; base < total; base += stride) {
    const long long job = base + grp;
    const bool live = job < total;
    const long long tok = live ? job % tokens : 0;
    const int h0 = live ? (int)(job / tokens) * per : 0, h1 = live ? min(heads, h0 + per) : 0;
    const int b = (int)(tok / a.T);
    const long long t = tok % a.T;
    float c[VE], s[VE];
    if (a.rot) angles<VE>(a, a.positions ? a.positions[tok] : a.offset + t, e0, c, s);
    for (int i = 0; i < per; ++i) {
      const int hh = h0 + i;
      const bool on = hh < h1;
      const bool isq = hh < a.q.H;
      const NormRopeTensor& p = isq ? a.q : a.k;
      const int h = isq ? hh : hh - a.q.H;
      const long long xi = b * p.sb + h * p.sh + t * p.st + e0;
      const long long yi = (((long long)b * p.H + h) * a.T + t) * D + e0;
      float x[VE], w[VE], y[VE], o[VE];
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = 0.f, w[j] = 1.f;
      if (on) {
        Vec<IO>::load(reinterpret_cast<const IO*>(p.x) + xi, x);
        if (p.w)
#pragma unroll
          for (int j = 0; j < VE; ++j) w[j] = p.w[e0 + j];
      }
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < VE; ++j) sum = fmaf(x[j], x[j], sum);
      const float total_sq = row_sum<LPR>(sum);
      const float r = on ? inv_size(a, total_sq) : 0.f;  // idle lanes add nothing, whatever ε is
      if (!BWD) {
#pragma unroll
        for (int j = 0; j < VE; ++j) y[j] = x[j] * r * w[j];
        if (a.rot) {
          others<VE>(a, l, aligned, rows[grp], y, o);
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (e0 + j < a.rot) y[j] = fmaf(y[j], c[j], o[j] * s[j]);
        }
        if (on) Vec<IO>::store(reinterpret_cast<IO*>(p.y) + yi, y);
      } else {
        float g[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) g[j] = 0.f;
        if (on && p.gy) Vec<IO>::load(reinterpret_cast<const IO*>(p.gy) + yi, g);
        if (a.rot) {  // the transpose: the same cosines, the sines' sign turned
          others<VE>(a, l, aligned, rows[grp], g, o);
#pragma unroll
          for (int j = 0; j < VE; ++j)
            if (e0 + j < a.rot) g[j] = fmaf(g[j], c[j], -o[j] * s[j]);
        }
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const float xr = x[j] * r;
          if (isq) accq[j] = fmaf(g[j], xr, accq[j]);
          else acck[j] = fmaf(g[j], xr, acck[j]);
          g[j] *= w[j];
          dot = fmaf(g[j], xr, dot);
        }
        dot = row_sum<LPR>(dot);
        if (a.norm == kNormNone) dot = 0.f;
        else if (a.norm == kNormRms) dot /= (float)D;
#pragma unroll
        for (int j = 0; j < VE; ++j) y[j] = r * (g[j] - x[j] * r * dot);
        if (on) Vec<IO>::store(reinterpret_cast<IO*>(p.gx) + b * p.gsb + h * p.gsh + t * p.gst + e0, y);
      }
    }
  }
  if (BWD && a.part) {  // the block's weight gradients, in a fixed order
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < VE; ++j) rows[grp][e0 + j] = m ? acck[j] : accq[j];
      __syncthreads();
      for (int i = threadIdx.x; i < D; i += kThreads) {
        float x = 0.f;
        for (int n = 0; n < GROUPS; ++n) x += rows[n][i];
        a.part[((size_t)blockIdx.x * 2 + m) * D + i] = x;
      }
    }
  }
}

// Sums the blocks' partials: one warp per weight, lanes over blocks, then exchanges.
__global__ void __launch_bounds__(32) kla_norm_rope_sum_kernel(const NormRopeArgs a, int blocks) {
  const int i = blockIdx.x % a.D, m = blockIdx.x / a.D;
  float* out = m ? a.gwk : a.gwq;
  if (!out) return;
  float x = 0.f;
  for (int b = threadIdx.x; b < blocks; b += 32) x += a.part[((size_t)b * 2 + m) * a.D + i];
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  if (threadIdx.x == 0) out[i] = x;
}

// How many groups share a token's heads, and the blocks. A token's angles cost
// about as much as several rows, so a group takes all heads unless that leaves
// the device short of warps (about 32 an SM).
void geometry(int B, int heads, int T, int D, int io, int num_sms, bool bwd, int* splits, unsigned* blocks) {
  const long long gpb = kThreads * (io == IO_BF16 ? 8 : 4) / D, tokens = (long long)B * T;
  const long long want = (long long)num_sms * 4 * gpb;
  long long s = tokens > 0 ? (want + tokens - 1) / tokens : 1;
  s = std::min<long long>(std::max<long long>(s, 1), std::max(heads, 1));
  const long long per = (heads + s - 1) / s;
  s = per > 0 ? (heads + per - 1) / per : 1;
  *splits = (int)s;
  long long n = (tokens * s + gpb - 1) / gpb;
  n = std::min<long long>(n, bwd ? num_sms * 8LL : 1LL << 30);
  *blocks = (unsigned)std::max<long long>(n, 1);
}

template <typename IO, bool BWD>
void launch_d(const NormRopeArgs& a, int splits, unsigned blocks, cudaStream_t s) {
  switch (a.D) {
    case 16: kla_norm_rope_kernel<IO, 16, BWD><<<blocks, kThreads, 0, s>>>(a, splits); break;
    case 32: kla_norm_rope_kernel<IO, 32, BWD><<<blocks, kThreads, 0, s>>>(a, splits); break;
    case 64: kla_norm_rope_kernel<IO, 64, BWD><<<blocks, kThreads, 0, s>>>(a, splits); break;
    default: kla_norm_rope_kernel<IO, 128, BWD><<<blocks, kThreads, 0, s>>>(a, splits); break;
  }
}

}  // namespace

size_t norm_rope_partial_bytes(int B, int Hq, int Hk, int T, int D, int num_sms) {
  unsigned blocks = 0, most = 0;
  int splits = 0;
  for (int io = 0; io < 2; ++io) {
    geometry(B, Hq + Hk, T, D, io, num_sms, true, &splits, &blocks);
    most = std::max(most, blocks);
  }
  return (size_t)most * 2 * D * sizeof(float);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, int num_sms, cudaStream_t s) {
  int splits = 0;
  unsigned blocks = 0;
  geometry(a.B, a.q.H + a.k.H, a.T, a.D, a.io, num_sms, false, &splits, &blocks);
  if (a.io == IO_BF16) launch_d<__nv_bfloat16, false>(a, splits, blocks, s);
  else launch_d<float, false>(a, splits, blocks, s);
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_backward(const NormRopeArgs& a, int num_sms, cudaStream_t s) {
  int splits = 0;
  unsigned blocks = 0;
  geometry(a.B, a.q.H + a.k.H, a.T, a.D, a.io, num_sms, true, &splits, &blocks);
  if (a.io == IO_BF16) launch_d<__nv_bfloat16, true>(a, splits, blocks, s);
  else launch_d<float, true>(a, splits, blocks, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.part) return e;
  kla_norm_rope_sum_kernel<<<2 * a.D, 32, 0, s>>>(a, (int)blocks);
  return cudaGetLastError();
}

}  // namespace kla
