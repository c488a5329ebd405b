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
// few lane exchanges, and the other members of a lane's pairs are in the lane
// itself (neighbouring pairs) or in one other lane (halves), fetched as they
// were read. A group keeps one token and goes through heads, four rows (two
// backward) in flight at a time, so that the angles, which cost as much as
// several rows, are computed once, and with the weights folded in a rotated
// entry is r (x wc + x' ws). Input strides are free: a projection's [B,T,H,D]
// is read in place and leaves as [B,H,T,D].
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

// 16 bytes of a row
template <typename IO>
struct Row {
  static constexpr int N = 16 / sizeof(IO);
  uint4 v;
  __device__ __forceinline__ void load(const void* p, long long i) {
    v = *reinterpret_cast<const uint4*>(reinterpret_cast<const IO*>(p) + i);
  }
  __device__ __forceinline__ void values(float (&x)[N]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (N == 4) {
        x[i] = __uint_as_float(u[i]);
      } else {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ void store(void* p, long long i, const float (&x)[N]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (N == 4) {
        u[j] = __float_as_uint(x[j]);
      } else {
        const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<IO*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
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

// The other member of element e's pair (e itself where it is not rotated).
__device__ __forceinline__ int other(const NormRopeArgs& a, int e) {
  if (e >= a.rot) return e;
  if (a.layout) return e ^ 1;
  return e < a.rot / 2 ? e + a.rot / 2 : e - a.rot / 2;
}

// The angles of a lane's elements, as y = x·c + other·s with the sign of the
// element's place in its pair in s.
template <int VE>
__device__ __forceinline__ void angles(const NormRopeArgs& a, long long pos, int e0, float (&c)[VE], float (&s)[VE]) {
  const int R = a.rot / 2;
#pragma unroll
  for (int j = 0; j < VE; ++j) {
    const int e = e0 + j;
    if (a.layout && (j & 1)) {  // a pair's second
      c[j] = c[j - 1];
      s[j] = -s[j - 1];
      continue;
    }
    c[j] = 1.f;
    s[j] = 0.f;
    if (e < a.rot) {
      const int i = a.layout ? e / 2 : (e < R ? e : e - R);
      float sn, cs;
      sincospif(2.f * turn_of(pos, a.inv_freq[i]), &sn, &cs);
      c[j] = cs * a.rot_scale;
      s[j] = (a.layout || e < R ? -sn : sn) * a.rot_scale;
    }
  }
}

// The other members of a lane's pairs, zero where nothing is rotated. `aligned`: halves that are whole lanes.
template <typename IO>
__device__ __forceinline__ void others(const NormRopeArgs& a, int e0, bool aligned, float* row, const Row<IO>& v,
                                       const float (&x)[Row<IO>::N], float (&o)[Row<IO>::N]) {
  constexpr int VE = Row<IO>::N;
  if (a.layout) {
#pragma unroll
    for (int j = 0; j < VE; ++j) o[j] = e0 + j < a.rot ? x[j ^ 1] : 0.f;
  } else if (aligned) {
    const int R = a.rot / 2, d = R / VE, lane = threadIdx.x & 31;
    const int from = e0 < R ? lane + d : (e0 < a.rot ? lane - d : lane);
    Row<IO> w;
    w.v.x = __shfl_sync(~0u, v.v.x, from);
    w.v.y = __shfl_sync(~0u, v.v.y, from);
    w.v.z = __shfl_sync(~0u, v.v.z, from);
    w.v.w = __shfl_sync(~0u, v.v.w, from);
    if (e0 >= a.rot) w.v = make_uint4(0, 0, 0, 0);
    w.values(o);
  } else {  // through the group's row in shared memory
#pragma unroll
    for (int j = 0; j < VE; ++j) row[e0 + j] = x[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VE; ++j) o[j] = e0 + j < a.rot ? row[other(a, e0 + j)] : 0.f;
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
  return rsqrtf(fmaf(sum, a.norm == kNormRms ? 1.f / (float)a.D : 1.f, a.eps));
}

// A block takes GROUPS tokens and one of `splits` ranges of the heads of q
// followed by those of k; BWD also sums its weight gradients. Lanes without a
// token go along, so that every lane of a warp takes part in its exchanges.
template <typename IO, int D, bool BWD>
__global__ void __launch_bounds__(kThreads) kla_norm_rope_kernel(const NormRopeArgs a, int splits) {
  constexpr int VE = Row<IO>::N, LPR = D / VE, GROUPS = kThreads / LPR, U = BWD ? 2 : 4;
  __shared__ float rows[GROUPS][D];
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR, e0 = l * VE;
  const bool aligned = (a.rot / 2) % VE == 0;
  const int heads = a.q.H + a.k.H, per = (heads + splits - 1) / splits;
  const long long tokens = (long long)a.B * a.T, groups = (tokens + GROUPS - 1) / GROUPS;
  float acc[2][BWD ? VE : 1] = {};
  for (long long job = blockIdx.x; job < groups * splits; job += gridDim.x) {
    const int h0 = (int)(job / groups) * per, h1 = min(heads, h0 + per);
    const long long tok = job % groups * GROUPS + grp;
    const bool live = tok < tokens;
    const long long at = live ? tok : 0;
    const int b = (int)(at / a.T);
    const long long t = at % a.T;
    float c[VE], s[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) c[j] = 1.f, s[j] = 0.f;
    if (a.rot) angles<VE>(a, a.positions ? a.positions[at] : a.offset + t, e0, c, s);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const NormRopeTensor& p = m ? a.k : a.q;
      const int lo = m ? max(h0 - a.q.H, 0) : h0, hi = m ? h1 - a.q.H : min(h1, a.q.H);
      if (lo >= hi) continue;
      float w[VE], wc[VE], ws[VE];  // forward: the weights are part of the rotation
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        w[j] = p.w ? p.w[e0 + j] : 1.f;
        wc[j] = w[j] * c[j];
        ws[j] = (p.w ? p.w[other(a, e0 + j)] : 1.f) * s[j];
      }
      const long long x0 = b * p.sb + t * p.st + e0, y0 = ((long long)b * p.H * a.T + t) * D + e0;
      for (int h = lo; h < hi; h += U) {
        Row<IO> xv[U], gv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          xv[u].v = gv[u].v = make_uint4(0, 0, 0, 0);
          if (live && h + u < hi) {
            xv[u].load(p.x, x0 + (h + u) * p.sh);
            if (BWD && p.gy) gv[u].load(p.gy, y0 + (long long)(h + u) * a.T * D);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool on = live && h + u < hi;
          float x[VE], o[VE], y[VE];
          xv[u].values(x);
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < VE; ++j) sum = fmaf(x[j], x[j], sum);
          sum = row_sum<LPR>(sum);
          const float r = on ? inv_size(a, sum) : 0.f;  // idle lanes add nothing, whatever ε is
          if (!BWD) {
            if (a.rot) {
              others<IO>(a, e0, aligned, rows[grp], xv[u], x, o);
#pragma unroll
              for (int j = 0; j < VE; ++j) y[j] = r * fmaf(x[j], wc[j], o[j] * ws[j]);
            } else {
#pragma unroll
              for (int j = 0; j < VE; ++j) y[j] = r * (x[j] * w[j]);
            }
            if (on) Row<IO>::store(p.y, y0 + (long long)(h + u) * a.T * D, y);
          } else {
            float g[VE];
            gv[u].values(g);
            if (a.rot) {  // the transpose: the same cosines, the sines' sign turned
              others<IO>(a, e0, aligned, rows[grp], gv[u], g, o);
#pragma unroll
              for (int j = 0; j < VE; ++j) g[j] = fmaf(g[j], c[j], -o[j] * s[j]);
            }
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              x[j] *= r;
              acc[m][j] = fmaf(g[j], x[j], acc[m][j]);
              g[j] *= w[j];
              dot = fmaf(g[j], x[j], dot);
            }
            dot = row_sum<LPR>(dot);
            if (a.norm == kNormNone) dot = 0.f;
            else if (a.norm == kNormRms) dot *= 1.f / (float)D;
#pragma unroll
            for (int j = 0; j < VE; ++j) y[j] = r * fmaf(-x[j], dot, g[j]);
            if (on) Row<IO>::store(p.gx, b * p.gsb + (h + u) * p.gsh + t * p.gst + e0, y);
          }
        }
      }
    }
  }
  if (BWD && a.part) {  // the block's weight gradients, in a fixed order
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < VE; ++j) rows[grp][e0 + j] = acc[m][j];
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

// How many blocks share a token's heads, and the blocks. A token's angles cost
// about as much as several rows, so a block takes all heads unless that leaves
// the device short of blocks (four an SM; backward, where every block leaves
// partial sums, no more than that).
void geometry(int B, int heads, int T, int D, int io, int num_sms, bool bwd, int* splits, unsigned* blocks) {
  const long long gpb = kThreads * (io == IO_BF16 ? 8 : 4) / D, groups = ((long long)B * T + gpb - 1) / gpb;
  const long long want = (long long)num_sms * 4;
  long long s = groups > 0 ? (want + groups - 1) / groups : 1;
  s = std::min<long long>(std::max<long long>(s, 1), std::max(heads, 1));
  const long long per = (heads + s - 1) / s;
  s = per > 0 ? (heads + per - 1) / per : 1;
  *splits = (int)s;
  const long long n = std::min<long long>(groups * s, bwd ? want : 1LL << 30);
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
