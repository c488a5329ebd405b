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
// were read. A group keeps one token and goes through heads, the next two rows on
// their way while two are worked on (one, four and other numbers of blocks an
// SM measured slower), so that the angles, which cost as much as
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

// 16 bytes of a row, and its values in pairs for the packed arithmetic
template <typename IO>
struct Row {
  static constexpr int N = 16 / sizeof(IO), P = N / 2;
  uint32_t u[4];
  __device__ __forceinline__ void zero() { u[0] = u[1] = u[2] = u[3] = 0; }
  __device__ __forceinline__ void load(const IO* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
  }
  __device__ __forceinline__ void pairs(f2 (&x)[P]) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (N == 4) x[i] = f2_make(__uint_as_float(u[2 * i]), __uint_as_float(u[(2 * i + 1) & 3]));
      else x[i] = f2_make(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
  }
  static __device__ __forceinline__ void store(IO* p, const f2 (&x)[P]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (N == 4) {
        u[2 * i] = __float_as_uint(f2_lo(x[i]));
        u[(2 * i + 1) & 3] = __float_as_uint(f2_hi(x[i]));
      } else {
        const __nv_bfloat162 y = __floats2bfloat162_rn(f2_lo(x[i]), f2_hi(x[i]));
        u[i] = *reinterpret_cast<const uint32_t*>(&y);
      }
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

// The other member of element e's pair (e itself where it is not rotated).
__device__ __forceinline__ int other(const NormRopeArgs& a, int e) {
  if (e >= a.rot) return e;
  if (a.layout) return e ^ 1;
  return e < a.rot / 2 ? e + a.rot / 2 : e - a.rot / 2;
}

// Where a lane finds the other members of its pairs: in itself (neighbouring
// pairs, or no rotation), in one other lane (halves that are whole lanes), or
// anywhere in the row.
enum Mode { kInLane, kOtherLane, kAnywhere };

// The other members, zero where nothing is rotated (`mask`).
template <typename IO, int MODE>
__device__ __forceinline__ Row<IO> others(const NormRopeArgs& a, int e0, int from, const uint32_t (&mask)[4], IO* row,
                                          const Row<IO>& x) {
  constexpr int VE = Row<IO>::N;
  Row<IO> o;
  if (MODE == kInLane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o.u[j] = VE == 4 ? x.u[j ^ 1] : __byte_perm(x.u[j], 0, 0x1032);
  } else if (MODE == kOtherLane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o.u[j] = __shfl_sync(~0u, x.u[j], from);
  } else {
    *reinterpret_cast<uint4*>(row + e0) = make_uint4(x.u[0], x.u[1], x.u[2], x.u[3]);
    __syncwarp();
    IO y[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) y[j] = row[other(a, e0 + j)];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (VE == 4) o.u[j] = *reinterpret_cast<const uint32_t*>(&y[j]);
      else o.u[j] = (uint32_t)*reinterpret_cast<const uint16_t*>(&y[(2 * j) % VE]) |
                    (uint32_t)*reinterpret_cast<const uint16_t*>(&y[(2 * j + 1) % VE]) << 16;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) o.u[j] &= mask[j];
  return o;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) x += __shfl_xor_sync(~0u, x, m);
  return x;
}

// The y index of a block says whether it works on q or on k. It takes GROUPS
// tokens and `per` of the heads at a time; BWD also sums its weight gradients.
// Lanes without a token go along, so that every lane of a warp takes part in
// its exchanges. NORMED false: the gradients without a norm, which know nothing
// of x, whatever x holds (a kernel of its own: a branch or a mask in the other
// took 3% of the headline's gradients).
template <typename IO, int D, bool BWD, int MODE, bool NORMED>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 3) kla_norm_rope_kernel(const NormRopeArgs a, int per) {
  constexpr int VE = Row<IO>::N, P = VE / 2, LPR = D / VE, GROUPS = kThreads / LPR, U = 2;
  __shared__ __align__(16) float rows[GROUPS][D];  // halves that cut lanes; the block's weight gradients
  __shared__ float2 turns[GROUPS][D / 2];          // cosine and sine of every pair of every token
  const NormRopeTensor p = blockIdx.y ? a.k : a.q;
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR, e0 = l * VE, R = a.rot / 2;
  const long long tokens = (long long)a.B * a.T, groups = (tokens + GROUPS - 1) / GROUPS;
  const long long jobs = groups * ((p.H + per - 1) / per), ystep = (long long)a.T * D;
  IO* row = reinterpret_cast<IO*>(rows[grp]);
  int from = threadIdx.x & 31;
  if (e0 < a.rot) from += e0 < R ? R / VE : -(R / VE);
  uint32_t mask[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = e0 + j * VE / 4;
    mask[j] = e < a.rot ? 0xffffffffu : 0u;
  }
  const float f = a.norm == kNormNone ? 0.f : a.norm == kNormRms ? 1.f / (float)D : 1.f;
  f2 w[BWD ? P : 1], acc[BWD ? P : 1] = {};
  if (BWD)
#pragma unroll
    for (int j = 0; j < P; ++j) w[j] = p.w ? f2_make(p.w[e0 + 2 * j], p.w[e0 + 2 * j + 1]) : f2_make(1.f, 1.f);
  for (long long job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int h0 = (int)(job / groups) * per, n = min(p.H - h0, per);
    const long long first = job % groups * GROUPS, tok = first + grp;
    const bool live = tok < tokens;
    const long long at = live ? tok : 0;
    const int b = (int)(at / a.T);
    const long long t = at % a.T;
    const IO* x = reinterpret_cast<const IO*>(p.x) + b * p.sb + t * p.st + h0 * p.sh + e0;
    const long long y0 = (((long long)b * p.H + h0) * a.T + t) * D + e0;
    const bool with_g = BWD && p.gy;
    const IO* gy = reinterpret_cast<const IO*>(p.gy) + (with_g ? y0 : 0);
    IO* out = BWD ? reinterpret_cast<IO*>(p.gx) + b * p.gsb + t * p.gst + h0 * p.gsh + e0 : reinterpret_cast<IO*>(p.y) + y0;
    const long long ostep = BWD ? p.gsh : ystep;
    Row<IO> nx[U], ng[U];
    auto fetch = [&](int left) {  // the next U rows, or those that are left
#pragma unroll
      for (int u = 0; u < U; ++u) {
        nx[u].zero();
        if (BWD) ng[u].zero();
        if (live && u < left) {
          nx[u].load(x);
          if (with_g) ng[u].load(gy);
        }
        x += p.sh;
        if (BWD) gy += ystep;
      }
    };
    fetch(n);  // the first rows ahead of the angles
    f2 c[P], s[P];
    __syncthreads();  // the last job's angles are read
    for (int i = threadIdx.x; i < GROUPS * R; i += kThreads) {
      const int m = i / R, k = i % R;
      const long long q = min(first + m, tokens - 1);
      float sn, cs;
      sincospif(2.f * turn_of(a.positions ? a.positions[q] : a.offset + q % a.T, a.inv_freq[k]), &sn, &cs);
      turns[m][k] = make_float2(cs * a.rot_scale, sn * a.rot_scale);
    }
    __syncthreads();
    // y = x·c + other·s, with the sign of the element's place in its pair in s, and forward the weights in both
#pragma unroll
    for (int j = 0; j < P; ++j) {
      float cj[2], sj[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = e0 + 2 * j + i;
        const bool lead = a.layout ? !(e & 1) : e < R;
        float2 y = make_float2(1.f, 0.f);
        if (e < a.rot) y = turns[grp][a.layout ? e / 2 : (lead ? e : e - R)];
        cj[i] = y.x;
        sj[i] = lead != BWD ? -y.y : y.y;  // backward: the transpose
        if (!BWD && p.w) cj[i] *= p.w[e], sj[i] *= p.w[other(a, e)];
      }
      c[j] = f2_make(cj[0], cj[1]);
      s[j] = f2_make(sj[0], sj[1]);
    }
    for (int i = 0; i < n; i += U) {
      Row<IO> xr[U], gr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        xr[u] = nx[u];
        if (BWD) gr[u] = ng[u];
      }
      if (i + U < n) fetch(n - i - U);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool on = live && i + u < n;
        f2 v[P], o[P], y[P], sum2 = 0;
        xr[u].pairs(v);
#pragma unroll
        for (int j = 0; j < P; ++j) sum2 = f2_fma(v[j], v[j], sum2);
        const float sum = row_sum<LPR>(f2_lo(sum2) + f2_hi(sum2));
        float r = rsqrtf(fmaf(sum, f, a.eps));
        if (a.norm == kNormNone) r = 1.f;
        if (!on) r = 0.f;  // idle lanes add nothing, whatever ε is
        const f2 r2 = f2_make(r, r);
        others<IO, MODE>(a, e0, from, mask, row, BWD ? gr[u] : xr[u]).pairs(o);
        if (!BWD) {
#pragma unroll
          for (int j = 0; j < P; ++j) y[j] = f2_mul(r2, f2_fma(v[j], c[j], f2_mul(o[j], s[j])));
        } else {
          f2 g[P], dot2 = 0;
          gr[u].pairs(g);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            g[j] = f2_fma(g[j], c[j], f2_mul(o[j], s[j]));
            v[j] = f2_mul(v[j], r2);
            acc[j] = f2_fma(g[j], v[j], acc[j]);
            g[j] = f2_mul(g[j], w[j]);
            dot2 = f2_fma(g[j], v[j], dot2);
          }
          if (NORMED) {
            const float dot = -f * row_sum<LPR>(f2_lo(dot2) + f2_hi(dot2));
            const f2 d2 = f2_make(dot, dot);
#pragma unroll
            for (int j = 0; j < P; ++j) g[j] = f2_mul(r2, f2_fma(v[j], d2, g[j]));
          }
#pragma unroll
          for (int j = 0; j < P; ++j) y[j] = g[j];
        }
        if (on) Row<IO>::store(out, y);
        out += ostep;
      }
    }
  }
  if (BWD && a.part) {  // the block's weight gradients, in a fixed order
    __syncthreads();
#pragma unroll
    for (int j = 0; j < P; ++j) rows[grp][e0 + 2 * j] = f2_lo(acc[j]), rows[grp][e0 + 2 * j + 1] = f2_hi(acc[j]);
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
      float v = 0.f;
      for (int n = 0; n < GROUPS; ++n) v += rows[n][i];
      a.part[((size_t)blockIdx.x * 2 + blockIdx.y) * D + i] = v;
    }
  }
}

// Sums the blocks' partials: one warp per weight, lanes over blocks, then exchanges.
__global__ void __launch_bounds__(32) kla_norm_rope_sum_kernel(const NormRopeArgs a, int blocks) {
  const int i = blockIdx.x % a.D, m = blockIdx.x / a.D;
  float* out = m ? a.gwk : a.gwq;
  if (!out) return;  // (k's sums of a call without k are zero: its blocks were not launched)
  if (m && a.k.H == 0) blocks = 0;
  float x = 0.f;
  for (int b = threadIdx.x; b < blocks; b += 32) x += a.part[((size_t)b * 2 + m) * a.D + i];
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  if (threadIdx.x == 0) out[i] = x;
}

// How many heads a block takes with its tokens' angles, and the blocks of q's
// and of k's grid. Angles cost about as much as a few rows, so it is all of
// them unless that leaves the device short of blocks (four an SM; backward,
// where every block leaves partial sums, no more than that).
void geometry(int B, int Hq, int Hk, int T, int D, int io, int num_sms, bool bwd, int* per, unsigned* blocks) {
  const long long gpb = kThreads * (io == IO_BF16 ? 8 : 4) / D, groups = ((long long)B * T + gpb - 1) / gpb;
  const long long want = (long long)num_sms * (Hk > 0 ? 2 : 4), heads = std::max(std::max(Hq, Hk), 1);
  const long long s = std::min(std::max(groups > 0 ? (want + groups - 1) / groups : 1, 1LL), heads);
  *per = (int)((heads + s - 1) / s);
  const long long n = groups * ((heads + *per - 1) / *per);
  *blocks = (unsigned)std::max(std::min(n, bwd ? want : 1LL << 30), 1LL);
}

template <typename IO, int D, bool BWD, bool NORMED>
void launch_rows(const NormRopeArgs& a, dim3 grid, int per, cudaStream_t s) {
  if (a.layout || a.rot == 0) kla_norm_rope_kernel<IO, D, BWD, kInLane, NORMED><<<grid, kThreads, 0, s>>>(a, per);
  else if (a.rot / 2 % Row<IO>::N == 0) kla_norm_rope_kernel<IO, D, BWD, kOtherLane, NORMED><<<grid, kThreads, 0, s>>>(a, per);
  else kla_norm_rope_kernel<IO, D, BWD, kAnywhere, NORMED><<<grid, kThreads, 0, s>>>(a, per);
}

template <typename IO, int D, bool BWD>
void launch_mode(const NormRopeArgs& a, dim3 grid, int per, cudaStream_t s) {
  if (BWD && a.norm == kNormNone) launch_rows<IO, D, BWD, !BWD>(a, grid, per, s);
  else launch_rows<IO, D, BWD, true>(a, grid, per, s);
}

template <typename IO, bool BWD>
cudaError_t launch_io(const NormRopeArgs& a, int num_sms, unsigned* blocks, cudaStream_t s) {
  int per = 1;
  geometry(a.B, a.q.H, a.k.H, a.T, a.D, a.io, num_sms, BWD, &per, blocks);
  const dim3 grid(*blocks, a.k.H > 0 ? 2 : 1);
  switch (a.D) {
    case 16: launch_mode<IO, 16, BWD>(a, grid, per, s); break;
    case 32: launch_mode<IO, 32, BWD>(a, grid, per, s); break;
    case 64: launch_mode<IO, 64, BWD>(a, grid, per, s); break;
    default: launch_mode<IO, 128, BWD>(a, grid, per, s); break;
  }
  return cudaGetLastError();
}

}  // namespace

size_t norm_rope_partial_bytes(int B, int Hq, int Hk, int T, int D, int num_sms) {
  unsigned blocks = 0, most = 0;
  int per = 0;
  for (int io = 0; io < 2; ++io) {
    geometry(B, Hq, Hk, T, D, io, num_sms, true, &per, &blocks);
    most = std::max(most, blocks);
  }
  return (size_t)most * 2 * D * sizeof(float);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, int num_sms, cudaStream_t s) {
  unsigned blocks = 0;
  return a.io == IO_BF16 ? launch_io<__nv_bfloat16, false>(a, num_sms, &blocks, s)
                         : launch_io<float, false>(a, num_sms, &blocks, s);
}

cudaError_t launch_norm_rope_backward(const NormRopeArgs& a, int num_sms, cudaStream_t s) {
  unsigned blocks = 0;
  const cudaError_t e = a.io == IO_BF16 ? launch_io<__nv_bfloat16, true>(a, num_sms, &blocks, s)
                                        : launch_io<float, true>(a, num_sms, &blocks, s);
  if (e != cudaSuccess || !a.part) return e;
  kla_norm_rope_sum_kernel<<<2 * a.D, 32, 0, s>>>(a, (int)blocks);
  return cudaGetLastError();
}

}  // namespace kla
