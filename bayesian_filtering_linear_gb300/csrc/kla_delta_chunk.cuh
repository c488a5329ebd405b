// Shared pieces of the chunked gated delta rule (kla_delta_chunk.cu,
// kla_delta_backward.cu): the workspace, tile loads and per-chunk gates.
#pragma once

#include "kla_launch.h"
#include "kla_umma.cuh"

namespace kla {
namespace delta {

using namespace umma;

constexpr int C = 64;             // tokens of a chunk
constexpr int kThreads = 256;     // of the kernels that take a chunk each
// Floats of a chunk's gates: cumulative log2 of the decay in two, decay from the start, to the end, β; then what the
// chunk's whole decay is more than the float that has it (and three that fill 16 bytes).
constexpr int kGates = 5 * C + 4;
constexpr int kMaxBytes = 227 * 1024 - 4096;  // shared memory of a block, less its static part
constexpr float kMinLog = -104.f; // e^-104 is 0 in fp32: smaller logs change nothing but the sums' exactness

template <typename IO>
constexpr int kParts = sizeof(IO) == 2 ? 1 : 3;  // bf16 parts that hold an input exactly (fp32: to 24 bits)

__host__ __device__ constexpr int pad64(int d) { return d <= 64 ? 64 : 128; }

// Per chunk of every value head, padded to whole chunks and to widths of 64:
// blocks of 64 × 64 (a column of blocks per 64 columns, one or two rows of
// them) in the order of the fragments that 256 threads hold of them, so that
// a warp's stores and loads are whole lines (see Fragment). W and Wr only the
// chain reads: they are its operand's tiles, DK / 64 of 128 rows (in turns 16
// rows of the largest part and 16 of the middle one), then as many of the
// smallest part's 64 rows.
struct Workspace {
  float* gates;  // [chunks][kGates]
  char* W;       // [chunks] tiles: −M (β G K)
  float* S;      // [chunks][DK][DV]: the state before each chunk
  float* U;      // [chunks][64][DV]: first M (β V), then U
  char* Wr;      // [chunks] tiles: Mᵀ (E K)
  float* Z;      // [chunks][DK][DV]: first Qᵀ(G O'), then the gradient of the state after each chunk
  float* R;      // [chunks][64][DV]: first Mᵀ Pᵀ O', then dR
  float* part;   // [B·H][T][2][dk]: gradients of q and k by value head (shared key heads)
};

__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <typename IO>
__device__ __forceinline__ float2 load_two(const IO* p);
template <>
__device__ __forceinline__ float2 load_two<float>(const float* p) { return *reinterpret_cast<const float2*>(p); }
template <>
__device__ __forceinline__ float2 load_two<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void store_two(float* p, float x, float y) { *reinterpret_cast<float2*>(p) = make_float2(x, y); }
__device__ __forceinline__ void store_two(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = bf16_pair(x, y);
}
// Rows [0, len) of 64 (the rest zero) of an io array [.][d], columns c0 to
// c0 + W (those from d on zero), as tiles of kParts<IO> parts, by THREADS
// threads: fetch() brings a thread's share into registers, all loads in flight
// together, and put() writes the parts.
template <typename IO, int W, int THREADS>
struct TileLoad {
  static constexpr int N = C * W / 8 / THREADS, PARTS = kParts<IO>, PART = W / 64 * kTileBytes;
  uint4 v[N * sizeof(IO) / 2];
  __device__ __forceinline__ void fetch(const IO* src, int len, int d, int c0, int tid) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = tid + j * THREADS, r = i / (W / 8), c = i % (W / 8) * 8;
      const bool in = r < len && c0 + c < d;
      const uint4* p = reinterpret_cast<const uint4*>(src + (size_t)r * d + c0 + c);
#pragma unroll
      for (int e = 0; e < (int)sizeof(IO) / 2; ++e)
        v[j * sizeof(IO) / 2 + e] = in ? p[e] : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void put(char* tile, int tid) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = tid + j * THREADS, r = i / (W / 8), c = i % (W / 8) * 8;
      char* t = tile + (c >> 6) * kTileBytes;
      if (PARTS == 1) {
        *reinterpret_cast<uint4*>(t + r * 128 + ((((c >> 3) ^ r) & 7) << 4)) = v[j];
      } else {
        float x[8];
        eight(j, x);
        store_eight<PARTS>(t, PART, r, c & 63, x);
      }
    }
  }
  // the thread's j-th eight values
  __device__ __forceinline__ void eight(int j, float (&x)[8]) const {
#pragma unroll
    for (int e = 0; e < (int)sizeof(IO) / 2; ++e) {
      const uint4 y = v[j * sizeof(IO) / 2 + e];
      const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (PARTS == 1) {
          x[2 * m] = __uint_as_float(u[m] << 16);
          x[2 * m + 1] = __uint_as_float(u[m] & 0xffff0000u);
        } else {
          x[4 * e + m] = __uint_as_float(u[m]);
        }
      }
    }
  }
};

// A thread's sixteen values of a 64 × 64 block as they come from TMEM: rows
// r and r + 8, columns c + 8 j and the next, j < 4 (value 4 j + 2 o + e is row
// r + 8 o, column c + 8 j + e).
constexpr int kBlock = 64 * 64;
struct Lanes {
  int quad, half, lane, r, c;
  __device__ __forceinline__ Lanes(int tid)
      : quad((tid >> 5) & 3), half(tid >> 7), lane(tid & 31), r(16 * quad + (lane >> 2)), c(32 * half + 2 * (lane & 3)) {}
};
// rows of block rb of an array of DK rows (TMEM spreads 64 rows over 16 lanes of each quadrant, 128 over all)
template <int DK>
__device__ __forceinline__ int block_row(const Lanes& l, int rb) {
  return (DK == 64 ? 16 * l.quad : 32 * l.quad + 16 * rb) + (l.lane >> 2);
}
template <int J>
struct Columns {  // J of the four eights of columns, from the j0-th
  float v[4 * J];
  __device__ __forceinline__ void load(const float* block, int tid, int j0 = 0) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float4 x = reinterpret_cast<const float4*>(block)[(j0 + j) * 256 + tid];
      v[4 * j] = x.x, v[4 * j + 1] = x.y, v[4 * j + 2] = x.z, v[4 * j + 3] = x.w;
    }
  }
  __device__ __forceinline__ void store(float* block, int tid, int j0 = 0) const {
#pragma unroll
    for (int j = 0; j < J; ++j)
      reinterpret_cast<float4*>(block)[(j0 + j) * 256 + tid] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  }
  // into a column of tiles as parts, from row r and column c
  template <int PARTS>
  __device__ __forceinline__ void put(char* tile, int part, int r, int c) const {
#pragma unroll
    for (int e = 0; e < 4 * J; e += 2) store_pair<PARTS>(tile, part, r + (e & 2) * 4, c + (e >> 2) * 8, v[e], v[e + 1]);
  }
};

using Fragment = Columns<4>;

// Four lanes that hold columns 2 q and 2 q + 1 of four eights turn them so that lane q holds all of eight q (and back).
__device__ __forceinline__ void turn_four(uint32_t (&u)[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
  uint32_t a = __shfl_xor_sync(~0u, odd ? u[0] : u[1], 1), b = __shfl_xor_sync(~0u, odd ? u[2] : u[3], 1);
  if (odd) u[0] = a, u[2] = b;
  else u[1] = a, u[3] = b;
  a = __shfl_xor_sync(~0u, high ? u[0] : u[2], 2), b = __shfl_xor_sync(~0u, high ? u[1] : u[3], 2);
  if (high) u[0] = a, u[1] = b;
  else u[2] = a, u[3] = b;
}
// A fragment to and from rows of an io array of width d: columns from c0 on, rows below len (all lanes of a warp call).
template <typename IO>
__device__ __forceinline__ void store_rows(IO* out, const Lanes& l, int c0, int len, int d, const float (&v)[16]) {
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int r = l.r + 8 * o;
    if (sizeof(IO) == 2) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = bf16_pair(v[4 * j + 2 * o], v[4 * j + 2 * o + 1]);
      turn_four(u, l.lane);
      const int c = c0 + 32 * l.half + 8 * (l.lane & 3);
      if (r < len && c < d) *reinterpret_cast<uint4*>(out + (size_t)r * d + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r < len && c0 + l.c + 8 * j < d) store_two(out + (size_t)r * d + c0 + l.c + 8 * j, v[4 * j + 2 * o], v[4 * j + 2 * o + 1]);
    }
  }
}
template <typename IO>
__device__ __forceinline__ void load_rows(const IO* in, const Lanes& l, int c0, int len, int d, float (&v)[16]) {
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int r = l.r + 8 * o;
    if (sizeof(IO) == 2) {
      const int c = c0 + 32 * l.half + 8 * (l.lane & 3);
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < len && c < d) x = *reinterpret_cast<const uint4*>(in + (size_t)r * d + c);
      uint32_t u[4] = {x.x, x.y, x.z, x.w};
      turn_four(u, l.lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[4 * j + 2 * o] = __uint_as_float(u[j] << 16);
        v[4 * j + 2 * o + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 x = make_float2(0.f, 0.f);
        if (r < len && c0 + l.c + 8 * j < d) x = load_two(in + (size_t)r * d + c0 + l.c + 8 * j);
        v[4 * j + 2 * o] = x.x, v[4 * j + 2 * o + 1] = x.y;
      }
    }
  }
}

constexpr float kLog2e = 1.44269504f, kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e);
// 2^x by the hardware's instruction (2 ulp)
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^(h + l), the decay of a whole chunk, as the sum of two floats where it is next to 1: one float is off by up to 2^-25
// there, and over thousands of chunks with the same decay all of it would add up. e^x = 1 + x + x²/2 + … + x^8/8!.
__device__ __forceinline__ float whole_decay(float h, float l, float& low) {
  constexpr float kLn2 = 0.693147182f, kLn2Low = (float)(0.69314718055994531 - (double)kLn2);
  low = 0.f;
  if (!(h > -0.5f && h < 0.5f)) return exp2_of(h + l);
  const float x = h * kLn2, xl = fmaf(h, kLn2, -x) + fmaf(h, kLn2Low, l * kLn2);
  float p = fmaf(x, 1.f / 40320.f, 1.f / 5040.f);
  p = fmaf(x, p, 1.f / 720.f);
  p = fmaf(x, p, 1.f / 120.f);
  p = fmaf(x, p, 1.f / 24.f);
  p = fmaf(x, p, 1.f / 6.f);
  p = x * x * fmaf(x, p, 0.5f);
  const float s = x + p, y = 1.f + s;
  low = (s - (y - 1.f)) + ((p - (s - x)) + xl);
  return y;
}
// The decays D_ts of a thread's fragment from the cumulative logs (zero above the diagonal).
__device__ __forceinline__ void decays(const float2* logs, const Lanes& l, float (&D)[16]) {
  if (32 * l.half > 16 * l.quad + 15) {  // all of the warp's fragment is above it
#pragma unroll
    for (int e = 0; e < 16; ++e) D[e] = 0.f;
    return;
  }
  const float2 t[2] = {logs[l.r], logs[l.r + 8]};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int s = l.c + 8 * j;
    const float4 y = *reinterpret_cast<const float4*>(logs + s);  // of tokens s and s + 1
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const float d0 = (t[o].x - y.x) + (t[o].y - y.y), d1 = (t[o].x - y.z) + (t[o].y - y.w);
      D[4 * j + 2 * o] = s <= l.r + 8 * o ? exp2_of(d0) : 0.f;
      D[4 * j + 2 * o + 1] = s + 1 <= l.r + 8 * o ? exp2_of(d1) : 0.f;
    }
  }
}

// Everything of a block that starts a chunk: which one, and its rows.
struct Where {
  long long bh, key;
  int n, t0, len;
  size_t chunk;
};
// (in 32 bits, as a grid counts its blocks)
__device__ __forceinline__ Where where(const DeltaArgs& a, unsigned chunk) {
  const unsigned N = ((unsigned)a.T + C - 1) / C, bh = chunk / N, b = bh / a.H;
  Where w;
  w.chunk = chunk;
  w.bh = bh;
  w.n = (int)(chunk - bh * N);
  w.key = (long long)b * a.Hk + (bh - b * a.H) / ((unsigned)a.H / a.Hk);
  w.t0 = w.n * C;
  w.len = min(C, a.T - w.t0);
  return w;
}

// A chunk's rows of an io array on their way into L2.
template <typename IO>
__device__ __forceinline__ void prefetch_rows(const void* p, long long head, const Where& at, int T, int d) {
  prefetch(reinterpret_cast<const IO*>(p) + ((size_t)head * T + at.t0) * d, at.len * d * (int)sizeof(IO));
}

// Launches with dynamic shared memory; all of an SM's L1 is asked for as shared memory, so that as many blocks fit as
// their sizes allow.
template <typename F, typename... Args>
cudaError_t run(F kernel, int smem, dim3 blocks, int threads, cudaStream_t s, const Args&... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, threads, smem, s>>>(args...);
  return cudaGetLastError();
}

Workspace workspace(void* base, int B, int Hk, int H, int T, int dk, int dv, bool backward, size_t* bytes);
// The gates, W and M (β V); with d also Wr, Mᵀ Pᵀ O' and Qᵀ(G O').
cudaError_t launch_prepare(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, cudaStream_t s);
// The states before the chunks and U, with d also the gradients of the states after them and dR: one block per head
// and 64 or 32 columns, and direction.
cudaError_t launch_chain(const DeltaArgs& a, const DeltaGradArgs* d, const Workspace& w, int num_sms, cudaStream_t s);

}  // namespace delta
}  // namespace kla
