// Matrix products of fp32 accuracy on the tensor cores (sm_103a), for 64-token
// chunks: operands are tiles of 64 columns in shared memory, each kept as one
// to three bf16 parts (x = hi + mid + lo holds 24 bits), products of parts go
// through tcgen05.mma with fp32 accumulators in TMEM, and results come back to
// registers in the 16x256b form: lane l of a warp has rows l/4 and l/4 + 8 of
// its 16, columns 2(l%4) and 2(l%4) + 1 of every eight.
//
// A tile is rows of 128 bytes (64 bf16) with the 128-byte swizzle: 16-byte
// unit u of row r is at r·128 + (u ^ (r & 7))·16 from a 1024-byte boundary. The
// same tile serves as a K-major operand (rows are M or N, columns are K) or as
// an MN-major one (rows are K, columns are M or N), so nothing is transposed.
#pragma once

#include "kla_device.cuh"

namespace kla {
namespace umma {

constexpr int kTileBytes = 64 * 128;  // 64 rows

// ---- barriers ---------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// The phase ends when `bytes` of bulk copies have come in; they start here, 16-byte aligned, from global memory.
__device__ __forceinline__ void mbar_expect(uint64_t* bar, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, int bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
               "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
// Global memory on its way into L2, 16-byte aligned.
__device__ __forceinline__ void prefetch(const void* from, int bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t addr, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(done) : "r"(addr), "r"(parity) : "memory");
  return done != 0;
}
__device__ __forceinline__ uint64_t nanoseconds() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase of the given parity, for two seconds at most; then it
// gives up: `ok` turns false, and later waits return at once. A block that has
// such a thread overwrites its outputs at its end (fill_nan).
__device__ __forceinline__ void mbar_wait(uint64_t* bar, uint32_t parity, bool& ok) {
#ifdef KLA_RAN_OUT  // a test's build: every wait is waited for, and counts as run out for the threads that this names
  bool real = true;
  if (KLA_RAN_OUT) ok = false;
#else
  bool& real = ok;
#endif
  const uint32_t addr = smem_addr(bar);
  if (!real || mbar_try(addr, parity)) return;
  const uint64_t start = nanoseconds();
  while (!mbar_try(addr, parity))
    if (nanoseconds() - start > 2000000000ull) {
      real = ok = false;
      return;
    }
}
// Thread and block read anew: what follows a wait that ran out keeps no registers of the way before it.
__device__ __forceinline__ unsigned thread_again() {
  unsigned x;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(x));
  return x;
}
__device__ __forceinline__ unsigned block_again() {
  unsigned x;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(x));
  return x;
}
// Rows of an output that came of a wait that ran out: no numbers.
template <typename T>
__device__ __forceinline__ void fill_nan(T* out, int rows, int cols, size_t stride, int tid, int threads) {
  for (int i = tid; i < rows * cols; i += threads) out[i / cols * stride + i % cols] = from_f32<T>(__int_as_float(0x7fc00000));
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- TMEM ---------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, int cols) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, int cols) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
// 16 lanes × 32 columns from `addr` (lane in the upper half)
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// One lane of a converged warp. Products are issued by a warp that takes the
// branch as a whole, with values the compiler knows to be the same in all its
// lanes: descriptors then stay in uniform registers (inside a branch of one
// thread each product cost 60 to 100 cycles to issue).
__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }

// 16 lanes × 16 columns, the sum of three blocks `apart` columns from one another, the last one first.
__device__ __forceinline__ void tmem_load_sum(uint32_t addr, int apart, float (&v)[8]) {
  uint32_t r[24];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%25];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%26];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23])
      : "r"(addr), "r"(addr + apart), "r"(addr + 2 * apart)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = (__uint_as_float(r[16 + i]) + __uint_as_float(r[8 + i])) + __uint_as_float(r[i]);
}
// Both sixteen lanes of a quadrant with one wait: x from addr on, y from 16 lanes further.
__device__ __forceinline__ void tmem_load_both(uint32_t addr, float (&x)[16], float (&y)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
        "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31])
      : "r"(addr), "r"(addr + (16u << 16))
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = __uint_as_float(r[i]);
    y[i] = __uint_as_float(r[16 + i]);
  }
}
// The same, each the sum of three blocks of columns
__device__ __forceinline__ void tmem_load_both_sum(uint32_t addr, int apart, float (&x)[8], float (&y)[8]) {
  uint32_t r[48];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%48];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%49];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%16,%17,%18,%19,%20,%21,%22,%23}, [%50];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%24,%25,%26,%27,%28,%29,%30,%31}, [%51];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%32,%33,%34,%35,%36,%37,%38,%39}, [%52];\n\t"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%40,%41,%42,%43,%44,%45,%46,%47}, [%53];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
        "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]),
        "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]), "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]),
        "=&r"(r[40]), "=&r"(r[41]), "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47])
      : "r"(addr), "r"(addr + apart), "r"(addr + 2 * apart), "r"(addr + (16u << 16)), "r"(addr + apart + (16u << 16)), "r"(addr + 2 * apart + (16u << 16))
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = (__uint_as_float(r[16 + i]) + __uint_as_float(r[8 + i])) + __uint_as_float(r[i]);
    y[i] = (__uint_as_float(r[40 + i]) + __uint_as_float(r[32 + i])) + __uint_as_float(r[24 + i]);
  }
}

// ---- products -------------------------------------------------------------------
// A tile operand of PARTS parts, `part` bytes apart, K-major (rows are M or N)
// or MN-major (rows are K). `block`: bytes between its 64-column tiles.
template <int PARTS, bool MN>
struct Operand {
  uint32_t addr;  // shared-memory address of part 0
  int part, block;
};
// D[M×N] (+)= A·B over K of depth, issued by one thread. Sixteen of K are 32
// bytes along a K-major row (the next tile after 64) or 16 rows of an MN-major
// tile. Products of parts that weigh less than the last kept part are left out
// (i + j ≥ the larger number of parts). The small products go first: the
// accumulator is cut to 24 bits after every instruction, which costs nothing
// while it is small (64³ with 3 × 3 parts: 1.2e-6 of the largest value with the
// large products first).
template <int M, int N, int K, int PA, bool AMN, int PB, bool BMN>
__device__ __forceinline__ void mma_weight(uint32_t d, const Operand<PA, AMN>& a, const Operand<PB, BMN>& b, int w,
                                           uint32_t& acc) {  // the products of parts i + j = w
  constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)AMN << 15) | ((uint32_t)BMN << 16) |
                             ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
  // descriptor: address, distance of 64-column blocks (MN-major), of eight rows, version 1, 128-byte swizzle
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  const uint32_t la = ((a.addr & 0x3ffff) >> 4) | ((uint32_t)(AMN ? a.block >> 4 : 1) << 16);
  const uint32_t lb = ((b.addr & 0x3ffff) >> 4) | ((uint32_t)(BMN ? b.block >> 4 : 1) << 16);
#pragma unroll
  for (int i = 0; i < PA; ++i) {
    const int j = w - i;
    if (j < 0 || j >= PB) continue;
#pragma unroll
    for (int k = 0; k < K / 16; ++k) {
      const uint32_t oa = i * a.part + (AMN ? k * 2048 : (k >> 2) * a.block + (k & 3) * 32);
      const uint32_t ob = j * b.part + (BMN ? k * 2048 : (k >> 2) * b.block + (k & 3) * 32);
      asm volatile(
          "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\t"
          "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
          "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d), "r"(la + (oa >> 4)),
          "r"(lb + (ob >> 4)), "r"(hi), "r"(idesc), "r"(acc)
          : "memory");
      acc = 1u;
    }
  }
}
template <int M, int N, int K, int PA, bool AMN, int PB, bool BMN>
__device__ __forceinline__ void mma(uint32_t d, const Operand<PA, AMN>& a, const Operand<PB, BMN>& b,
                                    bool accumulate = false) {
  uint32_t acc = accumulate ? 1u : 0u;
#pragma unroll
  for (int w = (PA > PB ? PA : PB) - 1; w >= 0; --w) mma_weight<M, N, K>(d, a, b, w, acc);
}
// D = A·B + C·E, the small products of both first.
template <int M, int N, int K, int PA, bool AMN, int PB, bool BMN>
__device__ __forceinline__ void mma_sum(uint32_t d, const Operand<PA, AMN>& a, const Operand<PB, BMN>& b,
                                        const Operand<PA, AMN>& c, const Operand<PB, BMN>& e) {
  uint32_t acc = 0;
#pragma unroll
  for (int w = (PA > PB ? PA : PB) - 1; w >= 0; --w) {
    mma_weight<M, N, K>(d, a, b, w, acc);
    mma_weight<M, N, K>(d, c, e, w, acc);
  }
}
// `bar` gets one arrival when every product issued so far is done.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// ---- parts ------------------------------------------------------------------------
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two neighbouring columns of row r as PARTS bf16 pairs into the tile.
template <int PARTS>
__device__ __forceinline__ void store_pair(char* tile, int part_bytes, int r, int c, float x, float y) {
  char* p = tile + r * 128 + ((((c >> 3) ^ r) & 7) << 4) + (c & 7) * 2;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const uint32_t u = bf16_pair(x, y);
    *reinterpret_cast<uint32_t*>(p + i * part_bytes) = u;
    if (i + 1 < PARTS) {
      x -= __uint_as_float(u << 16);
      y -= __uint_as_float(u & 0xffff0000u);
    }
  }
}
// Eight neighbouring columns.
template <int PARTS>
__device__ __forceinline__ void store_eight(char* tile, int part_bytes, int r, int c, float (&x)[8]) {
  char* p = tile + r * 128 + ((((c >> 3) ^ r) & 7) << 4);
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = bf16_pair(x[2 * j], x[2 * j + 1]);
      x[2 * j] -= __uint_as_float(u[j] << 16);
      x[2 * j + 1] -= __uint_as_float(u[j] & 0xffff0000u);
    }
    *reinterpret_cast<uint4*>(p + i * part_bytes) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

}  // namespace umma
}  // namespace kla
