// kda_latent_tc.cuh -- what the latent attention's tensor-core kernels share:
// operands in shared memory in the 128-byte swizzle, as TMA writes them, and
// copies from tensor maps of three and four dimensions.  Internal to libkda.
//
// A chunk is [rows][64 channels] of bf16: 128 bytes a row, the 16-byte pieces of a
// row exchanged by the row's number modulo 8.  The same bytes serve as a K-major
// operand (rows are M or N, channels are K: groups of 8 rows 1024 bytes apart, a
// step of 16 channels is 32 bytes) and as an MN-major one (channels are M or N,
// rows are K: 64 channels a chunk, a step of 16 rows is 2048 bytes).
#pragma once

#include <cudaTypedefs.h>

#include "kda_latent.cuh"
#include "kda_tc_common.cuh"

namespace kda {
namespace latent {

constexpr int kChunkCols = 64;           // channels of a chunk
constexpr uint32_t kRowBytes = 128;

// Byte offset of a 16-byte piece (8 channels) in a chunk.
__device__ __forceinline__ uint32_t piece_off(int row, int piece) {
  return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4));
}

// Operand descriptor in the 128-byte swizzle.  lbo: bytes to the next 64 channels
// (MN-major); 8 rows are 1024 bytes.  A step through shared memory adds its bytes / 16:
// the one thread that issues the products makes a descriptor per chunk, not per
// instruction (made for each of them, an instruction took 146 cycles to issue).
constexpr uint64_t kStepK = 32 / 16, kStepRows = 2048 / 16;   // K = 16, K-major and MN-major
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t addr, uint32_t lbo) {
  uint64_t d = (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Into L2 alone.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// A wait that the other threads of the CTA can end: it gives up after `clocks`, or once
// one of them has; whoever gives up first says so in *fail.  Threads that share barriers
// of their own go on all the same, without waiting, so that all of them come to the end.
struct Waits {
  volatile int *fail;
  long long clocks;
  // About a second, and what the rows of a tile take where they are made again key by key.
  __device__ __forceinline__ Waits(int *f, long long keys)
      : fail(f), clocks(tc::kWaitLimit + (min(keys, 1ll << 20) << 16)) {}
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(bar, parity)) {
      if (*fail) return false;
      if (clock64() - t0 > clocks) {
        *fail = 1;
        return false;
      }
    }
    return true;
  }
};

// One thread of a warp that is whole.  (The compiler then knows that the branch holds
// one thread; behind `lane == 0` it readies each product's uniform registers for many.)
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
}

// A place in a ring of slots: the slot and how many times it has been used, modulo 2.
struct Slot {
  int at;
  uint32_t lap;
  __device__ __forceinline__ void next(int slots) {
    if (++at == slots) {
      at = 0;
      lap ^= 1u;
    }
  }
};

// The launch's 384 threads have 168 registers each (504 of three warpgroups); the two
// that work on rows take 216, the third keeps 72: 504.
__device__ __forceinline__ void few_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
}
__device__ __forceinline__ void many_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
}

// Columns [from, to) of 32 that begin at `at`, as bits.
__device__ __forceinline__ uint32_t column_bits(int from, int to, int at) {
  const int a = min(max(from - at, 0), 32), z = min(max(to - at, 0), 32);
  const uint32_t below = z >= 32 ? 0xffffffffu : (1u << z) - 1u;
  return a >= 32 ? 0u : below & (0xffffffffu << a);
}

// D (+)= A B over one K = 16 step, A in tensor memory (bf16, two a column).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                            uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

// 32 columns of this thread's lane, without waiting.
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// No use of the registers is scheduled before this.
__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                 "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t taddr, uint32_t (&r)[32]) {
  tmem_ld32_nw(taddr, r);
  tc::tmem_wait_ld();
  reg_fence32(r);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A tensor map of bf16 in the 128-byte swizzle: `rank` dimensions (the first one
// contiguous channels), strides in elements of the others, a box of 64 channels.
bool make_swizzled_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims,
                       const long long *strides, const uint32_t *box);

// The map of a prompt's tensor [B,T,heads,n], boxes of `rows` tokens of one head.
bool prompt_map(CUtensorMap *m, const void *x, const Strides &s, const Prompt &p, int heads, int n,
                int rows);

}  // namespace latent
}  // namespace kda
