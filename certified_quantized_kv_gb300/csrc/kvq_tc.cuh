// kvq_tc.cuh -- barriers, tensor memory (TMEM) and the MMAs of the 5th-generation tensor cores, as the kernels that use them
// take them: binary16 operands, fp32 accumulators, M = 128, one CTA.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kvq {

constexpr unsigned long long TC_WAIT_NS = 2000000000ull;   // bounded waits: 2 s

__device__ __forceinline__ uint32_t tc_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ unsigned long long tc_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool tc_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// A wait that runs out, in any warp, lets all further ones pass: the CTA finishes with outputs that are NaN.  (The clock is
// read once in 256 tries: it takes longer than they do.)
__device__ __forceinline__ void tc_wait_slow(uint32_t bar, uint32_t parity, volatile int* failed) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t n = 0; !tc_try(bar, parity); ++n) {
    if ((n & 255) != 255) continue;
    const unsigned long long t = tc_ns();
    if (*failed) return;
    if (t0 == 0) t0 = t;
    if (t - t0 > TC_WAIT_NS) *failed = 1;
  }
}
__device__ __forceinline__ void tc_wait(uint32_t bar, uint32_t parity, volatile int* failed) {
  if (!tc_try(bar, parity)) tc_wait_slow(bar, parity, failed);
}
__device__ __forceinline__ void tc_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
// (the whole warp comes here, so that the compiler keeps addresses in uniform registers, which these instructions take: one
// thread by itself needed 200 cycles per MMA)
__device__ __forceinline__ void tc_commit(uint32_t bar, bool leader) {
  if (leader) asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory operand of 128-byte rows of 64 elements, 16-byte pieces XORed with the row's number modulo 8 (128-byte
// swizzle), eight rows to 1024 bytes: the descriptor's halves.  `lead`: bytes between blocks of 64 elements along M or N
// where those are contiguous (values: rows are tokens, the contraction's index).
constexpr uint32_t TC_DESC_HIGH = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t tc_desc(uint32_t addr, uint32_t lead) { return (addr >> 4) | (lead >> 4) << 16; }
// fp32 accumulators, binary16 operands, M 128; B's contiguous index: the contraction's, or (turned) N
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool turned) {
  return 1u << 4 | (turned ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}
template <uint32_t IDESC>
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t x, uint32_t y, bool add, bool leader) {
  if (leader)
    asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n"
                 :: "r"(d), "r"(x), "r"(y), "r"(IDESC), "r"((uint32_t)add), "r"(TC_DESC_HIGH) : "memory");
}
template <uint32_t IDESC>
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t x, uint32_t y, bool add, bool leader) {
  if (leader)
    asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n"
                 :: "r"(d), "r"(x), "r"(y), "r"(IDESC), "r"((uint32_t)add), "r"(TC_DESC_HIGH) : "memory");
}
__device__ __forceinline__ bool tc_elect() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}

// 32 columns of this warp's 32 lanes, a lane's in one thread
__device__ __forceinline__ void tc_ld32(uint32_t (&v)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
        "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(at));
}
__device__ __forceinline__ void tc_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :: "r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
         "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t (&v)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(at));
}
__device__ __forceinline__ void tc_ld8(uint32_t (&v)[8], uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(at));
}
// (the loaded registers are tied to the wait, so that nothing reads them before it)
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]) :: "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]),
        "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]) :: "memory");
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]),
        "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]),
        "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
        "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31]) :: "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// piece `c` (16 bytes, eight elements) of row r of an operand of `rows` rows
__device__ __forceinline__ uint32_t tc_place(int rows, int r, int c) {
  return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

}  // namespace kvq
