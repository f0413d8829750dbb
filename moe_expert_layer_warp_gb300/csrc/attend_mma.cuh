// attend_mma.cuh — what attention needs of tcgen05 and TMA beyond the expert
// kernels' tcgen05.cuh and common.cuh: fp16 operands, A from tensor memory, B
// with rows along K, whole K-blocks issued by a converged warp.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace moe {

// (dst: an address in the shared window)
MOE_DEV void tma_load_4d_at(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar)),
      "l"(policy)
      : "memory");
}

namespace umma {

// Instruction descriptor, fp32 accumulators: A and B both fp16 (f16) or both
// bf16, A K-major, B K-major or with rows that run along K (b_mn: N contiguous).
MOE_DEV uint32_t idesc_f16(int M, int N, bool f16, bool b_mn) {
  const uint32_t t = f16 ? 0u : 1u;
  return (1u << 4) | (t << 7) | (t << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A shared-memory descriptor in two words: the high one is the same for every
// 128-byte-swizzled tile with 8-row groups 1024 bytes apart, and the low one
// moves with the address (16-byte units; it never carries, shared memory ends
// below 2^18). A tile whose rows run along K (row k holds 64 elements of N,
// 128 bytes) gives the distance of the next 64 elements of N as n_stride; its
// K-step of 16 advances the address by 2048 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
MOE_DEV uint32_t desc_lo(uint32_t smem_byte_addr, uint32_t n_stride) {
  return ((smem_byte_addr >> 4) & 0x3FFFu) | ((n_stride ? n_stride >> 4 : 1u) << 16);
}

// Four K-steps (64 elements of K) in one go, issued by one elected lane of a
// converged warp; `alo`, `blo` are the low words of the operands' descriptors
// at the first step. With the whole sequence in one block and the operands
// equal in every lane, issuing an MMA costs less than the MMA takes; from a
// divergent branch with a 64-bit descriptor each it cost 75 cycles apiece.
// mma4_ss: A and B both K-major tiles in shared memory.
MOE_DEV void mma4_ss(uint32_t tmem_d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
      "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n\t"
      "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n\t"
      "add.s64 a, a, 2;\n\tadd.s64 b, b, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, 1;\n\t}"
      ::"r"(tmem_d), "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

// mma4_ts: A from tensor memory (row r is lane r, two 16-bit elements per
// column along K), B a tile whose rows run along K (desc_lo with n_stride).
MOE_DEV void mma4_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t blo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b32 a, %1;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t"
      "add.s32 a, a, 8;\n\tadd.s64 b, b, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, 1;\n\t"
      "add.s32 a, a, 8;\n\tadd.s64 b, b, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, 1;\n\t"
      "add.s32 a, a, 8;\n\tadd.s64 b, b, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, 1;\n\t}"
      ::"r"(tmem_d), "r"(tmem_a), "r"(blo), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}

// umma::commit by the lane that mma4_ss and mma4_ts elect.
MOE_DEV void commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_addr(bar))
      : "memory");
}

MOE_DEV void ld_x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// The reverse of ld_x32: 32 consecutive columns of the thread's lane.
MOE_DEV void st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}

MOE_DEV void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace umma
}  // namespace moe
