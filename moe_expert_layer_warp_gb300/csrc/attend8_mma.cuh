// attend8_mma.cuh — what attention over a cache in 8 bits needs of tcgen05
// beyond attend_mma.cuh: products of 8-bit operands, whose rows may run along K
// or across it, and short loads and stores of tensor memory.
#pragma once

#include "attend_mma.cuh"

namespace moe {
namespace umma {

// Instruction descriptor of kind::f8f6f4 (whose operands' types are independent):
// A e4m3, B e4m3 or e5m2, fp32 accumulators; mn: both with rows that run along K
// (else both K-major). M 64 or 128, N a multiple of 16.
MOE_DEV uint32_t idesc_f8(int M, int N, bool b_e5m2, bool mn) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | (mn ? 3u << 15 : 0u) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The high word of a shared-memory descriptor: tiles of rows of 128 or 64 bytes,
// swizzled at that width, 8-row groups 1024 or 512 bytes apart.
template <int kRow>
constexpr uint32_t kDescHi8 =
    ((kRow * 8u) >> 4) | (1u << 14) | ((kRow == 128 ? 2u : 4u) << 29);

// kSteps K-steps of 32 elements, issued by one elected lane of a converged warp
// (see mma4_ss). alo, blo: low words of the operands' descriptors at the first
// step; kA, kB: what a step adds to them, in 16-byte units.
template <int kSteps, uint32_t kAHi, uint32_t kBHi, int kA, int kB>
MOE_DEV void mma_f8(uint32_t tmem_d, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t acc) {
  static_assert(kSteps == 2 || kSteps == 4, "steps");
  if constexpr (kSteps == 4) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, %7;\n\tadd.s64 b, b, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.s64 a, a, %7;\n\tadd.s64 b, b, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t"
        "add.s64 a, a, %7;\n\tadd.s64 b, b, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t}"
        ::"r"(tmem_d), "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "n"(kAHi), "n"(kBHi), "n"(kA),
        "n"(kB)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %6};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, %7;\n\tadd.s64 b, b, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, 1;\n\t}"
        ::"r"(tmem_d), "r"(alo), "r"(blo), "r"(idesc), "r"(acc), "n"(kAHi), "n"(kBHi), "n"(kA),
        "n"(kB)
        : "memory");
  }
}

// 4 consecutive columns of the thread's lane (16: tcgen05.cuh), and one, and the
// reverse for that.
MOE_DEV void ld_x4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}
MOE_DEV uint32_t ld_x1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
               : "=r"(r)
               : "r"(taddr)
               : "memory");
  return r;
}
MOE_DEV void st_x1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%1], {%0};" ::"r"(v), "r"(taddr) : "memory");
}

}  // namespace umma
}  // namespace moe
