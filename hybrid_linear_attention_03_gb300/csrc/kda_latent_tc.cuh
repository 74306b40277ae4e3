// kda_latent_tc.cuh -- what the latent-attention kernels on the tensor cores share
// beyond kda_attend_tc.cuh.
#pragma once

#include "kda_attend_tc.cuh"
#include "kda_latent.cuh"

namespace kda {
namespace kv {
namespace {

// Descriptors of bf16 operands swizzled over 128 bytes (sdesc_sw128, sdesc_sw128_mn) differ in their low words
// alone, which hold the address: products take those, and steps through an operand are 32-bit additions.
// (As 64-bit numbers the descriptors of a loop of products spilled, and a product took three times as long to issue.)
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t lbo) {
    return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) & 0x3FFFu) << 16;
}
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
// Likewise of e4m3 values, rows of 128 of them.
__device__ __forceinline__ void mma_lo_e4m3(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], A bf16 with two K values a column.
__device__ __forceinline__ void mma_lo_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}

// wait_for of two and three barriers, looked at one after the other without waiting in between, which takes little
// longer than one look.  The first one is passed before the others are looked at for good: where its passing is what
// makes a wait by parity for them sound, it stands first.
struct Awaited {
    uint64_t *bar;
    uint32_t parity;
};
__device__ __forceinline__ void wait_all(bool &ok, uint32_t *err, Awaited a, Awaited b, Awaited c) {
#ifndef KDA_ATTEND_LOOKS
    const bool in_a = mbar_try_wait(a.bar, a.parity), in_b = mbar_try_wait(b.bar, b.parity), in_c = mbar_try_wait(c.bar, c.parity);
    if (in_a && in_b && in_c) return;
#endif
    wait_for(ok, a.bar, a.parity, err);
    wait_for(ok, b.bar, b.parity, err);
    wait_for(ok, c.bar, c.parity, err);
}
// Tile t's barrier of a ring.
__device__ __forceinline__ Awaited of_tile(uint64_t *bars, uint32_t t) { return Awaited{&bars[t % kBars], (t / kBars) & 1}; }

// The products of one warp in one piece: those of two warps that issue at the same time would go by turns, and both
// be done when the later one is.  A place in shared memory that holds 1 while taken; whoever waits too long goes on, which
// costs time and nothing else.  One lane.
__device__ __forceinline__ void take_turn(uint32_t *place) {
    for (int i = 0; i < 4096 && atomicCAS(place, 0u, 1u) != 0u; ++i) {
    }
}
__device__ __forceinline__ void end_turn(uint32_t *place) { *reinterpret_cast<volatile uint32_t *>(place) = 0; }

}  // namespace
}  // namespace kv
}  // namespace kda
