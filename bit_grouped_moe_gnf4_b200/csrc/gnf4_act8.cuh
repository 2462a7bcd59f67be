// Reading an 8-bit activation checkpoint: the codes' values (format in gnf4_act8.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gnf4_common.cuh"

namespace gnf4 {

// one step of a block, 2^(s-133), as a bf16 pattern: a subnormal for s < 7, NaN for s = 255
__device__ __forceinline__ uint32_t act8_step_bf16(uint32_t s) {
    return s == 255u ? 0x7FC0u : s >= 7u ? (s - 6u) << 7 : 1u << s;
}

// Two codes, in bytes 0 and 2 of `codes` (the others are not looked at), times a pair of
// steps, as bf16 numbers; exact throughout. bf16 holds 128 + the low seven bits of a code as
// 0x4300 plus those bits, and 128 or 256, by the code's sign, is what is too much.
__device__ __forceinline__ uint32_t act8_pair(uint32_t codes, uint32_t steps) {
    const uint32_t low = (codes & 0x007F007Fu) | 0x43004300u, off = (codes & 0x00800080u) | 0x43004300u;
    uint32_t c, d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(low), "r"(off));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(c), "r"(steps));
    return d;
}

}  // namespace gnf4
