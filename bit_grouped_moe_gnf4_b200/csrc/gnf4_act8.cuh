// Reading an 8-bit activation checkpoint: the codes' values (format in gnf4_act8.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gnf4_common.cuh"

namespace gnf4 {

// one step of a block, 2^(s-133): an fp32 subnormal for s < 7, NaN for s = 255
__device__ __forceinline__ float act8_step(uint32_t s) {
    if (s == 255u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(s >= 7u ? (s - 6u) << 23 : 1u << (s + 16u));
}

// The values of 8 codes, exact: 128 + c is placed in the low mantissa byte of 2^23, and
// 2^23 + 128 taken off again leaves c.
__device__ __forceinline__ void act8_values(const uint2& q, float step, float (&f)[8]) {
    const uint32_t u[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = (__uint_as_float(prmt(u[i >> 2], 0x4B000000u, 0x7440u + (i & 3))) - 8388736.0f) * step;
}

}  // namespace gnf4
