// 8-bit activation checkpoints and the SwiGLU's backward pass.
//
// Format (OCP MXINT8: int8 elements, one e8m0 scale per 32 along the row): for a block of
// 32 bf16 values, s is the exponent field of the largest magnitude (floor(log2) + 127, 0
// for zeros and subnormals), a code c is the value in steps of 2^(s-133), rounded to
// nearest even and clamped to +-127, and it stands for c * 2^(s-133). bf16 has 8
// significant bits, so the largest value of a block is at most 127.5 steps and no value is
// off by more than half a step; every c * 2^(s-133) is itself a bf16 number. A block with
// an infinity or a NaN has s = 255 and codes 0, and all of it reads back as NaN.
//
// All four kernels stream 16-byte vectors of 8 bf16 (8 codes are 8 bytes); four
// neighbouring lanes hold one block of 32, so a block's scale is two shuffles. The arithmetic
// is about 4 instructions an element for the codes and 15 for the SwiGLU's gradients, which keeps
// issue three quarters busy beside HBM in all but the decoding kernel (32768 rows, under ncu with
// cold caches: codes 0.72 an issue slot and DRAM 67 %, values 0.48 and 59 %, SwiGLU with codes 0.77 and 54
// %, its gradients from codes 0.76 and 61 %); among other passes they run at 0.93 to 0.98 of the
// copy rate (2048 columns to codes and back 63.5 us, 62.0 at that rate).
#include <cstdint>
#include <cuda_runtime.h>

#include "gnf4_act8.cuh"
#include "gnf4_kernels.h"

namespace gnf4 {

namespace {

// small CTAs, as many as the data has, one pass each (a grid of a few CTAs an SM that strides over it
// was 2 to 14 % slower: 41 us against 36 for the codes of 32768 x 2048, 42 against 39 for the SwiGLU)
constexpr int kActThreads = 128;
constexpr int kActVecs = 4;            // 16-byte vectors per thread (loads issued together)
constexpr int kSwigluActVecs = 2;      // the SwiGLU kernels hold three or four arrays per vector

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// the block's scale: the largest exponent field of the 32 values held by four lanes
__device__ __forceinline__ uint32_t block_scale(const uint4& v) {
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7F807F80u, v.y & 0x7F807F80u),
                          __vmaxu2(v.z & 0x7F807F80u, v.w & 0x7F807F80u));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return m >> 7;
}

// four codes in the low bytes of c; 128 and -128 are one pattern there and become +-127
__device__ __forceinline__ uint32_t pack_codes(const uint32_t* c) {
    uint32_t w = prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u);
    const uint32_t y = w ^ 0x80808080u;
    if ((y - 0x01010101u) & ~y & 0x80808080u) {          // a byte is 0x80: the block's largest value rounded up
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((c[i] & 0xFFu) == 0x80u) w ^= ((int32_t)(c[i] << 9) < 0 ? 0xFFu : 0x01u) << (8 * i);
    }
    return w;
}

// A code is the value times 2^(133-s), at most 127.5 of either sign, rounded to nearest even:
// the fused multiply-add onto 1.5 * 2^23 leaves the integer in the low mantissa bits (two's
// complement, bit 22 clear for a negative one), with one rounding.
__device__ __forceinline__ uint2 encode8(const uint4& v, uint32_t s) {
    if (s == 255u) return make_uint2(0u, 0u);
    uint32_t c[8];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    // 2^(133-s) is an fp32 number for s >= 6; below that in two exact steps
    const float up = __uint_as_float((260u - max(s, 6u)) << 23);
    const float more = s < 6u ? __uint_as_float((133u - s) << 23) : 1.0f;
    if (s < 6u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[2 * i] = __float_as_uint(fmaf(lo_f(w[i]) * more, up, 12582912.0f));
            c[2 * i + 1] = __float_as_uint(fmaf(hi_f(w[i]) * more, up, 12582912.0f));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[2 * i] = __float_as_uint(fmaf(lo_f(w[i]), up, 12582912.0f));
            c[2 * i + 1] = __float_as_uint(fmaf(hi_f(w[i]), up, 12582912.0f));
        }
    }
    return make_uint2(pack_codes(c), pack_codes(c + 4));
}

__device__ __forceinline__ uint4 decode8(const uint2& q, uint32_t s) {
    const uint32_t step = act8_step_bf16(s) * 0x00010001u;
    return make_uint4(act8_pair(prmt(q.x, 0u, 0x0100u), step), act8_pair(prmt(q.x, 0u, 0x0302u), step),
                      act8_pair(prmt(q.y, 0u, 0x0100u), step), act8_pair(prmt(q.y, 0u, 0x0302u), step));
}

// r = i / d in 32 bits: a multiplication and two shifts (the round-up method of Granlund
// and Montgomery, 1994)
struct Divider {
    uint32_t d, m, s;
    __device__ uint32_t operator()(uint32_t i) const {
        const uint32_t t = __umulhi(m, i);
        return (t + ((i - t) >> 1)) >> s;
    }
    __device__ int64_t operator()(int64_t i) const { return i / (int64_t)d; }
};

// total: 16-byte vectors; a multiple of 4, so the four lanes of a block are all in range or all out
__global__ void __launch_bounds__(kActThreads) quantize_act8_kernel(const uint4* __restrict__ x, uint2* __restrict__ codes,
                                                                    uint8_t* __restrict__ scales, int64_t total) {
    const int64_t base = (int64_t)blockIdx.x * (kActThreads * kActVecs) + threadIdx.x;
    uint4 v[kActVecs];
#pragma unroll
    for (int j = 0; j < kActVecs; ++j) {
        const int64_t i = base + j * kActThreads;
        v[j] = i < total ? __ldg(x + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < kActVecs; ++j) {
        const int64_t i = base + j * kActThreads;
        const uint32_t s = block_scale(v[j]);
        if (i < total) {
            codes[i] = encode8(v[j], s);
            if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
        }
    }
}

__global__ void __launch_bounds__(kActThreads) dequantize_act8_kernel(const uint2* __restrict__ codes,
                                                                      const uint8_t* __restrict__ scales,
                                                                      uint4* __restrict__ out, int64_t total) {
    const int64_t base = (int64_t)blockIdx.x * (kActThreads * kActVecs) + threadIdx.x;
    uint2 q[kActVecs];
    uint32_t s[kActVecs];
#pragma unroll
    for (int j = 0; j < kActVecs; ++j) {
        const int64_t i = base + j * kActThreads;
        if (i < total) {
            q[j] = __ldg(codes + i);
            s[j] = __ldg(scales + (i >> 2));
        }
    }
#pragma unroll
    for (int j = 0; j < kActVecs; ++j) {
        const int64_t i = base + j * kActThreads;
        if (i < total) out[i] = decode8(q[j], s[j]);
    }
}

__device__ __forceinline__ uint32_t silu_word(uint32_t g, uint32_t u) {
    return pack_bf16x2(silu_mul(lo_f(g), lo_f(u)), silu_mul(hi_f(g), hi_f(u)));
}

// out = silu(gate) * up with the same instructions as gnf4_swiglu, and the checkpoint of
// both halves. I8 = I / 8 vectors a row and half (a multiple of 4: blocks never straddle).
template <typename IDX>
__global__ void __launch_bounds__(kActThreads) swiglu_act8_kernel(const uint4* __restrict__ h, uint4* __restrict__ out,
                                                                  uint2* __restrict__ codes,
                                                                  uint8_t* __restrict__ scales, Divider by, IDX total) {
    const IDX I8 = (IDX)by.d;
    const IDX base = (IDX)blockIdx.x * (kActThreads * kSwigluActVecs) + threadIdx.x;
    uint4 g[kSwigluActVecs], u[kSwigluActVecs];
    int64_t at[kSwigluActVecs];              // vector index of the gate in the [R, 2I] rows
#pragma unroll
    for (int j = 0; j < kSwigluActVecs; ++j) {
        const IDX i = base + (IDX)j * kActThreads;
        g[j] = u[j] = make_uint4(0u, 0u, 0u, 0u);
        at[j] = 0;
        if (i < total) {
            const IDX r = by(i);
            at[j] = (int64_t)i + (int64_t)r * I8;      // r * 2 I8 + (i - r I8)
            g[j] = __ldg(h + at[j]);
            u[j] = __ldg(h + at[j] + I8);
        }
    }
#pragma unroll
    for (int j = 0; j < kSwigluActVecs; ++j) {
        const IDX i = base + (IDX)j * kActThreads;
        const uint32_t sg = block_scale(g[j]), su = block_scale(u[j]);
        if (i < total) {
            out[i] = make_uint4(silu_word(g[j].x, u[j].x), silu_word(g[j].y, u[j].y),
                                silu_word(g[j].z, u[j].z), silu_word(g[j].w, u[j].w));
            codes[at[j]] = encode8(g[j], sg);
            codes[at[j] + I8] = encode8(u[j], su);
            if ((i & 3) == 0) {
                scales[at[j] >> 2] = (uint8_t)sg;
                scales[(at[j] + I8) >> 2] = (uint8_t)su;
            }
        }
    }
}

// With e = exp(-|g|) and v = 1 / (1 + e): sig = sigmoid(g) is v or e v by g's sign and 1 - sig
// the other one, so neither is a difference of near numbers. silu has the instructions of
// silu_mul (a fast division by 1 + e is a multiplication by v), so act has gnf4_swiglu's bits.
//   d_gate = d (u (sig + silu (1 - sig))),  d_up = d silu,  act = silu u
__device__ __forceinline__ void swiglu_grad(float g, float u, float d, float& dg, float& du, float& act) {
    const float e = exp_via_ex2(-fabsf(g));
    const float v = __fdividef(1.0f, 1.0f + e), ev = e * v;
    const float sig = g >= 0.0f ? v : ev, rest = g >= 0.0f ? ev : v;
    const float silu = (g >= 0.0f ? g : g * e) * v;
    dg = d * (u * fmaf(silu, rest, sig));
    du = d * silu;
    act = silu * u;
}

__device__ __forceinline__ void swiglu_grad_word(uint32_t g, uint32_t u, uint32_t d, uint32_t& dg, uint32_t& du,
                                                 uint32_t& act) {
    float a[2], b[2], c[2];
    swiglu_grad(lo_f(g), lo_f(u), lo_f(d), a[0], b[0], c[0]);
    swiglu_grad(hi_f(g), hi_f(u), hi_f(d), a[1], b[1], c[1]);
    dg = pack_bf16x2(a[0], a[1]);
    du = pack_bf16x2(b[0], b[1]);
    act = pack_bf16x2(c[0], c[1]);
}

// Q8: gate_up comes from its checkpoint. again (may be null): silu(gate) * up once more.
template <typename IDX, bool Q8>
__global__ void __launch_bounds__(kActThreads) swiglu_backward_kernel(const uint4* __restrict__ d,
                                                                      const uint4* __restrict__ h,
                                                                      const uint2* __restrict__ codes,
                                                                      const uint8_t* __restrict__ scales,
                                                                      uint4* __restrict__ dh, uint4* __restrict__ again,
                                                                      Divider by, IDX total) {
    const IDX I8 = (IDX)by.d;
    const IDX base = (IDX)blockIdx.x * (kActThreads * kSwigluActVecs) + threadIdx.x;
    uint4 g[kSwigluActVecs], u[kSwigluActVecs], dv[kSwigluActVecs];
    uint2 qg[kSwigluActVecs], qu[kSwigluActVecs];
    uint32_t sg[kSwigluActVecs], su[kSwigluActVecs];
    int64_t at[kSwigluActVecs];
#pragma unroll
    for (int j = 0; j < kSwigluActVecs; ++j) {
        const IDX i = base + (IDX)j * kActThreads;
        if (i < total) {
            const IDX r = by(i);
            at[j] = (int64_t)i + (int64_t)r * I8;
            dv[j] = __ldg(d + i);
            if (Q8) {
                qg[j] = __ldg(codes + at[j]);
                qu[j] = __ldg(codes + at[j] + I8);
                sg[j] = __ldg(scales + (at[j] >> 2));
                su[j] = __ldg(scales + ((at[j] + I8) >> 2));
            } else {
                g[j] = __ldg(h + at[j]);
                u[j] = __ldg(h + at[j] + I8);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kSwigluActVecs; ++j) {
        const IDX i = base + (IDX)j * kActThreads;
        if (i < total) {
            if (Q8) {
                g[j] = decode8(qg[j], sg[j]);
                u[j] = decode8(qu[j], su[j]);
            }
            uint4 dg, du, act;
            swiglu_grad_word(g[j].x, u[j].x, dv[j].x, dg.x, du.x, act.x);
            swiglu_grad_word(g[j].y, u[j].y, dv[j].y, dg.y, du.y, act.y);
            swiglu_grad_word(g[j].z, u[j].z, dv[j].z, dg.z, du.z, act.z);
            swiglu_grad_word(g[j].w, u[j].w, dv[j].w, dg.w, du.w, act.w);
            dh[at[j]] = dg;
            dh[at[j] + I8] = du;
            if (again) again[i] = act;
        }
    }
}

// the sizes that are let in (2^41 elements) make 2^30 CTAs at most
int act_grid(int64_t total, int per_thread) {
    const int64_t per_cta = (int64_t)kActThreads * per_thread;
    return (int)((total + per_cta - 1) / per_cta);
}

// I8 vectors a row, 1 < I8 < 2^31 (1 has no shift of its own: the 64-bit kernels take it)
Divider divider(int64_t I8) {
    Divider v{(uint32_t)I8, 0u, 0u};
    int l = 0;
    while ((1ll << l) < I8) ++l;
    if (l > 0) {
        v.m = (uint32_t)(((1ull << 32) * ((1ull << l) - (uint64_t)I8)) / (uint64_t)I8 + 1);
        v.s = (uint32_t)(l - 1);
    }
    return v;
}

// whether every index that the CTAs of `total` vectors form fits in 32 bits
bool fits_u32(int64_t total, int64_t I8) {
    return total <= (int64_t)UINT32_MAX - kActThreads * kSwigluActVecs && I8 > 1;
}

}  // namespace

cudaError_t launch_quantize_act8(const void* x, int64_t n, int8_t* codes, uint8_t* scales, cudaStream_t s) {
    const int64_t total = n / 8;
    quantize_act8_kernel<<<act_grid(total, kActVecs), kActThreads, 0, s>>>(
        reinterpret_cast<const uint4*>(x), reinterpret_cast<uint2*>(codes), scales, total);
    return cudaGetLastError();
}

cudaError_t launch_dequantize_act8(const int8_t* codes, const uint8_t* scales, int64_t n, void* out, cudaStream_t s) {
    const int64_t total = n / 8;
    dequantize_act8_kernel<<<act_grid(total, kActVecs), kActThreads, 0, s>>>(
        reinterpret_cast<const uint2*>(codes), scales, reinterpret_cast<uint4*>(out), total);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_act8(const void* gate_up, int64_t R, int64_t I, void* out, int8_t* codes, uint8_t* scales,
                               cudaStream_t s) {
    const int64_t I8 = I / 8, total = R * I8;
    const int grid = act_grid(total, kSwigluActVecs);
    const uint4* h = reinterpret_cast<const uint4*>(gate_up);
    uint4* o = reinterpret_cast<uint4*>(out);
    uint2* q = reinterpret_cast<uint2*>(codes);
    if (fits_u32(total, I8))
        swiglu_act8_kernel<uint32_t><<<grid, kActThreads, 0, s>>>(h, o, q, scales, divider(I8), (uint32_t)total);
    else
        swiglu_act8_kernel<int64_t><<<grid, kActThreads, 0, s>>>(h, o, q, scales, divider(I8), total);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_backward(const void* d_out, const void* gate_up, const int8_t* codes, const uint8_t* scales,
                                   int64_t R, int64_t I, void* d_gate_up, void* again, cudaStream_t s) {
    const int64_t I8 = I / 8, total = R * I8;
    const int grid = act_grid(total, kSwigluActVecs);
    const uint4* d = reinterpret_cast<const uint4*>(d_out);
    const uint4* h = reinterpret_cast<const uint4*>(gate_up);
    const uint2* q = reinterpret_cast<const uint2*>(codes);
    uint4* dh = reinterpret_cast<uint4*>(d_gate_up);
    uint4* a = reinterpret_cast<uint4*>(again);
    const bool small = fits_u32(total, I8);
    if (gate_up && small)
        swiglu_backward_kernel<uint32_t, false><<<grid, kActThreads, 0, s>>>(d, h, q, scales, dh, a, divider(I8), (uint32_t)total);
    else if (gate_up)
        swiglu_backward_kernel<int64_t, false><<<grid, kActThreads, 0, s>>>(d, h, q, scales, dh, a, divider(I8), total);
    else if (small)
        swiglu_backward_kernel<uint32_t, true><<<grid, kActThreads, 0, s>>>(d, h, q, scales, dh, a, divider(I8), (uint32_t)total);
    else
        swiglu_backward_kernel<int64_t, true><<<grid, kActThreads, 0, s>>>(d, h, q, scales, dh, a, divider(I8), total);
    return cudaGetLastError();
}

}  // namespace gnf4
