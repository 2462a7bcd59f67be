// Low-rank adapters beside a projection, for routed rows r sorted by adapter e:
//   forward    h_r = A_e x[tok r],           out[dest r] = base[dest r] + c_r B_e h_r
//   backward   g_r = c_r B_e^T dy[src r],    dx_r = base_dx_r + A_e^T g_r
//              dA_e = sum_r g_r x[tok r]^T,  dB_e = sum_r c_r dy[src r] h_r^T
// with c_r = scaling_e w_r. A [L, r, K], B [L, N, r].
//
// The forward, and the first line of the backward, are one chain of two products: the
// backward's has A and B swapped and both read along their other axis. Few rows go through
// gnf4_lora_rows.cu, many through gnf4_lora_stream.cu; the sums over an adapter's rows are in
// gnf4_lora_grads.cu and, for ranks above 32, gnf4_lora_grads_wide.cu. The rank is small, so all of
// it is bound by the rows it streams, by the adapters' bytes, by issue, or by latency. The products
// run on warp-level MMAs, but for the sums of the larger ranks, which run on tcgen05. The warp-level
// ones keep the tensor pipe busy for 14 to 20 % of the time over many rows at ranks up to 32, and
// longest at rank 64: 28 % over 4096 rows, 2880 -> 5760, 34 % in the backward's first half over 8192.
//
// Rounding: sums are fp32; long ones are cut into chains of matrix instructions, whose sums are added
// up rounded to nearest (kSumChain below, and kGradChain for the sums over rows). h (and g) enter the second product as two 16-bit terms, the value's
// rounding and that of its remainder: about 17 significant bits, so that what the caller sees
// is the one rounding of the output. For fp16 they are first scaled by a power of two per row,
// so that neither term leaves the type's range. The gradient sums take two terms for bf16
// results and three (24 bits) for fp32 results.
//
// This file: what the three have in common.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gnf4_common.cuh"
#include "gnf4_kernels.h"

namespace gnf4 {

constexpr int kLoraThreads = 256;
constexpr size_t kMaxSmem = 227 * 1024 - 512;      // dynamic shared memory of a CTA beside its static part
constexpr int kLoraWarps = kLoraThreads / 32;
// A matrix instruction cuts its accumulator off at 24 bits instead of rounding it (2^-25.8 of the sum on
// average, always to the same side), so after so many steps (two instructions each) of the first product
// a warp adds its accumulators to the partial sums and starts from nothing: up to 4096
// columns there is one such chain, 2^-20.8 short.
constexpr int kSumChain = 16;
constexpr long long kStallWaitCycles = 1LL << 17;   // where a test wants a wait to give up

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16x2(lo, hi);
    }
}

template <bool F16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        mma_bf16_16816(c, a0, a1, a2, a3, b0, b1);
}

// value = sum of TERMS bf16 (or fp16) numbers, each the rounding of what the ones before it
// leave; a value that is not finite stays in the first
template <int TERMS, bool F16>
__device__ __forceinline__ void split_pair(float v0, float v1, uint32_t (&o)[TERMS]) {
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        o[i] = pack16<F16>(v0, v1);
        const float2 f = unpack16<F16>(o[i]);
        v0 = isfinite(f.x) ? v0 - f.x : 0.0f;
        v1 = isfinite(f.y) ? v1 - f.y : 0.0f;
    }
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The sum over the cluster's CTAs of the four floats at `local` in their shared memory. All
// loads are issued before the first sum: one by one they would cost a microsecond each.
__device__ __forceinline__ float4 cluster_sum(const float* local, int size) {
    constexpr int kMost = 8;
    float4 v[kMost];
#pragma unroll
    for (int c = 0; c < kMost; ++c) {
        v[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < size) {
            uint32_t a;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(c));
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(v[c].x), "=f"(v[c].y), "=f"(v[c].z), "=f"(v[c].w) : "r"(a));
        }
    }
#pragma unroll
    for (int c = 1; c < kMost; ++c) {
        v[0].x += v[c].x;
        v[0].y += v[c].y;
        v[0].z += v[c].z;
        v[0].w += v[c].w;
    }
    return v[0];
}

// the grid behind this one may start where SMs are free (it waits for this one before it reads its results)
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// the grid before this one (the rows kernel of the same call) may still run: wait for it
__device__ __forceinline__ void wait_for_previous_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// rows of adapter e, kept inside [0, R] whatever the offsets hold
__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t R) { return v < 0 ? 0 : v > R ? R : v; }

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// 16 bytes to shared memory, zeros if bytes is 0
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&d)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&d)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(addr) : "memory");
}

// at most one partial tile of `rows` rows for every adapter that has a row
inline int64_t most_tiles(const LoraRowsArgs& a, int rows) {
    const int64_t active = a.R < a.L ? a.R : a.L;
    return active + (a.R - active) / rows;
}


// the streaming kernel's launch (ranks up to 64)
cudaError_t launch_lora_stream(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s);

}  // namespace gnf4
