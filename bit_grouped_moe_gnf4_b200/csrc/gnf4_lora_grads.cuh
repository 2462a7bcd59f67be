// What the two kernels of the adapters' gradients share: which item of the work a CTA has, and
// the launch.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "gnf4_lora.cuh"

namespace gnf4 {

// CTAs (or clusters) of one adapter for one gradient; none for a gradient that is not asked for
__host__ __device__ __forceinline__ int grad_items(const LoraGradSide& d, int cols) {
    return d.out ? (d.C + cols - 1) / cols : 0;
}

// adapters of more than p.heavy rows, at most
__host__ __device__ __forceinline__ int most_heavy(const LoraGradArgs& p) {
    const int64_t n = p.R / p.heavy;
    return n < p.L ? (int)n : p.L;
}

// An accumulating matrix instruction cuts its sum off at 24 bits instead of rounding it, so a chain of
// them falls short by up to 2^-23 of the sum each (2^-25.8 on average), always to the same side:
// 2^20 rows of one adapter, all products positive, left fp32 gradients 1.9e-4 (ranks up to 32) and
// 7.3e-4 of their value short. So the accumulators are emptied into totals that are added up in fp32,
// rounded to nearest: with three terms (fp32 results) after 48 instructions, 2^-20 short, with two
// (bf16 results) after 4096, 2^-13.8, which the result's 2^-9 hides.
template <int TERMS>
constexpr int kGradChain = TERMS == 3 ? 8 : 1024;        // stages of 32 rows

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Called by a whole warp, first of all: a CTA of a kernel that allocates tensor memory has its SM to
// itself until it gives up its permit to.
template <int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t* to) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(to)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS>
__device__ __forceinline__ void tmem_free(uint32_t at) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "n"(COLS));
}
// 16 columns of this warp's lanes
__device__ __forceinline__ void tmem_load16(float (&v)[16], uint32_t at) {
    uint32_t u[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(u[k]);
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
          "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]) : "memory");
}
// 4 columns
__device__ __forceinline__ float4 tmem_load4(uint32_t at) {
    float4 v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    return v;
}
__device__ __forceinline__ void tmem_store4(uint32_t at, const float (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}

struct GradItem {
    int e;                      // the adapter; L: nothing to do
    int col0, parts, part;      // first column; of how many parts of the rows this CTA has which
    bool side_b;
};
struct GradSearch {             // in shared memory
    int warp[kLoraWarps], adapter;
};

// A cluster has one unit of the work. Without p.heavy a unit is an item (an adapter's `cols`
// columns for one of the gradients), its rows shared by the cluster's CTAs. With p.heavy, the
// items of adapters of more rows than that are such units, and the others' items go one to a CTA:
// a routing that prefers a few adapters would leave the whole call waiting for the CTAs of the
// largest. Only the units of heavy adapters, of which there are as many as the rows can make,
// look for theirs; a CTA of the others has its item by its number, and nothing to do if the item
// is a heavy adapter's. dB's units come first: they need nothing of the rows kernel and fill the
// SMs that it leaves.
__device__ __forceinline__ GradItem grad_item(const LoraGradArgs& p, int cols, GradSearch* find) {
    const int CS = (int)cluster_size(), crank = (int)cluster_rank();
    const int na = grad_items(p.a, cols), nb = grad_items(p.b, cols), unit = (int)(blockIdx.x / CS);
    GradItem it;
    if (p.heavy == 0) {
        it.side_b = unit < p.L * nb;
        const int n = it.side_b ? nb : na, item = it.side_b ? unit : unit - p.L * nb;
        it.e = item / n;
        it.col0 = item % n * cols;
        it.parts = CS;
        it.part = crank;
        return it;
    }
    auto is_heavy = [&](int q) { return clamp_row(p.offsets[q + 1], p.R) - clamp_row(p.offsets[q], p.R) > p.heavy; };
    const int most = most_heavy(p), units_b = most * nb + (p.L * nb + CS - 1) / CS;
    it.side_b = unit < units_b;
    const int n = it.side_b ? nb : na;
    int item = it.side_b ? unit : unit - units_b;
    const bool shared = item < most * n;
    if (!shared) item = (item - most * n) * CS + crank;
    it.e = item / n;                                     // of the heavy adapters, or of all
    it.col0 = item % n * cols;
    it.parts = shared ? CS : 1;
    it.part = shared ? crank : 0;
    if (!shared) {
        if (it.e < p.L && is_heavy(it.e)) it.e = p.L;
        return it;
    }
    // the it.e-th heavy adapter, counted over runs of neighbouring ones, a run a thread
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (p.L + kLoraThreads - 1) / kLoraThreads;
    const int e0 = min(tid * per, p.L), e1 = min(e0 + per, p.L);
    int mine = 0;
    for (int q = e0; q < e1; ++q) mine += is_heavy(q);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) find->warp[warp] = upto;
    if (tid == 0) find->adapter = p.L;
    __syncthreads();
    int before = upto - mine;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) before += w < warp ? find->warp[w] : 0;
    int k = it.e - before;
    if (k >= 0 && k < mine)
        for (int q = e0; q < e1; ++q)
            if (is_heavy(q) && k-- == 0) find->adapter = q;
    __syncthreads();
    it.e = find->adapter;
    return it;
}

// The end of an item: a CTA's sums, RP rows (ranks) by CW columns at s_red, SC columns side by side in a
// row of STRIDE floats and RP rows below one another, are added up over the cluster and stored.
template <int RP, int CW, int SC, int STRIDE, int TERMS>
__device__ __forceinline__ void store_sums(const LoraGradArgs& p, const LoraGradSide& d, const GradItem& it, float* s_red) {
    const int tid = threadIdx.x, e = it.e, col0 = it.col0, parts = it.parts, part = it.part;
    // the cluster's CTAs share the columns out and add up theirs, in place: no other CTA reads those
    const int own = CW / parts, own0 = part * own;
    if (parts > 1) {
        cluster_arrive();
        cluster_wait();
        for (int i = tid; i < RP * own / 4; i += kLoraThreads) {
            const int j = i / (own / 4), n = own0 + 4 * (i % (own / 4));
            float* at = s_red + (size_t)(n / SC) * RP * STRIDE + j * STRIDE + n % SC;
            *reinterpret_cast<float4*>(at) = cluster_sum(at, parts);
        }
        cluster_arrive();                                // a CTA's sums are read until here
        __syncthreads();
    }
    // eight at a time along the gradient's contiguous axis: its columns (dA) or the rank (dB); C
    // and r are multiples of 8
    for (int i = tid; i < own * RP / 8; i += kLoraThreads) {
        // dA: (rank, columns n..); dB: (column, ranks j..), the pieces of a column's ranks in turn
        const int j = d.transposed ? 8 * (i % (RP / 8)) : i / (own / 8);
        const int n = own0 + (d.transposed ? i / (RP / 8) : 8 * (i % (own / 8)));
        if (j >= p.r || col0 + n >= d.C) continue;
        const float* at = s_red + (size_t)(n / SC) * RP * STRIDE + j * STRIDE + n % SC;
        const int next = d.transposed ? STRIDE : 1;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = at[k * next];
        const int64_t o = (int64_t)e * p.r * d.C + (d.transposed ? (int64_t)(col0 + n) * p.r + j : (int64_t)j * d.C + col0 + n);
        if constexpr (TERMS == 3) {
            float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(d.out) + o);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(d.out) + o) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
    }
    if (parts > 1) cluster_wait();
}

// a cluster of cs CTAs for each unit that the rows can make
template <void (*KERNEL)(LoraGradArgs)>
cudaError_t launch_grads_kernel(const LoraGradArgs& a, int cols, int cs, int smem, cudaStream_t s) {
    static std::atomic<bool> attr_set[64];
    const int dev = current_device();
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const int na = grad_items(a.a, cols), nb = grad_items(a.b, cols);
    int64_t clusters = (int64_t)a.L * (na + nb);
    if (a.heavy) {
        clusters = most_heavy(a) * (int64_t)(na + nb) + (a.L * (int64_t)nb + cs - 1) / cs + (a.L * (int64_t)na + cs - 1) / cs;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * cs));
    cfg.blockDim = dim3(kLoraThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.after_rows ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, KERNEL, a);
}

// The rows from which an adapter is heavy: four times the average's, 256 at least, and a 32nd of
// all, so that the units kept for heavy adapters stay few; 0 if there is no room for one. An
// average below 8 rows, or fewer than 1024 in all, has no search: what one adapter with all rows
// would cost is then less than what the call costs for its adapters anyway. us of a backward pass at
// 2048 and 1536 columns, rank 16, without and with the search, the rows spread evenly and then
// all one adapter's: 2048 adapters, 32768 rows 392 to 431 and 1188 to 455, 4096 rows 383 to 420
// and 253 to 213; 200 adapters, 4096 rows 47 to 51 and 179 to 61, 2048 rows 43 to 47 and 89 to
// 45, 1024 rows 37 to 41 and 55 to 32; 128 adapters, 32768 rows 123 to 125 and 1545 to 440.
inline int heavy_rows(int64_t R, int64_t avg) {
    int64_t heavy = 4 * avg > 256 ? 4 * avg : 256;
    if (heavy < R / 32) heavy = R / 32;
    return avg < 8 || R < 1024 || heavy >= R ? 0 : (int)heavy;
}

// Whether a CTA (or `warps` of its warps that share the rows of a stage) can get more rows than a chain
// has: all rows may be one adapter's, which the cs CTAs of its cluster share, or a single CTA
// has the rows from which an adapter is heavy. The kernels with totals take longer, us of a backward
// pass with fp32 results at 2048 and 1536 columns, without and with them: 128 adapters, 32768 rows,
// rank 16 131.7 and 136.2, rank 32 174.0 and 179.9; 64 adapters, 8192 rows, rank 64 87.5 and 92.7,
// rank 128 219 and 222; one adapter of 65536 rows, rank 32 414 and 429, rank 64 575 and 624.
inline bool past_chain(const LoraGradArgs& a, int cs, int warps, int chain) {
    const int64_t most = a.heavy * (int64_t)cs > a.R ? a.heavy * (int64_t)cs : a.R;
    return most > (int64_t)32 * chain * warps * cs;
}

// ranks above 32 (gnf4_lora_grads_wide.cu)
cudaError_t launch_lora_grads_wide(const LoraGradArgs& a, bool f32, cudaStream_t s);

}  // namespace gnf4
