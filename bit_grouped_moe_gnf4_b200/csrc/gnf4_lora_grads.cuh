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

// ranks above 32 (gnf4_lora_grads_wide.cu)
cudaError_t launch_lora_grads_wide(const LoraGradArgs& a, bool f32, cudaStream_t s);

}  // namespace gnf4
