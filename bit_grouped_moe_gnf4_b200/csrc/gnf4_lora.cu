// Low-rank adapters beside a projection, for routed rows r sorted by adapter e:
//   forward    h_r = A_e x[tok r],           out[dest r] = base[dest r] + c_r B_e h_r
//   backward   g_r = c_r B_e^T dy[src r],    dx_r = base_dx_r + A_e^T g_r
//              dA_e = sum_r g_r x[tok r]^T,  dB_e = sum_r c_r dy[src r] h_r^T
// with c_r = scaling_e w_r. A [L, r, K], B [L, N, r].
//
// The rank is small, so every product is bound by the rows it streams (or, with few rows,
// by the adapters' bytes and latency), not by the tensor pipe: warp-level MMAs fed straight
// from 16-byte global loads, whose fragment layouts are reached by permuting the contraction
// index and the output columns instead of passing the operands through shared memory.
//
// lora_rows_kernel does the two products of the forward, or the first two of the backward
// (the same chain with A and B swapped and both read along their other axis), in one
// launch: a cluster of CTAs owns a tile of 16 or 32 rows of one adapter; its warps split the
// contraction of the first product, the partial sums meet in shared memory (and through
// distributed shared memory when the cluster has more than one CTA), and then the warps
// split the output columns of the second. x, base and out are touched once.
//
// lora_grads_kernel sums over an adapter's rows (below).
//
// Rounding: sums are fp32. h (and g) enter the second product as two 16-bit terms (value
// and remainder: about 17 significant bits, so that what the caller sees is the one
// rounding of the output); for fp16 they are first scaled by a power of two per row, so
// that neither term leaves the type's range. The gradient sums take two terms for bf16
// results and three (24 bits) for fp32 results.
#include <atomic>
#include <climits>
#include <cstdint>
#include <type_traits>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gnf4_act8.cuh"
#include "gnf4_kernels.h"

namespace gnf4 {

namespace {

constexpr int kLoraThreads = 256;
constexpr size_t kMaxSmem = 227 * 1024 - 512;      // dynamic shared memory of a CTA beside its static part
constexpr int kLoraWarps = kLoraThreads / 32;

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

// lane (g, t) holds row g, columns 2t, 2t+1 of an 8x8 matrix; afterwards rows 2t, 2t+1 of column g
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint2 ldg8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

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

struct Tile {
    int e, rows;
    int64_t row0;
};

// Tile `tile` of the list of all adapters' tiles of BM rows: each thread counts the tiles of
// a run of neighbouring adapters, a block scan places them, and the thread whose run covers
// the tile writes it down. s_tile->rows is 0 when the list is shorter.
template <int BM>
__device__ __forceinline__ void find_tile(const int64_t* offsets, int L, int64_t R, int tile, Tile* s_tile, int* s_warp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (L + kLoraThreads - 1) / kLoraThreads;
    const int e0 = min(tid * per, L), e1 = min(e0 + per, L);
    int mine = 0;
    int64_t lo = e0 < e1 ? clamp_row(offsets[e0], R) : 0;
    const int64_t first = lo;
    for (int e = e0; e < e1; ++e) {
        const int64_t hi = clamp_row(offsets[e + 1], R);
        if (hi > lo) mine += (int)((hi - lo + BM - 1) / BM);
        lo = hi;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) s_warp[warp] = incl;
    if (tid == 0) s_tile->rows = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += s_warp[w];
    int at = incl - mine;
    if (tile >= at && tile < incl) {
        lo = first;
        for (int e = e0; e < e1; ++e) {
            const int64_t hi = clamp_row(offsets[e + 1], R);
            const int n = hi > lo ? (int)((hi - lo + BM - 1) / BM) : 0;
            if (tile < at + n) {
                s_tile->e = e;
                s_tile->row0 = lo + (int64_t)(tile - at) * BM;
                s_tile->rows = (int)min((int64_t)BM, hi - s_tile->row0);
                break;
            }
            at += n;
            lo = hi;
        }
    }
    __syncthreads();
}

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

// RP: rank padded to 16, 32, 64 or 128; MT: 16-row MMA tiles of a CTA
template <int RP, int MT>
struct RowsShape {
    static constexpr int BM = 16 * MT, NT = RP / 8, KS = RP / 16;
    static constexpr int kPlane = RP + (RP >= 64 ? 32 : 0);          // 16-bit elements a row; conflict-free fragment loads
    static constexpr int kRed = RP + 8;                              // floats a row
    static constexpr size_t red = sizeof(float) * 4 * BM * kRed;     // partial sums of four warps
    static constexpr size_t plane = sizeof(uint16_t) * 2 * BM * kPlane;
    static constexpr size_t smem = red + plane + sizeof(float) * BM;
    static constexpr int kCtas = RP * MT <= 64 ? 2 : 1;              // that an SM's registers are to hold
};

// BWD: the backward's chain (first factor [L, C, r], second [L, r, O]) instead of the forward's
// ([L, r, C], [L, O, r]). A row that does not exist is computed from an address that does and
// not stored (rows do not mix), so only the last piece of an axis that is no multiple of 32
// is guarded element by element.
template <int RP, int MT, bool BWD, bool F16>
__global__ void __launch_bounds__(kLoraThreads, RowsShape<RP, MT>::kCtas) lora_rows_kernel(const LoraRowsArgs p) {
    using S = RowsShape<RP, MT>;
    constexpr int BM = S::BM, NT = S::NT, KS = S::KS;
    constexpr int V = RP >= 32 ? 4 : 2;           // rank tiles in one vector of the backward's first factor
    constexpr int G = RP >= 32 ? 2 : 1;           // MMA steps in one vector of the forward's second factor
    extern __shared__ __align__(16) uint8_t smem[];
    float* s_red = reinterpret_cast<float*>(smem);
    uint16_t* s_plane = reinterpret_cast<uint16_t*>(smem + S::red);
    float* s_fac = reinterpret_cast<float*>(smem + S::red + S::plane);
    __shared__ Tile s_tile;
    __shared__ int s_warp[kLoraWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int CS = (int)cluster_size(), crank = (int)cluster_rank();
    if (BWD) let_next_grid_start();
    find_tile<BM>(p.offsets, p.L, p.R, (int)(blockIdx.x / CS), &s_tile, s_warp);
    const int rows = s_tile.rows, e = s_tile.e;
    const int64_t row0 = s_tile.row0;
    if (rows == 0) return;                       // the same in every CTA of the cluster
    const int part = crank * kLoraWarps + warp, parts = CS * kLoraWarps;

    // ---- first product: [BM, C] x [C, r], the contraction split over all warps of the cluster
    {
        const uint16_t* src[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t r = row0 + min(16 * m + 8 * h + g, rows - 1);
                const int64_t at = p.src_row ? (int64_t)__ldg(p.src_row + r) : r;
                src[m][h] = p.src + (at >= 0 && at < p.n_src ? at * p.C : 0) + 8 * t;
            }
        // forward: rank row 8c + g, 16 bytes along the contraction; backward: contraction row
        // 8 (g>>1) + 2q + (g&1), its rank along the lanes' t
        const uint16_t* down = p.down + (int64_t)e * p.r * p.C +
                               (BWD ? (int64_t)(8 * (g >> 1) + (g & 1)) * p.r + 2 * V * t : (int64_t)g * p.C + 8 * t);
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][c][j] = 0.0f;
        auto step = [&](int k0, auto guard) {
            constexpr bool GUARD = decltype(guard)::value;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            const bool in = !GUARD || k0 + 8 * t < p.C;
            uint4 a[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) a[m][h] = in ? ldg16(src[m][h] + k0) : zero;
            // b[c]: this lane's contraction indices k0 + 8t .. 8t+7 of rank tile c, as four pairs
            uint32_t b[NT][4];
            if constexpr (!BWD) {
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const uint4 x = in && 8 * c < p.r ? ldg16(down + (int64_t)(8 * c) * p.C + k0) : zero;
                    b[c][0] = x.x, b[c][1] = x.y, b[c][2] = x.z, b[c][3] = x.w;
                }
            } else {
                // a transposed 8x8 matrix gives each lane its two rows of one column
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool inq = !GUARD || k0 + 8 * (g >> 1) + 2 * q + (g & 1) < p.C;
#pragma unroll
                    for (int v = 0; v < NT / V; ++v) {
                        const bool ok = inq && 8 * V * v + 2 * V * t < p.r;
                        const uint16_t* at = down + (int64_t)(k0 + 2 * q) * p.r + 8 * V * v;
                        if constexpr (V == 4) {
                            const uint4 x = ok ? ldg16(at) : zero;
                            b[V * v][q] = x.x, b[V * v + 1][q] = x.y, b[V * v + 2][q] = x.z, b[V * v + 3][q] = x.w;
                        } else {
                            const uint2 x = ok ? ldg8(at) : make_uint2(0u, 0u);
                            b[V * v][q] = x.x, b[V * v + 1][q] = x.y;
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) b[c][q] = transpose8x8(b[c][q]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    mma16<F16>(acc[m][c], a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y, b[c][0], b[c][1]);
                    mma16<F16>(acc[m][c], a[m][0].z, a[m][1].z, a[m][0].w, a[m][1].w, b[c][2], b[c][3]);
                }
        };
        const int whole = p.C / 32;
        const int st0 = (int)((int64_t)whole * part / parts), st1 = (int)((int64_t)whole * (part + 1) / parts);
#pragma unroll 2
        for (int st = st0; st < st1; ++st) step(32 * st, std::false_type{});
        if (part == parts - 1 && (p.C & 31)) step(32 * whole, std::true_type{});
        // partial sums: tile c, column index n of the MMA is rank 8c + n (forward), or
        // 8 V (c / V) + 2 V (n >> 1) + 2 (c % V) + (n & 1) (backward). The upper four warps put
        // theirs down, the lower four add their own on top.
        float* mine = s_red + (size_t)(warp & 3) * BM * S::kRed;
#pragma unroll
        for (int turn = 0; turn < 2; ++turn) {
            if ((warp < 4) == (turn == 1)) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            const int j = BWD ? 8 * V * (c / V) + 2 * V * t + 2 * (c % V) : 8 * c + 2 * t;
                            float2* at = reinterpret_cast<float2*>(mine + (16 * m + 8 * h + g) * S::kRed + j);
                            float2 v = make_float2(acc[m][c][2 * h], acc[m][c][2 * h + 1]);
                            if (turn == 1) {
                                const float2 o = *at;
                                v.x += o.x;
                                v.y += o.y;
                            }
                            *at = v;
                        }
            }
            __syncthreads();
        }
    }
    if (CS > 1) {
        // the CTA's sum in the first of the four places
        for (int i = tid; i < BM * RP; i += kLoraThreads) {
            float* at = s_red + (i / RP) * S::kRed + i % RP;
            *at = (at[0] + at[BM * S::kRed]) + (at[2 * BM * S::kRed] + at[3 * BM * S::kRed]);
        }
        cluster_arrive();
        cluster_wait();
    }
    // ---- the sums, their 16-bit terms and each row's output factor: RP / 4 lanes a row
    {
        constexpr int LPR = RP / 4 < 32 ? RP / 4 : 32, PER = RP / LPR;       // lanes a row, ranks a lane
        const float scal = p.scaling ? __ldg(p.scaling + e) : 1.0f;
        for (int i = tid; i < BM * LPR; i += kLoraThreads) {
            const int local = i / LPR, j = PER * (i % LPR);
            const int64_t r = row0 + local;
            float v[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) v[k] = 0.0f;
            float fac = scal;
            bool have = local < rows;
            if (have && p.weight) fac *= __ldg(p.weight + r);
            if (have && p.src_row) {
                const int at = __ldg(p.src_row + r);
                have = at >= 0 && at < p.n_src;                              // else h is zero
            }
            if (local < rows && j < p.r) {
                const float* at = s_red + local * S::kRed + j;
                if (have && CS > 1) {
#pragma unroll
                    for (int k = 0; k < PER; k += 4) {
                        const float4 a = cluster_sum(at + k, CS);
                        v[k] = a.x, v[k + 1] = a.y, v[k + 2] = a.z, v[k + 3] = a.w;
                    }
                } else if (have) {
#pragma unroll
                    for (int k = 0; k < PER; k += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(at + k);
                        const float4 b = *reinterpret_cast<const float4*>(at + k + BM * S::kRed);
                        const float4 c = *reinterpret_cast<const float4*>(at + k + 2 * BM * S::kRed);
                        const float4 d = *reinterpret_cast<const float4*>(at + k + 3 * BM * S::kRed);
                        v[k] = (a.x + b.x) + (c.x + d.x);
                        v[k + 1] = (a.y + b.y) + (c.y + d.y);
                        v[k + 2] = (a.z + b.z) + (c.z + d.z);
                        v[k + 3] = (a.w + b.w) + (c.w + d.w);
                    }
                }
                if (BWD) {
#pragma unroll
                    for (int k = 0; k < PER; ++k) v[k] *= fac;
                }
                if (crank == 0 && p.mid) {
#pragma unroll
                    for (int k = 0; k < PER; k += 4)
                        *reinterpret_cast<float4*>(p.mid + r * p.r + j + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                }
            }
            if (BWD) fac = 1.0f;
            if constexpr (F16) {
                // the row's largest value to [1, 2): both terms stay normal or fall below 2^-24 of it
                float big = 0.0f;
#pragma unroll
                for (int k = 0; k < PER; ++k) big = fmaxf(big, fabsf(v[k]));
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                const uint32_t ex = __float_as_uint(big) >> 23;
                if (ex > 0u && ex < 254u) {
                    const float shrink = __uint_as_float((254u - ex) << 23);
#pragma unroll
                    for (int k = 0; k < PER; ++k) v[k] *= shrink;
                    fac *= __uint_as_float(ex << 23);
                }
            }
#pragma unroll
            for (int k = 0; k < PER; k += 4) {
                uint32_t x[2], y[2];
                split_pair<2, F16>(v[k], v[k + 1], x);
                split_pair<2, F16>(v[k + 2], v[k + 3], y);
#pragma unroll
                for (int term = 0; term < 2; ++term)
                    *reinterpret_cast<uint2*>(s_plane + (size_t)(term * BM + local) * S::kPlane + j + k) = make_uint2(x[term], y[term]);
            }
            if (j == 0) s_fac[local] = fac;
        }
    }
    if (CS > 1) cluster_arrive();                // this CTA has read its peers' sums; they may not leave before
    __syncthreads();

    // ---- second product: [BM, r] x [r, O] on top of base, the columns split over all warps
    {
        // where this lane's rows g and g + 8 of each MMA tile go, or -1
        int dst[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int local = 16 * m + 8 * h + g;
                int b = -1;
                if (local < rows) b = p.dst_row ? __ldg(p.dst_row + row0 + local) : (int)(row0 + local);
                dst[m][h] = b < p.n_dst ? b : -1;
            }
        const uint16_t* up = p.up + (int64_t)e * p.r * p.O;
        const uint32_t plane0 = smem_addr(s_plane) + (uint32_t)(g * S::kPlane + 4 * G * t) * 2u;
        auto piece = [&](int n0, auto guard) {
            constexpr bool GUARD = decltype(guard)::value;
            const bool in = !GUARD || n0 + 8 * t < p.O;
            uint4 bs[MT][2];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    bs[m][h] = p.base && in && dst[m][h] >= 0
                                   ? *reinterpret_cast<const uint4*>(p.base + (int64_t)dst[m][h] * p.O + n0 + 8 * t)
                                   : make_uint4(0u, 0u, 0u, 0u);
            // b[c][q]: column n0 + 4g + c; the rank indices of MMA step q held by this lane are
            // 4t .. 4t+3 (RP = 16) or 32 (q >> 1) + 8t + 4 (q & 1) + 0..3
            uint2 b[4][KS];
            const int col = n0 + 4 * g;
            const bool inc = !GUARD || col < p.O;
            if constexpr (!BWD) {
                const uint16_t* at = up + (int64_t)col * p.r + 4 * G * t;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int q = 0; q < KS; q += G) {
                        const bool ok = inc && 16 * q + 4 * G * t < p.r;
                        if constexpr (G == 2) {
                            const uint4 v = ok ? ldg16(at + c * p.r + 16 * q) : make_uint4(0u, 0u, 0u, 0u);
                            b[c][q] = make_uint2(v.x, v.y);
                            b[c][q + 1] = make_uint2(v.z, v.w);
                        } else {
                            b[c][q] = ok ? ldg8(at + c * p.r) : make_uint2(0u, 0u);
                        }
                    }
            } else {
#pragma unroll
                for (int q = 0; q < KS; ++q) {
                    const int j = 16 * G * (q / G) + 4 * G * t + 4 * (q % G);
                    const bool ok = inc && j < p.r;                // r is a multiple of 8: all four or none
                    const uint16_t* at = up + (int64_t)j * p.O + col;
                    uint2 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = ok ? ldg8(at + (int64_t)i * p.O) : make_uint2(0u, 0u);
                    b[0][q] = make_uint2(prmt(v[0].x, v[1].x, 0x5410u), prmt(v[2].x, v[3].x, 0x5410u));
                    b[1][q] = make_uint2(prmt(v[0].x, v[1].x, 0x7632u), prmt(v[2].x, v[3].x, 0x7632u));
                    b[2][q] = make_uint2(prmt(v[0].y, v[1].y, 0x5410u), prmt(v[2].y, v[3].y, 0x5410u));
                    b[3][q] = make_uint2(prmt(v[0].y, v[1].y, 0x7632u), prmt(v[2].y, v[3].y, 0x7632u));
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float acc[4][4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[c][j] = 0.0f;
#pragma unroll
                for (int term = 0; term < 2; ++term)
#pragma unroll
                    for (int q = 0; q < KS; q += G) {
                        uint2 a0[G], a1[G];
                        const uint32_t at = plane0 + (uint32_t)((term * BM + 16 * m) * S::kPlane + 16 * q) * 2u;
                        if constexpr (G == 2) {
                            const uint4 x = lds16(at), y = lds16(at + 16 * S::kPlane);
                            a0[0] = make_uint2(x.x, x.y), a0[1] = make_uint2(x.z, x.w);
                            a1[0] = make_uint2(y.x, y.y), a1[1] = make_uint2(y.z, y.w);
                        } else {
                            a0[0] = lds8(at);
                            a1[0] = lds8(at + 16 * S::kPlane);
                        }
#pragma unroll
                        for (int i = 0; i < G; ++i)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                mma16<F16>(acc[c], a0[i].x, a1[i].x, a0[i].y, a1[i].y, b[c][q + i].x, b[c][q + i].y);
                    }
                // lane (g, t): columns n0 + 8t + 4i + c in acc[c][2h + i]
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (dst[m][h] < 0 || !in) continue;
                    const float f = s_fac[16 * m + 8 * h + g];
                    const uint32_t bw[4] = {bs[m][h].x, bs[m][h].y, bs[m][h].z, bs[m][h].w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int c = 0; c < 4; c += 2) {
                            const float2 v = unpack16<F16>(bw[2 * i + c / 2]);
                            o[2 * i + c / 2] = pack16<F16>(fmaf(f, acc[c][2 * h + i], v.x), fmaf(f, acc[c + 1][2 * h + i], v.y));
                        }
                    *reinterpret_cast<uint4*>(p.out + (int64_t)dst[m][h] * p.O + n0 + 8 * t) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        };
        const int whole = p.O / 32;
        const int st0 = (int)((int64_t)whole * part / parts), st1 = (int)((int64_t)whole * (part + 1) / parts);
#pragma unroll RP <= 16 ? 2 : 1
        for (int st = st0; st < st1; ++st) piece(32 * st, std::false_type{});
        if (part == parts - 1 && (p.O & 31)) piece(32 * whole, std::true_type{});
    }
    if (CS > 1) cluster_wait();
}

// ---------------------------------------------------------------------------
// the two products for many rows
// ---------------------------------------------------------------------------
// Persistent CTAs over the 32-row tiles. Producer warps keep a ring of stages filled by
// asynchronous copies, the rows' next 256 columns together with the factor's, straight
// through from the first product of a tile to the second and on to the next tile; eight
// consumer warps take 32 columns of every stage each, so that memory never waits for the
// warps to meet for the sums. All fragments come out of shared memory by ldmatrix.
__device__ unsigned g_lora_err;               // set when a wait of the stream gives up

template <int RP, int ROWS>
struct StreamShape {
    static constexpr int BM = ROWS, MT = BM / 16, NT = RP / 8, KS = RP / 16;
    static constexpr int CW = 32 * kLoraWarps;                       // columns of a stage
    static constexpr int kProducers = 128;                           // threads
    static constexpr int kThreads = kLoraThreads + kProducers;
    static constexpr int kStages = RP == 16 ? (BM == 32 ? 6 : 4) : RP == 32 && BM == 32 ? 4 : 3;
    static constexpr int kRow = 2 * CW + 16;                         // bytes a row of CW columns
    static constexpr int kRank = RP == 16 ? 32 : 2 * RP + 16;        // bytes a row of the rank
    static constexpr int kFactor = CW * kRank > RP * kRow ? CW * kRank : RP * kRow;
    static constexpr int kStage = BM * kRow + kFactor;
    static constexpr int kRed = RP + 8;                              // floats a row
    static constexpr int kSums = RP <= 32 && BM == 32 ? 8 : 4;                   // warps' partial sums that are kept apart
    // Tiles whose row indices are kept: when the producers begin a tile they have issued all of
    // the ones before it, of at least two stages each, and all but kStages of those are released
    static constexpr int kTiles = 4;
    static_assert((kTiles - 1) * 2 >= kStages, "a tile's indices are overwritten after its last use");
    static constexpr int kInfo = 2 * BM + 4;                         // its source rows, destinations; adapter, first row, rows
    static constexpr size_t red = sizeof(float) * kSums * BM * kRed;
    static constexpr size_t plane = (size_t)2 * BM * (2 * RP + 16);
    static constexpr size_t fixed = (size_t)kStages * kStage + red + plane + sizeof(float) * BM + sizeof(int) * kInfo * kTiles;
    static constexpr size_t smem(int L) { return fixed + (size_t)(L + 1) * 8; }
    // byte offset of 16-byte piece c of row n of the rank: rows of 32 bytes swap their halves
    // every four rows, longer ones are padded, so that eight rows in a row never share a bank
    __device__ static uint32_t rank_at(int n, int c) {
        return RP == 16 ? (uint32_t)(n * 32 + 16 * (c ^ ((n >> 2) & 1))) : (uint32_t)(n * kRank + 16 * c);
    }
};

__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// arrives on the barrier once this thread's asynchronous copies so far have landed
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int RP, int ROWS, bool BWD, bool F16>
__global__ void __launch_bounds__(StreamShape<RP, ROWS>::kThreads, 1) lora_stream_kernel(const LoraRowsArgs p) {
    using S = StreamShape<RP, ROWS>;
    constexpr int BM = S::BM, MT = S::MT, NT = S::NT, KS = S::KS, CW = S::CW, NS = S::kStages, NP = S::kProducers;
    constexpr int kPlane = 2 * RP + 16;                              // bytes a row of h's terms
    extern __shared__ __align__(16) uint8_t smem[];
    float* s_red = reinterpret_cast<float*>(smem + NS * S::kStage);
    uint8_t* s_plane = smem + NS * S::kStage + S::red;
    float* s_fac = reinterpret_cast<float*>(s_plane + S::plane);
    int* s_info = reinterpret_cast<int*>(s_fac + BM);
    int* s_first = s_info + S::kInfo * S::kTiles;                    // first tile of each adapter
    int* s_off = s_first + p.L + 1;
    __shared__ uint64_t s_full[NS], s_empty[NS];
    __shared__ int s_abort;
    __shared__ int s_warp[S::kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_addr(s_full + i), NP + 1);
            mbar_init(smem_addr(s_empty + i), kLoraWarps);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (BWD) let_next_grid_start();
    // the adapters' tiles, a run of neighbouring adapters a thread
    {
        const int per = (p.L + S::kThreads - 1) / S::kThreads;
        const int e0 = min(tid * per, p.L), e1 = min(e0 + per, p.L);
        int mine = 0;
        int lo = e0 < e1 ? (int)clamp_row(p.offsets[e0], p.R) : 0;
        for (int e = e0; e < e1; ++e) {
            const int hi = (int)clamp_row(p.offsets[e + 1], p.R);
            s_off[e] = lo;
            s_first[e] = mine;                                       // within the run
            if (hi > lo) mine += (hi - lo + BM - 1) / BM;
            lo = hi;
        }
        if (e1 == p.L && e0 < e1) s_off[p.L] = lo;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += s_warp[w];
        for (int e = e0; e < e1; ++e) s_first[e] += incl - mine;
        if (tid == S::kThreads - 1) s_first[p.L] = incl;
        __syncthreads();
    }
    const int tiles = s_first[p.L];
    const int n1 = (p.C + CW - 1) / CW, n2 = (p.O + CW - 1) / CW;
    const uint32_t ring = smem_addr(smem);
    bool gone = false;                                               // a wait gave up: no more copies or sums
    int slot = 0;
    uint32_t phase = 0;                                              // of the slot's barriers, by turns of the ring
    auto advance = [&]() {
        if (++slot == NS) {
            slot = 0;
            phase ^= 1u;
        }
    };

    if (warp >= kLoraWarps) {
        // ------------------------------------------------------------ producers
        const int ptid = tid - kLoraThreads;
        int e = 0, row0 = 0, rows = 0;
        // the tile's adapter and rows, and the row index that this thread keeps for the tile: its
        // sources and then its destinations over the producers
        auto look_up = [&](int tile) -> int {
            if (tile >= tiles) return -1;
            int lo = 0, hi = p.L - 1;                                // the last adapter whose first tile <= tile
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_first[mid] <= tile) lo = mid; else hi = mid - 1;
            }
            e = lo;
            row0 = s_off[lo] + (tile - s_first[lo]) * BM;
            rows = min(BM, s_off[lo + 1] - row0);
            const int local = ptid & (BM - 1), r = row0 + local;
            if (ptid >= 2 * BM || local >= rows) return -1;
            if (ptid < BM) {
                const int at = p.src_row ? __ldg(p.src_row + r) : r;
                return at < p.n_src ? at : -1;
            }
            const int at = p.dst_row ? __ldg(p.dst_row + r) : r;
            return at < p.n_dst ? at : -1;
        };
        constexpr int CPR = CW / 8, CPJ = RP / 8;                    // 16-byte pieces of a row, of the rank
        const int c = ptid % CPR, jc = ptid % CPJ;
        int next = look_up(blockIdx.x);
        int buf = 0;
        bool wrapped = false;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf = (buf + 1) % S::kTiles) {
            int* info = s_info + S::kInfo * buf;
            if (ptid < 2 * BM) info[ptid] = next;
            if (ptid == 0) {
                info[2 * BM] = e;
                info[2 * BM + 1] = row0;
                info[2 * BM + 2] = rows;
            }
            const uint16_t* down = p.down + (int64_t)e * p.r * p.C;
            const uint16_t* up = p.up + (int64_t)e * p.r * p.O;
            named_sync(2, NP);
            // this thread's rows of the tile, read before any copy is issued: a read of shared memory
            // may not pass the copies before it, and would wait once for each
            constexpr int PER = BM * CPR / NP;
            const uint16_t* source[PER];
            const uint16_t* dest[PER];
            bool every = rows == BM;                                 // all rows exist (and their indices are in range)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int x = info[i * (NP / CPR) + ptid / CPR], y = info[BM + i * (NP / CPR) + ptid / CPR];
                source[i] = x >= 0 ? p.src + (int64_t)x * p.C + 8 * c : nullptr;
                dest[i] = y >= 0 && p.base ? p.base + (int64_t)y * p.O + 8 * c : nullptr;
                every = every && x >= 0 && y >= 0;
            }
            every = p.base && __all_sync(0xffffffffu, every);
            // the factors: where this thread's first piece lies in a stage, and the step to its next ones
            const uint16_t* by_columns = (BWD ? up : down) + (int64_t)(ptid / CPR) * (BWD ? p.O : p.C) + 8 * c;
            const uint16_t* by_ranks = (BWD ? down : up) + (int64_t)(ptid / CPJ) * p.r + 8 * jc;
            const int first_n = ptid / CPJ;
            const int first_place = BWD ? first_n : (first_n & ~31) | ((first_n & 3) << 3) | ((first_n >> 2) & 7);
            next = look_up(tile + gridDim.x);
            for (int q = 0; q < n1 + n2; ++q) {
                if (wrapped && !gone)
                    gone = __any_sync(0xffffffffu, !mbar_wait_bounded(smem_addr(s_empty + slot), phase ^ 1u, &s_abort,
                                                                      &g_lora_err, 1u));
                const bool first = q < n1;
                const int c0 = (first ? q : q - n1) * CW, width = first ? p.C : p.O;
                const uint32_t stage = ring + (uint32_t)(slot * S::kStage), factor = stage + BM * S::kRow;
                const uint32_t mine = stage + (uint32_t)((ptid / CPR) * S::kRow + 16 * c);
                const uint32_t mine_r = mine + BM * S::kRow, mine_c = factor + S::rank_at(first_place, jc);
                // whole: no piece of the stage is outside, so nothing is looked at per copy
                auto copies = [&](auto whole) {
                    constexpr bool WHOLE = decltype(whole)::value;
                    const bool inside = WHOLE || c0 + 8 * c < width;
                    if (WHOLE || first || p.base) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const uint16_t* row = first ? source[i] : dest[i];
                            const bool ok = WHOLE || (inside && row);
                            copy_async16(mine + (uint32_t)(i * (NP / CPR) * S::kRow), ok ? row + c0 : p.src, ok ? 16u : 0u);
                        }
                    }
                    if (first != BWD) {
                        // rank rows of CW columns
#pragma unroll
                        for (int i = 0; i < RP * CPR / NP; ++i) {
                            const bool ok = WHOLE || (inside && i * (NP / CPR) + ptid / CPR < p.r);
                            copy_async16(mine_r + (uint32_t)(i * (NP / CPR) * S::kRow),
                                         ok ? by_columns + (int64_t)(i * (NP / CPR)) * width + c0 : p.src, ok ? 16u : 0u);
                        }
                    } else {
                        // columns as rows of the rank; for the second product column 4i + c of a piece of 32
                        // lies at 8c + i, where the fragment of MMA tile c finds its eight columns in a row
                        constexpr int Q = NP / CPJ;                  // 16 or a multiple of 32
                        static_assert(Q == 16 || Q % 32 == 0, "places of a thread's columns");
                        const bool in_rank = 8 * jc < p.r;
#pragma unroll
                        for (int i = 0; i < CW / Q; ++i) {
                            const bool ok = WHOLE || (in_rank && c0 + i * Q + first_n < width);
                            const int step = BWD || Q % 32 == 0 ? i * Q : 32 * (i >> 1) + 4 * (i & 1);
                            copy_async16(mine_c + (uint32_t)(step * S::kRank),
                                         ok ? by_ranks + (int64_t)(c0 + i * Q) * p.r : p.src, ok ? 16u : 0u);
                        }
                    }
                };
                if (!gone) {
                    if (every && c0 + CW <= width && p.r == RP) copies(std::true_type{});
                    else copies(std::false_type{});
                }
                copy_arrive(smem_addr(s_full + slot));
                if (ptid == 0) mbar_arrive(smem_addr(s_full + slot));   // publishes the tile's info too
                advance();
                wrapped = wrapped || slot == 0;
            }
        }
        copy_commit();
        copy_wait<0>();
        return;
    }

    // ---------------------------------------------------------------- consumers
    auto wait_stage = [&]() {
        if (!gone)
            gone = __any_sync(0xffffffffu, !mbar_wait_bounded(smem_addr(s_full + slot), phase, &s_abort, &g_lora_err, 2u));
    };
    auto release_stage = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(s_empty + slot));
        advance();
    };
    // this lane's part of the addresses of an ldmatrix.x4 over a 16 x 16 block: its rows' halves
    // come first (by_row, by_col), or its columns' halves (by_n, by_k)
    const uint32_t by_row = (uint32_t)(lane & 15), by_col = (uint32_t)(lane >> 4) * 16u;
    const int by_n = (lane & 7) + 8 * (lane >> 4), by_k = (lane >> 3) & 1;
    const int k0 = 32 * warp;                                        // this warp's columns of every stage
    const uint32_t rows_frag = ring + by_row * S::kRow + 2 * k0 + by_col;
    // in the second product a warp has 16 of the rows and 64 or 128 of the columns: whole 128-byte lines
    constexpr int SUB = MT;                                          // in pieces of 32
    const int wm = warp % MT, n0 = 32 * SUB * (warp / MT);
    constexpr int TPR = kLoraThreads / BM;                           // threads that finish a row of sums
    const uint32_t plane0 = smem_addr(s_plane) + (16 * wm + by_row) * kPlane + by_col;
    int buf = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf = (buf + 1) % S::kTiles) {
        const int* info = s_info + S::kInfo * buf;
        wait_stage();                                                // the tile's info is there with its first stage
        const int e = gone ? 0 : info[2 * BM], row0 = gone ? 0 : info[2 * BM + 1], rows = gone ? 0 : info[2 * BM + 2];
        // the factor of the row that this thread finishes below
        const int mine_row = tid / TPR;
        float mine_fac = p.scaling ? __ldg(p.scaling + e) : 1.0f;
        if (p.weight && mine_row < rows) mine_fac *= __ldg(p.weight + row0 + mine_row);

        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][c][j] = 0.0f;
        for (int q = 0; q < n1; ++q) {
            if (q) wait_stage();
            const uint32_t at = (uint32_t)(slot * S::kStage), factor = ring + at + BM * S::kRow;
            if (!gone) {                                             // columns past the end are zeros in both
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t a[MT][4];
#pragma unroll
                    for (int m = 0; m < MT; ++m) ldmatrix4(a[m], rows_frag + at + 16 * m * S::kRow + 32 * half);
#pragma unroll
                    for (int c = 0; c < NT; c += 2) {
                        uint32_t b[4];                               // tile c: k 0-7, 8-15; tile c + 1: the same
                        if constexpr (!BWD)
                            ldmatrix4(b, factor + (8 * c + by_n) * S::kRow + 2 * k0 + 32 * half + 16 * by_k);
                        else
                            ldmatrix4_trans(b, factor + S::rank_at(k0 + 16 * half + (int)by_row, c + (lane >> 4)));
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            mma16<F16>(acc[m][c], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
                            mma16<F16>(acc[m][c + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
                        }
                    }
                }
            }
            release_stage();
        }
        // partial sums; with room for four only, the upper four warps put theirs down first and
        // the lower four add their own on top
        {
            float* mine = s_red + (size_t)(warp & (S::kSums - 1)) * BM * S::kRed;
#pragma unroll
            for (int turn = 0; turn < kLoraWarps / S::kSums; ++turn) {
                if (S::kSums == kLoraWarps || (warp < 4) == (turn == 1)) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                float2* o = reinterpret_cast<float2*>(mine + (16 * m + 8 * h + g) * S::kRed + 8 * c + 2 * t);
                                float2 v = make_float2(acc[m][c][2 * h], acc[m][c][2 * h + 1]);
                                if (turn == 1) {
                                    const float2 u = *o;
                                    v.x += u.x;
                                    v.y += u.y;
                                }
                                *o = v;
                            }
                }
                named_sync(1, kLoraThreads);
            }
        }
        // TPR threads a row: the sums, times the row's factor, and their 16-bit terms. fp16 terms are
        // of the row scaled by a power of two, its largest value in [1, 2) (or below, where the whole
        // row is below 2^-24, the type's smallest step), which s_fac takes back.
        {
            constexpr int PER = RP / TPR;
            const int j0 = PER * (tid % TPR);
            float v[PER];
            const bool have = mine_row < rows && info[mine_row] >= 0;            // no source row: zeros
            const float* from = s_red + mine_row * S::kRed + j0;
            float big = 0.0f;
#pragma unroll
            for (int k = 0; k < PER; ++k) v[k] = 0.0f;
            if (have) {
#pragma unroll
                for (int w = 0; w < S::kSums; w += 2)
#pragma unroll
                    for (int k = 0; k < PER; k += 2) {
                        const float2 x = *reinterpret_cast<const float2*>(from + k + w * BM * S::kRed);
                        const float2 y = *reinterpret_cast<const float2*>(from + k + (w + 1) * BM * S::kRed);
                        v[k] += x.x + y.x;
                        v[k + 1] += x.y + y.y;
                    }
            }
            if (p.mid && mine_row < rows) {
                const float f = BWD ? mine_fac : 1.0f;
#pragma unroll
                for (int k = 0; k < PER; k += 2)
                    if (j0 + k < p.r)
                        *reinterpret_cast<float2*>(p.mid + (int64_t)(row0 + mine_row) * p.r + j0 + k) = make_float2(f * v[k], f * v[k + 1]);
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                v[k] = j0 + k < p.r ? mine_fac * v[k] : 0.0f;
                big = fmaxf(big, fabsf(v[k]));
            }
            if constexpr (F16) {
#pragma unroll
                for (int o = TPR / 2; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                const uint32_t ex = min(max(__float_as_uint(big) >> 23, 103u), 253u);
                const float shrink = __uint_as_float((254u - ex) << 23);
#pragma unroll
                for (int k = 0; k < PER; ++k) v[k] *= shrink;
                if (tid % TPR == 0) s_fac[mine_row] = shrink;
            }
#pragma unroll
            for (int k = 0; k < PER; k += 2) {
                uint32_t o[2];
                split_pair<2, F16>(v[k], v[k + 1], o);
#pragma unroll
                for (int term = 0; term < 2; ++term)
                    *reinterpret_cast<uint32_t*>(s_plane + (size_t)(term * BM + mine_row) * kPlane + 2 * (j0 + k)) = o[term];
            }
        }
        named_sync(1, kLoraThreads);
        uint32_t a[2][KS][4];                                        // the terms of h
        float shrink[2], grow[2];                                    // the row's scale and its inverse (fp16)
        uint16_t* dst[2];                                            // this lane's first column of its rows, or null
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int k = 0; k < KS; ++k) ldmatrix4(a[term][k], plane0 + term * BM * kPlane + 32 * k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int local = 16 * wm + 8 * h + g, at = gone ? -1 : info[BM + local];
            dst[h] = at >= 0 ? p.out + (int64_t)at * p.O + n0 + 8 * t : nullptr;
            if constexpr (F16) {
                shrink[h] = s_fac[local];
                grow[h] = __uint_as_float((254u << 23) - __float_as_uint(shrink[h]));
            }
        }
        for (int q = 0; q < n2; ++q) {
            wait_stage();
            const uint32_t at = (uint32_t)(slot * S::kStage), factor = ring + at + BM * S::kRow;
            if (!gone && q * CW + n0 < p.O) {
                // the sums start from base: lane (g, t) has columns 32 s + 8t + 4i + c in o[s][c][2h + i]
                float o[SUB][4][4];
#pragma unroll
                for (int s = 0; s < SUB; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4 bs = make_uint4(0u, 0u, 0u, 0u);
                        if (p.base) bs = lds16(ring + at + (16 * wm + 8 * h + g) * S::kRow + 2 * (n0 + 32 * s + 8 * t));
                        const uint32_t w[4] = {bs.x, bs.y, bs.z, bs.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float2 v = unpack16<F16>(w[i]);
                            if constexpr (F16) {
                                v.x *= shrink[h];
                                v.y *= shrink[h];
                            }
                            o[s][2 * (i & 1)][2 * h + (i >> 1)] = v.x;
                            o[s][2 * (i & 1) + 1][2 * h + (i >> 1)] = v.y;
                        }
                    }
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int s = 0; s < SUB; ++s) {
                        uint32_t b[4][2];                            // MMA tile c: columns 4n + c of 32
                        if constexpr (!BWD) {
#pragma unroll
                            for (int c = 0; c < 4; c += 2) {
                                uint32_t d[4];
                                ldmatrix4(d, factor + S::rank_at(n0 + 32 * s + 8 * c + by_n, 2 * k + by_k));
                                b[c][0] = d[0], b[c][1] = d[1], b[c + 1][0] = d[2], b[c + 1][1] = d[3];
                            }
                        } else {
                            uint2 v[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[i] = lds8(factor + (16 * k + 2 * t + (i & 1) + 8 * (i >> 1)) * S::kRow + 2 * (n0 + 32 * s + 4 * g));
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                b[0][i] = prmt(v[2 * i].x, v[2 * i + 1].x, 0x5410u);
                                b[1][i] = prmt(v[2 * i].x, v[2 * i + 1].x, 0x7632u);
                                b[2][i] = prmt(v[2 * i].y, v[2 * i + 1].y, 0x5410u);
                                b[3][i] = prmt(v[2 * i].y, v[2 * i + 1].y, 0x7632u);
                            }
                        }
#pragma unroll
                        for (int term = 0; term < 2; ++term)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                mma16<F16>(o[s][c], a[term][k][0], a[term][k][1], a[term][k][2], a[term][k][3], b[c][0], b[c][1]);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int s = 0; s < SUB; ++s) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x = o[s][2 * (i & 1)][2 * h + (i >> 1)], y = o[s][2 * (i & 1) + 1][2 * h + (i >> 1)];
                            if constexpr (F16) {
                                x *= grow[h];
                                y *= grow[h];
                            }
                            w[i] = pack16<F16>(x, y);
                        }
                        if (dst[h] && q * CW + n0 + 32 * s + 8 * t < p.O)
                            *reinterpret_cast<uint4*>(dst[h] + q * CW + 32 * s) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            }
            release_stage();
        }
    }
}

// at most one partial tile of `rows` rows for every adapter that has a row
int64_t most_tiles(const LoraRowsArgs& a, int rows) {
    const int64_t active = a.R < a.L ? a.R : a.L;
    return active + (a.R - active) / rows;
}

template <int RP, int ROWS, bool BWD, bool F16>
cudaError_t launch_stream_t(const LoraRowsArgs& a, cudaStream_t s) {
    using S = StreamShape<RP, ROWS>;
    constexpr size_t most = S::smem(2048) < kMaxSmem ? S::smem(2048) : kMaxSmem;
    static std::atomic<bool> attr_set[64];           // per device: dynamic shared memory opted in
    const int dev = current_device();
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(lora_stream_kernel<RP, ROWS, BWD, F16>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = most_tiles(a, ROWS), sms = device_sm_count();
    lora_stream_kernel<RP, ROWS, BWD, F16><<<(unsigned)(tiles < sms ? tiles : sms), S::kThreads, S::smem(a.L), s>>>(a);
    return cudaGetLastError();
}

template <int RP, int ROWS>
cudaError_t launch_stream_m(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    if (bwd) return launch_stream_t<RP, ROWS, true, false>(a, s);
    return f16 ? launch_stream_t<RP, ROWS, false, true>(a, s) : launch_stream_t<RP, ROWS, false, false>(a, s);
}

// Tiles of 64 rows halve what the factors cost and keep more rows in flight, once there are
// enough of them for two rounds of the SMs (and the adapters' table fits beside a rank of 32)
template <int RP>
cudaError_t launch_stream(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    static_assert(StreamShape<RP, 32>::smem(2048) <= kMaxSmem, "shared memory of a CTA");
    if constexpr (RP <= 32)
        if (most_tiles(a, 64) >= 2 * (int64_t)device_sm_count() && StreamShape<RP, 64>::smem(a.L) <= kMaxSmem)
            return launch_stream_m<RP, 64>(a, bwd, f16, s);
    return launch_stream_m<RP, 32>(a, bwd, f16, s);
}

template <int RP, int MT, bool BWD, bool F16>
cudaError_t launch_rows_t(const LoraRowsArgs& a, cudaStream_t s) {
    constexpr int BM = 16 * MT;
    constexpr size_t smem = RowsShape<RP, MT>::smem;
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static std::atomic<bool> attr_set[64];           // per device: dynamic shared memory opted in
    const int dev = current_device();
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(lora_rows_kernel<RP, MT, BWD, F16>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = most_tiles(a, BM);
    int cs = 1;
    while (cs < 8 && tiles * cs * 2 <= 2 * (int64_t)device_sm_count()) cs *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * cs));
    cfg.blockDim = dim3(kLoraThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_rows_kernel<RP, MT, BWD, F16>, a);
}

template <int RP, int MT>
cudaError_t launch_rows_m(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    if (bwd) return launch_rows_t<RP, MT, true, false>(a, s);
    return f16 ? launch_rows_t<RP, MT, false, true>(a, s) : launch_rows_t<RP, MT, false, false>(a, s);
}

template <int RP>
cudaError_t launch_rows_r(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    const int64_t active = a.R < a.L ? a.R : a.L;
    if constexpr (RP <= 64)
        if (a.R >= 24 * active && a.R >= 16 * (int64_t)device_sm_count()) return launch_stream<RP>(a, bwd, f16, s);
    return a.R >= 24 * active ? launch_rows_m<RP, 2>(a, bwd, f16, s) : launch_rows_m<RP, 1>(a, bwd, f16, s);
}

// ---------------------------------------------------------------------------
// gradients of the adapters
// ---------------------------------------------------------------------------
// One gradient of one adapter: sum over its rows of left[r, j] right[row r, n], rows the MMA's
// contraction index. A CTA owns WC * SC columns (SC a warp) and walks the adapter's rows in
// stages of 32 WR: the rows of `right` are gathered into shared memory by 16-byte asynchronous
// copies, three stages deep (the gather's latency, index then row, is what a warp alone cannot
// hide), while `left` is read ahead by a stage into registers and split into its 16-bit terms
// once for all warps. Both fragments come out of shared memory transposed.
constexpr int kGradStages = 3;

template <int RP, int WR, int TERMS>
struct GradShape {
    static constexpr int CT = RP <= 32 ? 8 : 4;          // MMA column tiles of a warp's slab
    static constexpr int SC = 8 * CT;                    // its columns
    static constexpr int MT = RP / 16;
    static constexpr int WC = kLoraWarps / WR;
    static constexpr int CW = WC * SC;                   // columns of the CTA
    static constexpr int SR = 32 * WR;                   // rows of a stage
    static constexpr int kPitch16 = 2 * CW + 16;         // bytes a row in shared memory: bf16,
    static constexpr int kPitch8 = CW + 16;              // codes; conflict-free fragment loads
    static constexpr int kPlane = RP + 8;                // elements a row of a term plane
    static constexpr int kStride = SC + 4;               // floats of a row of the sum
    static constexpr int kLeft = (SR * RP / 4 + kLoraThreads - 1) / kLoraThreads;   // float4 of left a thread and stage
    static constexpr size_t stage_bytes = (size_t)SR * kPitch16;
    static constexpr size_t plane_bytes = (size_t)TERMS * SR * kPlane * 2;          // one of two buffers
    static constexpr size_t scale_bytes = (size_t)SR * (CW / 32) * 2;               // one of two buffers
    static constexpr size_t work = kGradStages * stage_bytes + 2 * plane_bytes + 2 * scale_bytes + 2 * SR * 4;
    static constexpr size_t sums = sizeof(float) * (size_t)kLoraWarps * RP * kStride;
    static constexpr size_t smem = work > sums ? work : sums;
};

template <int RP, int WR, int TERMS, bool Q8>
__device__ __forceinline__ void grad_body(const LoraGradArgs& p, const LoraGradSide& d, int e, int col0, uint8_t* smem) {
    using S = GradShape<RP, WR, TERMS>;
    constexpr int CT = S::CT, MT = S::MT, WC = S::WC, CW = S::CW, SR = S::SR;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int wc = warp % WC, wr = warp / WC;
    const int CS = (int)cluster_size(), crank = (int)cluster_rank();
    uint8_t* s_stage = smem;
    uint16_t* s_plane = reinterpret_cast<uint16_t*>(smem + kGradStages * S::stage_bytes);
    uint16_t* s_step = reinterpret_cast<uint16_t*>(smem + kGradStages * S::stage_bytes + 2 * S::plane_bytes);
    int* s_row = reinterpret_cast<int*>(smem + kGradStages * S::stage_bytes + 2 * S::plane_bytes + 2 * S::scale_bytes);
    const uint32_t stage0 = smem_addr(s_stage), plane0 = smem_addr(s_plane);

    const int64_t lo = clamp_row(p.offsets[e], p.R), hi = clamp_row(p.offsets[e + 1], p.R);
    const int rows = hi > lo ? (int)(hi - lo) : 0;
    const float scal = d.factor && p.scaling ? __ldg(p.scaling + e) : 1.0f;
    // stage i of this CTA: rows first(i) .. first(i) + SR - 1 of the adapter
    const int stages = (rows + SR * CS - 1) / (SR * CS);
    auto first = [&](int i) { return (i * CS + crank) * SR; };

    // the row of `right` behind row `local` of the adapter, or -1
    auto source_row = [&](int local) -> int {
        if (local >= rows) return -1;
        const int64_t r = lo + local;
        const int64_t at = d.row ? (int64_t)__ldg(d.row + r) : r;
        return at >= 0 && at < d.n ? (int)at : -1;
    };
    auto issue = [&](int i) {
        constexpr int CPR = (Q8 ? CW : 2 * CW) / 16;       // 16-byte pieces of a row
        const int* row = s_row + (i & 1) * SR;
        const uint32_t dst = stage0 + (uint32_t)((i % kGradStages) * S::stage_bytes);
        const int per = Q8 ? 16 : 8;
        constexpr int PER = SR * CPR / kLoraThreads;
        int source[PER];                                   // read before any copy is issued, which would hold them up
#pragma unroll
        for (int q = 0; q < PER; ++q) source[q] = row[(q * kLoraThreads + tid) / CPR];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int id = q * kLoraThreads + tid, r = id / CPR, c = id % CPR;
            const int at = source[q];
            const bool ok = at >= 0 && col0 + c * per < d.C;
            const void* src = Q8 ? (const void*)(d.codes + (ok ? (int64_t)at * d.C + col0 + c * per : 0))
                                 : (const void*)(d.right + (ok ? (int64_t)at * d.C + col0 + c * per : 0));
            copy_async16(dst + (uint32_t)(r * (Q8 ? S::kPitch8 : S::kPitch16) + c * 16), src, ok ? 16u : 0u);
        }
    };

    // `left` of the next stage, in registers until the stage before it is being worked on
    float4 left[S::kLeft];
    float fac[S::kLeft];
    uint32_t scale[(SR * (CW / 32) + kLoraThreads - 1) / kLoraThreads];
    auto fetch = [&](int i) {
#pragma unroll
        for (int q = 0; q < S::kLeft; ++q) {
            const int id = q * kLoraThreads + tid, local = first(i) + id / (RP / 4), j = 4 * (id % (RP / 4));
            left[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            fac[q] = scal;
            if (id < SR * RP / 4 && local < rows && j < p.r) {
                const int64_t r = lo + local;
                left[q] = *reinterpret_cast<const float4*>(d.left + r * p.r + j);
                if (d.factor && p.weight) fac[q] *= __ldg(p.weight + r);
            }
        }
        if constexpr (Q8) {
            constexpr int BPR = CW / 32;
#pragma unroll
            for (int q = 0; q < (SR * BPR + kLoraThreads - 1) / kLoraThreads; ++q) {
                const int id = q * kLoraThreads + tid;
                scale[q] = 0u;
                if (id < SR * BPR && col0 + 32 * (id % BPR) < d.C) {
                    const int at = source_row(first(i) + id / BPR);
                    if (at >= 0) scale[q] = __ldg(d.scales + (int64_t)at * (d.C / 32) + col0 / 32 + id % BPR);
                }
            }
        }
    };
    auto place = [&](int i) {
        uint16_t* plane = s_plane + (i & 1) * (S::plane_bytes / 2);
#pragma unroll
        for (int q = 0; q < S::kLeft; ++q) {
            const int id = q * kLoraThreads + tid;
            if (id < SR * RP / 4) {
                uint32_t a[TERMS], b[TERMS];
                split_pair<TERMS, false>(left[q].x * fac[q], left[q].y * fac[q], a);
                split_pair<TERMS, false>(left[q].z * fac[q], left[q].w * fac[q], b);
#pragma unroll
                for (int k = 0; k < TERMS; ++k)
                    *reinterpret_cast<uint2*>(plane + (size_t)(k * SR + id / (RP / 4)) * S::kPlane + 4 * (id % (RP / 4))) =
                        make_uint2(a[k], b[k]);
            }
        }
        if constexpr (Q8) {
#pragma unroll
            for (int q = 0; q < (SR * (CW / 32) + kLoraThreads - 1) / kLoraThreads; ++q) {
                const int id = q * kLoraThreads + tid;
                if (id < SR * (CW / 32)) s_step[(i & 1) * (S::scale_bytes / 2) + id] = (uint16_t)act8_step_bf16(scale[q]);
            }
        }
    };

    float acc[MT][CT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][c][j] = 0.0f;

    // prologue: two stages of copies under way, the first stage's left in place
    static_assert(kGradStages == 3, "the prologue and the row buffers are written for three stages");
    if (tid < SR) {
        s_row[tid] = source_row(first(0) + tid);
        s_row[SR + tid] = source_row(first(1) + tid);
    }
    __syncthreads();
    if (stages > 0) issue(0);
    copy_commit();
    if (stages > 1) issue(1);
    copy_commit();
    int next_row = tid < SR ? source_row(first(2) + tid) : -1;
    if (!d.factor) wait_for_previous_grid();            // dA's left comes from the rows kernel; the copies do not
    fetch(0);
    place(0);
    fetch(1);
    __syncthreads();                                    // s_row has been read
    if (tid < SR) s_row[tid] = next_row;                // stage 2's
    next_row = tid < SR ? source_row(first(3) + tid) : -1;

    for (int i = 0; i < stages; ++i) {
        copy_wait<1>();
        __syncthreads();                                // stage i is there; stage i - 1 is done with
        if (i + 2 < stages) issue(i + 2);
        copy_commit();
        place(i + 1);
        if (tid < SR) s_row[((i + 3) & 1) * SR + tid] = next_row;
        fetch(i + 2);
        next_row = tid < SR ? source_row(first(i + 4) + tid) : -1;

        const uint32_t x = stage0 + (uint32_t)((i % kGradStages) * S::stage_bytes);
        const uint32_t plane = plane0 + (uint32_t)((i & 1) * S::plane_bytes);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r0 = 32 * wr + 16 * half;
            uint32_t a[MT][TERMS][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int k = 0; k < TERMS; ++k)
                    ldmatrix4_trans(a[m][k], plane + (uint32_t)(((k * SR + r0 + (lane & 7) + 8 * (lane >> 4)) * S::kPlane +
                                                                 16 * m + 8 * ((lane >> 3) & 1)) * 2));
            if constexpr (!Q8) {
#pragma unroll
                for (int c = 0; c < CT; c += 2) {
                    uint32_t b[4];                       // two column tiles: rows 0-7 and 8-15 of each
                    ldmatrix4_trans(b, x + (uint32_t)((r0 + (lane & 15)) * S::kPitch16 +
                                                      (wc * S::SC + 8 * c + 8 * (lane >> 4)) * 2));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int k = 0; k < TERMS; ++k) {
                            mma_bf16_16816(acc[m][c], a[m][k][0], a[m][k][1], a[m][k][2], a[m][k][3], b[0], b[1]);
                            mma_bf16_16816(acc[m][c + 1], a[m][k][0], a[m][k][1], a[m][k][2], a[m][k][3], b[2], b[3]);
                        }
                }
            } else {
                uint32_t code_frag[CT][2];
                // this lane's rows 2t, 2t+1 and 2t+8, 2t+9, its CT columns from CT g on; MMA tile c takes
                // column c of them, a byte of either row of a pair, as two bf16 numbers
#pragma unroll
                for (int pair = 0; pair < 2; ++pair) {
                    const int row = r0 + 2 * t + 8 * pair;
                    const uint32_t at = x + (uint32_t)(row * S::kPitch8 + wc * S::SC + CT * g);
                    uint32_t w[2][CT / 4];
                    if constexpr (CT == 8) {
                        const uint2 u = lds8(at), v = lds8(at + S::kPitch8);
                        w[0][0] = u.x, w[0][1] = u.y, w[1][0] = v.x, w[1][1] = v.y;
                    } else {
                        w[0][0] = lds4(at), w[1][0] = lds4(at + S::kPitch8);
                    }
                    const uint16_t* st = s_step + (i & 1) * (S::scale_bytes / 2) + row * (CW / 32) + (wc * S::SC + CT * g) / 32;
                    const uint32_t step = (uint32_t)st[0] | (uint32_t)st[CW / 32] << 16;
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        code_frag[c][pair] = act8_pair(prmt(w[0][c / 4], w[1][c / 4], 0x0400u + 0x0101u * (c & 3)), step);
                }
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int k = 0; k < TERMS; ++k)
                            mma_bf16_16816(acc[m][c], a[m][k][0], a[m][k][1], a[m][k][2], a[m][k][3], code_frag[c][0], code_frag[c][1]);
            }
        }
    }
    copy_wait<0>();
    __syncthreads();                                     // the stages become the sums' space

    // column of the accumulators: tile c, MMA column n is 8 c + n, from codes CT n + c
    float* s_red = reinterpret_cast<float*>(smem);
    float* mine = s_red + (size_t)warp * RP * S::kStride;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                float* row = mine + (16 * m + 8 * h + g) * S::kStride;
                if constexpr (Q8) {
                    row[CT * (2 * t) + c] = acc[m][c][2 * h];
                    row[CT * (2 * t + 1) + c] = acc[m][c][2 * h + 1];
                } else {
                    *reinterpret_cast<float2*>(row + 8 * c + 2 * t) = make_float2(acc[m][c][2 * h], acc[m][c][2 * h + 1]);
                }
            }
    __syncthreads();
    if (WR > 1) {
        for (int i = tid; i < CW * RP; i += kLoraThreads) {
            const int w = i / (RP * S::SC), at = (i / S::SC % RP) * S::kStride + i % S::SC;
            float v = s_red[(size_t)w * RP * S::kStride + at];
#pragma unroll
            for (int q = 1; q < WR; ++q) v += s_red[(size_t)(q * WC + w) * RP * S::kStride + at];
            s_red[(size_t)w * RP * S::kStride + at] = v;
        }
        __syncthreads();
    }
    // the cluster's CTAs share the columns out and add up theirs, in place: no other CTA reads those
    const int own = CW / CS, own0 = crank * own;
    if (CS > 1) {
        cluster_arrive();
        cluster_wait();
        for (int i = tid; i < RP * own / 4; i += kLoraThreads) {
            const int j = i / (own / 4), n = own0 + 4 * (i % (own / 4));
            float* at = s_red + (size_t)(n / S::SC) * RP * S::kStride + j * S::kStride + n % S::SC;
            *reinterpret_cast<float4*>(at) = cluster_sum(at, CS);
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
        const float* at = s_red + (size_t)(n / S::SC) * RP * S::kStride + j * S::kStride + n % S::SC;
        const int next = d.transposed ? S::kStride : 1;
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
    if (CS > 1) cluster_wait();
    if (tid == 0) wait_for_previous_grid();              // whoever waits for this grid waits for that one too
}

// CTAs (or clusters) of one adapter for one gradient; none for a gradient that is not asked for
__host__ __device__ __forceinline__ int grad_items(const LoraGradSide& d, int cols) {
    return d.out ? (d.C + cols - 1) / cols : 0;
}

template <int RP, int WR, int TERMS, bool Q8>
__global__ void __launch_bounds__(kLoraThreads, RP <= 32 && WR == 1 ? 2 : 1) lora_grads_kernel(const LoraGradArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int CW = GradShape<RP, WR, TERMS>::CW;
    const int item = (int)(blockIdx.x / cluster_size());
    const int na = grad_items(p.a, CW), nb = grad_items(p.b, CW);
    // dB's items come first: they need nothing of the rows kernel and fill the SMs that it leaves
    if (item < nb * p.L) grad_body<RP, WR, TERMS, false>(p, p.b, item / nb, item % nb * CW, smem);
    else grad_body<RP, WR, TERMS, Q8>(p, p.a, (item - nb * p.L) / na, (item - nb * p.L) % na * CW, smem);
}

template <int RP, int WR, int TERMS, bool Q8>
cudaError_t launch_grads_t(const LoraGradArgs& a, int cs, cudaStream_t s) {
    using S = GradShape<RP, WR, TERMS>;
    static_assert(S::smem <= 227 * 1024, "shared memory of a CTA");
    static std::atomic<bool> attr_set[64];
    const int dev = current_device();
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(lora_grads_kernel<RP, WR, TERMS, Q8>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t items = (int64_t)a.L * (grad_items(a.a, S::CW) + grad_items(a.b, S::CW));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * cs));
    cfg.blockDim = dim3(kLoraThreads);
    cfg.dynamicSmemBytes = S::smem;
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
    return cudaLaunchKernelEx(&cfg, lora_grads_kernel<RP, WR, TERMS, Q8>, a);
}

template <int RP, int WR>
cudaError_t launch_grads_w(const LoraGradArgs& a, bool f32, int cs, cudaStream_t s) {
    if (a.a.codes) return f32 ? launch_grads_t<RP, WR, 3, true>(a, cs, s) : launch_grads_t<RP, WR, 2, true>(a, cs, s);
    return f32 ? launch_grads_t<RP, WR, 3, false>(a, cs, s) : launch_grads_t<RP, WR, 2, false>(a, cs, s);
}

template <int RP>
cudaError_t launch_grads_r(const LoraGradArgs& a, bool f32, cudaStream_t s) {
    // warps and then CTAs along the rows where the columns and adapters alone leave SMs idle
    constexpr int WR = RP <= 64 ? 4 : 2;
    const int64_t active = a.R < a.L ? (a.R > 0 ? a.R : 1) : a.L;
    const int64_t avg = (a.R + active - 1) / active;
    const int wide = GradShape<RP, 1, 2>::CW;
    const int64_t sms = device_sm_count();
    if (avg <= 64 || active * (grad_items(a.a, wide) + grad_items(a.b, wide)) >= 2 * sms)
        return launch_grads_w<RP, 1>(a, f32, 1, s);
    const int cols = GradShape<RP, WR, 2>::CW;
    const int64_t items = active * (grad_items(a.a, cols) + grad_items(a.b, cols));
    int cs = 1;
    while (cs < 8 && items * cs * 2 <= sms && avg >= 2 * cs * GradShape<RP, WR, 2>::SR) cs *= 2;
    return launch_grads_w<RP, WR>(a, f32, cs, s);
}

// bits: 1 offsets decrease or leave [0, R], 2 offsets[0] != 0, 4 and 8 a row index of the rows
// that exist is out of range, 16 a weight that is not finite
__global__ void check_lora_kernel(const int64_t* offsets, int L, int64_t R, const int32_t* a, int64_t na,
                                  const int32_t* b, int64_t nb, const float* w, unsigned* status) {
    unsigned bad = 0;
    const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t e = tid; e < L; e += stride)
        if (offsets[e + 1] < offsets[e] || offsets[e + 1] > R) bad |= 1u;
    if (tid == 0 && offsets[0] != 0) bad |= 2u;
    const int64_t n = clamp_row(offsets[L], R);
    for (int64_t r = tid; r < n; r += stride) {
        if (a && (a[r] < 0 || a[r] >= na)) bad |= 4u;
        if (b && (b[r] < 0 || b[r] >= nb)) bad |= 8u;
        if (w && !isfinite(w[r])) bad |= 16u;
    }
    if (bad) atomicOr(status, bad);
}

}  // namespace

unsigned take_lora_error(cudaError_t* err) {
    unsigned v = 0;
    const unsigned zero = 0;
    *err = cudaMemcpyFromSymbol(&v, g_lora_err, sizeof(v));
    if (*err == cudaSuccess && v) *err = cudaMemcpyToSymbol(g_lora_err, &zero, sizeof(zero));
    return v;
}

cudaError_t launch_lora_rows(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    if (a.r <= 16) return launch_rows_r<16>(a, bwd, f16, s);
    if (a.r <= 32) return launch_rows_r<32>(a, bwd, f16, s);
    if (a.r <= 64) return launch_rows_r<64>(a, bwd, f16, s);
    return launch_rows_r<128>(a, bwd, f16, s);
}

cudaError_t launch_lora_grads(const LoraGradArgs& a, bool f32, cudaStream_t s) {
    if (a.r <= 16) return launch_grads_r<16>(a, f32, s);
    if (a.r <= 32) return launch_grads_r<32>(a, f32, s);
    if (a.r <= 64) return launch_grads_r<64>(a, f32, s);
    return launch_grads_r<128>(a, f32, s);
}

cudaError_t launch_check_lora(const int64_t* offsets, int L, int64_t R, const int32_t* a, int64_t na, const int32_t* b,
                              int64_t nb, const float* w, unsigned* status, cudaStream_t s) {
    check_lora_kernel<<<64, 256, 0, s>>>(offsets, L, R, a, na, b, nb, w, status);
    return cudaGetLastError();
}

}  // namespace gnf4
