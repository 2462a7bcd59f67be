// The adapters' two products (gnf4_lora.cuh) for few rows, and the choice between this and the
// streaming kernel.
//
// A cluster of CTAs owns a tile of 16 rows of one adapter. All its warps split the contraction
// of the first product, the partial sums meet in shared memory (and through distributed
// shared memory when the cluster has more than one CTA), and then the warps split the output
// columns of the second. One launch; x, base and out are touched once, and h never leaves the
// SM unless it is asked for.
//
// What bounds it is latency: a chain of dependent loads (offsets, row index, row), a meeting
// of the warps, a second round of loads. Fragments come straight from 16-byte global loads:
// the contraction index and the output columns are permuted so that a lane's 16 bytes are its
// operands, which leaves no copy through shared memory in that chain. One token with a rank
// of 16, 2048 -> 2048: 5.5 us in a graph, launch included (8 CTAs share its 128 KB of
// adapter; one by one they took 5.8); 61 tokens of 61 adapters 7.0 us, 7.9 MB: 1.1 TB/s.
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "gnf4_lora.cuh"

namespace gnf4 {

namespace {

// lane (g, t) holds row g, columns 2t, 2t+1 of an 8x8 matrix; afterwards rows 2t, 2t+1 of column g
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint2 ldg8(const uint16_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

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

// RP: rank padded to 16, 32, 64 or 128
template <int RP>
struct RowsShape {
    static constexpr int BM = 16, NT = RP / 8, KS = RP / 16;
    static constexpr int kPlane = RP + (RP >= 64 ? 32 : 0);          // 16-bit elements a row; conflict-free fragment loads
    static constexpr int kRed = RP + 8;                              // floats a row
    static constexpr size_t red = sizeof(float) * 4 * BM * kRed;     // partial sums of four warps
    static constexpr size_t plane = sizeof(uint16_t) * 2 * BM * kPlane;
    static constexpr size_t smem = red + plane + sizeof(float) * BM;
    static constexpr int kCtas = RP <= 64 ? 2 : 1;                   // that an SM's registers are to hold
};

// BWD: the backward's chain (first factor [L, C, r], second [L, r, O]) instead of the forward's
// ([L, r, C], [L, O, r]). A row that does not exist is computed from an address that does and
// not stored (rows do not mix), so only the last piece of an axis that is no multiple of 32
// is guarded element by element. LONG: a warp's part of the contraction is more than one chain.
template <int RP, bool BWD, bool F16, bool LONG>
__global__ void __launch_bounds__(kLoraThreads, RowsShape<RP>::kCtas) lora_rows_kernel(const LoraRowsArgs p) {
    using S = RowsShape<RP>;
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
        const uint16_t* src[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
                const int64_t r = row0 + min(8 * h + g, rows - 1);
                const int64_t at = p.src_row ? (int64_t)__ldg(p.src_row + r) : r;
                src[h] = p.src + (at >= 0 && at < p.n_src ? at * p.C : 0) + 8 * t;
            }
        // forward: rank row 8c + g, 16 bytes along the contraction; backward: contraction row
        // 8 (g>>1) + 2q + (g&1), its rank along the lanes' t
        const uint16_t* down = p.down + (int64_t)e * p.r * p.C +
                               (BWD ? (int64_t)(8 * (g >> 1) + (g & 1)) * p.r + 2 * V * t : (int64_t)g * p.C + 8 * t);
        float acc[NT][4];
        auto step = [&](int k0, auto guard) {
            constexpr bool GUARD = decltype(guard)::value;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            const bool in = !GUARD || k0 + 8 * t < p.C;
            uint4 a[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) a[h] = in ? ldg16(src[h] + k0) : zero;
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
            for (int c = 0; c < NT; ++c) {
                    mma16<F16>(acc[c], a[0].x, a[1].x, a[0].y, a[1].y, b[c][0], b[c][1]);
                    mma16<F16>(acc[c], a[0].z, a[1].z, a[0].w, a[1].w, b[c][2], b[c][3]);
                }
        };
        const int whole = p.C / 32;
        const int st0 = (int)((int64_t)whole * part / parts), st1 = (int)((int64_t)whole * (part + 1) / parts);
        float* mine = s_red + (size_t)(warp & 3) * BM * S::kRed;
        const int chains = LONG ? (whole / parts + kSumChain) / kSumChain : 1;  // of the warp with the most steps
        for (int i = 0; i < chains; ++i) {
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[c][j] = 0.0f;
            const int from = st0 + i * kSumChain, to = LONG ? min(from + kSumChain, st1) : st1;
#pragma unroll 2
            for (int st = from; st < to; ++st) step(32 * st, std::false_type{});
            if (i == chains - 1 && part == parts - 1 && (p.C & 31)) step(32 * whole, std::true_type{});
            // partial sums: tile c, column index n of the MMA is rank 8c + n (forward), or
            // 8 V (c / V) + 2 V (n >> 1) + 2 (c % V) + (n & 1) (backward). The upper four warps put
            // theirs down, the lower four add their own on top.
#pragma unroll
            for (int turn = 0; turn < 2; ++turn) {
                if ((warp < 4) == (turn == 1)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            const int j = BWD ? 8 * V * (c / V) + 2 * V * t + 2 * (c % V) : 8 * c + 2 * t;
                            float2* at = reinterpret_cast<float2*>(mine + (8 * h + g) * S::kRed + j);
                            float2 v = make_float2(acc[c][2 * h], acc[c][2 * h + 1]);
                            if (turn == 1 || i > 0) {
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
    // ---- the sums, their 16-bit terms and each row's output factor: four ranks a thread
    {
        constexpr int TPR = RP / 4;
        const float scal = p.scaling ? __ldg(p.scaling + e) : 1.0f;
        for (int i = tid; i < BM * TPR; i += kLoraThreads) {             // whole warps
            const int local = i / TPR, j = 4 * (i % TPR);
            const int64_t r = row0 + local;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            float fac = scal;
            bool have = local < rows;
            if (have && p.weight) fac *= __ldg(p.weight + r);
            if (have && p.src_row) {
                const int at = __ldg(p.src_row + r);
                have = at >= 0 && at < p.n_src;                          // else h is zero
            }
            if (local < rows && j < p.r) {
                const float* at = s_red + local * S::kRed + j;
                if (have) {
                    float4 s;
                    if (CS > 1) {
                        s = cluster_sum(at, CS);
                    } else {
                        const float4 a = *reinterpret_cast<const float4*>(at);
                        const float4 b = *reinterpret_cast<const float4*>(at + BM * S::kRed);
                        const float4 c = *reinterpret_cast<const float4*>(at + 2 * BM * S::kRed);
                        const float4 d = *reinterpret_cast<const float4*>(at + 3 * BM * S::kRed);
                        s = make_float4((a.x + b.x) + (c.x + d.x), (a.y + b.y) + (c.y + d.y), (a.z + b.z) + (c.z + d.z),
                                        (a.w + b.w) + (c.w + d.w));
                    }
                    const float f = BWD ? fac : 1.0f;
                    v[0] = f * s.x, v[1] = f * s.y, v[2] = f * s.z, v[3] = f * s.w;
                }
                if (crank == 0 && p.mid)
                    *reinterpret_cast<float4*>(p.mid + r * p.r + j) = make_float4(v[0], v[1], v[2], v[3]);
            }
            if (BWD) fac = 1.0f;
            if constexpr (F16) {
                // the row's largest value to [1, 2): both terms stay normal or fall below 2^-24 of it
                float big = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
                for (int o = TPR / 2; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                const uint32_t ex = __float_as_uint(big) >> 23;
                if (ex > 0u && ex < 254u) {
                    const float shrink = __uint_as_float((254u - ex) << 23);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] *= shrink;
                    fac *= __uint_as_float(ex << 23);
                }
            }
            uint32_t x[2], y[2];
            split_pair<2, F16>(v[0], v[1], x);
            split_pair<2, F16>(v[2], v[3], y);
#pragma unroll
            for (int term = 0; term < 2; ++term)
                *reinterpret_cast<uint2*>(s_plane + (size_t)(term * BM + local) * S::kPlane + j) = make_uint2(x[term], y[term]);
            if (j == 0) s_fac[local] = fac;
        }
    }
    if (CS > 1) cluster_arrive();                // this CTA has read its peers' sums; they may not leave before
    __syncthreads();

    // ---- second product: [BM, r] x [r, O] on top of base, the columns split over all warps
    {
        // where this lane's rows g and g + 8 of each MMA tile go, or -1
        int dst[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
                const int local = 8 * h + g;
                int b = -1;
                if (local < rows) b = p.dst_row ? __ldg(p.dst_row + row0 + local) : (int)(row0 + local);
                dst[h] = b < p.n_dst ? b : -1;
            }
        const uint16_t* up = p.up + (int64_t)e * p.r * p.O;
        const uint32_t plane0 = smem_addr(s_plane) + (uint32_t)(g * S::kPlane + 4 * G * t) * 2u;
        auto piece = [&](int n0, auto guard) {
            constexpr bool GUARD = decltype(guard)::value;
            const bool in = !GUARD || n0 + 8 * t < p.O;
            uint4 bs[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                    bs[h] = p.base && in && dst[h] >= 0
                                   ? *reinterpret_cast<const uint4*>(p.base + (int64_t)dst[h] * p.O + n0 + 8 * t)
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
                    const uint32_t at = plane0 + (uint32_t)((term * BM) * S::kPlane + 16 * q) * 2u;
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
                if (dst[h] < 0 || !in) continue;
                const float f = s_fac[8 * h + g];
                const uint32_t bw[4] = {bs[h].x, bs[h].y, bs[h].z, bs[h].w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        const float2 v = unpack16<F16>(bw[2 * i + c / 2]);
                        o[2 * i + c / 2] = pack16<F16>(fmaf(f, acc[c][2 * h + i], v.x), fmaf(f, acc[c + 1][2 * h + i], v.y));
                    }
                *reinterpret_cast<uint4*>(p.out + (int64_t)dst[h] * p.O + n0 + 8 * t) = make_uint4(o[0], o[1], o[2], o[3]);
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

template <int RP, bool BWD, bool F16>
cudaError_t launch_rows_t(const LoraRowsArgs& a, cudaStream_t s) {
    using S = RowsShape<RP>;
    static_assert(S::smem <= 48 * 1024, "shared memory without an opt-in");
    // CTAs of a cluster until there is about one for every SM
    const int64_t tiles = most_tiles(a, S::BM);
    int cs = 1;
    while (cs < 8 && tiles * cs * 2 <= 2 * (int64_t)device_sm_count()) cs *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * cs));
    cfg.blockDim = dim3(kLoraThreads);
    cfg.dynamicSmemBytes = S::smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // the loop over chains takes 0.2 of 5.8 us of a token at 2048 columns, which are one chain
    if (a.C / 32 / (cs * kLoraWarps) < kSumChain) return cudaLaunchKernelEx(&cfg, lora_rows_kernel<RP, BWD, F16, false>, a);
    return cudaLaunchKernelEx(&cfg, lora_rows_kernel<RP, BWD, F16, true>, a);
}

template <int RP>
cudaError_t launch_rows(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    if (bwd) return launch_rows_t<RP, true, false>(a, s);
    return f16 ? launch_rows_t<RP, false, true>(a, s) : launch_rows_t<RP, false, false>(a, s);
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

cudaError_t launch_lora_rows(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    // Many rows stream: from a 16-row tile for every SM on, one CTA after another no longer hides
    // the chain of loads. 2048 -> 1536, us with events, direct and streaming, forward / backward:
    // rank 16, 2048 rows of 64 adapters 12.8 and 14.8 / 13.7 and 14.5, 2400 rows 14.8 and 13.5 /
    // 17.0 and 14.9, 32768 rows of 128 adapters 96.9 and 68.6 / 110.7 and 74.0; rank 64, 2048 rows
    // 18.0 and 22.0 / 25.0 and 23.8, 2400 rows 22.8 and 21.7 / 34.1 and 23.1, 32768 rows 151.7 and
    // 119.1 / 217.5 and 123.2. Ranks above 64 have no streaming kernel: its stages of 256 columns do not
    // fit beside them (stages of 128 would), so their rows' factors are read once per 16 rows:
    // 8192 rows of 64 adapters, rank 64 36.7 us, rank 72 91.8, rank 128 100.
    if (a.r <= 64 && (a.test_stall || a.R >= 16 * (int64_t)device_sm_count())) return launch_lora_stream(a, bwd, f16, s);
    if (a.r <= 16) return launch_rows<16>(a, bwd, f16, s);
    if (a.r <= 32) return launch_rows<32>(a, bwd, f16, s);
    if (a.r <= 64) return launch_rows<64>(a, bwd, f16, s);
    return launch_rows<128>(a, bwd, f16, s);
}

cudaError_t launch_check_lora(const int64_t* offsets, int L, int64_t R, const int32_t* a, int64_t na, const int32_t* b,
                              int64_t nb, const float* w, unsigned* status, cudaStream_t s) {
    check_lora_kernel<<<64, 256, 0, s>>>(offsets, L, R, a, na, b, nb, w, status);
    return cudaGetLastError();
}

}  // namespace gnf4
