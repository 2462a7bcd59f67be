// The adapters' two products (gnf4_lora.cuh) for many rows.
//
// Persistent CTAs, one an SM, over tiles of 32 or 64 rows. Four producer warps keep a ring of
// stages filled by 16-byte asynchronous copies, the rows' next 256 columns together with the
// factor's, straight through from the first product of a tile to the second and on to the
// next tile; eight consumer warps take 32 columns (in the second product 16 rows of 64 or 128
// columns) of every stage, so that memory never waits for the warps to meet for the sums. All
// fragments come out of shared memory by ldmatrix.
//
// What bounds it: an SM's share of memory. One CTA's copies reach 43 GB/s from DRAM (6.4 TB/s
// in all) and 72 GB/s from L2, and a stage takes what its rows and its factor take at these
// rates, one after the other: 32768 rows of 128 adapters, rank 16, 2048 -> 1536, 68 us, 335 MB
// of rows at 4.9 TB/s. At rank 64 the factor, read once a tile, is half of a stage: 4096 rows,
// 2880 -> 5760, 47 us, of which memory alone takes 38 (under ncu: issue slots 31 % busy, the tensor
// pipe 28 %, DRAM 21 %, stalls on fixed latency and loads 2.6 and 2.5 cycles an instruction).
// Leaving out the products, the meeting of the warps or the stores changed the first case by 1, 0 and 18 us.
#include <atomic>
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "gnf4_lora.cuh"

namespace gnf4 {

namespace {

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
        if (p.test_stall) return;                                    // no copies: the consumers' waits give up
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
            gone = __any_sync(0xffffffffu, !mbar_wait_bounded(smem_addr(s_full + slot), phase, &s_abort, &g_lora_err, 2u,
                                                              p.test_stall ? kStallWaitCycles : kWaitTimeoutCycles));
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

        for (int q0 = 0; q0 < n1; q0 += kSumChain) {
            float acc[MT][NT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[m][c][j] = 0.0f;
            for (int q = q0; q < min(q0 + kSumChain, n1); ++q) {
                if (q) wait_stage();
                const uint32_t at = (uint32_t)(slot * S::kStage), factor = ring + at + BM * S::kRow;
                if (!gone) {                                         // columns past the end are zeros in both
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t a[MT][4];
#pragma unroll
                        for (int m = 0; m < MT; ++m) ldmatrix4(a[m], rows_frag + at + 16 * m * S::kRow + 32 * half);
#pragma unroll
                        for (int c = 0; c < NT; c += 2) {
                            uint32_t b[4];                           // tile c: k 0-7, 8-15; tile c + 1: the same
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
                                if (turn == 1 || q0 > 0) {
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

// Tiles of 64 rows halve what the factors cost, but leave SMs idle in the last wave sooner. A
// wave of them takes 1.7 waves of 32 rows (ranks of 16 and 32, 2048 -> 1536: 19000 rows,
// three waves of 64 49.5 and 59.6 us, five of 32 48.0 and 58.5; 16384 rows of 128 adapters,
// two and four waves, 41.9 and 46.3 against 44.0 and 53.6); about half a tile of every adapter
// is empty. A table of many adapters does not fit beside 64 rows at rank 32.
template <int RP>
cudaError_t launch_stream(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    static_assert(StreamShape<RP, 32>::smem(2048) <= kMaxSmem, "shared memory of a CTA");
    if constexpr (RP <= 32) {
        const int64_t sms = device_sm_count(), active = a.R < a.L ? a.R : a.L;
        const int64_t waves32 = (a.R / 32 + active / 2 + sms - 1) / sms, waves64 = (a.R / 64 + active / 2 + sms - 1) / sms;
        if (17 * waves64 < 10 * waves32 && StreamShape<RP, 64>::smem(a.L) <= kMaxSmem)
            return launch_stream_m<RP, 64>(a, bwd, f16, s);
    }
    return launch_stream_m<RP, 32>(a, bwd, f16, s);
}

}  // namespace

unsigned take_lora_error(cudaError_t* err) {
    unsigned v = 0;
    const unsigned zero = 0;
    *err = cudaMemcpyFromSymbol(&v, g_lora_err, sizeof(v));
    if (*err == cudaSuccess && v) *err = cudaMemcpyToSymbol(g_lora_err, &zero, sizeof(zero));
    return v;
}

cudaError_t launch_lora_stream(const LoraRowsArgs& a, bool bwd, bool f16, cudaStream_t s) {
    if (a.r <= 16) return launch_stream<16>(a, bwd, f16, s);
    if (a.r <= 32) return launch_stream<32>(a, bwd, f16, s);
    return launch_stream<64>(a, bwd, f16, s);
}

}  // namespace gnf4
