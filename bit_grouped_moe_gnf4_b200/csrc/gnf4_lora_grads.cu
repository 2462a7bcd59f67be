// The gradients of the adapters (gnf4_lora.cuh): sums over an adapter's rows.
//
// One gradient of one adapter: sum over its rows of left[r, j] right[row r, n], rows the MMA's
// contraction index. A CTA owns WC * SC columns (SC a warp) and walks the adapter's rows in
// stages of 32 WR: the rows of `right` are gathered into shared memory by 16-byte asynchronous
// copies, three stages deep (the gather's latency, index then row, is what a warp alone cannot
// hide), while `left` is read ahead by a stage into registers and split into its 16-bit terms
// once for all warps. Both fragments come out of shared memory transposed. Over many rows the
// accumulators are emptied into totals in tensor memory from time to time (kGradChain).
//
// What bounds it is instruction issue: about 330 instructions a warp and stage of 32 rows (the
// copies' addresses, the split of left, the products; 450 with codes). 128 experts over 32768 rows,
// rank 16, 2048 checkpointed and 1536 columns: issue slots 46 % busy, the stalls led by fixed
// latency (1.9 cycles an instruction) and barriers (1.2), loads and shared memory 0.8 each, DRAM
// at 18 % of its rate, the tensor pipe at 18 %; 64 us. Warps that only copy beside warps
// that only multiply took 65 to 75 us there, with bulk copies of a row (52 to 67 cycles each
// from one CTA) or 16-byte ones.
#include <cstdint>
#include <cuda_runtime.h>

#include "gnf4_act8.cuh"
#include "gnf4_lora_grads.cuh"

namespace gnf4 {

namespace {

constexpr int kGradStages = 3;

template <int RP, int WR, int TERMS>
struct GradShape {
    static constexpr int CT = 8;                         // MMA column tiles of a warp's slab
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
    // codes take half a stage; their steps lie in the other half of the last one
    static constexpr size_t step_at = kGradStages * stage_bytes - 2 * scale_bytes;
    static_assert((kGradStages - 1) * stage_bytes + SR * kPitch8 <= step_at, "the steps behind the last stage's codes");
    static constexpr size_t work = kGradStages * stage_bytes + 2 * plane_bytes + 2 * SR * 4;
    static constexpr size_t sums = sizeof(float) * (size_t)kLoraWarps * RP * kStride;
    static constexpr size_t smem = work > sums ? work : sums;
    static constexpr int kTotals = 64 * MT;              // columns of tensor memory: a warp's accumulators lie on its 32 lanes
    // with so much shared memory beside them, the CTAs that an SM holds never want more columns than it has
    static_assert(smem >= kTotals * 456, "tensor memory of an SM");
};

// One item; more than one part of its rows are those of the CTAs of a cluster.
template <int RP, int WR, int TERMS, bool Q8, bool MANY>
__device__ __forceinline__ void grad_body(const LoraGradArgs& p, const LoraGradSide& d, const GradItem& it, uint8_t* smem,
                                          uint32_t* s_tmem) {
    const int e = it.e, col0 = it.col0, parts = it.parts, part = it.part;
    using S = GradShape<RP, WR, TERMS>;
    constexpr int CT = S::CT, MT = S::MT, WC = S::WC, CW = S::CW, SR = S::SR;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int wc = warp % WC, wr = warp / WC;
    uint8_t* s_stage = smem;
    uint16_t* s_plane = reinterpret_cast<uint16_t*>(smem + kGradStages * S::stage_bytes);
    uint16_t* s_step = reinterpret_cast<uint16_t*>(smem + S::step_at);
    int* s_row = reinterpret_cast<int*>(smem + kGradStages * S::stage_bytes + 2 * S::plane_bytes);
    const uint32_t stage0 = smem_addr(s_stage), plane0 = smem_addr(s_plane);

    const int64_t lo = clamp_row(p.offsets[e], p.R), hi = clamp_row(p.offsets[e + 1], p.R);
    const int rows = hi > lo ? (int)(hi - lo) : 0;
    const float scal = d.factor && p.scaling ? __ldg(p.scaling + e) : 1.0f;
    // stage i of this CTA: rows first(i) .. first(i) + SR - 1 of the adapter
    const int stages = (rows + SR * parts - 1) / (SR * parts);
    auto first = [&](int i) { return (i * parts + part) * SR; };

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

    // MANY: the accumulators are emptied into totals, which lie in tensor memory, from time to time
    auto totals = [&]() { return *s_tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(warp >> 2) * (S::kTotals / 2); };
    auto add_totals = [&]() {
        const uint32_t at = totals();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const float4 v = tmem_load4(at + 32 * m + 4 * c);
                acc[m][c][0] += v.x;
                acc[m][c][1] += v.y;
                acc[m][c][2] += v.z;
                acc[m][c][3] += v.w;
            }
    };
    auto empty = [&]() {
        const uint32_t at = totals();
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                tmem_store4(at + 32 * m + 4 * c, acc[m][c]);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][c][j] = 0.0f;
            }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    };

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
                    static_assert(CT == 8, "two words of codes a row");
                    const uint2 u = lds8(at), v = lds8(at + S::kPitch8);
                    const uint32_t w[2][CT / 4] = {{u.x, u.y}, {v.x, v.y}};
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
        if (MANY && (i + 1) % kGradChain<TERMS> == 0 && i + 1 < stages) {
            if (i + 1 > kGradChain<TERMS>) add_totals();
            empty();
        }
    }
    if (MANY && stages > kGradChain<TERMS>) add_totals();
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
    store_sums<RP, CW, S::SC, S::kStride, TERMS>(p, d, it, s_red);
}

template <int RP, int WR, int TERMS, bool Q8, bool MANY>
__global__ void __launch_bounds__(kLoraThreads, WR == 1 ? 2 : 1) lora_grads_kernel(const LoraGradArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ GradSearch find;
    __shared__ uint32_t s_tmem;
    using S = GradShape<RP, WR, TERMS>;
    if constexpr (MANY) {
        if (threadIdx.x < 32) tmem_alloc<S::kTotals>(&s_tmem);
        tc_before();
        __syncthreads();
        tc_after();
    }
    const GradItem it = grad_item(p, S::CW, &find);
    if (it.e < p.L) {
        if (it.side_b) grad_body<RP, WR, TERMS, false, MANY>(p, p.b, it, smem, &s_tmem);
        else grad_body<RP, WR, TERMS, Q8, MANY>(p, p.a, it, smem, &s_tmem);
    }
    if constexpr (MANY) {
        tc_before();
        __syncthreads();
        tc_after();
        if (threadIdx.x < 32) tmem_free<S::kTotals>(s_tmem);
    }
    // whoever waits for this grid waits for that one too; a CTA without an item leaves its place at once
    if (threadIdx.x == 0 && (it.e < p.L || blockIdx.x == 0)) wait_for_previous_grid();
}

template <int RP, int WR, int TERMS, bool Q8, bool MANY>
cudaError_t launch_grads_t(const LoraGradArgs& a, int cs, cudaStream_t s) {
    using S = GradShape<RP, WR, TERMS>;
    static_assert(S::smem <= kMaxSmem, "shared memory of a CTA");
    return launch_grads_kernel<lora_grads_kernel<RP, WR, TERMS, Q8, MANY>>(a, S::CW, cs, (int)S::smem, s);
}

template <int RP, int WR, int TERMS, bool Q8>
cudaError_t launch_grads_q(const LoraGradArgs& a, int cs, cudaStream_t s) {
    if (past_chain(a, cs, WR, kGradChain<TERMS>)) return launch_grads_t<RP, WR, TERMS, Q8, true>(a, cs, s);
    return launch_grads_t<RP, WR, TERMS, Q8, false>(a, cs, s);
}

template <int RP, int WR>
cudaError_t launch_grads_w(const LoraGradArgs& a, bool f32, int cs, cudaStream_t s) {
    if (a.a.codes) return f32 ? launch_grads_q<RP, WR, 3, true>(a, cs, s) : launch_grads_q<RP, WR, 2, true>(a, cs, s);
    return f32 ? launch_grads_q<RP, WR, 3, false>(a, cs, s) : launch_grads_q<RP, WR, 2, false>(a, cs, s);
}

// How the work is cut. First by columns, all the CTA's warps side by side (WR = 1), with a
// cluster of CTAs along an adapter's rows as long as they fit on the SMs at once and keep 128
// rows each. Where that leaves more than half of the SMs idle, narrow CTAs whose warps share
// the rows of a stage. us with events at 2048 and 1536 columns, wide and narrow, best cluster
// of each: rank 16, one adapter of 4096 rows 25.8 and 19.1, of 512 rows 10.9 and 10.9, four
// of 1024 rows 17.0 and 19.0, four of 4096 rows 36.9 and 46.0, sixteen of 512 rows 23.8 and
// 35.3; rank 32 and fp32 results, one of 4096 rows 37.2 and 26.9, four of 4096 rows 64.2 and
// 76.6.
template <int RP>
cudaError_t launch_grads_r(const LoraGradArgs& a, bool f32, cudaStream_t s) {
    constexpr int WR = 4;
    const int64_t active = a.R < a.L ? (a.R > 0 ? a.R : 1) : a.L;
    const int64_t avg = (a.R + active - 1) / active, sms = device_sm_count();
    const int64_t wide = active * (grad_items(a.a, GradShape<RP, 1, 2>::CW) + grad_items(a.b, GradShape<RP, 1, 2>::CW));
    const int64_t narrow = active * (grad_items(a.a, GradShape<RP, WR, 2>::CW) + grad_items(a.b, GradShape<RP, WR, 2>::CW));
    const int64_t room = 2 * sms;                    // wide CTAs that run at once
    int cs = 1;
    while (cs < 8 && wide * cs * 2 <= room && avg >= 128 * 2 * cs) cs *= 2;
    if (2 * wide * cs >= room || narrow > sms) {
        LoraGradArgs b = a;
        b.heavy = cs > 1 ? 0 : heavy_rows(a.R, avg);
        if (b.heavy == 0) return launch_grads_w<RP, 1>(a, f32, cs, s);
        // One CTA an item, and clusters for the heavy adapters. us of a backward pass at 2048 and 1536
        // columns, 128 adapters, 32768 rows, rank 16, without and with them: even rows 123 and 125,
        // shares like 1 / e 342 and 155 (203 with clusters of 2).
        return launch_grads_w<RP, 1>(b, f32, 4, s);
    }
    cs = 1;
    while (cs < 8 && narrow * cs * 2 <= sms && avg >= 128 * 2 * cs) cs *= 2;
    return launch_grads_w<RP, WR>(a, f32, cs, s);
}

}  // namespace

cudaError_t launch_lora_grads(const LoraGradArgs& a, bool f32, cudaStream_t s) {
    if (a.r <= 16) return launch_grads_r<16>(a, f32, s);
    if (a.r <= 32) return launch_grads_r<32>(a, f32, s);
    return launch_lora_grads_wide(a, f32, s);
}

}  // namespace gnf4
