// The gradients of the adapters for ranks above 32 (gnf4_lora_grads.cu has the formula),
// on the tensor cores' own memory.
//
// A CTA owns CW columns of one gradient of one adapter and walks the adapter's rows in stages of
// 32. D [terms x rank, CW] += left^T right, rows the contraction index: both operands lie in
// shared memory as they come, row by row, contiguous across the contraction, and one thread has
// tcgen05.mma read them there. The terms of `left` are rows of one MMA side by side (128 in all,
// three terms of rank 64 take two and of rank 128 three) and are added up when the accumulator
// leaves tensor memory, at the end and, with very many rows (kGradChain), from time to time. The rows of `right` are copied straight to their swizzled
// place by 16-byte asynchronous copies, two stages ahead; codes and `left` go through the threads
// that copied them, which make bf16 of the one and the terms of the other.
//
// Against warp-level MMAs, which read every fragment through registers: at rank 64, 2048 and 1536
// columns, 64 adapters, 8192 rows, a backward pass of 87 us instead of 118; one adapter of 4096
// rows 50 and 71; rank 128, 100 adapters, 4096 rows 229 and 258. At rank 16 their fragments are
// few, and the parts that stay (a CTA's start, the split of left, the last sum) cost more than
// they do: 155 and 135 us with 128 adapters, 32768 rows, so that ranks up to 32 keep them.
// What bounds it is the chain of a stage (copied, made, multiplied) and its issue: in the first
// case 22 M instructions, 0.39 a cycle and scheduler, half of the stalls on shared memory and
// barriers, the tensor pipe and DRAM at 8 %. Persistent CTAs whose copies run on into the next
// item: 84 us instead of 87 there, but 103 and not 90 with shares like 1 / e, and 145 and not
// 137 at rank 128 (64 adapters, 8192 rows, 1024 columns).
#include <cstdint>
#include <cuda_runtime.h>

#include "gnf4_act8.cuh"
#include "gnf4_lora_grads.cuh"

namespace gnf4 {

namespace {

constexpr int kGradRows = 32;                            // rows of a stage

template <int RP, int TERMS, bool Q8, bool MANY>
struct GradShape {
    static constexpr int CW = RP == 64 ? 256 : 128;       // columns of a CTA, two of which share an SM
    static constexpr int S = 3;                          // stages
    static constexpr int MM = 128;                       // rows of an MMA
    static constexpr int SLOTS = MM / RP;                // terms that fit into one
    static constexpr int MMAS = (TERMS + SLOTS - 1) / SLOTS;
    static constexpr int kLeft = (kGradRows * RP / 4 + kLoraThreads - 1) / kLoraThreads;   // float4 of left a thread and stage
    static constexpr int tile = kGradRows * CW * 2;      // bytes of the rows' columns as bf16
    static constexpr int raw = Q8 ? tile / 2 : tile;     // as they are copied
    static constexpr int left = kGradRows * RP * 4, weight = kGradRows * RP;
    static constexpr int stage = (raw + left + weight + 1023) / 1024 * 1024;
    static constexpr int plane = MMAS * MM * kGradRows * 2;
    static constexpr int made = plane + (Q8 ? tile : 0);
    static constexpr int kStride = CW + 4;               // floats of a row of the sums
    static constexpr int work = S * stage + made, sums = 4 * RP * kStride;
    // so much at least that no more CTAs share an SM than its 512 columns of tensor memory serve:
    // one that waited for columns would hold up its cluster, and clusters could so wait for
    // one another
    static constexpr int kCols = MANY && SLOTS == 1 ? 2 * CW : CW;      // of tensor memory: the accumulator, and totals behind it
    static constexpr int least = kCols * 456 - 1024;
    static constexpr int need = 128 + 1023 + (work > sums ? work : sums);       // behind GradControl, at a multiple of 1024
    static constexpr int smem = need > least ? need : least;
};

struct GradControl {
    uint64_t done;                                       // the MMAs of a stage are through
    uint32_t tmem;
    int abort;
    GradSearch find;
};
static_assert(sizeof(GradControl) <= 128, "the space before the stages");

__device__ unsigned g_grads_err;                         // set when a wait gives up

// A matrix in shared memory for the tensor cores, contiguous along M or N: atoms of 8 rows (of K)
// by 64 elements, swizzled by 128 bytes; `next` bytes to the next 64 elements, 1024 to the next 8 rows.
__device__ __forceinline__ uint64_t desc_across(uint32_t saddr, uint32_t next) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(next >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// byte of element m, row k of such a matrix of `rows` rows
__device__ __forceinline__ uint32_t across(int m, int k, int rows) {
    return (uint32_t)((m >> 6) * (rows * 128) + k * 128 + ((((m & 63) >> 3) ^ (k & 7)) << 4) + (m & 7) * 2);
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// One item; more than one part of its rows are those of the CTAs of a cluster.
template <int RP, int TERMS, bool Q8, bool MANY>
__device__ __forceinline__ void grad_body(const LoraGradArgs& p, const LoraGradSide& d, const GradItem& it, uint8_t* smem,
                                          GradControl* ctl) {
    const int e = it.e, col0 = it.col0, parts = it.parts, part = it.part;
    using S = GradShape<RP, TERMS, Q8, MANY>;
    constexpr int CW = S::CW, SR = kGradRows, D = S::S - 1;     // stages that the copies are ahead
    constexpr int LPR = S::raw / SR / 16, RPI = 32 / LPR;    // lanes that copy a row, rows a warp copies at a time
    constexpr int BPR = CW / 32;                             // a row's blocks of a checkpoint
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t stage0 = smem_addr(smem), made0 = stage0 + S::S * S::stage;

    const int64_t lo = clamp_row(p.offsets[e], p.R), hi = clamp_row(p.offsets[e + 1], p.R);
    const int rows = hi > lo ? (int)(hi - lo) : 0;
    const float scal = d.factor && p.scaling ? __ldg(p.scaling + e) : 1.0f;
    const float* weight = d.factor ? p.weight : nullptr;
    // stage i of this CTA: rows first(i) .. first(i) + SR - 1 of the adapter
    const int stages = (rows + SR * parts - 1) / (SR * parts);
    auto first = [&](int i) { return (i * parts + part) * SR; };

    // A warp copies rows 8 s + warp of a stage, s = 0..3. Lane 4 j + s knows where row s of the
    // j-th of eight stages lies in `right` (-1: nowhere).
    auto source_rows = [&](int i0) -> int {
        const int local = first(i0 + (lane >> 2)) + 8 * (lane & 3) + warp;
        if (local >= rows) return -1;
        const int64_t r = lo + local, at = d.row ? (int64_t)__ldg(d.row + r) : r;
        return at >= 0 && at < d.n ? (int)at : -1;
    };
    // and that row's scales, a byte each
    uint32_t scale_now[(BPR + 3) / 4], scale_next[(BPR + 3) / 4];
    auto scales_of = [&](int at, uint32_t (&out)[(BPR + 3) / 4]) {
#pragma unroll
        for (int w = 0; w < (BPR + 3) / 4; ++w) out[w] = 0u;
#pragma unroll
        for (int b = 0; b < BPR; ++b)
            if (at >= 0 && col0 + 32 * b < d.C)
                out[b / 4] |= (uint32_t)__ldg(d.scales + (int64_t)at * (d.C / 32) + col0 / 32 + b) << 8 * (b & 3);
    };

    // a copied piece: codes wait where their own thread finds them again, bf16 in the MMA's order
    const int chunk = lane % LPR, sub = lane / LPR;
    const int col = col0 + chunk * (Q8 ? 16 : 8);
    const bool col_ok = col < d.C;
    auto copy_right = [&](int i, int row) {
        const uint32_t dst = stage0 + (uint32_t)(i % S::S * S::stage);
#pragma unroll
        for (int q = 0; q < 4 / RPI; ++q) {
            const int s = q * RPI + sub;
            const int at = __shfl_sync(0xffffffffu, row, 4 * (i & 7) + s);
            const bool ok = at >= 0 && col_ok;
            const int64_t o = ok ? (int64_t)at * d.C + col : 0;
            if constexpr (Q8) copy_async16(dst + (uint32_t)((q * kLoraThreads + tid) * 16), d.codes + o, ok ? 16u : 0u);
            else copy_async16(dst + across(8 * chunk, 8 * s + warp, SR), d.right + o, ok ? 16u : 0u);
        }
    };
    // left, four elements a piece, and the row's weight: read again by the thread that copied them
    auto copy_left = [&](int i) {
        const uint32_t dst = stage0 + (uint32_t)(i % S::S * S::stage + S::raw);
#pragma unroll
        for (int q = 0; q < S::kLeft; ++q) {
            const int id = q * kLoraThreads + tid, local = first(i) + id / (RP / 4), j = 4 * (id % (RP / 4));
            if (id < SR * RP / 4) {
                const bool ok = local < rows && j < p.r;
                copy_async16(dst + (uint32_t)(id * 16), d.left + (ok ? (lo + local) * p.r + j : 0), ok ? 16u : 0u);
                if (weight && ok) copy_async4(dst + (uint32_t)(S::left + id * 4), weight + lo + local);
            }
        }
    };
    // the stage's left, split into terms: of 16 SLOTS matrix rows of MMA q the first 16 hold term
    // q * SLOTS of 16 ranks, the next 16 (where there are two SLOTS) the next term of the same ranks
    auto make_left = [&](int i) {
        const uint32_t from = stage0 + (uint32_t)(i % S::S * S::stage + S::raw);
        const uint32_t to = made0;
#pragma unroll
        for (int q = 0; q < S::kLeft; ++q) {
            const int id = q * kLoraThreads + tid, k = id / (RP / 4), j = 4 * (id % (RP / 4));
            if (id >= SR * RP / 4) break;
            const uint4 v = lds16(from + (uint32_t)(id * 16));
            float f = first(i) + k < rows ? scal : 0.0f;
            if (weight && first(i) + k < rows) f *= __uint_as_float(lds4(from + (uint32_t)(S::left + id * 4)));
            uint32_t a[TERMS], b[TERMS];
            split_pair<TERMS, false>(__uint_as_float(v.x) * f, __uint_as_float(v.y) * f, a);
            split_pair<TERMS, false>(__uint_as_float(v.z) * f, __uint_as_float(v.w) * f, b);
#pragma unroll
            for (int t = 0; t < TERMS; ++t) {
                const uint32_t at = to + (uint32_t)(t / S::SLOTS * S::MM * SR * 2) + across(16 * S::SLOTS * (j / 16) + 16 * (t % S::SLOTS) + j % 16, k, SR);
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(a[t]), "r"(b[t]) : "memory");
            }
        }
    };
    // the stage's codes as bf16
    auto make_right = [&](int i) {
        const uint32_t from = stage0 + (uint32_t)(i % S::S * S::stage);
        const uint32_t to = made0 + S::plane;
#pragma unroll
        for (int q = 0; q < 4 / RPI; ++q) {
            const int s = q * RPI + sub;
            uint32_t sc = 0u;
#pragma unroll
            for (int w = 0; w < (BPR + 3) / 4; ++w) {
                const uint32_t v = __shfl_sync(0xffffffffu, scale_now[w], 4 * (i & 7) + s);
                if (w == chunk / 8) sc = v;
            }
            const uint32_t step = act8_step_bf16(sc >> 8 * (chunk / 2 & 3) & 255u) * 0x10001u;
            const uint4 v = lds16(from + (uint32_t)((q * kLoraThreads + tid) * 16));
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c] = act8_pair(prmt(u[c / 2], 0u, c & 1 ? 0x0302u : 0x0100u), step);
#pragma unroll
            for (int c = 0; c < 2; ++c)
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + across(16 * chunk + 8 * c, 8 * s + warp, SR)),
                             "r"(o[4 * c]), "r"(o[4 * c + 1]), "r"(o[4 * c + 2]), "r"(o[4 * c + 3]) : "memory");
        }
    };

    // prologue: D stages of copies under way
    int row_now = -1, row_next = -1;
    if (stages > 0) row_now = source_rows(0);
    if (stages > 8) row_next = source_rows(8);
#pragma unroll
    for (int i = 0; i < D; ++i)
        if (i < stages) copy_right(i, row_now);
    if constexpr (Q8) scales_of(row_now, scale_now);
    if (!d.factor) wait_for_previous_grid();             // dA's left comes from the rows kernel; the copies above do not
#pragma unroll
    for (int i = 0; i < D; ++i) {
        if (i < stages) copy_left(i);
        copy_commit();
    }
    if constexpr (TERMS % S::SLOTS != 0) {               // the rows of the last MMA that no term fills
        static_assert(S::SLOTS <= 2 && S::MM * SR * 2 / 16 == 2 * kLoraThreads, "half of the matrix's 16-byte pieces");
        const int k = tid & 31, m = 32 * (tid >> 6) + 16 + 8 * (tid >> 5 & 1);
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                     ::"r"(made0 + (uint32_t)((S::MMAS - 1) * S::MM * SR * 2) + across(m, k, SR)), "r"(0u) : "memory");
    }

    const uint32_t tmem = ctl->tmem;
    bool gone = false;
    // MANY: totals that the accumulator is emptied into. 64 columns a thread of one rank, half of the accumulator's for the 32 lanes (matrix
    // rows) that a warp reads. With two SLOTS lanes 16 to 31 hold the other term of the ranks of lanes 0
    // to 15, each of a pair of lanes keeps one half of its columns, and the totals lie in
    // registers: the accumulators of two CTAs fill the SM's tensor memory. Else they lie behind the accumulator.
    constexpr int CHAIN = kGradChain<TERMS>;
    const int quarter = warp & 3, half = warp >> 2;
    const bool upper = S::SLOTS == 2 && lane >= 16;
    const uint32_t sums = tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)(half * (CW / 2));
    constexpr bool REGS = MANY && S::SLOTS == 2;
    float total[REGS ? 64 : 1];
#pragma unroll
    for (int c = 0; c < (REGS ? 64 : 1); ++c) total[c] = 0.0f;
    // 16 of this thread's columns of the accumulator, terms added up, from column c on
    auto read = [&](int c, float (&v)[16]) {
        tmem_load16(v, sums + c);
        if constexpr (S::SLOTS == 2) {
            float w[16];
            tmem_load16(w, sums + 64 + c);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float other = __shfl_xor_sync(0xffffffffu, upper ? v[k] : w[k], 16);
                v[k] = (upper ? w[k] : v[k]) + other;
            }
        }
    };
    auto empty = [&](bool first) {
        tc_after();
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            float v[16];
            read(c, v);
            if constexpr (REGS) {
#pragma unroll
                for (int k = 0; k < 16; ++k) total[c + k] += v[k];
            } else {
                if (!first) {
                    float u[16];
                    tmem_load16(u, sums + CW + c);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] += u[k];
                }
                tmem_store16(sums + CW + c, v);
            }
        }
        if constexpr (!REGS) asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_before();
    };
    auto wait_made = [&](int i) {                        // the MMAs of stage i are through
        if (!gone)
            gone = !mbar_wait_bounded(smem_addr(&ctl->done), (uint32_t)(i & 1), &ctl->abort, &g_grads_err, 1u,
                                      p.test_stall ? kStallWaitCycles : kWaitTimeoutCycles);
    };
    for (int i = 0; i < stages; ++i) {
        copy_wait<D - 1>();
        if (i > 0) wait_made(i - 1);
        if ((i + D & 7) == 0) {
            row_now = row_next;
            row_next = i + D + 8 < stages ? source_rows(i + D + 8) : -1;
        }
        if (i + D < stages) {
            copy_right(i + D, row_now);
            copy_left(i + D);
        }
        copy_commit();
        if constexpr (MANY) {
            if (i > 0 && i % CHAIN == 0) empty(i == CHAIN);              // the next product starts from nothing
        }
        make_left(i);
        if constexpr (Q8) {
            if (i && (i & 7) == 0) {
#pragma unroll
                for (int w = 0; w < (BPR + 3) / 4; ++w) scale_now[w] = scale_next[w];
            }
            if ((i & 7) == 4) scales_of(row_next, scale_next);
            make_right(i);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        if (tid == 0 && !gone && !p.test_stall) {
            tc_after();
            const uint32_t a = made0;
            const uint32_t b = Q8 ? a + S::plane : stage0 + (uint32_t)(i % S::S * S::stage);
            // fp32 sums of bf16 products; both operands contiguous across K
            constexpr uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | 1u << 16 | (uint32_t)(CW / 8) << 17 | (uint32_t)(S::MM / 16) << 24;
#pragma unroll
            for (int k = 0; k < SR / 16; ++k)
#pragma unroll
                for (int m = 0; m < S::MMAS; ++m)
                    asm volatile(
                        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                        ::"r"(tmem), "l"(desc_across(a + (uint32_t)(m * S::MM * SR * 2 + k * 2048), SR * 128)),
                          "l"(desc_across(b + (uint32_t)(k * 2048), SR * 128)), "r"(idesc), "r"((uint32_t)((MANY ? i % CHAIN : i) | k | m)) : "memory");
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                         ::"r"(smem_addr(&ctl->done)) : "memory");
        }
    }
    copy_wait<0>();
    if (stages > 0) wait_made(stages - 1);
    tc_after();
    __syncthreads();                                     // the stages become the sums' space

    float* s_red = reinterpret_cast<float*>(smem);
    static_assert(CW / 2 == 64 * S::SLOTS, "columns of a thread's totals");
    {
        const int j = S::SLOTS == 2 ? 16 * quarter + (lane & 15) : 32 * quarter + lane;
        float4* to = reinterpret_cast<float4*>(s_red + j * S::kStride + half * (CW / 2) + (upper ? 64 : 0));
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = 0.0f;
            if (stages > 0) {                            // else nothing was ever written there
                read(c, v);
                if constexpr (REGS) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] += total[c + k];
                } else if (MANY && stages > CHAIN) {
                    float u[16];
                    tmem_load16(u, sums + CW + c);
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] += u[k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) to[c / 4 + k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
    }
    __syncthreads();
    store_sums<RP, CW, CW, S::kStride, TERMS>(p, d, it, s_red);
}

template <int RP, int TERMS, bool Q8, bool MANY>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_grads_wide_kernel(const LoraGradArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* buffers = smem + ((0u - smem_addr(smem) - (uint32_t)sizeof(GradControl) & 1023u) + sizeof(GradControl));
    using S = GradShape<RP, TERMS, Q8, MANY>;
    constexpr int CW = S::CW;
    GradControl* ctl = reinterpret_cast<GradControl*>(smem);
    if (threadIdx.x < 32) tmem_alloc<S::kCols>(&ctl->tmem);
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&ctl->done), 1);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const GradItem it = grad_item(p, CW, &ctl->find);
    if (it.e < p.L) {
        if (it.side_b) grad_body<RP, TERMS, false, MANY>(p, p.b, it, buffers, ctl);
        else grad_body<RP, TERMS, Q8, MANY>(p, p.a, it, buffers, ctl);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (threadIdx.x < 32) tmem_free<S::kCols>(ctl->tmem);
    // whoever waits for this grid waits for that one too; a CTA without an item leaves its place at once
    if (threadIdx.x == 0 && (it.e < p.L || blockIdx.x == 0)) wait_for_previous_grid();
}

template <int RP, int TERMS, bool Q8, bool MANY>
cudaError_t launch_wide_t(const LoraGradArgs& a, int cs, cudaStream_t s) {
    using S = GradShape<RP, TERMS, Q8, MANY>;
    constexpr int own = S::smem, other = GradShape<RP, TERMS, false, MANY>::smem;
    constexpr int smem = own > other ? own : other;
    static_assert(2 * (smem + 1024) <= 228 * 1024, "shared memory of an SM");
    return launch_grads_kernel<lora_grads_wide_kernel<RP, TERMS, Q8, MANY>>(a, S::CW, cs, smem, s);
}

template <int RP, int TERMS, bool Q8>
cudaError_t launch_wide_q(const LoraGradArgs& a, int cs, cudaStream_t s) {
    if (past_chain(a, cs, 1, kGradChain<TERMS>)) return launch_wide_t<RP, TERMS, Q8, true>(a, cs, s);
    return launch_wide_t<RP, TERMS, Q8, false>(a, cs, s);
}

template <int RP>
cudaError_t launch_wide_w(const LoraGradArgs& a, bool f32, int cs, cudaStream_t s) {
    if (a.a.codes) return f32 ? launch_wide_q<RP, 3, true>(a, cs, s) : launch_wide_q<RP, 2, true>(a, cs, s);
    return f32 ? launch_wide_q<RP, 3, false>(a, cs, s) : launch_wide_q<RP, 2, false>(a, cs, s);
}

// A cluster along an adapter's rows as long as they fit on the SMs at once and keep 128 rows each
// (one adapter of 512 rows, rank 128: 44 us, and 48 with 64 rows each). Else adapters of four
// times the average's rows share a cluster of 2, which is an SM: of 4, 93 us and not 87 in the
// first case above, 98 and not 90 with shares like 1 / e.
template <int RP>
cudaError_t launch_wide_r(const LoraGradArgs& a, bool f32, cudaStream_t s) {
    constexpr int CW = GradShape<RP, 2, false, false>::CW;
    const int64_t active = a.R < a.L ? (a.R > 0 ? a.R : 1) : a.L;
    const int64_t avg = (a.R + active - 1) / active, room = 2 * (int64_t)device_sm_count();
    const int64_t items = active * (grad_items(a.a, CW) + grad_items(a.b, CW));
    int cs = 1;
    while (cs < 8 && items * cs * 2 <= room && avg >= 128 * 2 * cs) cs *= 2;
    LoraGradArgs b = a;
    b.heavy = cs > 1 ? 0 : heavy_rows(a.R, avg);
    return launch_wide_w<RP>(b, f32, b.heavy ? 2 : cs, s);
}

}  // namespace

unsigned take_grads_error(cudaError_t* err) {
    unsigned v = 0;
    const unsigned zero = 0;
    *err = cudaMemcpyFromSymbol(&v, g_grads_err, sizeof(v));
    if (*err == cudaSuccess && v) *err = cudaMemcpyToSymbol(g_grads_err, &zero, sizeof(zero));
    return v;
}

cudaError_t launch_lora_grads_wide(const LoraGradArgs& a, bool f32, cudaStream_t s) {
    return a.r <= 64 ? launch_wide_r<64>(a, f32, s) : launch_wide_r<128>(a, f32, s);
}

}  // namespace gnf4
