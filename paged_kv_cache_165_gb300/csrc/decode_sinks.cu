// decode_sinks.cu -- paged attention with a sliding window whose first tokens stay visible (sinks), for bf16
// caches of d in {64, 128, 256} and bs in {16, 32}; other caches: decode_sinks_simt.cu.
//
// The query row at position p of a sequence sees the keys t <= p with t < S or t > p - W: two runs of tokens.
// The pages between them are left out of the count (sinks_span in decode_kparams.cuh), so that a chunk of
// pages is again a run of consecutive numbers and only table entries and masks know of the gap.
//
// This kernel, for up to eight (query row, head) pairs per sequence and KV head (more with d = 256): one CTA per
// (sequence, KV head, group of pairs, chunk of pages).  Every warp streams its own pages (round robin) through a
// private ring of TMA stages and attends all of the CTA's pairs to each, so that a page leaves HBM once per KV head
// and no warp waits for another.  Eight pairs make a tile of the m16n8k16 bf16 MMAs: bound by HBM, tcgen05's 128
// rows would be a sixteenth used (and measured 188 us where this takes 172).  More pairs: decode_sinks_umma.cu.
// 64 sequences, window 4096 + 4, 32 heads on 8 of 128: 172 us, 6.25 TB/s, 92% of the measured copy rate.
//
// Precision: the results are as exact as fp32 arithmetic on the bf16 cache.  q and the softmax weights enter
// the tensor cores as three bf16 parts (8 + 8 + 8 bits, all of an fp32 number): rows 0-7 of an MMA hold the
// first parts of a tile's pairs, rows 8-15 the second ones, and another MMA the third parts (of two tiles at
// once where there are two).  Sums inside the tensor cores are short -- d products of a score, the tokens of one
// page of an output -- and the running output is kept and rescaled in fp32 registers, since a long chain of
// tensor-core sums drifts by its truncations.
//
// V rows that no pair of the CTA sees may hold NaN or infinities and are cleared in shared memory (their
// weights are 0, but 0 times NaN is not); K rows need nothing, their scores are replaced.
#include <algorithm>
#include <atomic>
#include <math.h>

#include "common.cuh"
#include "decode_kparams.cuh"
#include "decode_sinks.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// D = A B (+ C) of m16n8k16 with the accumulator apart, so that a zero one costs no moves.
__device__ __forceinline__ void mma_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <int D, int BS, int TILES>
struct SinksCfg {
    // two blocks an SM with 96 KB of rings each: a deeper ring and fewer, longer blocks than three of 64 KB (window decode
    // 171 us against 181).  d = 256: rings of 64 KB, two blocks; with pages of 32, 128 KB and one block (kBlocks)
    static constexpr int NW = D == 256 ? 2 : BS * D == 4096 ? 3 : 4;                          // warps
    static constexpr int ST = D == 256 ? 2 : 98304 / (NW * 4 * BS * D);                       // stages of a warp's ring
    static constexpr int NT = BS / 8, KT = BS / 16, KS = D / 16;     // score tiles, k-steps of P.V and of q.K
    static constexpr int PANELS = D / 64;
    static constexpr int kPageBytes = BS * D * 2, kStageBytes = 2 * kPageBytes;
    static constexpr bool kQShared = TILES > 1 || D == 256;          // q parts in shared memory (else in registers)
    static constexpr int kPairs = TILES * 8;
    static constexpr int kRingBytes = NW * ST * kStageBytes;
    static constexpr int kMergeBytes = (NW * (D + 2) + 1) * kPairs * 4;   // the warps' states, in the ring
    static constexpr int kOffQ = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kQBytes = kQShared ? TILES * KS * 32 * 24 : 0;
    static constexpr int kOffBar = (kOffQ + kQBytes + 15) / 16 * 16;
    static constexpr int kSmemBytes = 1024 + kOffBar + NW * ST * 8;
    static constexpr int kBlocks = 2 * (kSmemBytes + 1024) <= 233472 ? 2 : 1;   // per SM
};
static_assert(SinksCfg<64, 16, 1>::kBlocks == 2 && SinksCfg<64, 32, 1>::kBlocks == 2 && SinksCfg<128, 16, 1>::kBlocks == 2 &&
                  SinksCfg<128, 32, 1>::kBlocks == 2 && SinksCfg<256, 16, 1>::kBlocks == 2 && SinksCfg<256, 16, 2>::kBlocks == 2 &&
                  SinksCfg<256, 32, 1>::kBlocks == SinksCfg<256, 32, 2>::kBlocks,
              "plan_sinks");

// One warp's pages for T tiles of pairs (MAXT: of the CTA's layout); leaves its states (running maximum and sum in
// base 2, unnormalised outputs) in shared memory.
template <int D, int BS, int MAXT, int T>
__device__ __forceinline__ void attend_pages(const CUtensorMap &tm_k, const CUtensorMap &tm_v, const DecodeKParams &p,
                                             const SinksWork &w, uint8_t *smem, uint64_t *bars) {
    using C = SinksCfg<D, BS, MAXT>;
    constexpr int NW = C::NW, ST = C::ST, NT = C::NT, KT = C::KT, KS = C::KS, NP = D / 16;
    constexpr int LT = T / 2;                                // accumulators of third parts, two tiles each
    constexpr bool kQRegs = T == 1 && D <= 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int kvh = w.kvh, npairs = w.npairs, pg0 = w.pg0, S = p.sinks;
    uint4 *s_qhm = reinterpret_cast<uint4 *>(smem + C::kOffQ);                      // [tiles][KS][32]
    uint2 *s_qlo = reinterpret_cast<uint2 *>(smem + C::kOffQ + MAXT * KS * 32 * 16);
    // this warp's pages: pg0 + warp + NW * k; table entries 32 at a time ahead of the copies
    const int n_my = w.pg1 - pg0 > warp ? (w.pg1 - pg0 - warp + NW - 1) / NW : 0;
    auto entry = [&](int k) {
        return k < n_my ? __ldg(p.block_table + static_cast<size_t>(w.b) * p.MBS + page_entry(w.sp, pg0 + warp + k * NW)) : 0;
    };
    int tcur = entry(lane), tnext = entry(32 + lane), tbase = 0;
    const int oob_row = p.NB * p.Hkv * BS;   // a row past the end: TMA fills zeros
    auto issue = [&](int k) {   // whole warp (shuffle); lane 0 issues the copies
        while (k >= tbase + 32) {
            tcur = tnext;
            tbase += 32;
            tnext = entry(tbase + 32 + lane);
        }
        const int phys = __shfl_sync(kFull, tcur, k & 31);
        if (lane == 0) {
            int row = oob_row;
            if (phys < 0 || phys >= p.NB) raise_error(p.err, PKV_DEVERR_BLOCK);
            else row = (phys * p.Hkv + kvh) * BS;
            const int st = warp * ST + k % ST;
            const uint32_t bar = smem_addr(&bars[st]), dst = smem_addr(smem + st * C::kStageBytes);
            mbar_arrive_expect_tx(bar, C::kStageBytes);
#pragma unroll
            for (int pn = 0; pn < C::PANELS; ++pn) {
                tma_load_2d(dst + pn * BS * 128, &tm_k, pn * 64, row, bar);
                tma_load_2d(dst + C::kPageBytes + pn * BS * 128, &tm_v, pn * 64, row, bar);
            }
        }
    };
    int issued = min(ST, n_my);
    for (int k = 0; k < issued; ++k) issue(k);

    // q parts of a tile's pair 8t + g, k-step kk: elements 16 kk + 2 t4 (+ 8); every load before the first use
    const float *q_row[T];
#pragma unroll
    for (int t = 0; t < T; ++t) q_row[t] = 8 * t + g < npairs ? p.q + w.row_of(p, 8 * t + g) * D + 2 * t4 : nullptr;
    uint4 qhm[kQRegs ? KS : 1];
    uint2 qlo[kQRegs ? KS : 1];
    {
        constexpr int kMine = kQRegs ? KS : (T * KS + NW - 1) / NW;   // (tile, k-step) items of this warp
        const int first = kQRegs ? 0 : warp * kMine;
        float2 x[kMine][2];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int t = (first + i) / KS, kk = (first + i) % KS;
            const float *q = q_row[0];
#pragma unroll
            for (int u = 1; u < T; ++u)
                if (t == u) q = q_row[u];
            x[i][0] = x[i][1] = make_float2(0.f, 0.f);
            if (q != nullptr && first + i < T * KS) {
                x[i][0] = __ldg(reinterpret_cast<const float2 *>(q + kk * 16));
                x[i][1] = __ldg(reinterpret_cast<const float2 *>(q + kk * 16 + 8));
            }
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            uint4 hm;
            uint2 l;
            split3(x[i][0].x, x[i][0].y, hm.x, hm.y, l.x);
            split3(x[i][1].x, x[i][1].y, hm.z, hm.w, l.y);
            if constexpr (kQRegs) {
                qhm[i] = hm;
                qlo[i] = l;
            } else if (first + i < T * KS) {
                s_qhm[(first + i) * 32 + lane] = hm;
                s_qlo[(first + i) * 32 + lane] = l;
            }
        }
        if constexpr (!kQRegs) __syncthreads();
    }

    float2 o[T][NP * 2];   // running outputs of pair 8t + g: columns 8n + 2 t4, + 1
    float m_run[T], l_run[T];
    int lo_r[T], hi_r[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int n = 0; n < NP * 2; ++n) o[t][n] = make_float2(0.f, 0.f);
        m_run[t] = -INFINITY;
        l_run[t] = 0.f;
        const int pos = w.position(p, min(8 * t + g, npairs - 1));
        lo_r[t] = w.lo_of(p, pos);
        hi_r[t] = w.hi_of(pos);
    }

    int k = 0;
    for (; k < n_my; ++k) {
        const int st = warp * ST + k % ST;
        const bool arrived = mbar_wait_bounded(smem_addr(&bars[st]), (k / ST) & 1);
        if (!__all_sync(kFull, arrived)) {
            if (lane == 0) raise_error(p.err, PKV_DEVERR_TIMEOUT);
            break;
        }
        uint8_t *stage = smem + st * C::kStageBytes;
        const int v0 = (pg0 + warp + k * NW) * BS;   // the page's first token
        const bool whole = v0 + BS <= w.all_hi && (v0 >= w.all_lo || v0 + BS <= S);   // every row sees all of it
        if (!whole) {
            for (int i = lane; i < BS * (D / 8); i += 32) {
                const int r = i / (D / 8), c16 = i % (D / 8), v = v0 + r;
                if (v >= w.hi || (v >= S && v < w.lo))
                    *reinterpret_cast<uint4 *>(stage + C::kPageBytes + (c16 >> 3) * BS * 128 + r * 128 + (c16 & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();   // before the stage's next copies
            __syncwarp();
        }
        const uint32_t k_s = smem_addr(stage), v_s = k_s + C::kPageBytes;
        const int mi = lane >> 3, r8 = lane & 7;

        // scores: rows g (first parts) and g + 8 (second) of each tile; third parts of two tiles in another
        // accumulator, of a single one onto its own
        float s[T][NT][4], sl[LT > 0 ? LT : 1][NT][4];
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            uint32_t kb[NT][2];
#pragma unroll
            for (int np = 0; np < NT / 2; ++np)
                ldsm_x4(k_s + swz128(BS, np * 16 + (mi >> 1) * 8 + r8, kk * 16 + (mi & 1) * 8), kb[2 * np][0], kb[2 * np][1],
                        kb[2 * np + 1][0], kb[2 * np + 1][1]);
            uint2 l[T];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                uint4 a;
                if constexpr (kQRegs) {
                    a = qhm[kk];
                    l[t] = qlo[kk];
                } else {
                    a = s_qhm[(t * KS + kk) * 32 + lane];
                    l[t] = s_qlo[(t * KS + kk) * 32 + lane];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (kk == 0) mma_new(s[t][n], a.x, a.y, a.z, a.w, kb[n][0], kb[n][1]);
                    else mma_bf16_16816(s[t][n], a.x, a.y, a.z, a.w, kb[n][0], kb[n][1]);
                }
            }
            if constexpr (T == 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16_16816(s[0][n], l[0].x, 0u, l[0].y, 0u, kb[n][0], kb[n][1]);
            } else {
#pragma unroll
                for (int t = 0; t < LT; ++t)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (kk == 0) mma_new(sl[t][n], l[2 * t].x, l[2 * t + 1].x, l[2 * t].y, l[2 * t + 1].y, kb[n][0], kb[n][1]);
                        else mma_bf16_16816(sl[t][n], l[2 * t].x, l[2 * t + 1].x, l[2 * t].y, l[2 * t + 1].y, kb[n][0], kb[n][1]);
                    }
            }
        }

        // online softmax (base 2) of pair 8t + g; weights in three parts
        uint32_t phm[T][KT][4], plo[T][KT][2];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float sc[NT][2], mx = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = s[t][n][2 + e];
                    if constexpr (T > 1) x += sl[t / 2][n][(t & 1) * 2 + e];
                    sc[n][e] = (s[t][n][e] + x) * p.scale_log2;
                    if (!whole) {
                        const int v = v0 + n * 8 + 2 * t4 + e;
                        if (v >= hi_r[t] || (v >= S && v < lo_r[t])) sc[n][e] = -INFINITY;
                    }
                    mx = fmaxf(mx, sc[n][e]);
                }
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            const float m_new = fmaxf(m_run[t], mx);
            const float m_ref = m_new == -INFINITY ? 0.f : m_new;   // a row that has seen no key yet
            const float alpha = ex2_approx(m_run[t] - m_ref);
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[n][e] = ex2_approx(sc[n][e] - m_ref);
                    sum += sc[n][e];
                }
            l_run[t] = l_run[t] * alpha + sum;
            m_run[t] = m_new;
            if (__any_sync(kFull, alpha != 1.f)) {   // only when a running maximum moved
#pragma unroll
                for (int n = 0; n < NP * 2; ++n) {
                    o[t][n].x *= alpha;
                    o[t][n].y *= alpha;
                }
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                split3(sc[2 * kt][0], sc[2 * kt][1], phm[t][kt][0], phm[t][kt][1], plo[t][kt][0]);
                split3(sc[2 * kt + 1][0], sc[2 * kt + 1][1], phm[t][kt][2], phm[t][kt][3], plo[t][kt][1]);
            }
        }

        // O += P V, the page's part summed apart
#pragma unroll
        for (int np = 0; np < NP; ++np) {
            uint32_t vb[KT][4];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
                ldsm_x4_trans(v_s + swz128(BS, kt * 16 + (mi & 1) * 8 + r8, np * 16 + (mi >> 1) * 8), vb[kt][0], vb[kt][1], vb[kt][2],
                              vb[kt][3]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float c[T][4], cl[LT > 0 ? LT : 1][4];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const uint32_t b0 = vb[kt][2 * h], b1 = vb[kt][2 * h + 1];
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        if (kt == 0) mma_new(c[t], phm[t][kt][0], phm[t][kt][1], phm[t][kt][2], phm[t][kt][3], b0, b1);
                        else mma_bf16_16816(c[t], phm[t][kt][0], phm[t][kt][1], phm[t][kt][2], phm[t][kt][3], b0, b1);
                    }
                    if constexpr (T == 1) {
                        mma_bf16_16816(c[0], plo[0][kt][0], 0u, plo[0][kt][1], 0u, b0, b1);
                    } else {
#pragma unroll
                        for (int t = 0; t < LT; ++t) {
                            if (kt == 0) mma_new(cl[t], plo[2 * t][kt][0], plo[2 * t + 1][kt][0], plo[2 * t][kt][1], plo[2 * t + 1][kt][1], b0, b1);
                            else mma_bf16_16816(cl[t], plo[2 * t][kt][0], plo[2 * t + 1][kt][0], plo[2 * t][kt][1], plo[2 * t + 1][kt][1], b0, b1);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    float2 x = make_float2(c[t][2], c[t][3]);
                    if constexpr (T > 1) x = add2(x, make_float2(cl[t / 2][(t & 1) * 2], cl[t / 2][(t & 1) * 2 + 1]));
                    o[t][2 * np + h] = add2(o[t][2 * np + h], add2(make_float2(c[t][0], c[t][1]), x));
                }
            }
        }
        __syncwarp();
        if (k + ST < n_my) {
            issue(k + ST);
            issued = k + ST + 1;
        }
    }
    if (k < n_my) {
        // a copy did not arrive in time: wait (bounded) for those in flight, so that none lands later
        for (int kk = k; kk < issued; ++kk) mbar_wait_bounded(smem_addr(&bars[warp * ST + kk % ST]), (kk / ST) & 1);
    }

    // ---- the warps' outputs meet in shared memory (the ring is free now), each scaled to the pairs' common maximum
    // and sum, so that they only remain to be added
    __syncthreads();
    float *lse2 = reinterpret_cast<float *>(smem);       // [pairs], as finish_sinks wants it
    float *ow = lse2 + C::kPairs;                        // [NW][pairs][D]
    float *ml = ow + NW * C::kPairs * D;                 // [NW][pairs][2]
#pragma unroll
    for (int t = 0; t < T; ++t) {
        float l = l_run[t];
        l += __shfl_xor_sync(kFull, l, 1);
        l += __shfl_xor_sync(kFull, l, 2);
        if (t4 == 0) *reinterpret_cast<float2 *>(ml + 2 * (warp * C::kPairs + 8 * t + g)) = make_float2(m_run[t], l);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < T; ++t) {
        float2 all[NW];
        float M = -INFINITY;
#pragma unroll
        for (int v = 0; v < NW; ++v) {
            all[v] = *reinterpret_cast<const float2 *>(ml + 2 * (v * C::kPairs + 8 * t + g));
            M = fmaxf(M, all[v].x);
        }
        const float ref = M == -INFINITY ? 0.f : M;
        float l = 0.f;
#pragma unroll
        for (int v = 0; v < NW; ++v) l += all[v].y * ex2_approx(all[v].x - ref);
        if (warp == 0 && t4 == 0) lse2[8 * t + g] = M + log2f(l);
        // no key of this chunk: an empty partial
        const float f = l == 0.f ? 0.f : ex2_approx(m_run[t] - ref) / l;
        float *to = ow + (warp * C::kPairs + 8 * t + g) * D + 2 * t4;
#pragma unroll
        for (int n = 0; n < NP * 2; ++n) *reinterpret_cast<float2 *>(to + n * 8) = make_float2(o[t][n].x * f, o[t][n].y * f);
    }
    __syncthreads();
}

template <int D, int BS, int TILES>
__global__ void __launch_bounds__(SinksCfg<D, BS, TILES>::NW * 32, SinksCfg<D, BS, TILES>::kBlocks)
    decode_sinks_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const DecodeKParams p, const int groups) {
    using C = SinksCfg<D, BS, TILES>;
    constexpr int NW = C::NW, ST = C::ST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);

    pdl_launch_dependents();   // a merge kernel after this one waits for the whole grid
    __shared__ SinksWork s_work;   // what is seldom needed takes no registers
    SinksWork w;
    if (!sinks_work<D, BS, C::kPairs>(p, groups, w)) return;
    if (threadIdx.x == 0) s_work = w;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        for (int s = 0; s < ST; ++s) mbar_init(smem_addr(&bars[warp * ST + s]), 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    __syncwarp();
    // only as many tiles as the CTA has pairs for (rows of a sequence and heads of a KV head differ)
    if (TILES == 1 || w.npairs <= 8) attend_pages<D, BS, TILES, 1>(tm_k, tm_v, p, s_work, smem, bars);
    else attend_pages<D, BS, TILES, TILES>(tm_k, tm_v, p, s_work, smem, bars);
    __shared__ int s_last;
    finish_sinks<D, C::kPairs, NW>(smem, &s_last, p, s_work, groups);
}

template <int D, int BS, int TILES>
cudaError_t launch(const DecodeKParams &kp, const CUtensorMap &tk, const CUtensorMap &tv, int groups, cudaStream_t stream) {
    using C = SinksCfg<D, BS, TILES>;
    static std::atomic<unsigned long long> ready{0};   // one bit a device: shared memory opted in
    auto kernel = decode_sinks_kernel<D, BS, TILES>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit);
    }
    kernel<<<dim3(static_cast<unsigned>(kp.splits) * groups, kp.Hkv, kp.B), C::NW * 32, C::kSmemBytes, stream>>>(tk, tv, kp, groups);
    return cudaGetLastError();
}

template <int D, int BS>
cudaError_t launch_tiles(const DecodeKParams &kp, const CUtensorMap &tk, const CUtensorMap &tv, const SinksPlan &plan,
                         cudaStream_t stream) {
    if constexpr (D == 256) {
        if (plan.tiles == 2) return launch<D, BS, 2>(kp, tk, tv, plan.groups, stream);
    }
    return launch<D, BS, 1>(kp, tk, tv, plan.groups, stream);
}

}  // namespace

SinksPlan plan_sinks(int B, int rows, int max_q, int Hq, int Hkv, int d, int bs, int pages, int NB, pkv_dtype dt, int num_splits,
                     int sm_count, bool aligned) {
    SinksPlan plan{};
    auto finish = [&] {
        plan.workspace_bytes = plan.splits > 1 ? PKV_DECODE_COUNTER_BYTES + static_cast<size_t>(rows) * Hq * plan.splits *
                                                                                (static_cast<size_t>(d) + 1) * sizeof(float)
                                               : 0;
        return plan;
    };
    auto simt = [&] {
        plan = SinksPlan{};
        plan_sinks_simt(plan, rows, Hq, Hkv, d, bs, pages, num_splits, sm_count);
        return finish();
    };
    if (dt != PKV_BF16 || (d != 64 && d != 128 && d != 256) || (bs != 16 && bs != 32) || !aligned ||
        static_cast<long long>(NB + 1) * Hkv * bs >= (1ll << 31))
        return simt();
    const long long pairs = static_cast<long long>(max_q) * (Hq / Hkv), tiles = (pairs + 7) / 8;
    plan.umma = pairs > kSinksMmaPairs && d <= 128;
    // more than eight pairs on tcgen05 (16 heads a KV head 22.7 us against 24.8 on warp MMAs, 1 to 4 rows of 8 104
    // against 155), eight and fewer on warp MMAs (above); d = 256 on these alone, two tiles a block at most
    plan.tiles = plan.umma ? kSinksUmmaPairs / 8 : tiles == 1 ? 1 : 2;
    const long long groups = (tiles + plan.tiles - 1) / plan.tiles;
    const long long units = static_cast<long long>(B) * Hkv * groups;
    if (units < 1) return simt();
    // blocks at a time: two an SM, but where their rings are too large for that
    const int per_sm = d == 256 && bs == 32 ? SinksCfg<256, 32, 2>::kBlocks : 2;
    const long long slots = static_cast<long long>(per_sm) * std::max(sm_count, 1);
    // Chunks of a sequence by a model of the time in tokens: a block costs its tokens and 512 more, a wave of blocks
    // as much as a block, a second wave at least half of one; more chunks than one cost a quarter of a wave where
    // they make several, and more than eight the merge kernel, 256 tokens.  (512 units of 4112 tokens, 1 to 4
    // chunks: 172, 187, 190 and 184 us; 64 units of 2096: 37, 25, 24 and 22 us, five chunks 29; with d = 256, pages of 32
    // and one block an SM 152 units of 2080: 78, 90 and 96, 64 units of 8220: 273, 145 and 192.)  No chunk is longer
    // than 16384 tokens, so that a long sequence among short ones does not end the launch alone.
    int splits = 1;
    if (num_splits > 0) {
        splits = std::min(num_splits, pages);
    } else {
        double best = 0;
        const long long tokens = static_cast<long long>(pages) * bs, least = std::min<long long>((tokens + 16383) / 16384, pages);
        auto consider = [&](long long n) {
            if (n < least || n > pages || n > kDecodeMaxChunks) return;
            double waves = static_cast<double>(units) * n / slots;
            waves = waves <= 1 ? 1 : std::max(waves, 1.5) + (n > 1 ? 0.25 : 0.0);
            const double cost = waves * (512.0 + static_cast<double>((pages + n - 1) / n) * bs) + (n > kSinksFusedChunks ? 256.0 : 0.0);
            if (best == 0 || cost < best) {
                best = cost;
                splits = static_cast<int>(n);
            }
        };
        for (int n = 1; n <= kSinksFusedChunks; ++n) consider(n);
        consider(least);
        if (slots / units > kSinksFusedChunks) consider(slots / units);
    }
    int chunk = (pages + splits - 1) / splits;
    if (plan.umma) chunk = (chunk + kSinksUmmaKeys / bs - 1) / (kSinksUmmaKeys / bs) * (kSinksUmmaKeys / bs);   // whole key tiles
    chunk = std::max(chunk, (pages + kDecodeMaxChunks - 1) / kDecodeMaxChunks);
    splits = (pages + chunk - 1) / chunk;
    // no more blocks than the call's rows can fill: max_q may be any bound (2^31 - 1 for none at all), and a block's first pair,
    // group * pairs of a block, has to stay below 2^31
    const long long launched = std::min(groups, (static_cast<long long>(rows) * (Hq / Hkv) + 8 * plan.tiles - 1) / (8 * plan.tiles));
    if (launched * splits > 0x7fffffffll) return simt();
    plan.mma = true;
    plan.groups = static_cast<int>(launched);
    plan.chunk_pages = chunk;
    plan.splits = splits;
    plan.fused_merge = splits > 1 && splits <= kSinksFusedChunks &&
                       units <= static_cast<long long>(PKV_DECODE_COUNTER_BYTES / sizeof(unsigned));
    return finish();
}

cudaError_t launch_decode_sinks(const DecodeArgs &a, const SinksPlan &plan, pkv_dtype dt, cudaStream_t stream) {
    DecodeKParams kp{};
    kp.out = a.out;
    kp.lse = a.lse;
    kp.q = a.q;
    kp.block_table = a.block_table;
    kp.context_lens = a.context_lens;
    kp.err = a.err;
    kp.B = a.B;
    kp.Hq = a.Hq;
    kp.Hkv = a.Hkv;
    kp.m = a.Hq / a.Hkv;
    kp.MBS = a.MBS;
    kp.NB = a.NB;
    kp.chunk_pages = plan.chunk_pages;
    kp.splits = plan.splits;
    kp.scale_log2 = a.scale * kDecLog2e;
    kp.window = a.window;
    kp.sinks = a.sinks;
    kp.cu_q = a.cu_q;
    kp.rows = a.rows;
    kp.max_q = a.max_q;
    if (plan.splits > 1) {
        uint8_t *ws = static_cast<uint8_t *>(a.workspace);
        kp.counters = plan.fused_merge ? reinterpret_cast<unsigned *>(ws) : nullptr;
        kp.ws_o = reinterpret_cast<float *>(ws + PKV_DECODE_COUNTER_BYTES);
        kp.ws_lse = kp.ws_o + static_cast<size_t>(a.rows) * a.Hq * plan.splits * a.d;
    }
    cudaError_t e;
    if (!plan.mma) {
        e = launch_decode_sinks_simt(kp, a.k_cache, a.v_cache, dt, a.d, a.bs, plan.block_heads, stream);
        if (e != cudaSuccess || plan.splits == 1 || plan.fused_merge) return e;
        return launch_decode_merge(kp, a.d, a.bs, static_cast<unsigned>(a.rows * a.Hq), stream);
    }
    CUtensorMap tk, tv;
    const uint64_t dims[2] = {static_cast<uint64_t>(a.d), static_cast<uint64_t>(a.NB) * a.Hkv * a.bs};
    const uint64_t strides[1] = {static_cast<uint64_t>(a.d) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(a.bs)};
    if (!encode_map_bf16(&tk, a.k_cache, 2, dims, strides, box) || !encode_map_bf16(&tv, a.v_cache, 2, dims, strides, box))
        return cudaErrorInvalidValue;
    if (plan.umma)
        e = launch_decode_sinks_umma(kp, tk, tv, a.d, a.bs, plan.groups, stream);
    else if (a.bs == 16)
        e = a.d == 64    ? launch_tiles<64, 16>(kp, tk, tv, plan, stream)
            : a.d == 128 ? launch_tiles<128, 16>(kp, tk, tv, plan, stream)
                         : launch_tiles<256, 16>(kp, tk, tv, plan, stream);
    else
        e = a.d == 64    ? launch_tiles<64, 32>(kp, tk, tv, plan, stream)
            : a.d == 128 ? launch_tiles<128, 32>(kp, tk, tv, plan, stream)
                         : launch_tiles<256, 32>(kp, tk, tv, plan, stream);
    if (e != cudaSuccess || plan.splits == 1 || plan.fused_merge) return e;
    return launch_decode_merge(kp, a.d, a.bs, static_cast<unsigned>(a.rows * a.Hq), stream);
}

}  // namespace pkv
