// decode_sinks_umma.cu -- paged attention with a window and first tokens that stay visible (sinks) on the
// 5th-generation tensor cores (tcgen05), for more than eight (query row, head) pairs per sequence and KV head:
// verification of drafts, rows of a prompt, many heads a KV head; d in {64, 128}, bs in {16, 32}.
//
// What is computed, which tokens a row sees and how the gap between the sinks and the window is left out stand in
// decode_sinks.cu; so does the precision, fp32's: q and the softmax weights enter as three bf16 parts, and the sums
// inside the tensor core are short (d products of a score, the 64 tokens of a tile of an output), each tile's
// product being added to a running output in fp32 registers.
//
// One block of 8 warps per (sequence, KV head, group of 32 pairs, chunk of pages), two blocks an SM, so that one
// block's start (lengths, table, queries, the first tile: some microseconds) runs beside the other's tiles.
//   Rows.  The 128 rows of the MMAs are 32 pairs times four: pair 8g + i has its first part in row 32g + i, its second in
//     row 32g + 8 + i, its third in row 32g + 16 + i; rows 32g + 24 + i are zero.  The three rows of a pair, added,
//     are the product with the fp32 number; with the 16-lane tensor-memory shapes the thread that owns a pair's
//     keys holds all of them, so nothing is exchanged.
//   Warps 4 and 5 (TMA) bring K and V tiles of 64 tokens into two rings, one {64, bs} box a lane.
//   Warps 6 and 7 (one lane each issues): S_t = Q K_t^T (Q in shared memory) into one of two tensor-memory buffers, and
//     O_t = P_t V_t, P_t written over S_t.
//   Warps 0-3 (softmax): warp g owns pairs 8g .. 8g + 7, four threads a pair; thread t holds keys 8k + 2 (t % 4), + 1 of
//     each tile.  It reads S_t, masks, takes the running maximum, writes the weights' parts, then adds O_{t-1} to
//     its output -- while the tensor core computes S_{t+1}.
// Every wait is bounded and shares an abort flag, as in decode_umma.cu.
//
// 64 sequences of 512 to 8192 tokens, 1 to 4 rows of 64 heads on 8 of 128, window 2048 + 16: 104 us, 5.3 TB/s of what the
// rows see (the warp-MMA kernel: 155).  What bounds it: one full wave of 304 long blocks runs at 6.45 TB/s, 95% of the
// measured copy rate (198 us; 148 with the pages in L2), but 512 blocks of 33 tiles are one and two thirds, each with its
// start and end; a block alone on its SM takes 0.9 us a tile with its pages in L2 and 1.1 from HBM.  Measured without
// gain: four more warps for the outputs (104 us), two groups of softmax warps with tiles in turn (103; 16 heads a KV head
// 24 for 23), queries in tensor memory, seven slots and O by 64 columns (114), two chunks a sequence (116), four slots
// instead of five (106).
#include <atomic>
#include <math.h>

#include "common.cuh"
#include "decode_kparams.cuh"
#include "decode_sinks.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

template <int D, int BS>
struct SinksUmmaCfg {
    static constexpr int kBM = 128, kTK = kSinksUmmaKeys, kPPT = kTK / BS, PANELS = D / 64, kPairs = kSinksUmmaPairs;
    static constexpr int kSlotBytes = kTK * D * 2;                    // one K or V tile: panels of [64][128 B]
    static constexpr int NK = D == 128 ? 2 : 6, NV = D == 128 ? 3 : 6;   // slots of the rings; a V tile waits for its weights
    static constexpr int kQBytes = kBM * D * 2;                       // panels of [128][128 B]
    static constexpr int kOffQ = 0, kOffK = kQBytes, kOffV = kOffK + NK * kSlotBytes, kOffBar = kOffV + NV * kSlotBytes;
    // barriers: Q built; K full / free per slot; V full / free per slot; S full x2; O full x2; P full; drain x2
    static constexpr int kQ = 0, kKFull = 1, kKFree = kKFull + NK, kVFull = kKFree + NK, kVFree = kVFull + NV,
                         kSFull = kVFree + NV, kOFull = kSFull + 2, kPFull = kOFull + 2, kDrain = kPFull + 1, kNumBars = kDrain + 2;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;           // TMEM slot, abort flag, and the end's flag
    static constexpr int kOffWork = (kOffMisc + 16 + 15) / 16 * 16;   // the block's SinksWork
    // all shared memory is dynamic and starts on the swizzle's 1024 bytes (checked), none of it spent on aligning
    static constexpr int kSmemBytes = kOffWork + static_cast<int>(sizeof(SinksWork));
    static constexpr int kTmemCols = 256;                             // two S buffers (P over them), O
    static constexpr int kSCol = 0, kOCol = 2 * kTK;
    static constexpr int kThreads = 256;
    // the end of a block: log-sum-exps and outputs, over the rings
    static constexpr int kFinishBytes = (kPairs + kPairs * D) * 4;
    static_assert(kFinishBytes <= kOffBar, "the end of a block fits the rings");
    static_assert(kOCol + D <= kTmemCols && 2 * (kSmemBytes + 1024) <= 233472, "two blocks an SM");
    static_assert(kPPT * PANELS <= 32 && 32 % kPPT == 0, "one box per loader lane; tiles within 32 pages");
};

template <int D, int BS>
__global__ void __launch_bounds__(256, 2)
    decode_sinks_umma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DecodeKParams p,
                             const int groups) {
    using C = SinksUmmaCfg<D, BS>;
    constexpr int BM = C::kBM, TK = C::kTK, PPT = C::kPPT, PANELS = C::PANELS, NK = C::NK, NV = C::NV;

    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    auto bar = [&](int k) { return smem_addr(&bars[k]); };

    pdl_launch_dependents();   // a merge kernel after this one waits for the whole grid
    if (smem_addr(smem) % 1024 != 0) {
        if (threadIdx.x == 0) raise_error(p.err, PKV_DEVERR_LAYOUT);
        return;
    }
    SinksWork &s_work = *reinterpret_cast<SinksWork *>(smem + C::kOffWork);   // for the block's end: no registers meanwhile
    SinksWork w;
    if (!sinks_work<D, BS, C::kPairs>(p, groups, w)) return;
    if (threadIdx.x == 0) s_work = w;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pages = max(0, w.pg1 - w.pg0), ntiles = (pages + PPT - 1) / PPT;
    const int v_first = w.pg0 * BS, v_end = w.pg1 * BS, S = p.sinks;   // tokens of the pages read

    if (threadIdx.x == 0) {
        mbar_init(bar(C::kQ), 4);
        for (int s = 0; s < NK; ++s) {
            mbar_init(bar(C::kKFull + s), 1);
            mbar_init(bar(C::kKFree + s), 1);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(bar(C::kVFull + s), 1);
            mbar_init(bar(C::kVFree + s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(bar(C::kSFull + x), 1);
            mbar_init(bar(C::kOFull + x), 1);
            mbar_init(bar(C::kDrain + x), 1);
        }
        mbar_init(bar(C::kPFull), 4);
        *abort = 0;
        fence_barrier_init();
        tma_prefetch_map(&tm_k);
        tma_prefetch_map(&tm_v);
    }
    if (warp == 0) tmem_alloc(smem_addr(tslot), C::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tslot;
    const uint32_t sQ = smem_addr(smem + C::kOffQ);
    auto sK = [&](int s) { return smem_addr(smem + C::kOffK + s * C::kSlotBytes); };
    auto sV = [&](int s) { return smem_addr(smem + C::kOffV + s * C::kSlotBytes); };

    // what the softmax warps keep to the end
    float m_run = -INFINITY, l_run = 0.f;
    float2 o[D / 8];   // columns 64 cc + 8k + 2 c4, + 1 in o[8 cc + k]
    bool ok = true;

    if (warp == 4 || warp == 5) {
        // ---- TMA: tile t into slot t % N of its ring once the slot's last tile is used.  Lane i < PPT * PANELS copies panel
        // i % PANELS of page i / PANELS; a page past the chunk is placed outside the cache (zeros)
        const bool is_k = warp == 4;
        const int N = is_k ? NK : NV;
        const int full0 = is_k ? C::kKFull : C::kVFull, free0 = is_k ? C::kKFree : C::kVFree;
        const CUtensorMap *map = is_k ? &tm_k : &tm_v;
        const int32_t *tbl = p.block_table + static_cast<size_t>(w.b) * p.MBS;
        auto entry = [&](int k) { return k < pages ? __ldg(tbl + page_entry(w.sp, w.pg0 + k)) : -1; };
        int tcur = entry(lane), tnext = entry(32 + lane), tbase = 0;
        const int oob_row = p.NB * p.Hkv * BS;
        const int pg = lane / PANELS, pn = lane % PANELS;
        int t = 0;
        for (; t < ntiles; ++t) {
            bool fr = true;
            if (lane == 0 && t >= N) fr = wait_or_abort(bar(free0 + t % N), ((t - N) / N) & 1, abort, p.err);
            if (!__shfl_sync(kFull, fr ? 1 : 0, 0)) break;
            const int s = t % N;
            if (t * PPT >= tbase + 32) {   // a tile never straddles 32 pages
                tbase += 32;
                tcur = tnext;
                tnext = entry(tbase + 32 + lane);
            }
            const int k = t * PPT + pg;
            const int phys = __shfl_sync(kFull, tcur, k & 31);
            if (lane == 0) mbar_arrive_expect_tx(bar(full0 + s), C::kSlotBytes);
            __syncwarp();
            if (lane < PPT * PANELS) {
                int row = oob_row;
                if (k < pages) {
                    if (phys < 0 || phys >= p.NB) {
                        if (is_k && pn == 0) raise_error(p.err, PKV_DEVERR_BLOCK);
                    } else {
                        row = (phys * p.Hkv + w.kvh) * BS;
                    }
                }
                tma_load_2d((is_k ? sK(s) : sV(s)) + pn * TK * 128 + pg * BS * 128, map, pn * 64, row, bar(full0 + s));
            }
        }
        // before teardown every copy issued must have landed (bounded)
        if (lane == 0)
            for (int u = max(0, t - N); u < t; ++u)
                if (!mbar_wait_bounded(bar(full0 + u % N), (u / N) & 1)) raise_error(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 6 || warp == 7) {
        // ---- MMA issue.  Warp 6: S_t into buffer t & 1 once K_t has landed and O_{t-2} is done (P_{t-2}, in that
        // buffer, has been read).  Warp 7: O_t once P_t is written (O_{t-1} has then been read) and V_t has landed.
        if (lane == 0) {
            const bool is_s = warp == 6;
            bool issued = false, alive = true;
            if (is_s) {
                const uint32_t idesc = umma_idesc_bf16(BM, TK, 0);
                alive = wait_or_abort(bar(C::kQ), 0, abort, p.err);
                for (int t = 0; t < ntiles && alive; ++t) {
                    const int s = t % NK, x = t & 1;
                    alive = wait_or_abort(bar(C::kKFull + s), (t / NK) & 1, abort, p.err);
                    if (alive && t >= 2) alive = wait_or_abort(bar(C::kOFull + x), ((t - 2) >> 1) & 1, abort, p.err);
                    if (!alive) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t ad = umma_desc_sw128(sQ + (kk / 4) * BM * 128 + (kk % 4) * 32, 16, 1024);
                        const uint64_t bd = umma_desc_sw128(sK(s) + (kk / 4) * TK * 128 + (kk % 4) * 32, 16, 1024);
                        umma_bf16(tmem + C::kSCol + x * TK, ad, bd, idesc, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(bar(C::kSFull + x));
                    umma_commit(bar(C::kKFree + s));
                    issued = true;
                }
            } else {
                const uint32_t idesc = umma_idesc_bf16(BM, D, 1);
                for (int t = 0; t < ntiles && alive; ++t) {
                    const int s = t % NV, x = t & 1;
                    alive = wait_or_abort(bar(C::kPFull), t & 1, abort, p.err) &&
                            wait_or_abort(bar(C::kVFull + s), (t / NV) & 1, abort, p.err);
                    if (!alive) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < TK / 16; ++kk) {
                        const uint64_t bd = umma_desc_sw128(sV(s) + kk * 16 * 128, TK * 128, 1024);
                        umma_bf16_ts(tmem + C::kOCol, tmem + C::kSCol + x * TK + kk * 8, bd, idesc, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(bar(C::kOFull + x));
                    umma_commit(bar(C::kVFree + s));
                    issued = true;
                }
            }
            if (*abort && issued) {   // let this thread's MMAs finish (bounded) before teardown
                const int drain = C::kDrain + (is_s ? 1 : 0);
                umma_commit(bar(drain));
                if (!mbar_wait_bounded(bar(drain), 0)) raise_error(p.err, PKV_DEVERR_TIMEOUT);
            }
        }
    } else {
        // ---- softmax.  First the queries' parts into shared memory, 8 elements of a pair at a time
        for (int i = threadIdx.x; i < C::kPairs * (D / 8); i += 128) {
            const int pair = i / (D / 8), c = i % (D / 8);   // 16-byte chunk of the row
            float2 x[4] = {};
            if (pair < w.npairs) {
                const float *q = p.q + w.row_of(p, pair) * D + c * 8;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = __ldg(reinterpret_cast<const float2 *>(q + 2 * e));
            }
            uint32_t part[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split3(x[e].x, x[e].y, part[0][e], part[1][e], part[2][e]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = 32 * (pair >> 3) + 8 * u + (pair & 7);
                *reinterpret_cast<uint4 *>(smem + C::kOffQ + (c >> 3) * BM * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                    u < 3 ? make_uint4(part[u < 3 ? u : 0][0], part[u < 3 ? u : 0][1], part[u < 3 ? u : 0][2], part[u < 3 ? u : 0][3])
                          : make_uint4(0, 0, 0, 0);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kQ));

        const int c4 = lane & 3, pair = 8 * warp + (lane >> 2);
        const int pos = w.position(p, min(pair, w.npairs - 1));
        const int lo_r = w.lo_of(p, pos), hi_r = min(w.hi_of(pos), v_end);
        // lanes of the pairs' first and second parts, and of the third ones
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * warp) << 16), lanes3 = tmem + (static_cast<uint32_t>(32 * warp + 16) << 16);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n] = make_float2(0.f, 0.f);
        // O_t of a tile, its three rows added, onto the running output
        auto fold = [&](int t) {
            if (ok) ok = __all_sync(kFull, wait_or_abort(bar(C::kOFull + (t & 1)), (t >> 1) & 1, abort, p.err));
            if (!ok) return;
            tc_fence_after_sync();
#pragma unroll
            for (int cc = 0; cc < D / 64; ++cc) {
                uint32_t a[32], b[32];
                tmem_ld_16x256b_x8(lanes + C::kOCol + cc * 64, a);
                tmem_ld_16x256b_x8(lanes3 + C::kOCol + cc * 64, b);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 lower = add2(make_float2(__uint_as_float(a[4 * k + 2]), __uint_as_float(a[4 * k + 3])),
                                              make_float2(__uint_as_float(b[4 * k]), __uint_as_float(b[4 * k + 1])));
                    o[8 * cc + k] = add2(o[8 * cc + k],
                                         add2(make_float2(__uint_as_float(a[4 * k]), __uint_as_float(a[4 * k + 1])), lower));
                }
            }
        };
        for (int t = 0; t < ntiles; ++t) {
            const int x = t & 1, v0 = v_first + t * TK;
            if (ok) ok = __all_sync(kFull, wait_or_abort(bar(C::kSFull + x), (t >> 1) & 1, abort, p.err));
            // every row sees all of the tile?
            const bool whole = v0 + TK <= min(w.all_hi, v_end) && (v0 >= w.all_lo || v0 + TK <= S);
            if (ok && !whole) {
                // V rows that no pair sees hold whatever the slots hold (NaN, Inf): cleared once they have landed
                ok = __all_sync(kFull, wait_or_abort(bar(C::kVFull + t % NV), (t / NV) & 1, abort, p.err));
                if (ok) {
                    uint8_t *vt = smem + C::kOffV + (t % NV) * C::kSlotBytes;
                    for (int i = threadIdx.x; i < TK * PANELS * 8; i += 128) {
                        const int r = i / (PANELS * 8), c = i % (PANELS * 8), v = v0 + r;
                        if (v >= w.hi || (v >= S && v < w.lo))
                            *reinterpret_cast<uint4 *>(vt + (c >> 3) * TK * 128 + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
            }
            if (!ok) continue;   // (uniform in the warp) what remains of its work is skipped
            tc_fence_after_sync();
            float2 sc[8];   // keys v0 + 8k + 2 c4, + 1
            {
                uint32_t a[32], b[32];
                tmem_ld_16x256b_x8(lanes + C::kSCol + x * TK, a);
                tmem_ld_16x256b_x8(lanes3 + C::kSCol + x * TK, b);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 lower = add2(make_float2(__uint_as_float(a[4 * k + 2]), __uint_as_float(a[4 * k + 3])),
                                              make_float2(__uint_as_float(b[4 * k]), __uint_as_float(b[4 * k + 1])));
                    sc[k] = add2(make_float2(__uint_as_float(a[4 * k]), __uint_as_float(a[4 * k + 1])), lower);
                    sc[k].x *= p.scale_log2;
                    sc[k].y *= p.scale_log2;
                }
            }
            if (!whole) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int v = v0 + 8 * k + 2 * c4;
                    if (v >= hi_r || (v >= S && v < lo_r)) sc[k].x = -INFINITY;
                    if (v + 1 >= hi_r || (v + 1 >= S && v + 1 < lo_r)) sc[k].y = -INFINITY;
                }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fmaxf(sc[k].x, sc[k].y));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            const float m_new = fmaxf(m_run, mx), m_ref = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = ex2_approx(m_run - m_ref);
            float sum = 0.f;
            uint32_t p12[16], p3[16];   // first and second parts; third parts and zeros
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float e0 = ex2_approx(sc[k].x - m_ref), e1 = ex2_approx(sc[k].y - m_ref);
                sum += e0 + e1;
                split3(e0, e1, p12[2 * k], p12[2 * k + 1], p3[2 * k]);
                p3[2 * k + 1] = 0u;
            }
            l_run = l_run * alpha + sum;
            m_run = m_new;
            tmem_st_16x128b_x8(lanes + C::kSCol + x * TK, p12);
            tmem_st_16x128b_x8(lanes3 + C::kSCol + x * TK, p3);
            if (t > 0) fold(t - 1);   // before P_t is announced: O_t replaces O_{t-1}
            if (!ok) continue;
            if (__any_sync(kFull, alpha != 1.f)) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n].x *= alpha;
                    o[n].y *= alpha;
                }
            }
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kPFull));
        }
        if (ntiles > 0) fold(ntiles - 1);
    }
    tc_fence_before_sync();
    const bool failed = __syncthreads_or(!ok || *abort) != 0;   // every MMA and copy is done
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, C::kTmemCols);
    if (failed) return;
    float *lse2 = reinterpret_cast<float *>(smem), *ow = lse2 + C::kPairs;   // as finish_sinks wants them
    if (warp < 4) {
        const int c4 = lane & 3, pair = 8 * warp + (lane >> 2);
        float l = l_run;
        l += __shfl_xor_sync(kFull, l, 1);
        l += __shfl_xor_sync(kFull, l, 2);
        const float f = l == 0.f ? 0.f : 1.f / l;   // no key of this chunk: an empty partial
        if (c4 == 0) lse2[pair] = m_run + log2f(l);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2 *>(ow + pair * D + (n >> 3) * 64 + (n & 7) * 8 + 2 * c4) = make_float2(o[n].x * f, o[n].y * f);
    }
    __syncthreads();
    finish_sinks<D, C::kPairs, 1>(smem, reinterpret_cast<int *>(smem + C::kOffMisc + 8), p, s_work, groups);
}

template <int D, int BS>
cudaError_t launch(const DecodeKParams &kp, const CUtensorMap &tk, const CUtensorMap &tv, int groups, cudaStream_t stream) {
    using C = SinksUmmaCfg<D, BS>;
    static std::atomic<unsigned long long> ready{0};   // one bit a device: shared memory opted in
    auto kernel = decode_sinks_umma_kernel<D, BS>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit);
    }
    kernel<<<dim3(static_cast<unsigned>(kp.splits) * groups, kp.Hkv, kp.B), C::kThreads, C::kSmemBytes, stream>>>(tk, tv, kp, groups);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_sinks_umma(const DecodeKParams &kp, const CUtensorMap &tk, const CUtensorMap &tv, int d, int bs, int groups,
                                     cudaStream_t stream) {
    if (d == 128) return bs == 16 ? launch<128, 16>(kp, tk, tv, groups, stream) : launch<128, 32>(kp, tk, tv, groups, stream);
    if (d == 64) return bs == 16 ? launch<64, 16>(kp, tk, tv, groups, stream) : launch<64, 32>(kp, tk, tv, groups, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pkv
