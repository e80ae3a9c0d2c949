// decode_q4_mma.cuh -- the warp-MMA kernel over a 4-bit cache (decode_q4.cu says what is computed).
#pragma once

#include <algorithm>

#include "decode_q4.cuh"
#include "decode_q4_rows.cuh"

namespace pkv {
namespace {

constexpr int kLeastSteps = 4;       // 32-key steps that a warp of one takes at least (128 keys)
// ============================================================== warp-MMA path
//
// attend_q4_mma_kernel (d a multiple of 32, bs 8, 16 or 32).  A unit is a tile of eight, or up to four, (query row,
// head) pairs of one sequence and KV head with the keys they see; a warp takes 32 keys at a time from a
// private ring of bulk copies (a page is one contiguous run).  Per 32 keys and warp, with m16n8k16
// f16 MMAs and fp32 accumulators:
//   scores S (rows: 8 query rows hi, 8 lo; 8 keys per tile): a code c in the low bits of an f16 is the
//     subnormal c * 2^-24, four bits further up c * 2^-20, exactly: four masks and a shift turn a word
//     of eight codes into MMA operands, no conversion.  q is scaled by a power of two per row (odd
//     elements by another 1/16) and enters as f16 hi + lo (2^-23 relative); the head dimension is taken
//     in the order in which the masks deliver the codes, each group in MMA steps of its own so that its
//     scale multiplies the sum; zero * sum(q in group) is added in fp32.
//   output O^T = V^T P^T: V^T is the A operand (16 dimensions x 16 keys), pairs of keys from a
//     transposing ldmatrix over 16-bit units; P^T is what the lane already holds for its row, times
//     the group's scale, as f16 hi + lo.  The tensor core cuts its sums off instead of rounding them,
//     relative to its operands' exponents.  Over many keys that adds up, and the zeros' term cancels
//     most of a sum of non-negative codes (subnormal codes summed over a warp's range, 4 x 131072
//     tokens: 1.1e-3 of the result).  So V's codes are centred and brought into the normal range by
//     one multiply-add, and a stage's 32 keys are summed and added to O in fp32, together with the
//     rescaling: 1e-7 of the result, for 10% of the time.  The zeros' term is summed in fp32.
//   Scales and zeros are widened to fp32 once per key by the lane of that number and read back
//   from shared memory.
//   Up to four rows (decode_q4_rows.cuh) change the places of K and q, S^T = K Q^T, and need half the
//   MMAs and exponentials: 4 x 65536 tokens of four KV heads 39.1 us for four rows, 49.9 for five;
//   MHA step 82.5 -> 68.3 us (4.2 TB/s), windows of 4096 tokens, four heads per KV head, 100.5 -> 78.9
//   (4.3 TB/s).  Eight rows: four sequences of 131072 tokens 162 us (3.7 TB/s), 70B-shaped step 99 us.
//   About 750 instructions a stage and warp, 224 of them to take the codes out of their words; half of
//   the issue slots used, the rest are the latencies of a stage's chain at three warps per scheduler.
// The f16 range of the weights: p * scale is kept below 2^14 by shifting the softmax reference by
// the largest scale seen so far, E = ceil(log2 max scale): w = 2^(s - m - E + 14); l, O and the
// zeros' term carry the same factor, which cancels, and a growing E rescales like a growing max.
//
// Two ways to share the work:
//   balanced: the 32-key steps of all units in a row (sequence, tile, KV head), an equal range for
//     every warp that the device holds at once; a range may end one unit and begin the next.  A
//     unit's parts meet in the workspace and the last to arrive merges them.  Nothing in a block
//     waits for another warp, so the start of a warp's next unit hides behind its neighbours.
//   chunks: one block for each unit and chunk, its four warps taking the steps in turn and merging
//     in shared memory; a few chunks merge in place, many in decode_merge_kernel.

constexpr int kMmaWarps = 4, kStages = 2;
constexpr int kUnitCost = 3;   // a unit's start (queries, first copies, its part written) in 32-key steps

template <int D, int BS, int G, typename Rows>
struct MmaCfg {
    static constexpr int PPS = kStageKeys / BS;      // pages per stage
    static constexpr int kPageBytes = BS * (D / 2 + 4 * G);
    static constexpr int kStageBytes = 2 * PPS * kPageBytes;   // K pages, then V pages
    static constexpr int kRingBytes = kMmaWarps * kStages * kStageBytes;
    static constexpr int kMergeBytes = kMmaWarps * Rows::ROWS * (2 + D) * 4;
    static constexpr int kScanBytes = (kMaxBalanced + 1) * 4;
    static constexpr int kUsed = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kDataBytes = (kUsed > kScanBytes ? kUsed : kScanBytes) + 15 & ~15;
    static constexpr int kQOff = kDataBytes;                            // query fragments [warp][step][lane]
    static constexpr int kParOff = kQOff + kMmaWarps * Rows::kQBytes;         // [warp][group][scale, zero][key]
    static constexpr int kParBytes = G * 2 * kStageKeys * 4;
    static constexpr int kBarOff = kParOff + kMmaWarps * kParBytes;
    static constexpr int kSmemBytes = kBarOff + kMmaWarps * kStages * 8;
    static constexpr int kBlocksPerSm = Rows::kBlocksPerSm;
    static_assert(kBlocksPerSm * (kSmemBytes + 2048) <= 228 * 1024, "the blocks fit an SM");
    static_assert(kPageBytes % 16 == 0, "bulk copies");
};

// The warps' states of a tile's R rows, in shared memory ([NW][R] references and sums, then
// [NW][R][D] outputs), merged and written: the result where the unit has one part, else this
// normalised part; with arrival counters the unit's last part merges them all.
template <int D, int NW, int R>
__device__ __forceinline__ void finish_rows(uint8_t *smem, const AttendQ4Params &P, const RowSpan *rows, const Parts &u) {
    const DecodeKParams &p = P.k;
    float *mw = reinterpret_cast<float *>(smem);
    float *lw = mw + NW * R;
    float *ow = lw + NW * R;
    for (int idx = threadIdx.x; idx < R * (D / 4); idx += NW * 32) {
        const int h = idx / (D / 4), c = idx % (D / 4) * 4;
        if (rows[h].bi < 0) continue;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, mw[w * R + h]);
        const float base = M == -INFINITY ? 0.f : M;   // the row sees none of this part's keys
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2f(mw[w * R + h] - base);
            const float4 o = *reinterpret_cast<const float4 *>(ow + (w * R + h) * D + c);
            L += lw[w * R + h] * f;
            acc.x += o.x * f;
            acc.y += o.y * f;
            acc.z += o.z * f;
            acc.w += o.w * f;
        }
        const bool empty = M == -INFINITY && L == 0.f;   // else scores of NaN, which the maximum ignores: lse NaN
        const float inv = empty ? 0.f : 1.f / L;
        const float4 r = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const float lse2 = empty ? -INFINITY : M + log2f(L);
        if (u.n == 1) {
            *reinterpret_cast<float4 *>(p.out + static_cast<size_t>(rows[h].bi) * D + c) = r;
            if (c == 0 && p.lse != nullptr) p.lse[rows[h].bi] = lse2 * kDecLn2;
        } else {
            const size_t at = static_cast<size_t>(rows[h].bi) * p.splits + u.own;
            *reinterpret_cast<float4 *>(p.ws_o + at * D + c) = r;
            if (c == 0) p.ws_lse[at] = lse2;
        }
    }
    if (u.n == 1 || u.counter == nullptr) return;
    __shared__ int s_last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned prev = atomicAdd(u.counter, 1u);
        s_last = prev + 1 == static_cast<unsigned>(u.n);
        if (s_last) *u.counter = 0u;   // every part of this call has arrived
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int idx = threadIdx.x; idx < R * (D / 4); idx += NW * 32) {
        const int h = idx / (D / 4), c = idx % (D / 4) * 4;
        if (rows[h].bi < 0) continue;
        const size_t at = static_cast<size_t>(rows[h].bi) * p.splits;
        float M = -INFINITY;
        for (int i = 0; i < u.n; ++i) M = fmaxf(M, __ldcg(p.ws_lse + at + i));
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < u.n; ++i) {
            const float w = exp2f(__ldcg(p.ws_lse + at + i) - M);
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + (at + i) * D + c));
            L += w;
            acc.x += w * o.x;
            acc.y += w * o.y;
            acc.z += w * o.z;
            acc.w += w * o.w;
        }
        const float inv = 1.f / L;
        *reinterpret_cast<float4 *>(p.out + static_cast<size_t>(rows[h].bi) * D + c) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (c == 0 && p.lse != nullptr) p.lse[rows[h].bi] = (M + log2f(L)) * kDecLn2;
    }
}

// Row h of a balanced part, in units of D floats of ws_o and of one float of ws_lse: a warp's first
// unit may have begun in the warp before (slot 0), its last may go on (slot 1).
template <int R>
__device__ __forceinline__ size_t part_at(const Parts &u, int h, int i) {
    return (static_cast<size_t>(u.first + i) * 2 + (i == 0)) * R + h;
}

// The last warp to arrive merges a balanced unit's parts: lane l holds row l % R of every SUB-th part's
// weight (and bi, that row's place), and every lane four columns of all rows.
template <int D, int R>
__device__ __forceinline__ void merge_unit(const AttendQ4Params &P, int bi, const Parts &u, int lane) {
    constexpr int SUB = 32 / R;
    const DecodeKParams &p = P.k;
    const int row = lane % R, sub = lane / R;
    float M = -INFINITY, L = 0.f;
    for (int i = sub; i < u.n; i += SUB) M = fmaxf(M, __ldcg(p.ws_lse + part_at<R>(u, row, i)));
#pragma unroll
    for (int sh = R; sh < 32; sh *= 2) M = fmaxf(M, __shfl_xor_sync(kFull, M, sh));
    const float base = M == -INFINITY ? 0.f : M;   // a row past the sequence's last
    for (int i = sub; i < u.n; i += SUB) L += exp2f(__ldcg(p.ws_lse + part_at<R>(u, row, i)) - base);
#pragma unroll
    for (int sh = R; sh < 32; sh *= 2) L += __shfl_xor_sync(kFull, L, sh);
    if (lane < R && bi >= 0 && p.lse != nullptr) p.lse[bi] = (M + log2f(L)) * kDecLn2;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 128) {   // 128 columns at a time
        const int col = c0 + lane * 4;
        float4 acc[R];
#pragma unroll
        for (int h = 0; h < R; ++h) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < u.n; i0 += SUB) {
            const float w = i0 + sub < u.n ? exp2f(__ldcg(p.ws_lse + part_at<R>(u, row, i0 + sub)) - base) : 0.f;
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                if (i0 + j >= u.n) break;
                const float *src = p.ws_o + part_at<R>(u, 0, i0 + j) * D + col;
#pragma unroll
                for (int h = 0; h < R; ++h) {
                    const float f = __shfl_sync(kFull, w, j * R + h);
                    const float4 o = col < D ? __ldcg(reinterpret_cast<const float4 *>(src + h * D)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    acc[h].x = fmaf(f, o.x, acc[h].x);
                    acc[h].y = fmaf(f, o.y, acc[h].y);
                    acc[h].z = fmaf(f, o.z, acc[h].z);
                    acc[h].w = fmaf(f, o.w, acc[h].w);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < R; ++h) {
            const float inv = 1.f / __shfl_sync(kFull, L, h);
            const int at = __shfl_sync(kFull, bi, h);
            if (at >= 0 && col < D)
                *reinterpret_cast<float4 *>(p.out + static_cast<size_t>(at) * D + col) =
                    make_float4(acc[h].x * inv, acc[h].y * inv, acc[h].z * inv, acc[h].w * inv);
        }
    }
}

// A step's new token (K: side 0, V: side 1) quantised into its row by one warp.
template <int D, int G>
__device__ __forceinline__ void write_new_row(const AttendQ4Params &p, int b, int kvh, long long row_page, int off, int bs,
                                              int side, int lane) {
    constexpr int WORDS = D / 8, LANES = WORDS / G;
    const size_t src = (static_cast<size_t>(b) * p.k.Hkv + kvh) * D + lane * 8;
    const void *rows = side ? p.k.v_new : p.k.k_new;
    __half2 par;
    uint32_t code[1];
    if (p.new_bf16) {
        Q4Loaded<__nv_bfloat16, 1> x;
        q4_load<false, 1>(lane < WORDS ? static_cast<const __nv_bfloat16 *>(rows) + src : nullptr, x.v);
        q4_quantise_loaded<LANES, 1>(x.v, par, code);
    } else {
        Q4Loaded<float, 1> x;
        q4_load<false, 1>(lane < WORDS ? static_cast<const float *>(rows) + src : nullptr, x.v);
        q4_quantise_loaded<LANES, 1>(x.v, par, code);
    }
    if (lane >= WORDS) return;
    uint8_t *page = (side ? p.vc : p.kc) + row_page;
    reinterpret_cast<uint32_t *>(page)[off * WORDS + lane] = code[0];
    if (lane % LANES == 0) reinterpret_cast<__half2 *>(page + bs * WORDS * 4)[off * G + lane / LANES] = par;
}

template <int D, int BS, int G, typename Rows>
__global__ void __launch_bounds__(kMmaWarps * 32, Rows::kBlocksPerSm)
    attend_q4_mma_kernel(const __grid_constant__ AttendQ4Params P) {
    using Cfg = MmaCfg<D, BS, G, Rows>;
    constexpr int R = Rows::ROWS, NW = kMmaWarps, PPS = Cfg::PPS;
    const DecodeKParams &p = P.k;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RowSpan s_rows[R];   // chunks: the tile's rows

    pdl_launch_dependents();   // a merge kernel after this one waits for the whole grid
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kBarOff) + warp * kStages;
    uint8_t *ring = smem + warp * kStages * Cfg::kStageBytes;
    Rows rows;
    if constexpr (Rows::kQBytes > 0)
        rows.qfrag = reinterpret_cast<uint4 *>(smem + Cfg::kQOff + warp * Rows::kQBytes) + lane;   // [step][lane]
    float *par = reinterpret_cast<float *>(smem + Cfg::kParOff + warp * Cfg::kParBytes);
    if (lane == 0) {
        for (int st = 0; st < kStages; ++st) mbar_init(smem_addr(&bars[st]), 1);
        fence_barrier_init();
    }
    int cnt = 0;        // stages this warp has consumed
    unsigned bad = 0;   // bit (stage * PPS + page): a page to be read as zeros

    // ---- balanced: this warp's share [x, x1) of the steps of all units, each unit kUnitCost steps
    // longer than its keys for its start.  Warps are as many as fit the device at once; fewer when
    // that would leave them less than kLeastSteps each, but one for every unit.  They are numbered so
    // that neighbours lie in different blocks.
    const int wid = warp * gridDim.x + blockIdx.x;
    int x = 0, x1 = 1, Q = 1, warps = 1, b = 0, unit = 0, step = 0;
    if (P.balanced) {
        int *pre = reinterpret_cast<int *>(smem);   // steps before each sequence
        __shared__ int s_sum[2][NW];
        const int per = (p.B + NW * 32 - 1) / (NW * 32), first = threadIdx.x * per;
        int steps = 0, units = 0;
        for (int i = first; i < min(p.B, first + per); ++i) {
            const SeqRows sq = seq_rows(P, i, BS, false);
            const int n = sq.pages > 0 ? p.Hkv * ((sq.nq * p.m + R - 1) / R) : 0;
            pre[i + 1] = n * ((sq.pages + PPS - 1) / PPS + kUnitCost);
            steps += pre[i + 1];
            units += n;
        }
        int before = steps;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int y = __shfl_up_sync(kFull, before, sh);
            if (lane >= sh) before += y;
            units += __shfl_xor_sync(kFull, units, sh);
        }
        if (lane == 31) s_sum[0][warp] = before, s_sum[1][warp] = units;
        __syncthreads();
        Q = units = 0;
        before -= steps;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += s_sum[0][w];
            Q += s_sum[0][w];
            units += s_sum[1][w];
        }
        if (threadIdx.x == 0) pre[0] = 0;
        for (int i = first; i < min(p.B, first + per); ++i) pre[i + 1] = before += pre[i + 1];
        warps = min(static_cast<int>(gridDim.x) * NW, max(units, Q / kLeastSteps));
        x = static_cast<int>(min(static_cast<long long>(Q), static_cast<long long>(wid) * Q / max(warps, 1)));
        x1 = static_cast<int>(min(static_cast<long long>(Q), (wid + 1ll) * Q / max(warps, 1)));
        __syncthreads();
        for (int st = kMaxBalanced / 2; st > 0; st >>= 1)
            if (b + st < p.B && pre[b + st] <= x) b += st;
        if (x < x1) {
            const SeqRows sq = seq_rows(P, b, BS, false);
            const int span = (sq.pages + PPS - 1) / PPS + kUnitCost;
            unit = (x - pre[b]) / span;
            step = (x - pre[b]) - unit * span;
        }
        // rows that see nothing, bad lengths and rows
        for (int i = blockIdx.x; i < p.B; i += gridDim.x) {
            const SeqRows sq = seq_rows(P, i, BS, threadIdx.x == 0);
            for (int h = 0; h < p.Hkv; ++h) clear_rows(P, sq, h, D);
            if (threadIdx.x == 0 && p.new_slots != nullptr && sq.L == 0 && __ldg(p.new_slots + i) >= 0)
                raise_error(p.err, PKV_DEVERR_SLOT);
        }
        fence_proxy_async_smem();   // the copies that will land there come after these writes and reads
        __syncthreads();            // the scan's memory becomes the ring
    }

    while (x < x1) {
        // ---- the next segment: a unit and its pages [c0, c1)
        int kvh, tile, c0, c1, turn = 0, turns = 1;   // this warp takes every turns-th step from turn on
        Parts part{};
        SeqRows sq;
        if (P.balanced) {
            sq = seq_rows(P, b, BS, false);
            int units = p.Hkv * ((sq.nq * p.m + R - 1) / R);
            while (sq.pages == 0 || unit == units) {   // on to the next sequence that has keys
                ++b;
                unit = 0;
                sq = seq_rows(P, b, BS, false);
                units = p.Hkv * ((sq.nq * p.m + R - 1) / R);
            }
            kvh = unit % p.Hkv;
            tile = unit / p.Hkv;
            // positions [step, end) of the unit's span, the first kUnitCost of which hold no keys
            const int len = (sq.pages + PPS - 1) / PPS, end = min(len + kUnitCost, step + (x1 - x));
            const int first = x - step + kUnitCost;   // the position of the unit's first keys
            c0 = sq.first + max(0, step - kUnitCost) * PPS;
            c1 = min(sq.first + sq.pages, sq.first + max(0, end - kUnitCost) * PPS);
            x += end - step;
            step = 0;
            ++unit;
            if (c0 >= c1) continue;   // the share ends before the unit's keys
            // the warp whose share holds position y is ((y + 1) * warps - 1) / Q
            part.first = static_cast<int>(((first + 1ll) * warps - 1) / Q);
            part.n = static_cast<int>((static_cast<long long>(first + len) * warps - 1) / Q) - part.first + 1;
            part.own = wid - part.first;
            part.counter = p.counters + part.first;   // at most one unit goes on from a warp into the next
        } else {
            tile = blockIdx.x % p.head_tiles;
            const int split = blockIdx.x / p.head_tiles;
            kvh = blockIdx.y;
            b = blockIdx.z;
            sq = seq_rows(P, b, BS, threadIdx.x == 0 && split == 0 && kvh == 0 && tile == 0);
            if (split == 0 && tile == 0) clear_rows(P, sq, kvh, D);
            if (!sq.ok || R * tile >= sq.nq * p.m) return;
            // pages that any row of the sequence sees; this chunk's
            c0 = sq.first + split * p.chunk_pages;
            c1 = min(sq.first + sq.pages, c0 + p.chunk_pages);
            if (c0 >= c1) {
                // a new token for a sequence that holds none has no position: flagged, not written
                if (split == 0 && p.new_slots != nullptr && threadIdx.x == 0 && sq.L == 0 && __ldg(p.new_slots + b) >= 0)
                    raise_error(p.err, PKV_DEVERR_SLOT);
                return;
            }
            part.own = split;
            part.n = (sq.pages + p.chunk_pages - 1) / p.chunk_pages;
            part.counter = p.counters == nullptr ? nullptr : p.counters + (b * p.Hkv + kvh) * p.head_tiles + tile;
            x = x1;
            turn = warp;
            turns = NW;
            if (threadIdx.x < R) s_rows[threadIdx.x] = tile_row(P, sq, kvh, R * tile + threadIdx.x);
        }
        const RowSpan t_first = tile_row(P, sq, kvh, R * tile), t_last = tile_row(P, sq, kvh, min(R * tile + R - 1, sq.nq * p.m - 1));
        const RowSpan me = tile_row(P, sq, kvh, R * tile + Rows::row(lane));
        const int pg0 = max(c0, t_first.lo / BS), pg1 = min(c1, (t_last.len + BS - 1) / BS);
        const int tok_end = pg1 * BS;   // the segment's keys end here

        if (p.new_slots != nullptr && c1 == sq.first + sq.pages) {
            // the step's new token: the warp (chunks: the block's first two) whose segment holds the
            // sequence's last page writes its K and V rows there before any copy of the page
            const long long slot = __ldg(p.new_slots + b);
            if (slot >= 0) {
                const int pos = sq.L - 1, phys = __ldg(p.block_table + static_cast<size_t>(b) * p.MBS + pos / BS);
                if (phys < 0 || phys >= p.NB || slot != static_cast<long long>(phys) * BS + pos % BS) {
                    if (turn == 0 && lane == 0) raise_error(p.err, PKV_DEVERR_SLOT);
                } else {
                    for (int side = turn; side < 2; side += turns)
                        write_new_row<D, G>(P, b, kvh, (static_cast<long long>(phys) * p.Hkv + kvh) * Cfg::kPageBytes,
                                            pos % BS, BS, side, lane);
                }
            }
            fence_proxy_async_global();
            if (turns > 1) __syncthreads();
            else __syncwarp();
            fence_proxy_async_global();
        }

        // the queries' loads start before the block table's
        const int q_bi = tile_row(P, sq, kvh, R * tile + Rows::query_row(lane)).bi;
        rows.load(q_bi >= 0 ? p.q + static_cast<size_t>(q_bi) * D : nullptr, lane);

        // ---- this warp's stages: steps of PPS pages turn, turn + turns, ... of [pg0, pg1)
        const int steps = pg1 > pg0 ? (pg1 - pg0 + PPS - 1) / PPS : 0;
        const int n_my = steps > turn ? (steps - turn + turns - 1) / turns : 0;
        const int32_t *tbl = p.block_table + static_cast<size_t>(b) * p.MBS;
        // lane l: copy l of a stage's 2 * PPS (K pages, then V pages), its page's id loaded a stage ahead
        int pg = pg0 + turn * PPS + lane % PPS, phys = pg < pg1 ? __ldg(tbl + pg) : -1;
        auto issue = [&](int k) {   // the whole warp, k = 0, 1, ...
            const int st = (cnt + k) % kStages;
            const uint32_t bar = smem_addr(&bars[st]);
            const bool there = lane < 2 * PPS && pg < pg1, ok = there && phys >= 0 && phys < p.NB;
            const unsigned copies = __ballot_sync(kFull, ok), absent = __ballot_sync(kFull, there && !ok);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, __popc(copies) * Cfg::kPageBytes);
                if (absent != 0) raise_error(p.err, PKV_DEVERR_BLOCK);
            }
            bad = (bad & ~(((1u << PPS) - 1) << (st * PPS))) | ((absent & ((1u << PPS) - 1)) << (st * PPS));
            __syncwarp();   // the expected bytes are announced before any copy
            if (ok)
                bulk_load(smem_addr(ring + st * Cfg::kStageBytes + lane * Cfg::kPageBytes),
                          (lane < PPS ? P.kc : P.vc) + (static_cast<size_t>(phys) * p.Hkv + kvh) * Cfg::kPageBytes,
                          Cfg::kPageBytes, bar);
            pg += turns * PPS;
            phys = pg < pg1 ? __ldg(tbl + pg) : -1;
        };
        int issued = min(kStages, n_my);
        for (int k = 0; k < issued; ++k) issue(k);

        rows.begin(p.scale_log2, P.q_sign, lane);   // while the copies fly

        int k = 0;
        for (; k < n_my; ++k) {
            const int st = (cnt + k) % kStages;
            const bool arrived = mbar_wait_bounded(smem_addr(&bars[st]), ((cnt + k) / kStages) & 1);
            if (!__all_sync(kFull, arrived)) {
                if (lane == 0) raise_error(p.err, PKV_DEVERR_TIMEOUT);
                break;
            }
            const uint8_t *kpages = ring + st * Cfg::kStageBytes;
            const uint8_t *vpages = kpages + PPS * Cfg::kPageBytes;
            const int tok0 = (pg0 + (turn + k * turns) * PPS) * BS;
            // does every row of the tile see every key of the stage?
            const bool whole = tok0 >= t_last.lo && tok0 + kStageKeys <= min(t_first.len, tok_end);
            // this lane's key: parameters of keys that no row sees (which may be anything) and of
            // pages that are not there become 0; codes are finite whatever they are
            const bool seen = tok0 + lane >= t_first.lo && tok0 + lane < min(t_last.len, tok_end) &&
                              !(bad >> (st * PPS + lane / BS) & 1);
            rows.stage(kpages, vpages, par, seen, tok0, whole ? -1 : tok_end, me, lane);
            __syncwarp();
            if (k + kStages < n_my) {
                issue(k + kStages);
                issued = k + kStages + 1;
            }
        }
        const bool gave_up = k < n_my;
        if (gave_up) {
            // A copy did not arrive in time: wait (bounded) for the copies still in flight so that
            // none lands after the block exits.
            for (int kk = k; kk < issued; ++kk) mbar_wait_bounded(smem_addr(&bars[(cnt + kk) % kStages]), ((cnt + kk) / kStages) & 1);
        }
        cnt += n_my;

        rows.end();

        if (P.balanced) {
            if (gave_up) return;   // lanes together; the block's other warps go on
            // no key of this part for the row; a sum of NaN has keys whose scores are NaN, which ref ignores
            const bool empty = rows.ref == -INFINITY && rows.l == 0.f;
            const float inv = empty ? 0.f : 1.f / rows.l, lse2 = empty ? -INFINITY : rows.ref + log2f(rows.l);
            if (Rows::owner(lane)) {
                if (part.n > 1) p.ws_lse[part_at<R>(part, Rows::row(lane), part.own)] = me.bi >= 0 ? lse2 : -INFINITY;
                else if (me.bi >= 0 && p.lse != nullptr) p.lse[me.bi] = lse2 * kDecLn2;
            }
#pragma unroll
            for (int r = 0; r < Rows::OUT; ++r) {
                const float il = Rows::of_out_row(inv, r, lane);
                const int bi = Rows::of_out_row(me.bi, r, lane);
                float *dst = part.n > 1 ? p.ws_o + part_at<R>(part, Rows::out_row(r, lane), part.own) * D
                                        : p.out + static_cast<size_t>(max(bi, 0)) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const float4 y = rows.output(c, r, lane);
                    if (part.n > 1 || bi >= 0)
                        *reinterpret_cast<float4 *>(dst + 32 * c + 4 * g) = make_float4(y.x * il, y.y * il, y.z * il, y.w * il);
                }
            }
            if (part.n > 1) {
                __threadfence();
                __syncwarp();
                int last = 0;
                if (lane == 0) {
                    last = atomicAdd(part.counter, 1u) + 1 == static_cast<unsigned>(part.n);
                    if (last) *part.counter = 0u;   // every part of this call has arrived
                }
                if (__shfl_sync(kFull, last, 0)) {
                    __threadfence();
                    merge_unit<D, R>(P, Rows::of_merge_row(me.bi, lane), part, lane);
                }
            }
            continue;
        }

        // ---- the warps' (ref, l, O) through shared memory (the ring is free now)
        if (__syncthreads_or(gave_up)) return;
        float *mw = reinterpret_cast<float *>(smem);
        float *lw = mw + NW * R;
        float *ow = lw + NW * R;
        if (Rows::owner(lane)) {
            mw[warp * R + Rows::row(lane)] = rows.ref;
            lw[warp * R + Rows::row(lane)] = rows.l;
        }
#pragma unroll
        for (int r = 0; r < Rows::OUT; ++r)
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                *reinterpret_cast<float4 *>(ow + (warp * R + Rows::out_row(r, lane)) * D + 32 * c + 4 * g) = rows.output(c, r, lane);
        __syncthreads();
        finish_rows<D, NW, R>(smem, P, s_rows, part);
    }
}

template <int D, int BS, int G, typename Rows>
cudaError_t launch_mma_as(const AttendQ4Params &P, dim3 grid, cudaStream_t stream) {
    using Cfg = MmaCfg<D, BS, G, Rows>;
    static std::atomic<unsigned long long> done{0};
    auto kernel = attend_q4_mma_kernel<D, BS, G, Rows>;
    const cudaError_t e = set_smem_once(kernel, Cfg::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kMmaWarps * 32, Cfg::kSmemBytes, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace
}  // namespace pkv
