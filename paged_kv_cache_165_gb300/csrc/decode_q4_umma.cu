// decode_q4_umma.cu -- attention over a 4-bit cache for many query rows x heads on one KV head
// (MQA, large GQA groups, verification, chunks of new tokens) on the 5th-generation tensor cores
// (tcgen05).
//
// What is computed is the attention of decode_q4.cu (scale and zero factored out of the products;
// limoncc.com "大语言模型研究15——注意力机制优化之KV缓存" §3.1, §3.3; online softmax, plumephp.com
// "KV Cache 优化与注意力机制加速" §2.2-§2.3).  A tile is up to 64 (query row, head) pairs ("slots")
// of one sequence and KV head; its 128 rows are the slots' f16 hi and lo parts, 8 lanes apart in
// 16-lane groups, as in decode_umma.cu.  Keys are taken TK = 128 / G at a time, so that the sums of
// a key tile's G scale groups fill one 128-column buffer.  One block per SM, 14 warps:
//   warp 9 (loader): the pages' runs (codes and parameters) into a ring of packed tiles, one bulk
//     copy per K or V page.
//   warps 10-13 (converters): codes to f16 -- K's by masks alone: in the low bits of an f16 a code is
//     the subnormal code * 2^-24, four bits further up code * 2^-20; V's centred and brought into the
//     normal range by one more multiply-add -- written as 128-byte-swizzled tiles; parameters widened
//     to fp32.  A word's elements lie in the order 0 4 1 5 2 6 3 7 (as the masks deliver them); K's odd
//     ones are 16 times too large: the queries are laid out and scaled to match.
//   warp 8 (one lane issues): S = Q K^T per group into one of two buffers, and O_g += P_g V_g, with Q
//     and P in tensor memory.
//   warps 0-7 (softmax): thread (w, lane) owns slot 8 g + lane / 4 of lane group g = 2 (w % 4) + w / 4
//     and every fourth key pair: s = sum_g scale_g S_g + zero_g sum(q_g), then the weights times each
//     group's V scale as f16 hi + lo into tensor memory; the zeros' part of the output in fp32.
// The f16 range: queries are scaled by a power of two per slot; the weights' reference is shifted by
// E = ceil(log2 of the largest V scale) - 7, so that weight * scale stays below 2^15 although O is
// rescaled only when the running maximum grew by more than 2^8.
// The tensor core cuts its sums off instead of rounding them, so it adds up 1024 keys; the softmax warps
// then take O into fp32 sums in shared memory (4 x 131072 tokens: off by 2e-7 of the result instead of
// 2.2e-6, in the same time).
//
// Work: balanced (an equal range of all units' key tiles for every block, which may end one unit and
// begin the next; the loader and the converters run ahead into it) or one block per unit and chunk,
// as the warp-MMA kernel.
// Bound by the chain of a key tile (scores, softmax, weights, output: some 2000 cycles for 128 keys,
// tensor pipe 26%), plus 13 us of start and merge: 4 x 131072 tokens, 64 heads on one KV head, 56 us for
// 71.7 MB (1.3 TB/s).  Sixteen softmax warps took 68 us (half the registers each).
// Every wait is bounded and shares an abort flag, as in decode_umma.cu.
#include "decode_q4.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

template <int D, int BS, int G>
struct Cfg {
    static constexpr int TK = 128 / G, PPT = TK / BS, WORDS = D / 8, DG = D / G;
    static constexpr int kCodeBytes = BS * D / 2, kPageBytes = BS * (D / 2 + 4 * G);
    static constexpr int kTileBytes = TK * D * 2;               // an f16 K or V tile
    static constexpr int kPackedBytes = 2 * PPT * kPageBytes;   // a packed tile: K pages, V pages
    static constexpr int kParRow = TK + 16;                     // parameters: four runs of TK / 4, padded apart
    static constexpr int kParFloats = 4 * G * kParRow;          // K scale, K zero, V scale, V zero
    static constexpr int NT = kTileBytes > 16384 ? 2 : 4;       // f16 tiles of a ring: 64 KB
    static constexpr int kFold = 1024 / TK;                     // key tiles that the tensor core sums up
    static constexpr int kSumBytes = kQ4UmmaSlots * D * 4;      // the sums of those before, in fp32
    static constexpr int kRest = 232448 - 1024 - 64 - 256 - 4 * 16384 * 2 - kSumBytes - NT * (kParFloats + 4) * 4;
    static constexpr int NS = kRest >= 4 * kPackedBytes ? 4 : 3;   // packed tiles
    static constexpr int kOffK = 0, kOffV = kOffK + NT * kTileBytes, kOffS = kOffV + NT * kTileBytes;
    static constexpr int kOffPar = kOffS + NS * kPackedBytes;
    static constexpr int kOffMax = kOffPar + NT * kParFloats * 4;   // V's largest |scale| [tile][converter warp]
    static constexpr int kOffBar = kOffMax + NT * 4 * 4;
    static constexpr int kSFull = 0, kSFree = NS, kKFull = 2 * NS, kKFree = kKFull + NT, kVFull = kKFree + NT,
                         kVFree = kVFull + NT, kQ = kVFree + NT, kScore = kQ + 1, kP = kScore + 2, kO = kP + 1,
                         kDrain = kO + 1, kBars = kDrain + 2;
    static constexpr int kOffSum = kOffBar + (kBars * 8 + 15) / 16 * 16;
    static constexpr int kOffMisc = kOffSum + kSumBytes;   // TMEM address, abort flag, bad pages [NS], the share
    static constexpr int kSmemBytes = 1024 + kOffMisc + 64;
    static constexpr int kSCol = 0, kOCol = 256, kPCol = kOCol + D, kQCol = kPCol + 64;
    static constexpr int kThreads = 448;
    static_assert(kPageBytes % 16 == 0 && kPackedBytes % 16 == 0 && DG >= 64, "layout");
    static_assert(kQCol + D / 2 <= 512, "tensor memory budget");
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// Instruction descriptor of kind::f16: f16 A and B, fp32 D, M x N, B K-major or MN-major.
__device__ __forceinline__ uint32_t idesc_f16(int M, int N, int b_mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// A block's segments: units (sequence, tile of slots, KV head) and their page ranges.
struct Share {
    int x, x1, Q, blocks;   // balanced: key tiles [x, x1) of Q, and the blocks that have any
    int b, unit, step;
};
struct Segment {
    SeqRows sq;
    int b, kvh, slot0, slots, pg0, pg1, lo, tok_end;
    Parts part;
};

template <int BS, int PPT>
__device__ __forceinline__ bool next_segment(const AttendQ4Params &P, Share &s, Segment &g, bool report) {
    const DecodeKParams &p = P.k;
    if (s.x >= s.x1) return false;
    int tile, c0, c1;
    g.part = Parts{};
    if (P.balanced) {
        g.sq = seq_rows(P, s.b, BS, false);
        int len = (g.sq.pages + PPT - 1) / PPT;
        int units = p.Hkv * ((g.sq.nq * p.m + kQ4UmmaSlots - 1) / kQ4UmmaSlots);
        while (g.sq.pages == 0 || s.unit == units) {   // on to the next sequence that has keys
            ++s.b;
            s.unit = 0;
            g.sq = seq_rows(P, s.b, BS, false);
            len = (g.sq.pages + PPT - 1) / PPT;
            units = p.Hkv * ((g.sq.nq * p.m + kQ4UmmaSlots - 1) / kQ4UmmaSlots);
        }
        g.b = s.b;
        g.kvh = s.unit % p.Hkv;
        tile = s.unit / p.Hkv;
        const int end = min(len, s.step + (s.x1 - s.x)), start = s.x - s.step;
        c0 = g.sq.first + s.step * PPT;
        c1 = min(g.sq.first + g.sq.pages, g.sq.first + end * PPT);
        g.part.first = static_cast<int>(((start + 1ll) * s.blocks - 1) / s.Q);
        g.part.n = static_cast<int>((static_cast<long long>(start + len) * s.blocks - 1) / s.Q) - g.part.first + 1;
        g.part.own = blockIdx.x - g.part.first;
        g.part.counter = p.counters + g.part.first;   // at most one unit goes on from a block into the next
        s.x += end - s.step;
        s.step = 0;
        ++s.unit;
    } else {
        s.x = s.x1;
        tile = blockIdx.x % p.head_tiles;
        const int split = blockIdx.x / p.head_tiles;
        g.kvh = blockIdx.y;
        g.b = blockIdx.z;
        g.sq = seq_rows(P, g.b, BS, report && split == 0 && g.kvh == 0 && tile == 0);
        if (!g.sq.ok || kQ4UmmaSlots * tile >= g.sq.nq * p.m) return false;
        c0 = g.sq.first + split * p.chunk_pages;
        c1 = min(g.sq.first + g.sq.pages, c0 + p.chunk_pages);
        if (c0 >= c1) return false;
        g.part.own = split;
        g.part.n = (g.sq.pages + p.chunk_pages - 1) / p.chunk_pages;
    }
    g.slot0 = kQ4UmmaSlots * tile;
    g.slots = min(kQ4UmmaSlots, g.sq.nq * p.m - g.slot0);
    const RowSpan a = tile_row(P, g.sq, g.kvh, g.slot0), z = tile_row(P, g.sq, g.kvh, g.slot0 + g.slots - 1);
    g.lo = a.lo;
    g.pg0 = max(c0, a.lo / BS);
    g.pg1 = min(c1, (z.len + BS - 1) / BS);
    g.tok_end = min(z.len, g.pg1 * BS);
    return true;
}

// Row h of a balanced part, in units of D floats of ws_o and of one float of ws_lse.
__device__ __forceinline__ size_t part_at(const Parts &u, int h, int i) {
    return (static_cast<size_t>(u.first + i) * 2 + (i == 0)) * kQ4UmmaSlots + h;
}

template <int D, int BS, int G>
__global__ void __launch_bounds__(448, 1) attend_q4_umma_kernel(const __grid_constant__ AttendQ4Params P) {
    using C = Cfg<D, BS, G>;
    constexpr int TK = C::TK, PPT = C::PPT, WORDS = C::WORDS, NT = C::NT, NS = C::NS;
    const DecodeKParams &p = P.k;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    auto bar = [&](int k) { return smem_addr(&bars[k]); };
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    volatile int *s_last = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 8);
    volatile unsigned *s_bad = reinterpret_cast<volatile unsigned *>(smem + C::kOffMisc + 16);   // [NS]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(bar(C::kSFull + i), 1);
            mbar_init(bar(C::kSFree + i), 4);
        }
        for (int i = 0; i < NT; ++i) {
            mbar_init(bar(C::kKFull + i), 4);
            mbar_init(bar(C::kKFree + i), 1);
            mbar_init(bar(C::kVFull + i), 4);
            mbar_init(bar(C::kVFree + i), 1);
        }
        mbar_init(bar(C::kQ), 8);
        mbar_init(bar(C::kScore), 1);
        mbar_init(bar(C::kScore + 1), 1);
        mbar_init(bar(C::kP), 8);
        mbar_init(bar(C::kO), 1);
        mbar_init(bar(C::kDrain), 1);
        mbar_init(bar(C::kDrain + 1), 1);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(smem_addr(tslot), 512);

    // ---- this block's share.  Balanced: as many blocks as units, or enough for four key tiles each,
    // when the keys are few.
    Share share{0, 1, 1, 1, 0, 0, 0};
    if (P.balanced) {
        int *pre = reinterpret_cast<int *>(smem);   // key tiles before each sequence; the K ring is free yet
        __shared__ int s_sum[2][14];
        const int per = (p.B + C::kThreads - 1) / C::kThreads, first = threadIdx.x * per;
        int steps = 0, units = 0;
        for (int i = first; i < min(p.B, first + per); ++i) {
            const SeqRows sq = seq_rows(P, i, BS, false);
            const int n = sq.pages > 0 ? p.Hkv * ((sq.nq * p.m + kQ4UmmaSlots - 1) / kQ4UmmaSlots) : 0;
            pre[i + 1] = n * ((sq.pages + PPT - 1) / PPT);
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
        int Q = 0;
        units = 0;
        before -= steps;
        for (int w = 0; w < 14; ++w) {
            if (w < warp) before += s_sum[0][w];
            Q += s_sum[0][w];
            units += s_sum[1][w];
        }
        if (threadIdx.x == 0) pre[0] = 0;
        for (int i = first; i < min(p.B, first + per); ++i) pre[i + 1] = before += pre[i + 1];
        share.Q = Q;
        share.blocks = min(static_cast<int>(gridDim.x), max(units, Q / 4));
        const int blocks = max(share.blocks, 1);
        share.x = static_cast<int>(min(static_cast<long long>(Q), static_cast<long long>(blockIdx.x) * Q / blocks));
        share.x1 = static_cast<int>(min(static_cast<long long>(Q), (blockIdx.x + 1ll) * Q / blocks));
        __syncthreads();
        for (int st = kMaxBalanced / 2; st > 0; st >>= 1)
            if (share.b + st < p.B && pre[share.b + st] <= share.x) share.b += st;
        if (share.x < share.x1) {
            const SeqRows sq = seq_rows(P, share.b, BS, false);
            const int len = (sq.pages + PPT - 1) / PPT;
            share.unit = (share.x - pre[share.b]) / len;
            share.step = (share.x - pre[share.b]) - share.unit * len;
        }
        // rows that see nothing, bad lengths and rows
        for (int i = blockIdx.x; i < p.B; i += gridDim.x) {
            const SeqRows sq = seq_rows(P, i, BS, threadIdx.x == 0);
            for (int h = 0; h < p.Hkv; ++h) clear_rows(P, sq, h, D);
        }
    } else if (blockIdx.x == 0) {
        clear_rows(P, seq_rows(P, blockIdx.z, BS, false), blockIdx.y, D);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    pdl_launch_dependents();   // a merge kernel may be scheduled; it waits for this grid
    const uint32_t tmem = *tslot;
    auto sK = [&](int i) { return smem + C::kOffK + i * C::kTileBytes; };
    auto sV = [&](int i) { return smem + C::kOffV + i * C::kTileBytes; };
    auto sS = [&](int i) { return smem + C::kOffS + i * C::kPackedBytes; };
    float *par = reinterpret_cast<float *>(smem + C::kOffPar);
    float *vmax = reinterpret_cast<float *>(smem + C::kOffMax);

    Segment g;
    int T = 0;   // key tiles of the segments so far (ring positions run on across segments)
    if (warp == 9) {
        // ---- loader: lane l copies page l % PPT of K (l < PPT) or V
        bool alive = true;
        int done = 0;
        while (alive && next_segment<BS, PPT>(P, share, g, false)) {
            const int32_t *tbl = p.block_table + static_cast<size_t>(g.b) * p.MBS + g.pg0;
            const int pages = max(0, g.pg1 - g.pg0), n = (pages + PPT - 1) / PPT;
            int tcur = lane < pages ? __ldg(tbl + lane) : -1, tnext = 32 + lane < pages ? __ldg(tbl + 32 + lane) : -1;
            for (int t = 0; t < n; ++t, ++done) {
                const int st = (T + t) % NS;
                bool fr = true;
                if (lane == 0 && T + t >= NS) fr = wait_or_abort(bar(C::kSFree + st), ((T + t) / NS - 1) & 1, abort, p.err);
                alive = __shfl_sync(kFull, fr ? 1 : 0, 0);
                if (!alive) break;
                const int at = t * PPT;
                if (at > 0 && at % 32 == 0) {
                    tcur = tnext;
                    tnext = at + 32 + lane < pages ? __ldg(tbl + at + 32 + lane) : -1;
                }
                const int pg = lane % PPT, phys = __shfl_sync(kFull, tcur, (at + pg) & 31);
                const bool there = lane < 2 * PPT && at + pg < pages, ok = there && phys >= 0 && phys < p.NB;
                const unsigned copies = __ballot_sync(kFull, ok), absent = __ballot_sync(kFull, there && !ok);
                if (lane == 0) {
                    s_bad[st] = absent & ((1u << PPT) - 1);
                    if (absent != 0) raise_error(p.err, PKV_DEVERR_BLOCK);
                    mbar_arrive_expect_tx(bar(C::kSFull + st), __popc(copies) * C::kPageBytes);
                }
                __syncwarp();   // the expected bytes are announced before any copy
                if (ok)
                    bulk_load(smem_addr(sS(st) + lane * C::kPageBytes),
                              (lane < PPT ? P.kc : P.vc) + (static_cast<size_t>(phys) * p.Hkv + g.kvh) * C::kPageBytes,
                              C::kPageBytes, bar(C::kSFull + st));
            }
            T += n;
        }
        // before teardown every copy issued must have landed (bounded)
        if (lane == 0)
            for (int u = max(0, done - NS); u < done; ++u)
                if (!mbar_wait_bounded(bar(C::kSFull + u % NS), (u / NS) & 1)) raise_error(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp >= 10) {
        // ---- converters.  A 16-byte piece holds four words; lanes take (key, piece) pairs so that
        // eight lanes read eight different 16-byte banks and write eight different ones of the
        // swizzled tile: d = 128: pieces 0, 1 of two keys with pieces 2, 3 of their neighbours
        const int w = warp - 10, ct = threadIdx.x - 320;
        bool alive = true;
        auto convert = [&](const uint8_t *pages, uint8_t *tile, auto centred) {
#pragma unroll
            for (int i = 0; i < TK * WORDS / 4 / 128; ++i) {
                int key, piece;
                if constexpr (D == 128) {
                    piece = lane & 3;
                    key = ((i * 4 + w) << 3) + ((lane >> 4) << 2) + ((lane >> 2) & 1) + 2 * ((piece >> 1) ^ ((lane >> 3) & 1));
                } else {
                    piece = lane & 1;
                    key = ((i * 4 + w) << 4) + (lane >> 1);
                }
                const uint4 u = *reinterpret_cast<const uint4 *>(pages + (key / BS) * C::kPageBytes + (key % BS) * (D / 2) + piece * 16);
                const uint32_t c[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t y = c[j] >> 8;
                    uint4 z = make_uint4(c[j] & 0x000f000fu, c[j] & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u);
                    if constexpr (decltype(centred)::value) centre(c[j], z.x, z.y), centre(y, z.z, z.w);
                    *reinterpret_cast<uint4 *>(tile + swz128(TK, key, (4 * piece + j) * 8)) = z;
                }
            }
            fence_proxy_async_smem();   // before the MMAs read the tile
            __syncwarp();
        };
        while (alive && next_segment<BS, PPT>(P, share, g, false)) {
            const int n = max(0, (g.pg1 - g.pg0 + PPT - 1) / PPT);
            for (int t = 0; t < n && alive; ++t) {
                const int r = T + t, st = r % NS, sl = r % NT;
                alive = __all_sync(kFull, wait_or_abort(bar(C::kSFull + st), (r / NS) & 1, abort, p.err));
                if (alive && r >= NT) alive = __all_sync(kFull, wait_or_abort(bar(C::kKFree + sl), (r / NT - 1) & 1, abort, p.err));
                if (!alive) break;
                convert(sS(st), sK(sl), std::false_type{});
                if (lane == 0) mbar_arrive(bar(C::kKFull + sl));
                if (r >= NT) alive = __all_sync(kFull, wait_or_abort(bar(C::kVFree + sl), (r / NT - 1) & 1, abort, p.err));
                if (!alive) break;
                // the parameters: those of keys that no slot sees, or of pages that are not there, as 0
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 2 * TK / 128; ++i) {
                    const int side = (i * 128 + ct) / TK, key = (i * 128 + ct) % TK, tok = g.pg0 * BS + t * TK + key;
                    const bool seen = tok >= g.lo && tok < g.tok_end && !(s_bad[st] >> (key / BS) & 1);
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(sS(st) + (side * PPT + key / BS) * C::kPageBytes + C::kCodeBytes) +
                                          (key % BS) * G;
                    const int at = ((key % 8) / 2) * (TK / 4 + 4) + key / 8 * 2 + (key & 1);
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        const uint32_t raw = seen ? src[gi] : 0u;
                        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&raw));
                        float *dst = par + sl * C::kParFloats + (2 * side * G + gi) * C::kParRow + at;
                        dst[0] = y.x;
                        dst[G * C::kParRow] = side == 1 ? fmaf(8.f, y.x, y.y) : y.y;   // V's codes are centred
                        if (side == 1) top = fmaxf(top, fabsf(y.x));
                    }
                }
                top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));   // non-negative floats order like their bits
                if (lane == 0) vmax[sl * 4 + w] = top;
                convert(sS(st) + PPT * C::kPageBytes, sV(sl), std::true_type{});
                if (lane == 0) {
                    mbar_arrive(bar(C::kVFull + sl));
                    mbar_arrive(bar(C::kSFree + st));
                }
            }
            T += n;
        }
    } else if (warp == 8) {
        // ---- MMA issue by one lane: S of tile t + 1, then the products of tile t, so that the next
        // scores are computed while the softmax of tile t runs.  S of tile t + 1 may overwrite that of
        // tile t - 1: its products were issued, so its weights are written and its scores read.
        if (lane == 0) {
            bool alive = true, issued = false;
            const uint32_t is = idesc_f16(128, TK, 0), io = idesc_f16(128, C::DG, 1);
            int qn = 0;
            auto scores = [&](int r) {   // S of ring tile r into buffer r & 1
                alive = wait_or_abort(bar(C::kKFull + r % NT), (r / NT) & 1, abort, p.err);
                if (!alive) return;
                tc_fence_after_sync();
                const uint32_t k = smem_addr(sK(r % NT));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const int gi = kk / (C::DG / 16);
                    umma_bf16_ts(tmem + C::kSCol + (r & 1) * 128 + gi * TK, tmem + C::kQCol + kk * 8,
                                 umma_desc_sw128(k + (kk / 4) * TK * 128 + (kk % 4) * 32, 16, 1024), is,
                                 kk % (C::DG / 16) > 0 ? 1u : 0u);
                }
                umma_commit(bar(C::kScore + (r & 1)));
                umma_commit(bar(C::kKFree + r % NT));
                issued = true;
            };
            auto products = [&](int r, bool fresh) {   // O += P V of ring tile r
                alive = wait_or_abort(bar(C::kP), r & 1, abort, p.err) &&
                        wait_or_abort(bar(C::kVFull + r % NT), (r / NT) & 1, abort, p.err);
                if (!alive) return;
                tc_fence_after_sync();
                const uint32_t v = smem_addr(sV(r % NT));
#pragma unroll
                for (int gi = 0; gi < G; ++gi)
#pragma unroll
                    for (int kk = 0; kk < TK / 16; ++kk)
                        umma_bf16_ts(tmem + C::kOCol + gi * C::DG, tmem + C::kPCol + gi * (TK / 2) + kk * 8,
                                     umma_desc_sw128(v + gi * (C::DG / 64) * TK * 128 + kk * 16 * 128, TK * 128, 1024), io,
                                     (!fresh || kk > 0) ? 1u : 0u);
                umma_commit(bar(C::kO));
                umma_commit(bar(C::kVFree + r % NT));
                issued = true;
            };
            while (alive && next_segment<BS, PPT>(P, share, g, false)) {
                const int n = max(0, (g.pg1 - g.pg0 + PPT - 1) / PPT);
                if (n > 0) {
                    alive = wait_or_abort(bar(C::kQ), qn & 1, abort, p.err);
                    ++qn;
                    if (alive) scores(T);
                    for (int t = 0; t < n && alive; ++t) {
                        if (t + 1 < n) scores(T + t + 1);
                        if (alive) products(T + t, t % C::kFold == 0);
                    }
                }
                T += n;
            }
            if (*abort && issued) {   // let the MMAs finish (bounded) before teardown
                umma_commit(bar(C::kDrain));
                if (!mbar_wait_bounded(bar(C::kDrain), 0)) raise_error(p.err, PKV_DEVERR_TIMEOUT);
            }
        }
    } else {
        // ---- softmax
        const int c4 = lane & 3, grp = 2 * (warp & 3) + (warp >> 2), slot = 8 * grp + (lane >> 2);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(16 * grp) << 16);
        float *sums = reinterpret_cast<float *>(smem + C::kOffSum) + threadIdx.x;   // [32 of a slot's sums][thread]
        bool ok = true;   // warp-uniform; a failed wait skips the warp's remaining work
        while (next_segment<BS, PPT>(P, share, g, threadIdx.x == 0)) {
            const int n = max(0, (g.pg1 - g.pg0 + PPT - 1) / PPT);
            const RowSpan me = tile_row(P, g.sq, g.kvh, g.slot0 + min(slot, g.slots - 1));
            const bool mine = slot < g.slots;
            float f = 0.f, qsum[G];
#pragma unroll
            for (int gi = 0; gi < G; ++gi) qsum[gi] = 0.f;
            if (n > 0 && ok) {
                // the queries: the four threads of a slot take every fourth word.  Word w goes to columns
                // 4 w .. 4 w + 3 of the slot's hi and lo rows: elements (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16
                const float *qrow = p.q + static_cast<size_t>(me.bi) * D;
                float amax = 0.f;
                if (mine)
                    for (int i = c4; i < D / 4; i += 4) {
                        const float4 y = __ldg(reinterpret_cast<const float4 *>(qrow) + i);
                        amax = fmaxf(fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y))), fmaxf(fabsf(y.z), fabsf(y.w)));
                    }
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
                // |q| * 2^up in [2^13, 2^14); a row of zeros (or of subnormals) keeps the factor finite
                const int up = min(13 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), 126);
                const float qs = pow2i(up) * P.q_sign;
                f = (p.scale_log2 * 0x1p24f) * pow2i(-up);
                // 16 lanes x 128 bits, 8 repeats: repeat k puts r[2k] at lane base + lane / 4, column 4 k + c4
                // and r[2k + 1] eight lanes further: word k of a half of eight, pair c4
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    uint32_t r[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float *src = qrow + (8 * h + k) * 8 + c4;
                        float2 y = mine ? make_float2(__ldg(src) * qs, __ldg(src + 4) * qs) : make_float2(0.f, 0.f);
                        qsum[h * 64 / C::DG] += y.x + y.y;
                        if (c4 & 1) y.x *= 0.0625f, y.y *= 0.0625f;
                        split2(y, r[2 * k], r[2 * k + 1]);
                    }
                    tmem_st_16x128b_x8(lane_base + C::kQCol + h * 32, r);
                }
#pragma unroll
                for (int gi = 0; gi < G; ++gi) {
                    qsum[gi] += __shfl_xor_sync(kFull, qsum[gi], 1);
                    qsum[gi] += __shfl_xor_sync(kFull, qsum[gi], 2);
                    qsum[gi] *= 0x1p-24f;
                }
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kQ));
            }

            float m_run = -INFINITY, ref = -INFINITY, l = 0.f, vtop = 0.f, vexp = -24.f;
            float2 zo[G];
#pragma unroll
            for (int gi = 0; gi < G; ++gi) zo[gi] = make_float2(0.f, 0.f);
            for (int t = 0; t < n; ++t) {
                const int r = T + t, sl = r % NT;
                // V full: this tile's parameters are written
                if (ok) ok = __all_sync(kFull, wait_or_abort(bar(C::kVFull + sl), (r / NT) & 1, abort, p.err));
                if (ok) ok = __all_sync(kFull, wait_or_abort(bar(C::kScore + (r & 1)), (r >> 1) & 1, abort, p.err));
                if (!ok) continue;
                tc_fence_after_sync();
                const float *pk = par + sl * C::kParFloats + c4 * (TK / 4 + 4), *pv = pk + 2 * G * C::kParRow;
                // sc[k]: the slot's scores of keys 8 k + 2 c4 + {0, 1} of the tile, in the MMAs' units
                float2 sc[TK / 8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {   // columns 64 h ..: keys (G = 1) or a group's sums (G = 2)
                    uint32_t s[32];
                    tmem_ld_16x256b_x8(lane_base + C::kSCol + (r & 1) * 128 + h * 64, s);
                    tmem_ld_wait();
                    const int gi = G == 1 ? 0 : h;
                    const float2 qz = make_float2(qsum[gi], qsum[gi]);
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const int kk = G == 1 ? 8 * h + k : k;
                        const float4 a = *reinterpret_cast<const float4 *>(pk + gi * C::kParRow + 2 * kk);
                        const float4 z = *reinterpret_cast<const float4 *>(pk + (G + gi) * C::kParRow + 2 * kk);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t *q = s + 4 * (k + e);
                            const float2 y = add2(make_float2(__uint_as_float(q[0]), __uint_as_float(q[1])),
                                                  make_float2(__uint_as_float(q[2]), __uint_as_float(q[3])));
                            const float2 zp = e ? make_float2(z.z, z.w) : make_float2(z.x, z.y);
                            const float2 base = gi == 0 ? mul2(zp, qz) : fma2(zp, qz, sc[kk + e]);
                            sc[kk + e] = fma2(e ? make_float2(a.z, a.w) : make_float2(a.x, a.y), y, base);
                        }
                    }
                }
                const int tok0 = g.pg0 * BS + t * TK, end = min(me.len, g.tok_end);
                const bool partial = tok0 < me.lo || tok0 + TK > end;   // of a tile
                if (partial) {
#pragma unroll
                    for (int k = 0; k < TK / 8; ++k) {
                        const int tok = tok0 + 8 * k + 2 * c4;
                        if (tok < me.lo || tok >= end) sc[k].x = -INFINITY;
                        if (tok + 1 < me.lo || tok + 1 >= end) sc[k].y = -INFINITY;
                    }
                }
                float mx = fmaxf(sc[0].x, sc[0].y);
#pragma unroll
                for (int k = 1; k < TK / 8; ++k) mx = fmaxf(mx, fmaxf(sc[k].x, sc[k].y));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2)) * f;
                const float4 vm = *reinterpret_cast<const float4 *>(vmax + sl * 4);
                const float top = fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w));
                if (top > vtop) {   // the same in every thread: the next power of two
                    vtop = top;
                    vexp = fmaxf(static_cast<float>(static_cast<int>((__float_as_uint(top) + 0x7fffffu) >> 23) - 127), -24.f);
                }
                // a slot that has seen no key yet keeps m = -inf and weight 0
                if (mx > m_run + 8.f || m_run == -INFINITY) m_run = mx;
                const float ref_new = m_run + (vexp - 7.f);
                const float alpha = ref == -INFINITY || ref_new == ref ? 1.f : ex2_approx(ref - ref_new);
                ref = ref_new;
                const float neg = ref == -INFINITY ? 0.f : -ref;
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < TK / 8; ++k) {
                    const float2 x = fma2(sc[k], make_float2(f, f), make_float2(neg, neg));
                    sc[k] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    sum = add2(sum, sc[k]);
                }
                l = l * alpha + (sum.x + sum.y);
#pragma unroll
                for (int gi = 0; gi < G; ++gi) zo[gi] = mul2(zo[gi], make_float2(alpha, alpha));
                // pair 4 k + c4 of the weights: P_hi for the hi row, P_lo for the lo row
                uint32_t pw[2][16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int gi = G == 1 ? 0 : h;
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const int kk = G == 1 ? 8 * h + k : k;
                        const float4 a = *reinterpret_cast<const float4 *>(pv + gi * C::kParRow + 2 * kk);
                        float4 z = *reinterpret_cast<const float4 *>(pv + (G + gi) * C::kParRow + 2 * kk);
                        if (partial) {   // a key that another slot sees may hold a NaN
                            z.x = sc[kk].x != 0.f ? z.x : 0.f, z.y = sc[kk].y != 0.f ? z.y : 0.f;
                            z.z = sc[kk + 1].x != 0.f ? z.z : 0.f, z.w = sc[kk + 1].y != 0.f ? z.w : 0.f;
                        }
                        split2(mul2(sc[kk], make_float2(a.x, a.y)), pw[h][2 * k], pw[h][2 * k + 1]);
                        split2(mul2(sc[kk + 1], make_float2(a.z, a.w)), pw[h][2 * k + 2], pw[h][2 * k + 3]);
                        zo[gi] = fma2(sc[kk], make_float2(z.x, z.y), fma2(sc[kk + 1], make_float2(z.z, z.w), zo[gi]));
                    }
                }
                // P V of the tile before must be done: the P columns are free and O is current
                if (t > 0) {
                    ok = __all_sync(kFull, wait_or_abort(bar(C::kO), (r - 1) & 1, abort, p.err));
                    if (!ok) continue;
                    tc_fence_after_sync();
                    const bool fold = t % C::kFold == 0;   // the products of this tile start O anew
                    if (fold || __any_sync(kFull, alpha != 1.f)) {
#pragma unroll
                        for (int cc = 0; cc < D / 64; ++cc) {
                            uint32_t o[32];
                            tmem_ld_16x256b_x8(lane_base + C::kOCol + cc * 64, o);
                            tmem_ld_wait();
                            if (fold || t > C::kFold) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    float *q = sums + (cc * 16 + e) * 256;
                                    float x = t > C::kFold ? *q : 0.f;
                                    if (fold) x += __uint_as_float(o[e / 2 * 4 + e % 2]) + __uint_as_float(o[e / 2 * 4 + 2 + e % 2]);
                                    *q = x * alpha;
                                }
                            }
                            if (!fold) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st_16x256b_x8(lane_base + C::kOCol + cc * 64, o);
                            }
                        }
                    }
                }
                tmem_st_16x128b_x8(lane_base + C::kPCol, pw[0]);
                tmem_st_16x128b_x8(lane_base + C::kPCol + 32, pw[1]);
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kP));
            }
            if (n > 0 && ok) ok = __all_sync(kFull, wait_or_abort(bar(C::kO), (T + n - 1) & 1, abort, p.err));

            // ---- the slot's sums over its four threads; O_hi + O_lo, unscaled, plus the zeros' part
            l += __shfl_xor_sync(kFull, l, 1);
            l += __shfl_xor_sync(kFull, l, 2);
            // the slot sees no key of this segment; a sum of NaN: it does, and ref ignores their scores
            const bool empty = ref == -INFINITY && l == 0.f;
            const float inv = empty ? 0.f : 1.f / l, lse2 = empty ? -INFINITY : ref + log2f(l);
            const bool whole = g.part.n == 1;
            const size_t at = whole        ? static_cast<size_t>(me.bi)
                              : P.balanced ? part_at(g.part, slot, g.part.own)
                                           : static_cast<size_t>(me.bi) * p.splits + g.part.own;
            float *dst = (whole ? p.out : p.ws_o) + at * D;
            const bool store = ok && (mine || (!whole && P.balanced));
            if (ok) tc_fence_after_sync();
#pragma unroll
            for (int cc = 0; cc < D / 64; ++cc) {
                const int gi = cc * 64 / C::DG;
                float z = zo[gi].x + zo[gi].y;
                z += __shfl_xor_sync(kFull, z, 1);
                z += __shfl_xor_sync(kFull, z, 2);
                uint32_t o[32];
                if (n > 0 && ok) {
                    tmem_ld_16x256b_x8(lane_base + C::kOCol + cc * 64, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (store)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {   // word 8 cc + k: elements c4 and c4 + 4
                        float *q = dst + cc * 64 + 8 * k + c4;
                        float x = __uint_as_float(o[4 * k]) + __uint_as_float(o[4 * k + 2]);
                        float y = __uint_as_float(o[4 * k + 1]) + __uint_as_float(o[4 * k + 3]);
                        if (n > C::kFold) {
                            x += sums[(cc * 16 + 2 * k) * 256];
                            y += sums[(cc * 16 + 2 * k + 1) * 256];
                        }
                        q[0] = fmaf(x, 0x1p9f, z) * inv;
                        q[4] = fmaf(y, 0x1p9f, z) * inv;
                    }
            }
            if (store && c4 == 0) {
                if (!whole) p.ws_lse[at] = mine ? lse2 : -INFINITY;
                else if (p.lse != nullptr) p.lse[me.bi] = lse2 * kDecLn2;
            }
            tc_fence_before_sync();   // O has been read before the next segment's products
            T += n;

            if (P.balanced && !whole) {
                // the block's part is written; the last block to arrive merges the unit's parts
                __threadfence();
                named_barrier(1, 256);
                if (threadIdx.x == 0) {
                    int last = 0;
                    if (*abort == 0) {
                        last = atomicAdd(g.part.counter, 1u) + 1 == static_cast<unsigned>(g.part.n);
                        if (last) *g.part.counter = 0u;   // every part of this call has arrived
                    }
                    *s_last = last;
                }
                named_barrier(1, 256);
                if (*s_last) {
                    __threadfence();
                    for (int h = warp; h < g.slots; h += 8) {
                        float M = -INFINITY, L = 0.f;
                        for (int i = lane; i < g.part.n; i += 32) M = fmaxf(M, __ldcg(p.ws_lse + part_at(g.part, h, i)));
#pragma unroll
                        for (int sh = 16; sh > 0; sh >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, sh));
                        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                        for (int i0 = 0; i0 < g.part.n; i0 += 32) {
                            const float wl = i0 + lane < g.part.n ? exp2f(__ldcg(p.ws_lse + part_at(g.part, h, i0 + lane)) - M) : 0.f;
                            L += wl;
                            const int m = min(32, g.part.n - i0);
#pragma unroll 8
                            for (int i = 0; i < m; ++i) {
                                const float wi = __shfl_sync(kFull, wl, i);
                                if (4 * lane < D) {
                                    const float4 y = __ldcg(reinterpret_cast<const float4 *>(p.ws_o + part_at(g.part, h, i0 + i) * D) + lane);
                                    acc.x = fmaf(wi, y.x, acc.x);
                                    acc.y = fmaf(wi, y.y, acc.y);
                                    acc.z = fmaf(wi, y.z, acc.z);
                                    acc.w = fmaf(wi, y.w, acc.w);
                                }
                            }
                        }
#pragma unroll
                        for (int sh = 16; sh > 0; sh >>= 1) L += __shfl_xor_sync(kFull, L, sh);
                        const RowSpan row = tile_row(P, g.sq, g.kvh, g.slot0 + h);
                        const float il = 1.f / L;
                        if (4 * lane < D)
                            reinterpret_cast<float4 *>(p.out + static_cast<size_t>(row.bi) * D)[lane] =
                                make_float4(acc.x * il, acc.y * il, acc.z * il, acc.w * il);
                        if (lane == 0 && p.lse != nullptr) p.lse[row.bi] = (M + log2f(L)) * kDecLn2;
                    }
                }
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D, int BS, int G>
cudaError_t launch_as(const AttendQ4Params &P, dim3 grid, cudaStream_t stream) {
    static std::atomic<unsigned long long> done{0};
    auto kernel = attend_q4_umma_kernel<D, BS, G>;
    const cudaError_t e = set_smem_once(kernel, Cfg<D, BS, G>::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    kernel<<<grid, Cfg<D, BS, G>::kThreads, Cfg<D, BS, G>::kSmemBytes, stream>>>(P);
    return cudaGetLastError();
}

}  // namespace

// Groups of at least 64 elements: a group's outputs are whole 128-byte panels of the V tile.
bool q4_umma_shape(int d, int group, int bs) { return (d == 64 || d == 128) && group >= 64 && (bs == 16 || bs == 32); }

cudaError_t launch_attend_q4_umma(const AttendQ4Params &P, int d, int bs, int G, dim3 grid, cudaStream_t stream) {
    if (d == 64) return bs == 16 ? launch_as<64, 16, 1>(P, grid, stream) : launch_as<64, 32, 1>(P, grid, stream);
    if (G == 1) return bs == 16 ? launch_as<128, 16, 1>(P, grid, stream) : launch_as<128, 32, 1>(P, grid, stream);
    return bs == 16 ? launch_as<128, 16, 2>(P, grid, stream) : launch_as<128, 32, 2>(P, grid, stream);
}

}  // namespace pkv
