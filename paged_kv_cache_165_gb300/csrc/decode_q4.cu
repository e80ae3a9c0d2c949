// decode_q4.cu -- attention of the newest query row(s) of every sequence over a paged cache
// held in 4 bits (q4_codes.cuh): value = zero + scale * code per group of elements.
//
// What is computed is the attention of decode.cu over those values (limoncc.com
// "大语言模型研究15——注意力机制优化之KV缓存" §3.1, §3.3; online softmax, plumephp.com
// "KV Cache 优化与注意力机制加速" §2.2-§2.3; rows at the end of the cache and windows,
// zwjcode.cn "KV Cache 的增量解码" §10, §13).  Scale and zero factor out of the products:
//   q . k_t = sum_g scale_tg (q_g . code_tg) + zero_tg sum(q_g)
//   sum_t p_t v_t = sum_t (p_t scale_tg) code_t + sum_t p_t zero_tg      (element in group g)
// so codes enter the products as the small integers they are, exactly.
#include <algorithm>
#include <atomic>

#include "decode_q4.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

constexpr int kLeastSteps = 4;       // 32-key steps that a warp of one takes at least (128 keys)

// ================================================================ CUDA-core path

// One warp per (query row, query head, chunk).  W lanes (a power of two, W * 8 >= d) hold one
// key's row, eight elements each, so 32 / W keys are taken at a time; every such slice of the
// warp keeps its own online softmax and they merge at the end.
template <int W>
__global__ void __launch_bounds__(128)
    attend_q4_simt_kernel(const uint8_t *__restrict__ kc, const uint8_t *__restrict__ vc, const DecodeKParams p,
                          int d, int bs, int lanes, int rows) {
    constexpr int KEYS = 32 / W;
    pdl_launch_dependents();   // the merge kernel after this one waits for the whole grid
    const int lane = threadIdx.x & 31;
    const long long unit = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (unit >= static_cast<long long>(rows) * p.Hq) return;
    const int row = static_cast<int>(unit / p.Hq), i = static_cast<int>(unit % p.Hq), split = blockIdx.y;
    const int kvh = i / p.m, j = lane % W, slice = lane / W;
    const SeqSpan sp = row_span(p, row, bs, lane == 0 && split == 0 && i == 0);
    const int nc = (sp.cnpages + p.chunk_pages - 1) / p.chunk_pages;
    const int c0 = sp.cpfirst + split * p.chunk_pages;
    const int c1 = min(sp.cpfirst + sp.cnpages, c0 + p.chunk_pages);
    const int pg0 = max(c0, sp.pfirst), pg1 = min(c1, sp.pfirst + sp.npages);
    const size_t bi = static_cast<size_t>(row) * p.Hq + i;
    if (c0 >= c1) {
        if (split == 0) {   // an empty sequence: out = 0, lse = -inf
            for (int e = lane; e < d; e += 32) p.out[bi * d + e] = 0.f;
            if (lane == 0 && p.lse != nullptr) p.lse[bi] = -INFINITY;
        }
        return;
    }
    if (pg0 >= pg1) {   // the chunk holds none of this row's keys: an empty partial
        for (int e = lane; e < d; e += 32) p.ws_o[(bi * p.splits + split) * d + e] = 0.f;
        if (lane == 0) p.ws_lse[bi * p.splits + split] = -INFINITY;
        return;
    }
    const int words = d / 8, G = words / lanes;
    const bool mine = j < words;
    float q[8], acc[8], qsum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q[e] = mine ? p.q[bi * d + j * 8 + e] : 0.f;
        qsum += q[e];
        acc[e] = 0.f;
    }
    float m_run = -INFINITY, l_run = 0.f;
    const int page_bytes = bs * (words * 4 + G * 4);
    for (int pg = pg0; pg < pg1; ++pg) {
        const int phys = __ldg(p.block_table + static_cast<size_t>(sp.b) * p.MBS + pg);
        const bool bad = phys < 0 || phys >= p.NB;
        if (bad && lane == 0) raise_error(p.err, PKV_DEVERR_BLOCK);
        const size_t base = bad ? 0 : (static_cast<size_t>(phys) * p.Hkv + kvh) * page_bytes;
        const uint32_t *kw = reinterpret_cast<const uint32_t *>(kc + base);
        const uint32_t *vw = reinterpret_cast<const uint32_t *>(vc + base);
        const int first = max(0, sp.lo - pg * bs), valid = min(bs, sp.len - pg * bs);
        for (int t0 = first; t0 < valid; t0 += KEYS) {
            const int t = t0 + slice;
            const bool see = t < valid, read = see && mine && !bad;
            uint32_t kcode = 0, vcode = 0;
            float2 kp = make_float2(0.f, 0.f), vp = kp;
            if (read) {
                kcode = __ldg(kw + t * words + j);
                vcode = __ldg(vw + t * words + j);
                kp = __half22float2(__ldg(reinterpret_cast<const __half2 *>(kw + bs * words) + t * G + j / lanes));
                vp = __half22float2(__ldg(reinterpret_cast<const __half2 *>(vw + bs * words) + t * G + j / lanes));
            }
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = fmaf(q[e], static_cast<float>((kcode >> (4 * e)) & 15u), dot);
            dot = read ? fmaf(dot, kp.x, qsum * kp.y) : 0.f;
#pragma unroll
            for (int sh = W / 2; sh > 0; sh >>= 1) dot += __shfl_xor_sync(kFull, dot, sh);
            const float s = see ? dot * p.scale_log2 : -INFINITY;
            const float m_new = fmaxf(m_run, s);
            const float alpha = m_run == -INFINITY ? 0.f : exp2f(m_run - m_new);
            const float w = see ? exp2f(s - m_new) : 0.f;
            l_run = l_run * alpha + w;
            const float ws = read ? w * vp.x : 0.f, wz = read ? w * vp.y : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[e] = fmaf(acc[e], alpha, fmaf(ws, static_cast<float>((vcode >> (4 * e)) & 15u), wz));
            m_run = m_new;
        }
    }
    // the slices' states, lanes j of every slice
    float M = m_run;
#pragma unroll
    for (int sh = W; sh < 32; sh <<= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, sh));
    const float f = m_run == -INFINITY ? 0.f : exp2f(m_run - M);
    float L = l_run * f;
#pragma unroll
    for (int sh = W; sh < 32; sh <<= 1) L += __shfl_xor_sync(kFull, L, sh);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        acc[e] *= f;
#pragma unroll
        for (int sh = W; sh < 32; sh <<= 1) acc[e] += __shfl_xor_sync(kFull, acc[e], sh);
    }
    float *dst = nc == 1 ? p.out + bi * d : p.ws_o + (bi * p.splits + split) * d;
    if (mine && slice == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[j * 8 + e] = acc[e] / L;
    }
    if (lane == 0) {
        const float lse2 = M + log2f(L);
        if (nc > 1) p.ws_lse[bi * p.splits + split] = lse2;
        else if (p.lse != nullptr) p.lse[bi] = lse2 * kDecLn2;
    }
}

// ============================================================== warp-MMA path
//
// attend_q4_mma_kernel (d 64 or 128, bs 16 or 32).  A unit is a tile of eight (query row, head)
// pairs of one sequence and KV head with the keys they see; a warp takes 32 keys at a time from a
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
//   from shared memory in pairs of keys.
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

constexpr int kMmaWarps = 4, kStageKeys = 32, kStages = 2;
constexpr int kUnitCost = 3;   // a unit's start (queries, first copies, its part written) in 32-key steps

template <int D, int BS, int G>
struct MmaCfg {
    static constexpr int WORDS = D / 8;              // code words per row
    static constexpr int PPS = kStageKeys / BS;      // pages per stage
    static constexpr int kCodeBytes = BS * D / 2;    // a page's codes; its parameters follow
    static constexpr int kPageBytes = BS * (D / 2 + 4 * G);
    static constexpr int kStageBytes = 2 * PPS * kPageBytes;   // K pages, then V pages
    static constexpr int kRingBytes = kMmaWarps * kStages * kStageBytes;
    static constexpr int kMergeBytes = kMmaWarps * 8 * (2 + D) * 4;
    static constexpr int kScanBytes = (kMaxBalanced + 1) * 4;
    static constexpr int kUsed = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kDataBytes = (kUsed > kScanBytes ? kUsed : kScanBytes) + 15 & ~15;
    static constexpr int kQOff = kDataBytes;                            // query fragments [warp][step][lane]
    static constexpr int kQBytes = (D / 16) * 512;
    static constexpr int kParOff = kQOff + kMmaWarps * kQBytes;         // [warp][group][scale, zero][key]
    static constexpr int kParBytes = G * 2 * kStageKeys * 4;
    static constexpr int kBarOff = kParOff + kMmaWarps * kParBytes;
    static constexpr int kSmemBytes = kBarOff + kMmaWarps * kStages * 8;
    // Three blocks (12 warps, 168 registers a thread) against four (128, with spills): 70B-shaped step
    // 91.4 against 94.2 us, MHA step 76.4 against 79.0, four sequences of 131072 tokens 142 against 139.
    static constexpr int kBlocksPerSm = 3;
    static_assert(kBlocksPerSm * (kSmemBytes + 2048) <= 228 * 1024, "three blocks fit an SM");
    static_assert(kPageBytes % 16 == 0, "bulk copies");
};

// D = A(16x16, f16, row) * B(16x8, f16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with C = 0, so that no registers are cleared first.
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void ldsm_x2_trans(uint32_t addr, uint32_t &r0, uint32_t &r1) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr));
}

// The warps' states of a tile's eight rows, in shared memory ([NW][8] references and sums, then
// [NW][8][D] outputs), merged and written: the result where the unit has one part, else this
// normalised part; with arrival counters the unit's last part merges them all.
template <int D, int NW>
__device__ __forceinline__ void finish_rows(uint8_t *smem, const AttendQ4Params &P, const RowSpan *rows, const Parts &u) {
    const DecodeKParams &p = P.k;
    float *mw = reinterpret_cast<float *>(smem);
    float *lw = mw + NW * 8;
    float *ow = lw + NW * 8;
    for (int idx = threadIdx.x; idx < 8 * (D / 4); idx += NW * 32) {
        const int h = idx / (D / 4), c = idx % (D / 4) * 4;
        if (rows[h].bi < 0) continue;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, mw[w * 8 + h]);
        const float base = M == -INFINITY ? 0.f : M;   // the row sees none of this part's keys
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2f(mw[w * 8 + h] - base);
            const float4 o = *reinterpret_cast<const float4 *>(ow + (w * 8 + h) * D + c);
            L += lw[w * 8 + h] * f;
            acc.x += o.x * f;
            acc.y += o.y * f;
            acc.z += o.z * f;
            acc.w += o.w * f;
        }
        const float inv = M == -INFINITY ? 0.f : 1.f / L;
        const float4 r = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const float lse2 = M == -INFINITY ? -INFINITY : M + log2f(L);
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
    for (int idx = threadIdx.x; idx < 8 * (D / 4); idx += NW * 32) {
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
__device__ __forceinline__ size_t part_at(const Parts &u, int h, int i) {
    return (static_cast<size_t>(u.first + i) * 2 + (i == 0)) * 8 + h;
}

// The last warp to arrive merges a balanced unit's parts: lane l holds row l % 8 of every fourth
// part's weight, and every lane four columns of all rows.
template <int D>
__device__ __forceinline__ void merge_unit(const AttendQ4Params &P, const RowSpan &me, const Parts &u, int lane) {
    const DecodeKParams &p = P.k;
    const int row = lane & 7, sub = lane >> 3, col = lane * 4;
    float M = -INFINITY, L = 0.f;
    for (int i = sub; i < u.n; i += 4) M = fmaxf(M, __ldcg(p.ws_lse + part_at(u, row, i)));
    M = fmaxf(M, __shfl_xor_sync(kFull, M, 8));
    M = fmaxf(M, __shfl_xor_sync(kFull, M, 16));
    const float base = M == -INFINITY ? 0.f : M;   // a row past the sequence's last
    float4 acc[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < u.n; i0 += 4) {
        const float w = i0 + sub < u.n ? exp2f(__ldcg(p.ws_lse + part_at(u, row, i0 + sub)) - base) : 0.f;
        L += w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (i0 + j >= u.n) break;
            const float *src = p.ws_o + part_at(u, 0, i0 + j) * D + col;
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float f = __shfl_sync(kFull, w, j * 8 + h);
                const float4 o = col < D ? __ldcg(reinterpret_cast<const float4 *>(src + h * D)) : make_float4(0.f, 0.f, 0.f, 0.f);
                acc[h].x = fmaf(f, o.x, acc[h].x);
                acc[h].y = fmaf(f, o.y, acc[h].y);
                acc[h].z = fmaf(f, o.z, acc[h].z);
                acc[h].w = fmaf(f, o.w, acc[h].w);
            }
        }
    }
    L += __shfl_xor_sync(kFull, L, 8);
    L += __shfl_xor_sync(kFull, L, 16);
    const int bi = __shfl_sync(kFull, me.bi, row * 4);   // lane 4 * r holds row r's
    if (lane < 8 && bi >= 0 && p.lse != nullptr) p.lse[bi] = (M + log2f(L)) * kDecLn2;
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        const float inv = 1.f / __shfl_sync(kFull, L, h);
        const int at = __shfl_sync(kFull, bi, h);
        if (at >= 0 && col < D)
            *reinterpret_cast<float4 *>(p.out + static_cast<size_t>(at) * D + col) =
                make_float4(acc[h].x * inv, acc[h].y * inv, acc[h].z * inv, acc[h].w * inv);
    }
}

// Words per thread and group of `N` consecutive 32-bit words from shared memory.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x, w[1] = u.y;
    } else if constexpr (N == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p), v = *reinterpret_cast<const uint4 *>(p + 16);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w, w[4] = v.x, w[5] = v.y, w[6] = v.z, w[7] = v.w;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
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

template <int D, int BS, int G>
__global__ void __launch_bounds__(kMmaWarps * 32, (MmaCfg<D, BS, G>::kBlocksPerSm))
    attend_q4_mma_kernel(const __grid_constant__ AttendQ4Params P) {
    using Cfg = MmaCfg<D, BS, G>;
    constexpr int NW = kMmaWarps, NT = kStageKeys / 8, PPS = Cfg::PPS, WORDS = Cfg::WORDS;
    constexpr int WPT = WORDS / (4 * G);         // K: words per lane and group
    constexpr int HPG = D / 32 / G;              // V: 32-dimension columns per group
    static_assert(WPT >= 1 && HPG >= 1, "a group has at least 32 elements");
    const DecodeKParams &p = P.k;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ RowSpan s_rows[8];   // chunks: the tile's rows

    pdl_launch_dependents();   // a merge kernel after this one waits for the whole grid
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kBarOff) + warp * kStages;
    uint8_t *ring = smem + warp * kStages * Cfg::kStageBytes;
    uint4 *qfrag = reinterpret_cast<uint4 *>(smem + Cfg::kQOff + warp * Cfg::kQBytes) + lane;   // [step][lane]
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
            const int n = sq.pages > 0 ? p.Hkv * ((sq.nq * p.m + 7) / 8) : 0;
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
        __syncthreads();   // the scan's memory becomes the ring
    }

    while (x < x1) {
        // ---- the next segment: a unit and its pages [c0, c1)
        int kvh, tile, c0, c1, turn = 0, turns = 1;   // this warp takes every turns-th step from turn on
        Parts part{};
        SeqRows sq;
        if (P.balanced) {
            sq = seq_rows(P, b, BS, false);
            int units = p.Hkv * ((sq.nq * p.m + 7) / 8);
            while (sq.pages == 0 || unit == units) {   // on to the next sequence that has keys
                ++b;
                unit = 0;
                sq = seq_rows(P, b, BS, false);
                units = p.Hkv * ((sq.nq * p.m + 7) / 8);
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
            if (!sq.ok || 8 * tile >= sq.nq * p.m) return;
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
            if (threadIdx.x < 8) s_rows[threadIdx.x] = tile_row(P, sq, kvh, 8 * tile + threadIdx.x);
        }
        const RowSpan t_first = tile_row(P, sq, kvh, 8 * tile), t_last = tile_row(P, sq, kvh, min(8 * tile + 7, sq.nq * p.m - 1));
        const RowSpan me = tile_row(P, sq, kvh, 8 * tile + g);
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
        float qv[G * WPT][8];
#pragma unroll
        for (int u = 0; u < G * WPT; ++u) {
            const float2 *src = reinterpret_cast<const float2 *>(p.q + static_cast<size_t>(max(me.bi, 0)) * D +
                                                                 8 * ((u / WPT) * (WORDS / G) + t4 * WPT + u % WPT));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = me.bi >= 0 ? __ldg(src + e) : make_float2(0.f, 0.f);
                qv[u][2 * e] = y.x;
                qv[u][2 * e + 1] = y.y;
            }
        }

        // ---- this warp's stages: steps of PPS pages turn, turn + turns, ... of [pg0, pg1)
        const int steps = pg1 > pg0 ? (pg1 - pg0 + PPS - 1) / PPS : 0;
        const int n_my = steps > turn ? (steps - turn + turns - 1) / turns : 0;
        const int32_t *tbl = p.block_table + static_cast<size_t>(b) * p.MBS;
        int tcur[PPS], tnext[PPS];
        auto load_ids = [&](int k, int (&t)[PPS]) {
#pragma unroll
            for (int i = 0; i < PPS; ++i) {
                const int pg = pg0 + (turn + k * turns) * PPS + i;
                t[i] = k < n_my && pg < pg1 ? __ldg(tbl + pg) : -1;
            }
        };
        load_ids(lane, tcur);
        load_ids(32 + lane, tnext);
        int tbase = 0;
        auto issue = [&](int k) {   // the whole warp
            while (k >= tbase + 32) {
                tbase += 32;
#pragma unroll
                for (int i = 0; i < PPS; ++i) tcur[i] = tnext[i];
                load_ids(tbase + 32 + lane, tnext);
            }
            const int st = (cnt + k) % kStages;
            const uint32_t bar = smem_addr(&bars[st]);
            // lane l: copy l of the stage's 2 * PPS (K pages, then V pages)
            const int i = lane % PPS, pg = pg0 + (turn + k * turns) * PPS + i;
            int phys = __shfl_sync(kFull, tcur[0], k & 31);
            if (PPS == 2) {
                const int second = __shfl_sync(kFull, tcur[PPS - 1], k & 31);
                if (i == 1) phys = second;
            }
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
        };
        int issued = min(kStages, n_my);
        for (int k = 0; k < issued; ++k) issue(k);

        // ---- query fragments, while the copies fly.  MMA steps 2u and 2u + 1 of word u = gi * WPT + i:
        // elements 8 * word + {0, 4}, {2, 6}, and their odd neighbours / 16
        float f, qsum[G];   // score (base 2) = MMA sum * f; the groups' sums of q in the MMAs' units
        {
            float(&v)[G * WPT][8] = qv, amax = 0.f;
#pragma unroll
            for (int u = 0; u < G * WPT; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[u][e]));
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
            // |q| * 2^up in [2^13, 2^14); a row of zeros (or of subnormals) keeps the factor finite
            const int up = min(13 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), 126);
            const float scale = pow2i(up);
            f = (p.scale_log2 * 0x1p24f) * pow2i(-up);
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < WPT; ++i) {
                    const int u = gi * WPT + i;
                    uint4 e, o;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[u][j] *= scale;
                        sum += v[u][j];
                    }
#pragma unroll
                    for (int j = 1; j < 8; j += 2) v[u][j] *= 0.0625f;
                    split2(v[u][0], v[u][4], e.x, e.y);
                    split2(v[u][2], v[u][6], e.z, e.w);
                    split2(v[u][1], v[u][5], o.x, o.y);
                    split2(v[u][3], v[u][7], o.z, o.w);
                    qfrag[(2 * u) * 32] = e;
                    qfrag[(2 * u + 1) * 32] = o;
                }
                sum += __shfl_xor_sync(kFull, sum, 1);
                sum += __shfl_xor_sync(kFull, sum, 2);
                qsum[gi] = sum * 0x1p-24f;
            }
        }

        float oT[D / 16][4];
        float2 zo[G];   // sums of weight * zero over this lane's keys
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) oT[mt][0] = oT[mt][1] = oT[mt][2] = oT[mt][3] = 0.f;
#pragma unroll
        for (int gi = 0; gi < G; ++gi) zo[gi] = make_float2(0.f, 0.f);
        float m_run = -INFINITY, l_run = 0.f;   // the running max, and l relative to `ref`
        float ref = -INFINITY;                  // m_run + E - 14
        float vs_max = 0.f, vs_exp = -24.f;     // the largest V scale seen; E, its exponent rounded up

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
            const int par_at = (lane / BS) * Cfg::kPageBytes + Cfg::kCodeBytes + (lane % BS) * G * 4;
            auto widen = [&](const uint8_t *pages, float centred) {
                uint32_t v[G];
                lds_words<G>(pages + par_at, v);
                float top = 0.f;
#pragma unroll
                for (int gi = 0; gi < G; ++gi) {
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&v[gi]));
                    par[gi * 64 + lane] = seen ? y.x : 0.f;
                    par[gi * 64 + 32 + lane] = seen ? fmaf(centred, y.x, y.y) : 0.f;
                    top = fmaxf(top, seen ? y.x : 0.f);
                }
                return top;
            };

            // ---- scores of row g for keys 8 * nt + 2 * t4 + {0, 1}
            widen(kpages, 0.f);
            __syncwarp();
            float2 s[NT];
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                float a[NT][4];
                uint32_t c[NT][WPT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    lds_words<WPT>(kpages + (nt * 8 / BS) * Cfg::kPageBytes + (nt * 8 % BS + g) * (D / 2) + gi * (D / 2 / G) +
                                       t4 * WPT * 4,
                                   c[nt]);
                }
#pragma unroll
                for (int i = 0; i < WPT; ++i) {
                    const uint4 e = qfrag[(2 * (gi * WPT + i)) * 32], o = qfrag[(2 * (gi * WPT + i) + 1) * 32];
                    // the tiles' chains side by side
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t x = c[nt][i] & 0x000f000fu, y = (c[nt][i] >> 8) & 0x000f000fu;
                        if (i == 0) mma16_first(a[nt], e.x, e.y, e.z, e.w, x, y);
                        else mma16(a[nt], e.x, e.y, e.z, e.w, x, y);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16(a[nt], o.x, o.y, o.z, o.w, c[nt][i] & 0x00f000f0u, (c[nt][i] >> 8) & 0x00f000f0u);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 sc = *reinterpret_cast<const float2 *>(par + gi * 64 + nt * 8 + 2 * t4);
                    const float2 ze = *reinterpret_cast<const float2 *>(par + gi * 64 + 32 + nt * 8 + 2 * t4);
                    const float2 qz = make_float2(qsum[gi], qsum[gi]);
                    const float2 y = gi == 0 ? mul2(ze, qz) : fma2(ze, qz, s[nt]);
                    s[nt] = fma2(sc, add2(make_float2(a[nt][0], a[nt][1]), make_float2(a[nt][2], a[nt][3])), y);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt] = mul2(s[nt], make_float2(f, f));
            if (!whole) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int tok = tok0 + nt * 8 + 2 * t4, end = min(me.len, tok_end);
                    if (tok < me.lo || tok >= end) s[nt].x = -INFINITY;
                    if (tok + 1 < me.lo || tok + 1 >= end) s[nt].y = -INFINITY;
                }
            }
            __syncwarp();   // K's parameters have been read

            // ---- the running reference: the rows' maxima and the largest V scale
            const float top = widen(vpages, 8.f);
            float mx = fmaxf(s[0].x, s[0].y);
#pragma unroll
            for (int nt = 1; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt].x, s[nt].y));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
            m_run = fmaxf(m_run, mx);
            if (__any_sync(kFull, top > vs_max)) {   // rarely after the first stage: the next power of two
                // non-negative floats order like their bits
                vs_max = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(fmaxf(top, vs_max))));
                vs_exp = fmaxf(static_cast<float>(static_cast<int>((__float_as_uint(vs_max) + 0x7fffffu) >> 23) - 127), -24.f);
            }
            const float ref_new = m_run + (vs_exp - 14.f);
            // a row that has seen no key yet has ref -inf: its weights are 0 whatever the base
            const float base = ref_new == -INFINITY ? 0.f : ref_new;
            const float alpha = ref == -INFINITY ? 1.f : ex2_approx(ref - base);   // nothing to rescale yet
            ref = ref_new;
            float2 psum = make_float2(0.f, 0.f), w[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 e = add2(s[nt], make_float2(-base, -base));
                w[nt] = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                psum = add2(psum, w[nt]);
            }
            l_run = l_run * alpha + (psum.x + psum.y);
            const float2 rescale = make_float2(__shfl_sync(kFull, alpha, 8 * t4), __shfl_sync(kFull, alpha, 8 * t4 + 4));
#pragma unroll
            for (int gi = 0; gi < G; ++gi) zo[gi] = mul2(zo[gi], make_float2(alpha, alpha));
            __syncwarp();   // V's parameters have been written

            // ---- O^T = O^T alpha + V^T P^T, 16 keys per step.  ldmatrix with transposition over 16-bit
            // units (four codes of a key) hands lane (g, t4) the units 8 * c + g of keys 2 * t4, 2 * t4 + 1
            // in one register: the pairs along the keys that the A operand wants
            constexpr int KT = kStageKeys / 16, N = HPG >= 2 ? 2 : 1;   // N columns of 32 dimensions at a time
            const uint32_t vrow = smem_addr(vpages) + (lane & 15) * (D / 2) + (HPG >= 2 ? (lane >> 4) * 16 : 0);
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                uint32_t ph[KT][2], pl[KT][2];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const float *src = par + gi * 64 + kt * 16 + 2 * t4;
                    const float2 wa = w[2 * kt], wb = w[2 * kt + 1];
                    split2(mul2(wa, *reinterpret_cast<const float2 *>(src)), ph[kt][0], pl[kt][0]);
                    split2(mul2(wb, *reinterpret_cast<const float2 *>(src + 8)), ph[kt][1], pl[kt][1]);
                    zo[gi] = fma2(wa, *reinterpret_cast<const float2 *>(src + 32),
                                  fma2(wb, *reinterpret_cast<const float2 *>(src + 40), zo[gi]));
                }
#pragma unroll
                for (int h = 0; h < HPG; h += N) {
                    const int c = gi * HPG + h;
                    float sum[2 * N][4];   // even and odd elements of each column
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        // registers: units 8 * c of keys 0..7, of keys 8..15, units 8 * (c + 1) likewise
                        const uint32_t rows = vrow + (kt * 16 / BS) * Cfg::kPageBytes + (kt * 16 % BS) * (D / 2) + c * 16;
                        uint32_t v[4], e[2 * N][2], o[2 * N][2];
                        if constexpr (N == 2) ldsm_x4_trans(rows, v[0], v[1], v[2], v[3]);
                        else ldsm_x2_trans(rows, v[0], v[1]);
#pragma unroll
                        for (int i = 0; i < 2 * N; ++i) {
                            centre(v[i], e[i][0], o[i][0]);
                            centre(v[i] >> 8, e[i][1], o[i][1]);
                        }
#pragma unroll
                        for (int lo = 0; lo < 2; ++lo) {   // the weights' high parts, then their low ones
                            const uint32_t b0 = lo ? pl[kt][0] : ph[kt][0], b1 = lo ? pl[kt][1] : ph[kt][1];
#pragma unroll
                            for (int i = 0; i < N; ++i) {
                                if (kt == 0 && lo == 0) {
                                    mma16_first(sum[2 * i], e[2 * i][0], e[2 * i][1], e[2 * i + 1][0], e[2 * i + 1][1], b0, b1);
                                    mma16_first(sum[2 * i + 1], o[2 * i][0], o[2 * i][1], o[2 * i + 1][0], o[2 * i + 1][1], b0, b1);
                                } else {
                                    mma16(sum[2 * i], e[2 * i][0], e[2 * i][1], e[2 * i + 1][0], e[2 * i + 1][1], b0, b1);
                                    mma16(sum[2 * i + 1], o[2 * i][0], o[2 * i][1], o[2 * i + 1][0], o[2 * i + 1][1], b0, b1);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i)
#pragma unroll
                        for (int r = 0; r < 4; r += 2) {
                            float(&acc)[4] = oT[2 * c + i];
                            const float2 y = fma2(make_float2(acc[r], acc[r + 1]), rescale, make_float2(sum[i][r], sum[i][r + 1]));
                            acc[r] = y.x;
                            acc[r + 1] = y.y;
                        }
                }
            }
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

        l_run += __shfl_xor_sync(kFull, l_run, 1);
        l_run += __shfl_xor_sync(kFull, l_run, 2);
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            zo[gi].x += zo[gi].y;
            zo[gi].x += __shfl_xor_sync(kFull, zo[gi].x, 1);
            zo[gi].x += __shfl_xor_sync(kFull, zo[gi].x, 2);
        }
        // this lane's outputs of rows 2 * t4 + r: dimensions 32 * c + 4 * g + {0, 1, 2, 3}
        auto outputs = [&](int c, int r) {
            const float z = __shfl_sync(kFull, zo[c / HPG].x, 8 * t4 + 4 * r);
            const float (&e)[4] = oT[2 * c], (&o)[4] = oT[2 * c + 1];
            return make_float4(fmaf(e[r], 0x1p9f, z), fmaf(o[r], 0x1p9f, z), fmaf(e[2 + r], 0x1p9f, z), fmaf(o[2 + r], 0x1p9f, z));
        };

        if (P.balanced) {
            if (gave_up) return;   // lanes together; the block's other warps go on
            const float inv = ref == -INFINITY ? 0.f : 1.f / l_run;   // no key of this part for the row
            const float lse2 = ref == -INFINITY ? -INFINITY : ref + log2f(l_run);
            if (t4 == 0 && me.bi >= 0) {
                if (part.n > 1) p.ws_lse[part_at(part, g, part.own)] = lse2;
                else if (p.lse != nullptr) p.lse[me.bi] = lse2 * kDecLn2;
            }
            if (t4 == 0 && me.bi < 0 && part.n > 1) p.ws_lse[part_at(part, g, part.own)] = -INFINITY;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float il = __shfl_sync(kFull, inv, 8 * t4 + 4 * r);
                const int bi = __shfl_sync(kFull, me.bi, 8 * t4 + 4 * r);
                float *dst = part.n > 1 ? p.ws_o + part_at(part, 2 * t4 + r, part.own) * D
                                        : p.out + static_cast<size_t>(max(bi, 0)) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const float4 y = outputs(c, r);
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
                    merge_unit<D>(P, me, part, lane);
                }
            }
            continue;
        }

        // ---- the warps' (ref, l, O) through shared memory (the ring is free now)
        if (__syncthreads_or(gave_up)) return;
        float *mw = reinterpret_cast<float *>(smem);
        float *lw = mw + NW * 8;
        float *ow = lw + NW * 8;
        if (t4 == 0) {
            mw[warp * 8 + g] = ref;
            lw[warp * 8 + g] = l_run;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
                *reinterpret_cast<float4 *>(ow + (warp * 8 + 2 * t4 + r) * D + 32 * c + 4 * g) = outputs(c, r);
        __syncthreads();
        finish_rows<D, NW>(smem, P, s_rows, part);
    }
}

template <int D, int BS, int G>
cudaError_t launch_mma_as(const AttendQ4Params &P, dim3 grid, cudaStream_t stream) {
    using Cfg = MmaCfg<D, BS, G>;
    static std::atomic<unsigned long long> done{0};
    auto kernel = attend_q4_mma_kernel<D, BS, G>;
    const cudaError_t e = set_smem_once(kernel, Cfg::kSmemBytes, done);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kMmaWarps * 32, Cfg::kSmemBytes, stream>>>(P);
    return cudaGetLastError();
}

cudaError_t launch_mma(const AttendQ4Params &P, int d, int bs, int G, dim3 grid, cudaStream_t stream) {
    if (bs == 16) {
        if (d == 64) return G == 1 ? launch_mma_as<64, 16, 1>(P, grid, stream) : launch_mma_as<64, 16, 2>(P, grid, stream);
        return G == 1   ? launch_mma_as<128, 16, 1>(P, grid, stream)
               : G == 2 ? launch_mma_as<128, 16, 2>(P, grid, stream)
                        : launch_mma_as<128, 16, 4>(P, grid, stream);
    }
    if (d == 64) return G == 1 ? launch_mma_as<64, 32, 1>(P, grid, stream) : launch_mma_as<64, 32, 2>(P, grid, stream);
    return G == 1   ? launch_mma_as<128, 32, 1>(P, grid, stream)
           : G == 2 ? launch_mma_as<128, 32, 2>(P, grid, stream)
                    : launch_mma_as<128, 32, 4>(P, grid, stream);
}

cudaError_t launch_simt(const AttendQ4Args &a, const DecodeKParams &kp, cudaStream_t stream) {
    const long long units = static_cast<long long>(a.rows) * a.Hq;
    const dim3 grid(static_cast<unsigned>((units + 3) / 4), static_cast<unsigned>(kp.splits));
    const int words = a.d / 8, lanes = a.group / 8;
#define PKV_Q4_SIMT(WW) attend_q4_simt_kernel<WW><<<grid, 128, 0, stream>>>(a.k_cache, a.v_cache, kp, a.d, a.bs, lanes, a.rows)
    if (words <= 4) PKV_Q4_SIMT(4);
    else if (words <= 8) PKV_Q4_SIMT(8);
    else if (words <= 16) PKV_Q4_SIMT(16);
    else PKV_Q4_SIMT(32);
#undef PKV_Q4_SIMT
    return cudaGetLastError();
}

// Units with at most this many chunks merge in the attention kernel.
constexpr int kFusedMergeMaxChunks = 8;

size_t partial_bytes(long long rows, int Hq, int splits, int d) {
    return splits > 1 ? PKV_DECODE_COUNTER_BYTES +
                            static_cast<size_t>(rows) * Hq * splits * (static_cast<size_t>(d) + 1) * sizeof(float)
                      : 0;
}

}  // namespace

namespace {
int q4_blocks_per_sm(int d, int bs, int G) {
    if (bs == 16) {
        if (d == 64) return G == 1 ? MmaCfg<64, 16, 1>::kBlocksPerSm : MmaCfg<64, 16, 2>::kBlocksPerSm;
        return G == 1 ? MmaCfg<128, 16, 1>::kBlocksPerSm : G == 2 ? MmaCfg<128, 16, 2>::kBlocksPerSm : MmaCfg<128, 16, 4>::kBlocksPerSm;
    }
    if (d == 64) return G == 1 ? MmaCfg<64, 32, 1>::kBlocksPerSm : MmaCfg<64, 32, 2>::kBlocksPerSm;
    return G == 1 ? MmaCfg<128, 32, 1>::kBlocksPerSm : G == 2 ? MmaCfg<128, 32, 2>::kBlocksPerSm : MmaCfg<128, 32, 4>::kBlocksPerSm;
}
// (Query row, head) pairs of a sequence and KV head that the warp-MMA kernel, which takes eight at a
// time, is faster for than the tcgen05 kernel, whose time hardly depends on them.  4 x 65536 tokens, one
// scale group a row: 24 pairs 37.3 us, the tcgen05 kernel 34.0 (32 pairs); 64 x 2048 tokens, four KV heads:
// 66.5 and 74.1.  Two groups: 32 pairs 48.7 us, 40 58.7, the tcgen05 kernel 47.5 (40 pairs); 87.3, 105.4
// and 100.9 (64 x 2048).
int q4_mma_slots(int G) { return G == 1 ? 24 : 32; }

// Rows of partial results of a balanced launch: two units for every warp or block.
size_t balanced_rows(const Q4Plan &plan) {
    return static_cast<size_t>(plan.blocks) * 2 * (plan.umma ? kQ4UmmaSlots : kMmaWarps * 8);
}
}  // namespace

Q4Plan plan_attend_q4(int B, int rows, int max_q, int Hq, int Hkv, int d, int group, int bs, int pages,
                      int num_splits, int sm_count, bool aligned) {
    Q4Plan plan{};
    const int m = Hq / Hkv, sms = std::max(sm_count, 1);
    const long long slots = static_cast<long long>(max_q) * m;
    plan.umma = q4_umma_shape(d, group, bs) && aligned && slots > q4_mma_slots(d / group) && slots < (1 << 20);
    plan.mma = !plan.umma && (d == 64 || d == 128) && (bs == 16 || bs == 32) && d / group <= 4 && aligned && slots < (1 << 20);
    const int per_tile = plan.umma ? kQ4UmmaSlots : 8;
    plan.tiles = plan.umma || plan.mma ? static_cast<int>((slots + per_tile - 1) / per_tile) : 1;
    const long long units = plan.umma || plan.mma ? static_cast<long long>(B) * Hkv * plan.tiles : static_cast<long long>(rows) * Hq;
    int chunk = pages;
    if (num_splits > 1) {
        chunk = (pages + num_splits - 1) / num_splits;
    } else if (num_splits == 0 && (plan.umma || plan.mma)) {
        // An equal share for every warp (umma: block) the device holds at once, unless the units are
        // so few that one would be left to merge parts from many: then, or with more sequences than a
        // block scans, equal chunks for one wave of blocks and a merge over many blocks.
        const int step = plan.umma ? 128 / (d / group) : kStageKeys;
        plan.blocks = plan.umma ? sms : q4_blocks_per_sm(d, bs, d / group) * sms;
        plan.balanced = B <= kMaxBalanced && (plan.umma ? plan.blocks <= 8 * units : plan.blocks * kMmaWarps <= 24 * units) &&
                        units * (static_cast<long long>(pages) * bs / step + 1 + kUnitCost) < (1ll << 30);
        const int least = 256 / bs;
        const long long per_unit = std::max(1ll, plan.blocks / std::max(units, 1ll));
        chunk = static_cast<int>(std::max<long long>(least, (pages + per_unit - 1) / per_unit));
    } else if (num_splits == 0) {
        // one warp per (row, head, chunk): several warps for each scheduler, no chunk shorter
        // than 128 keys
        const int least = std::max(1, 128 / bs);
        while (chunk > least && units * ((pages + chunk - 1) / chunk) < 32ll * sms) chunk = (chunk + 1) / 2;
    }
    chunk = std::max(chunk, (pages + kDecodeMaxChunks - 1) / kDecodeMaxChunks);
    if (plan.umma) {   // whole key tiles
        const int per = 128 / (d / group) / bs;
        chunk = (chunk + per - 1) / per * per;
    }
    plan.chunk_pages = std::max(chunk, 1);
    plan.splits = (pages + plan.chunk_pages - 1) / plan.chunk_pages;
    if (plan.balanced) {
        plan.splits = 1;   // the parts' number is known on the device only
        plan.workspace_bytes = PKV_DECODE_COUNTER_BYTES + balanced_rows(plan) * (d + 1) * sizeof(float);
        return plan;
    }
    plan.fused_merge = plan.mma && plan.splits > 1 && plan.splits <= kFusedMergeMaxChunks &&
                       units <= static_cast<long long>(PKV_DECODE_COUNTER_BYTES / sizeof(unsigned));
    plan.workspace_bytes = partial_bytes(rows, Hq, plan.splits, d);
    return plan;
}

bool q4_fuses_append(const Q4Plan &plan) { return plan.mma && plan.tiles == 1; }

cudaError_t launch_attend_q4(const AttendQ4Args &a, const Q4Plan &plan, cudaStream_t stream) {
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
    kp.cu_q = a.cu_q;
    if (plan.workspace_bytes > 0) {
        uint8_t *ws = static_cast<uint8_t *>(a.workspace);
        const size_t parts = plan.balanced ? balanced_rows(plan)
                                           : static_cast<size_t>(a.rows) * a.Hq * plan.splits;
        kp.ws_o = reinterpret_cast<float *>(ws + PKV_DECODE_COUNTER_BYTES);
        kp.ws_lse = kp.ws_o + parts * a.d;
    }
    cudaError_t e;
    if (plan.mma || plan.umma) {
        AttendQ4Params P{};
        kp.head_tiles = plan.tiles;
        if (plan.fused_merge || plan.balanced) kp.counters = static_cast<unsigned *>(a.workspace);
        if (a.new_slots != nullptr) {
            kp.k_new = a.k_new;
            kp.v_new = a.v_new;
            kp.new_slots = a.new_slots;
            P.new_bf16 = a.new_dt == PKV_BF16;
        }
        P.k = kp;
        P.kc = const_cast<uint8_t *>(a.k_cache);   // written only for a step's new tokens
        P.vc = const_cast<uint8_t *>(a.v_cache);
        P.rows = a.rows;
        P.max_q = a.max_q;
        P.balanced = plan.balanced;
        const dim3 grid = plan.balanced ? dim3(plan.blocks) : dim3(static_cast<unsigned>(plan.splits) * plan.tiles, a.Hkv, a.B);
        e = plan.umma ? launch_attend_q4_umma(P, a.d, a.bs, a.d / a.group, grid, stream)
                      : launch_mma(P, a.d, a.bs, a.d / a.group, grid, stream);
    } else {
        e = launch_simt(a, kp, stream);
    }
    if (e != cudaSuccess || plan.splits == 1 || plan.fused_merge) return e;
    return launch_decode_merge(kp, a.d, a.bs, static_cast<unsigned>(a.rows * a.Hq), stream);
}

}  // namespace pkv
