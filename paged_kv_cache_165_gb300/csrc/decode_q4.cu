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

#include "common.cuh"
#include "decode_kparams.cuh"
#include "internal.h"
#include "q4_codes.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct AttendQ4Params {
    DecodeKParams k;     // head_tiles: tiles of eight (query row, head) pairs per sequence and KV head
    uint8_t *kc, *vc;
    int rows, max_q;     // query rows of the call, and of a sequence at most
    int new_bf16;        // type of the step's new rows
};

template <typename Kernel>
cudaError_t set_smem_once(Kernel kernel, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    return cudaSuccess;
}

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
// attend_q4_mma_kernel (d 64 or 128, bs 16 or 32): one CTA per (sequence, KV head, tile of eight
// query rows x heads, chunk of blocks); four warps take 32 keys at a time, each with a private
// ring of bulk copies (a page is one contiguous run).  Per 32 keys and warp, with m16n8k16 f16
// MMAs and fp32 accumulators:
//   A code c in 0..15 placed in the low bits of an f16 is the subnormal c * 2^-24, and shifted
//   left by four bits it is c * 2^-20: both exact, so two masks turn a word of eight codes into
//   four f16 pairs (three logic operations and a shift per pair of pairs) with no conversion.
//   scores S (rows: 8 query rows hi, 8 lo; 8 keys per tile): q is scaled by a power of two per
//     row and enters as f16 hi + lo (2^-22 relative); the head dimension is taken in the order in
//     which the masks deliver the codes, each group in MMA steps of its own so that its scale
//     multiplies the sum; the zeros' term, sum_g zero_g * sum(q in g), is one k8 MMA whose B
//     operand is the (scale, zero) pairs as they lie in the page against A = (0, sum q).
//   output O^T = V^T P^T: V^T is the A operand (16 dimensions x 16 keys), words of two keys paired
//     by byte permutes; P^T is what the lane already holds for its row, times the group's scale,
//     as f16 hi + lo.  The zeros' term is summed in fp32.
// The f16 range of the weights: p * scale is kept below 2^14 by shifting the softmax reference by
// the largest scale seen so far, E = ceil(log2 max scale): w = 2^(s - m - E + 14); l, O and the
// zeros' term carry the same factor, which cancels, and a growing E rescales like a growing max.

constexpr int kMmaWarps = 4, kStageKeys = 32, kStages = 2;

template <int D, int BS, int G>
struct MmaCfg {
    static constexpr int WORDS = D / 8;              // code words per row
    static constexpr int PPS = kStageKeys / BS;      // pages per stage
    static constexpr int kCodeBytes = BS * D / 2;    // a page's codes; its parameters follow
    static constexpr int kPageBytes = BS * (D / 2 + 4 * G);
    static constexpr int kStageBytes = 2 * PPS * kPageBytes;   // K pages, then V pages
    static constexpr int kRingBytes = kMmaWarps * kStages * kStageBytes;
    static constexpr int kMergeBytes = kMmaWarps * 8 * (2 + D) * 4;
    static constexpr int kDataBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kQOff = kDataBytes;          // query fragments, the sums' ones, the rows' factors
    static constexpr int kBarOff = kQOff + (D / 16) * 512 + 256 + 32;
    static constexpr int kSmemBytes = kBarOff + kMmaWarps * kStages * 8;
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
__device__ __forceinline__ void mma8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0));
}

// x ~= hi + lo, hi = rn_f16(x), lo = rn_f16(x - hi); the low half holds x.x.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x.x, x.y);
    const float2 f = __half22float2(h);
    const float2 r = add2(x, make_float2(-f.x, -f.y));
    const __half2 l = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    split2(make_float2(x0, x1), hi, lo);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ void ldsm_x2_trans(uint32_t addr, uint32_t &r0, uint32_t &r1) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr));
}

__device__ __forceinline__ float2 par_of(uint32_t u) {   // (scale, zero)
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
__device__ __forceinline__ float scale_of(uint32_t u) {
    return __low2float(*reinterpret_cast<const __half2 *>(&u));
}

// 2^e as a float, e clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) {
    return __uint_as_float(static_cast<uint32_t>(min(max(e, -126), 127) + 127) << 23);
}

// A sequence's query rows r0 .. r0 + nq - 1 (checked), its length L and the pages [first, first +
// pages) that any of them sees; rows [z0, z1) see nothing and are written as out = 0, lse = -inf.
struct SeqRows {
    int r0, nq, L, first, pages, z0, z1, z2, z3;
    bool ok;
};

__device__ __forceinline__ SeqRows seq_rows(const AttendQ4Params &P, int b, int bs, bool report) {
    const DecodeKParams &p = P.k;
    SeqRows s{};
    s.L = checked_len(p, b, bs, report);
    s.ok = true;
    if (p.cu_q == nullptr) {
        s.r0 = b;
        s.nq = 1;
        if (s.L == 0) s.z0 = b, s.z1 = b + 1;
    } else {
        const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1);
        s.r0 = c0;
        s.nq = c1 - c0;
        s.ok = c0 >= 0 && c1 >= c0 && c1 <= P.rows && s.nq <= s.L && s.nq <= P.max_q;
        if (!s.ok) s.z0 = min(max(c0, 0), P.rows), s.z1 = min(max(c1, 0), P.rows);
        // rows before the first sequence or behind the last one belong to none
        if (b == 0 && c0 > 0) s.z2 = 0, s.z3 = min(c0, P.rows);
        if (b == p.B - 1 && c1 < P.rows) s.z2 = max(c1, 0), s.z3 = P.rows;
        if (report && (!s.ok || s.z3 > s.z2)) raise_error(p.err, PKV_DEVERR_CU_SEQLENS);
    }
    s.first = p.window > 0 ? max(0, s.L - s.nq + 1 - p.window) / bs : 0;
    s.pages = s.L > 0 && s.ok ? (s.L + bs - 1) / bs - s.first : 0;
    return s;
}

__device__ __forceinline__ void clear_rows(const AttendQ4Params &P, const SeqRows &s, int kvh, int d) {
    const DecodeKParams &p = P.k;
    for (int part = 0; part < 2; ++part) {
        const int z0 = part ? s.z2 : s.z0, z1 = part ? s.z3 : s.z1;
        for (int r = z0; r < z1; ++r) {
            const size_t at = static_cast<size_t>(r) * p.Hq + kvh * p.m;
            for (int i = threadIdx.x; i < p.m * d; i += blockDim.x) p.out[at * d + i] = 0.f;
            if (p.lse != nullptr)
                for (int i = threadIdx.x; i < p.m; i += blockDim.x) p.lse[at + i] = -INFINITY;
        }
    }
}

// Row v of a tile's (query row, head) pairs: head kvh * m + v % m of the sequence's query row
// v / m, which sees tokens [lo, len).  A row past the sequence's last repeats that one's span,
// with bi = -1.
struct RowSpan {
    int bi;        // (query row) * Hq + head
    int lo, len;
};
__device__ __forceinline__ RowSpan tile_row(const AttendQ4Params &P, const SeqRows &s, int kvh, int v) {
    const DecodeKParams &p = P.k;
    const int i = min(v / p.m, s.nq - 1);
    RowSpan r;
    r.len = s.L - s.nq + i + 1;
    r.lo = p.window > 0 ? max(0, r.len - p.window) : 0;
    r.bi = v < s.nq * p.m ? (s.r0 + i) * p.Hq + kvh * p.m + v % p.m : -1;
    return r;
}

// The warps' states of a tile's eight rows, in shared memory ([NW][8] references and sums, then
// [NW][8][D] outputs), merged and written: the result where the sequence has one chunk, else the
// chunk's normalised partial; with arrival counters the unit's last chunk merges them all.
template <int D, int NW>
__device__ __forceinline__ void finish_rows(uint8_t *smem, const AttendQ4Params &P, const RowSpan *rows, int unit,
                                            int split, int nc) {
    const DecodeKParams &p = P.k;
    float *mw = reinterpret_cast<float *>(smem);
    float *lw = mw + NW * 8;
    float *ow = lw + NW * 8;
    for (int idx = threadIdx.x; idx < 8 * (D / 4); idx += NW * 32) {
        const int h = idx / (D / 4), c = idx % (D / 4) * 4;
        if (rows[h].bi < 0) continue;
        const size_t bi = rows[h].bi;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, mw[w * 8 + h]);
        const float base = M == -INFINITY ? 0.f : M;   // the row sees none of this chunk's keys
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
        if (nc == 1) {
            *reinterpret_cast<float4 *>(p.out + bi * D + c) = r;
            if (c == 0 && p.lse != nullptr) p.lse[bi] = lse2 * kDecLn2;
        } else {
            *reinterpret_cast<float4 *>(p.ws_o + (bi * p.splits + split) * D + c) = r;
            if (c == 0) p.ws_lse[bi * p.splits + split] = lse2;
        }
    }
    if (nc == 1 || p.counters == nullptr) return;
    __shared__ int s_last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned prev = atomicAdd(p.counters + unit, 1u);
        s_last = prev + 1 == static_cast<unsigned>(nc);
        if (s_last) p.counters[unit] = 0u;   // every chunk of this call has arrived
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int idx = threadIdx.x; idx < 8 * (D / 4); idx += NW * 32) {
        const int h = idx / (D / 4), c = idx % (D / 4) * 4;
        if (rows[h].bi < 0) continue;
        const size_t bi = rows[h].bi;
        const float *ls = p.ws_lse + bi * p.splits, *po = p.ws_o + bi * p.splits * D + c;
        float M = -INFINITY;
        for (int i = 0; i < nc; ++i) M = fmaxf(M, __ldcg(ls + i));
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < nc; ++i) {
            const float w = exp2f(__ldcg(ls + i) - M);
            const float4 o = __ldcg(reinterpret_cast<const float4 *>(po + static_cast<size_t>(i) * D));
            L += w;
            acc.x += w * o.x;
            acc.y += w * o.y;
            acc.z += w * o.z;
            acc.w += w * o.w;
        }
        const float inv = 1.f / L;
        *reinterpret_cast<float4 *>(p.out + bi * D + c) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (c == 0 && p.lse != nullptr) p.lse[bi] = (M + log2f(L)) * kDecLn2;
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
    float x[8] = {};
    if (lane < WORDS) {
        if (p.new_bf16) q4_load8<__nv_bfloat16, false>(static_cast<const __nv_bfloat16 *>(side ? p.k.v_new : p.k.k_new) + src, x);
        else q4_load8<float, false>(static_cast<const float *>(side ? p.k.v_new : p.k.k_new) + src, x);
    }
    __half2 par;
    const uint32_t code = q4_quantise8(x, LANES, par);
    if (lane >= WORDS) return;
    uint8_t *page = (side ? p.vc : p.kc) + row_page;
    reinterpret_cast<uint32_t *>(page)[off * WORDS + lane] = code;
    if (lane % LANES == 0) reinterpret_cast<__half2 *>(page + bs * WORDS * 4)[off * G + lane / LANES] = par;
}

template <int D, int BS, int G>
__global__ void __launch_bounds__(kMmaWarps * 32, 4) attend_q4_mma_kernel(const __grid_constant__ AttendQ4Params P) {
    using Cfg = MmaCfg<D, BS, G>;
    constexpr int NW = kMmaWarps, NT = kStageKeys / 8, PPS = Cfg::PPS, WORDS = Cfg::WORDS;
    constexpr int WPT = WORDS / (4 * G);         // K: words per lane and group
    constexpr int KSTEPS = D / 16;
    constexpr int HPG = D / 32 / G;              // V: 32-dimension columns per group
    static_assert(WPT >= 1 && HPG >= 1, "a group has at least 32 elements");
    const DecodeKParams &p = P.k;

    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kBarOff);
    __shared__ RowSpan s_rows[8];

    pdl_launch_dependents();   // a merge kernel after this one waits for the whole grid
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int tile = blockIdx.x % p.head_tiles, split = blockIdx.x / p.head_tiles;
    const int kvh = blockIdx.y, b = blockIdx.z;
    const bool report = threadIdx.x == 0 && split == 0 && kvh == 0 && tile == 0;

    // ---- the sequence's rows and this tile's
    const SeqRows sq = seq_rows(P, b, BS, report);
    if (split == 0 && tile == 0) clear_rows(P, sq, kvh, D);
    if (!sq.ok || 8 * tile >= sq.nq * p.m) return;
    if (threadIdx.x < 8) s_rows[threadIdx.x] = tile_row(P, sq, kvh, 8 * tile + threadIdx.x);
    // pages that any row of the sequence sees; this chunk's, and those that this tile sees
    const int c0 = sq.first + split * p.chunk_pages, c1 = min(sq.first + sq.pages, c0 + p.chunk_pages);
    if (c0 >= c1) {
        // a new token for a sequence that holds none has no position: flagged, not written
        if (split == 0 && p.new_slots != nullptr && threadIdx.x == 0 && sq.L == 0 && __ldg(p.new_slots + b) >= 0)
            raise_error(p.err, PKV_DEVERR_SLOT);
        return;
    }
    const RowSpan t_first = tile_row(P, sq, kvh, 8 * tile), t_last = tile_row(P, sq, kvh, min(8 * tile + 7, sq.nq * p.m - 1));
    const int pg0 = max(c0, t_first.lo / BS), pg1 = min(c1, (t_last.len + BS - 1) / BS);
    const int tok_end = pg1 * BS;   // the chunk's keys end here

    if (p.new_slots != nullptr && c1 == sq.first + sq.pages) {
        // the step's new token: the CTA that reads the sequence's last page writes its K and V
        // rows there before any copy of the page
        if (warp < 2) {
            const long long slot = __ldg(p.new_slots + b);
            if (slot >= 0) {
                const int pos = sq.L - 1, phys = __ldg(p.block_table + static_cast<size_t>(b) * p.MBS + pos / BS);
                if (phys < 0 || phys >= p.NB || slot != static_cast<long long>(phys) * BS + pos % BS) {
                    if (warp == 0 && lane == 0) raise_error(p.err, PKV_DEVERR_SLOT);
                } else {
                    write_new_row<D, G>(P, b, kvh, (static_cast<long long>(phys) * p.Hkv + kvh) * Cfg::kPageBytes, pos % BS,
                                        BS, warp, lane);
                }
            }
            fence_proxy_async_global();
        }
        __syncthreads();
        fence_proxy_async_global();
    }

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(smem_addr(&bars[warp * kStages + s]), 1);
        fence_barrier_init();
    }
    __syncthreads();   // s_rows; the barriers are the warp's own

    // ---- this warp's stages: units of PPS pages warp, warp + NW, ... of [pg0, pg1)
    const int units = pg1 > pg0 ? (pg1 - pg0 + PPS - 1) / PPS : 0;
    const int n_my = units > warp ? (units - warp + NW - 1) / NW : 0;
    const int32_t *tbl = p.block_table + static_cast<size_t>(b) * p.MBS;
    int tcur[PPS], tnext[PPS];
    auto load_ids = [&](int k, int (&t)[PPS]) {
#pragma unroll
        for (int i = 0; i < PPS; ++i) {
            const int pg = pg0 + (warp + k * NW) * PPS + i;
            t[i] = k < n_my && pg < pg1 ? __ldg(tbl + pg) : -1;
        }
    };
    load_ids(lane, tcur);
    load_ids(32 + lane, tnext);
    int tbase = 0;
    unsigned bad = 0;   // bit (stage * PPS + page): a page to be read as zeros
    auto issue = [&](int k) {   // the whole warp; lane 0 starts the copies
        while (k >= tbase + 32) {
            tbase += 32;
#pragma unroll
            for (int i = 0; i < PPS; ++i) tcur[i] = tnext[i];
            load_ids(tbase + 32 + lane, tnext);
        }
        const int st = k % kStages;
        uint8_t *stage = smem + (warp * kStages + st) * Cfg::kStageBytes;
        const uint32_t bar = smem_addr(&bars[warp * kStages + st]);
        // lane l: copy l of the stage's 2 * PPS (K pages, then V pages)
        const int i = lane % PPS, pg = pg0 + (warp + k * NW) * PPS + i;
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
            bulk_load(smem_addr(stage + lane * Cfg::kPageBytes),
                      (lane < PPS ? P.kc : P.vc) + (static_cast<size_t>(phys) * p.Hkv + kvh) * Cfg::kPageBytes,
                      Cfg::kPageBytes, bar);
    };
    int issued = min(kStages, n_my);
    for (int k = 0; k < issued; ++k) issue(k);

    // ---- query fragments, for all warps, by warp 0 while the copies fly.  MMA step 2u (codes' even
    // nibbles) and 2u + 1 (odd nibbles, 16 times the value) of word u = gi * WPT + i: elements
    // 8 * word + {0, 4}, {2, 6} and {1, 5}, {3, 7}
    uint4 *qfrag = reinterpret_cast<uint4 *>(smem + Cfg::kQOff) + lane;    // [step][lane]
    uint2 *zfrag = reinterpret_cast<uint2 *>(smem + Cfg::kQOff + KSTEPS * 512) + lane;
    float *ffrag = reinterpret_cast<float *>(smem + Cfg::kQOff + KSTEPS * 512 + 256) + g;
    const RowSpan me = s_rows[g];
    if (warp == 0) {
        const float *qrow = p.q + static_cast<size_t>(me.bi >= 0 ? me.bi : 0) * D;
        float x[G * WPT][8], amax = 0.f, zsum = 0.f;
#pragma unroll
        for (int u = 0; u < G * WPT; ++u) {
            const int word = (u / WPT) * (WORDS / G) + t4 * WPT + u % WPT;
            const float2 *src = reinterpret_cast<const float2 *>(qrow + 8 * word);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = me.bi >= 0 ? __ldg(src + e) : make_float2(0.f, 0.f);
                x[u][2 * e] = v.x;
                x[u][2 * e + 1] = v.y;
                amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        // |q| * 2^sq in [2^13, 2^14); a row of zeros (or of subnormals) keeps the factor finite
        const int sq = min(13 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), 126);
        const float up = pow2i(sq);
        if (t4 == 0) *ffrag = (p.scale_log2 * 0x1p24f) * pow2i(-sq);   // score (base 2) = MMA sum * this
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < WPT; ++i) {
                const int u = gi * WPT + i;
                uint4 qe, qo;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[u][e] *= up;
                    sum += x[u][e];
                }
                split2(x[u][0], x[u][4], qe.x, qe.y);
                split2(x[u][2], x[u][6], qe.z, qe.w);
                split2(x[u][1] * 0.0625f, x[u][5] * 0.0625f, qo.x, qo.y);
                split2(x[u][3] * 0.0625f, x[u][7] * 0.0625f, qo.z, qo.w);
                qfrag[(2 * u) * 32] = qe;
                qfrag[(2 * u + 1) * 32] = qo;
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            if (gi == t4) zsum = sum;
        }
        // (0, sum of q over group t4) * 2^-8, which keeps 128 elements below 2^14; zero beyond G
        uint2 z;
        split2(0.f, zsum * 0x1p-8f, z.x, z.y);
        *zfrag = z;
    }
    __syncthreads();
    const uint2 za = *zfrag;
    const float f = *ffrag;

    float oT[D / 16][4];
    float2 zo[G];   // sums of weight * zero over this lane's keys
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) oT[mt][0] = oT[mt][1] = oT[mt][2] = oT[mt][3] = 0.f;
#pragma unroll
    for (int gi = 0; gi < G; ++gi) zo[gi] = make_float2(0.f, 0.f);
    float m_run = -INFINITY, l_run = 0.f;   // the running max, and l relative to `ref`
    float ref = -INFINITY;                  // m_run + E - 14
    unsigned vs_bits = 0;                   // the largest V scale seen (f16 bits)
    float vs_exp = -24.f;                   // E: its exponent, rounded up (fp16's smallest to begin with)

    int k = 0;
    for (; k < n_my; ++k) {
        const int st = k % kStages;
        const bool arrived = mbar_wait_bounded(smem_addr(&bars[warp * kStages + st]), (k / kStages) & 1);
        if (!__all_sync(kFull, arrived)) {
            if (lane == 0) raise_error(p.err, PKV_DEVERR_TIMEOUT);
            break;
        }
        uint8_t *kpages = smem + (warp * kStages + st) * Cfg::kStageBytes;
        uint8_t *vpages = kpages + PPS * Cfg::kPageBytes;
        const int tok0 = (pg0 + (warp + k * NW) * PPS) * BS;
        if (const unsigned zero = (bad >> (st * PPS)) & ((1u << PPS) - 1); zero != 0) {
#pragma unroll
            for (int i = 0; i < 2 * PPS; ++i)
                if (zero >> (i % PPS) & 1)
                    for (int c = lane * 16; c < Cfg::kPageBytes; c += 512)
                        *reinterpret_cast<uint4 *>(kpages + i * Cfg::kPageBytes + c) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();   // before a later copy into this stage
            __syncwarp();
        }
        // does every row of the tile see every key of the stage?
        const bool whole = tok0 >= t_last.lo && tok0 + kStageKeys <= min(t_first.len, tok_end);
        if (!whole) {
            // parameters of V rows that no row of the tile sees may be anything: zero them, so that
            // weight 0 contributes 0 (codes are finite whatever they are)
            const int tok = tok0 + lane, off = lane % BS;
            if (tok < t_first.lo || tok >= min(t_last.len, tok_end)) {
#pragma unroll
                for (int gi = 0; gi < G; ++gi)
                    reinterpret_cast<uint32_t *>(vpages + (lane / BS) * Cfg::kPageBytes + Cfg::kCodeBytes)[off * G + gi] = 0;
                fence_proxy_async_smem();
            }
            __syncwarp();
        }

        // ---- scores of row g for keys 8 * nt + 2 * t4 + {0, 1}
        float2 s[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint32_t *par = reinterpret_cast<const uint32_t *>(kpages + (nt * 8 / BS) * Cfg::kPageBytes + Cfg::kCodeBytes);
            float z[4] = {0.f, 0.f, 0.f, 0.f};
            mma8(z, za.x, za.y, t4 < G ? par[(nt * 8 % BS + g) * G + t4] : 0u);
            s[nt] = mul2(add2(make_float2(z[0], z[1]), make_float2(z[2], z[3])), make_float2(0x1p-16f, 0x1p-16f));
        }
#pragma unroll
        for (int gi = 0; gi < G; ++gi) {
            float a[NT][4];
            uint32_t c[NT][WPT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                a[nt][0] = a[nt][1] = a[nt][2] = a[nt][3] = 0.f;
                lds_words<WPT>(kpages + (nt * 8 / BS) * Cfg::kPageBytes + (nt * 8 % BS + g) * (D / 2) + gi * (D / 2 / G) +
                                   t4 * WPT * 4,
                               c[nt]);
            }
#pragma unroll
            for (int i = 0; i < WPT; ++i) {
                const uint4 qe = qfrag[(2 * (gi * WPT + i)) * 32], qo = qfrag[(2 * (gi * WPT + i) + 1) * 32];
                // the tiles' chains side by side
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16(a[nt], qe.x, qe.y, qe.z, qe.w, c[nt][i] & 0x000f000fu, (c[nt][i] >> 8) & 0x000f000fu);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16(a[nt], qo.x, qo.y, qo.z, qo.w, c[nt][i] & 0x00f000f0u, (c[nt][i] >> 8) & 0x00f000f0u);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint32_t *par = reinterpret_cast<const uint32_t *>(kpages + (nt * 8 / BS) * Cfg::kPageBytes + Cfg::kCodeBytes) +
                                      (nt * 8 % BS + 2 * t4) * G + gi;
                s[nt] = fma2(make_float2(scale_of(par[0]), scale_of(par[G])),
                             add2(make_float2(a[nt][0], a[nt][1]), make_float2(a[nt][2], a[nt][3])), s[nt]);
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

        // ---- the running reference: the rows' maxima and the largest V scale (lane: one key)
        float mx = fmaxf(s[0].x, s[0].y);
#pragma unroll
        for (int nt = 1; nt < NT; ++nt) mx = fmaxf(mx, fmaxf(s[nt].x, s[nt].y));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        m_run = fmaxf(m_run, mx);
        unsigned top = 0;   // positive f16 order like their bits
        {
            uint32_t v[G];
            lds_words<G>(vpages + (lane / BS) * Cfg::kPageBytes + Cfg::kCodeBytes + (lane % BS) * G * 4, v);
#pragma unroll
            for (int gi = 0; gi < G; ++gi) top = max(top, v[gi] & 0xffffu);
            top = __reduce_max_sync(kFull, top);
        }
        if (top > vs_bits) {   // rarely after the first stage: the next power of two, E = its exponent
            vs_bits = top;
            const uint32_t v = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
            vs_exp = static_cast<float>(static_cast<int>((v + 0x7fffffu) >> 23) - 127);
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
        if (__any_sync(kFull, alpha != 1.f)) {
            const float alpha_a = __shfl_sync(kFull, alpha, 8 * t4);
            const float alpha_b = __shfl_sync(kFull, alpha, 8 * t4 + 4);
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                oT[mt][0] *= alpha_a;
                oT[mt][1] *= alpha_b;
                oT[mt][2] *= alpha_a;
                oT[mt][3] *= alpha_b;
            }
#pragma unroll
            for (int gi = 0; gi < G; ++gi) zo[gi] = mul2(zo[gi], make_float2(alpha, alpha));
        }

        // ---- O^T += V^T P^T, 16 keys per step.  ldmatrix with transposition over 16-bit units
        // (four codes of a key) hands lane (g, t4) the units 8 * c + g of keys 2 * t4, 2 * t4 + 1 in
        // one register: the pairs along the keys that the A operand wants
        const uint32_t vrow = smem_addr(vpages) + (lane & 15) * (D / 2) + (lane >> 4) * 16;
#pragma unroll
        for (int kt = 0; kt < kStageKeys / 16; ++kt) {
            const uint32_t rows = vrow + (kt * 16 / BS) * Cfg::kPageBytes + (kt * 16 % BS) * (D / 2);
#pragma unroll
            for (int gi = 0; gi < G; ++gi) {
                uint32_t bh0, bl0, bh1, bl1;
                {
                    const uint32_t *par = reinterpret_cast<const uint32_t *>(vpages + (kt * 16 / BS) * Cfg::kPageBytes + Cfg::kCodeBytes) +
                                          (kt * 16 % BS + 2 * t4) * G + gi;
                    const float2 p0 = par_of(par[0]), p1 = par_of(par[G]), p2 = par_of(par[8 * G]), p3 = par_of(par[9 * G]);
                    const float2 wa = w[2 * kt], wb = w[2 * kt + 1];
                    split2(mul2(wa, make_float2(p0.x, p1.x)), bh0, bl0);
                    split2(mul2(wb, make_float2(p2.x, p3.x)), bh1, bl1);
                    zo[gi] = fma2(wa, make_float2(p0.y, p1.y), fma2(wb, make_float2(p2.y, p3.y), zo[gi]));
                }
#pragma unroll
                for (int h = 0; h < HPG; h += 2) {
                    // registers: units 8 * c of keys 0..7, of keys 8..15, units 8 * (c + 1) likewise
                    const int c = gi * HPG + h;
                    uint32_t v[4];
                    if constexpr (HPG >= 2) ldsm_x4_trans(rows + c * 16, v[0], v[1], v[2], v[3]);
                    else ldsm_x2_trans(rows - (lane >> 4) * 16 + c * 16, v[0], v[1]);
                    constexpr int N = HPG >= 2 ? 2 : 1;
#pragma unroll
                    for (int lo = 0; lo < 2; ++lo) {   // the weights' high parts, then their low ones
                        const uint32_t b0 = lo ? bl0 : bh0, b1 = lo ? bl1 : bh1;
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const uint32_t x = v[2 * i], y = v[2 * i + 1], x8 = x >> 8, y8 = y >> 8;
                            const int mt = 2 * (c + i);
                            mma16(oT[mt], x & 0x000f000fu, x8 & 0x000f000fu, y & 0x000f000fu, y8 & 0x000f000fu, b0, b1);
                            mma16(oT[mt + 1], x & 0x00f000f0u, x8 & 0x00f000f0u, y & 0x00f000f0u, y8 & 0x00f000f0u, b0, b1);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (k + kStages < n_my) {
            issue(k + kStages);
            issued = k + kStages + 1;
        }
    }
    if (k < n_my) {
        // A copy did not arrive in time: wait (bounded) for the copies still in flight so that
        // none lands after the block exits.
        for (int kk = k; kk < issued; ++kk)
            mbar_wait_bounded(smem_addr(&bars[warp * kStages + kk % kStages]), (kk / kStages) & 1);
    }

    l_run += __shfl_xor_sync(kFull, l_run, 1);
    l_run += __shfl_xor_sync(kFull, l_run, 2);
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
        zo[gi].x += zo[gi].y;
        zo[gi].x += __shfl_xor_sync(kFull, zo[gi].x, 1);
        zo[gi].x += __shfl_xor_sync(kFull, zo[gi].x, 2);
    }

    // ---- the warps' (ref, l, O) through shared memory (the ring is free now)
    __syncthreads();
    float *mw = reinterpret_cast<float *>(smem);
    float *lw = mw + NW * 8;
    float *ow = lw + NW * 8;
    if (t4 == 0) {
        mw[warp * 8 + g] = ref;
        lw[warp * 8 + g] = l_run;
    }
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
        const float za_ = __shfl_sync(kFull, zo[gi].x, 8 * t4), zb_ = __shfl_sync(kFull, zo[gi].x, 8 * t4 + 4);
#pragma unroll
        for (int h = 0; h < HPG; ++h) {
            const int c = gi * HPG + h, dim = 32 * c + 4 * g, mt = 2 * c;
            // even codes were c * 2^-24, odd ones c * 2^-20
            float *oa = ow + (warp * 8 + 2 * t4) * D + dim, *ob = oa + D;
            oa[0] = fmaf(oT[mt][0], 0x1p24f, za_);
            oa[1] = fmaf(oT[mt + 1][0], 0x1p20f, za_);
            oa[2] = fmaf(oT[mt][2], 0x1p24f, za_);
            oa[3] = fmaf(oT[mt + 1][2], 0x1p20f, za_);
            ob[0] = fmaf(oT[mt][1], 0x1p24f, zb_);
            ob[1] = fmaf(oT[mt + 1][1], 0x1p20f, zb_);
            ob[2] = fmaf(oT[mt][3], 0x1p24f, zb_);
            ob[3] = fmaf(oT[mt + 1][3], 0x1p20f, zb_);
        }
    }
    __syncthreads();
    finish_rows<D, NW>(smem, P, s_rows, (b * p.Hkv + kvh) * p.head_tiles + tile, split,
                       (sq.pages + p.chunk_pages - 1) / p.chunk_pages);
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

Q4Plan plan_attend_q4(int B, int rows, int max_q, int Hq, int Hkv, int d, int group, int bs, int pages,
                      int num_splits, int sm_count, bool aligned) {
    Q4Plan plan{};
    const int m = Hq / Hkv, sms = std::max(sm_count, 1);
    const long long tiles = (static_cast<long long>(max_q) * m + 7) / 8;
    plan.mma = (d == 64 || d == 128) && (bs == 16 || bs == 32) && d / group <= 4 && aligned && tiles < (1 << 18);
    plan.tiles = plan.mma ? static_cast<int>(tiles) : 1;
    const long long units = plan.mma ? static_cast<long long>(B) * Hkv * tiles : static_cast<long long>(rows) * Hq;
    int chunk = pages;
    if (num_splits > 1) {
        chunk = (pages + num_splits - 1) / num_splits;
    } else if (num_splits == 0 && plan.mma) {
        // about two waves of the CTAs an SM holds, chunks of at least 256 keys; and none of more
        // than 8192, so that a long sequence among short ones spreads
        const int least = 256 / bs, most = 8192 / bs;
        while (chunk > least && units * ((pages + chunk - 1) / chunk) < 8ll * sms) chunk = (chunk + 1) / 2;
        if (chunk > most) chunk = (pages + (pages + most - 1) / most - 1) / ((pages + most - 1) / most);
    } else if (num_splits == 0) {
        // one warp per (row, head, chunk): several warps for each scheduler, no chunk shorter
        // than 128 keys
        const int least = std::max(1, 128 / bs);
        while (chunk > least && units * ((pages + chunk - 1) / chunk) < 32ll * sms) chunk = (chunk + 1) / 2;
    }
    chunk = std::max(chunk, (pages + kDecodeMaxChunks - 1) / kDecodeMaxChunks);
    plan.chunk_pages = std::max(chunk, 1);
    plan.splits = (pages + plan.chunk_pages - 1) / plan.chunk_pages;
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
    if (plan.splits > 1) {
        uint8_t *ws = static_cast<uint8_t *>(a.workspace);
        kp.ws_o = reinterpret_cast<float *>(ws + PKV_DECODE_COUNTER_BYTES);
        kp.ws_lse = kp.ws_o + static_cast<size_t>(a.rows) * a.Hq * plan.splits * a.d;
    }
    cudaError_t e;
    if (plan.mma) {
        AttendQ4Params P{};
        kp.head_tiles = plan.tiles;
        if (plan.fused_merge) kp.counters = static_cast<unsigned *>(a.workspace);
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
        const dim3 grid(static_cast<unsigned>(plan.splits) * plan.tiles, a.Hkv, a.B);
        e = launch_mma(P, a.d, a.bs, a.d / a.group, grid, stream);
    } else {
        e = launch_simt(a, kp, stream);
    }
    if (e != cudaSuccess || plan.splits == 1 || plan.fused_merge) return e;
    return launch_decode_merge(kp, a.d, a.bs, static_cast<unsigned>(a.rows * a.Hq), stream);
}

}  // namespace pkv
