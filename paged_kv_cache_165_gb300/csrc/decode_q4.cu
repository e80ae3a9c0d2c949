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

#include "common.cuh"
#include "decode_kparams.cuh"
#include "internal.h"
#include "q4_codes.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

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

size_t partial_bytes(long long rows, int Hq, int splits, int d) {
    return splits > 1 ? PKV_DECODE_COUNTER_BYTES +
                            static_cast<size_t>(rows) * Hq * splits * (static_cast<size_t>(d) + 1) * sizeof(float)
                      : 0;
}

}  // namespace

Q4Plan plan_attend_q4(int B, int rows, int max_q, int Hq, int Hkv, int d, int group, int bs, int pages,
                      int num_splits, int sm_count, bool aligned) {
    (void)B, (void)max_q, (void)Hkv, (void)group, (void)aligned;
    Q4Plan plan{};
    int chunk = pages;
    if (num_splits > 1) {
        chunk = (pages + num_splits - 1) / num_splits;
    } else if (num_splits == 0) {
        // one warp per (row, head, chunk): several warps for each scheduler, no chunk shorter
        // than 128 keys
        const long long units = static_cast<long long>(rows) * Hq, target = 32ll * std::max(sm_count, 1);
        const int least = std::max(1, 128 / bs);
        while (chunk > least && units * ((pages + chunk - 1) / chunk) < target) chunk = (chunk + 1) / 2;
    }
    chunk = std::max(chunk, (pages + kDecodeMaxChunks - 1) / kDecodeMaxChunks);
    plan.chunk_pages = std::max(chunk, 1);
    plan.splits = (pages + plan.chunk_pages - 1) / plan.chunk_pages;
    plan.workspace_bytes = partial_bytes(rows, Hq, plan.splits, d);
    return plan;
}

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
    const cudaError_t e = launch_simt(a, kp, stream);
    if (e != cudaSuccess || plan.splits == 1) return e;
    return launch_decode_merge(kp, a.d, a.bs, static_cast<unsigned>(a.rows * a.Hq), stream);
}

}  // namespace pkv
