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
#include <cmath>

#include "decode_q4.cuh"
#include "decode_q4_mma.cuh"

namespace pkv {
namespace {

// ================================================================ CUDA-core path

// Query heads that a warp takes together, so that they share the codes' way into fp32.
int simt_heads(int m) { return m <= 2 ? m : 4; }

// A word's codes less 8, times 2^-9: elements (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void centred8(uint32_t w, float2 (&e)[4]) {
    uint32_t h[4];
    centre(w, h[0], h[1]);
    centre(w >> 8, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
}

// One warp per (query row, H query heads of a KV head, chunk).  W lanes (a power of two, W * 8 >= d)
// hold one key's row, eight elements each, so 32 / W keys are taken at a time, U such steps (16 keys at most)
// between two updates of the softmax; every such slice of the warp keeps its own online softmax and
// they merge at the end.  Bound by its arithmetic, shuffles most of all (64 x 2048 tokens, 32 heads on 8 of
// 128: 248 us, the warp-MMA kernel 45).
template <int W, int H>
__global__ void __launch_bounds__(128)
    attend_q4_simt_kernel(const uint8_t *__restrict__ kc, const uint8_t *__restrict__ vc, const DecodeKParams p,
                          int d, int bs, int lanes, int rows) {
    constexpr int KEYS = 32 / W, U = W == 4 ? 2 : 4;
    pdl_launch_dependents();   // the merge kernel after this one waits for the whole grid
    const int lane = threadIdx.x & 31, tiles = (p.m + H - 1) / H;
    const long long unit = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (unit >= static_cast<long long>(rows) * p.Hkv * tiles) return;
    const int row = static_cast<int>(unit / (p.Hkv * tiles)), part = static_cast<int>(unit % (p.Hkv * tiles));
    const int kvh = part / tiles, h0 = part % tiles * H, split = blockIdx.y, j = lane % W, slice = lane / W;
    const SeqSpan sp = row_span(p, row, bs, lane == 0 && split == 0 && part == 0);
    const int nc = (sp.cnpages + p.chunk_pages - 1) / p.chunk_pages;
    const int c0 = sp.cpfirst + split * p.chunk_pages;
    const int c1 = min(sp.cpfirst + sp.cnpages, c0 + p.chunk_pages);
    const int pg0 = max(c0, sp.pfirst), pg1 = min(c1, sp.pfirst + sp.npages);
    const size_t bi0 = static_cast<size_t>(row) * p.Hq + kvh * p.m + h0;
    const int heads = min(H, p.m - h0);
    if (c0 >= c1 || pg0 >= pg1) {
        // an empty sequence: out = 0, lse = -inf; a chunk with none of this row's keys: an empty partial
        if (c0 >= c1 && split > 0) return;
        for (int h = 0; h < heads; ++h) {
            const size_t at = c0 >= c1 ? bi0 + h : (bi0 + h) * p.splits + split;
            for (int e = lane; e < d; e += 32) (c0 >= c1 ? p.out : p.ws_o)[at * d + e] = 0.f;
            float *lse = c0 >= c1 ? p.lse : p.ws_lse;
            if (lane == 0 && lse != nullptr) lse[at] = -INFINITY;
        }
        return;
    }
    const int words = d / 8, G = words / lanes;
    const bool mine = j < words;
    float2 q[H][4], acc[H][4];
    float qsum[H], zero_sum[H], m_run[H], l_run[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const float *src = p.q + (bi0 + min(h, heads - 1)) * d + j * 8;
        qsum[h] = zero_sum[h] = l_run[h] = 0.f;
        m_run[h] = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q[h][e] = mine ? make_float2(src[e], src[e + 4]) : make_float2(0.f, 0.f);
            qsum[h] += q[h][e].x + q[h][e].y;
            acc[h][e] = make_float2(0.f, 0.f);
        }
    }
    const int page_bytes = bs * (words * 4 + G * 4);
    const int32_t *table = p.block_table + static_cast<size_t>(sp.b) * p.MBS;
    int next = __ldg(table + pg0);
    for (int pg = pg0; pg < pg1; ++pg) {
        const int phys = next;
        if (pg + 1 < pg1) next = __ldg(table + pg + 1);
        const bool bad = phys < 0 || phys >= p.NB;
        if (bad && lane == 0) raise_error(p.err, PKV_DEVERR_BLOCK);
        const size_t base = bad ? 0 : (static_cast<size_t>(phys) * p.Hkv + kvh) * page_bytes;
        const uint32_t *kw = reinterpret_cast<const uint32_t *>(kc + base);
        const uint32_t *vw = reinterpret_cast<const uint32_t *>(vc + base);
        const int first = max(0, sp.lo - pg * bs), valid = min(bs, sp.len - pg * bs);
        for (int t0 = first + slice; t0 - slice < valid; t0 += KEYS * U) {
            uint32_t kcode[U], vcode[U];
            float2 kp[U], vp[U];   // scale * 2^9 and the centred codes' zero
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + u * KEYS;
                kcode[u] = vcode[u] = 0;
                kp[u] = vp[u] = make_float2(0.f, 0.f);
                if (t < valid && mine && !bad) {
                    kcode[u] = __ldg(kw + t * words + j);
                    vcode[u] = __ldg(vw + t * words + j);
                    kp[u] = __half22float2(__ldg(reinterpret_cast<const __half2 *>(kw + bs * words) + t * G + j / lanes));
                    vp[u] = __half22float2(__ldg(reinterpret_cast<const __half2 *>(vw + bs * words) + t * G + j / lanes));
                }
            }
            float s[H][U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 e[4];
                centred8(kcode[u], e);
                const float zero = fmaf(8.f, kp[u].x, kp[u].y), scale = kp[u].x * 0x1p9f;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float2 y = fma2(q[h][0], e[0], fma2(q[h][1], e[1], fma2(q[h][2], e[2], mul2(q[h][3], e[3]))));
                    s[h][u] = fmaf(scale, y.x + y.y, zero * qsum[h]);
                }
            }
#pragma unroll
            for (int sh = W / 2; sh > 0; sh >>= 1)
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int u = 0; u < U; ++u) s[h][u] += __shfl_xor_sync(kFull, s[h][u], sh);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float m_new = m_run[h];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[h][u] = t0 + u * KEYS < valid ? s[h][u] * p.scale_log2 : -INFINITY;
                    m_new = fmaxf(m_new, s[h][u]);
                }
                const float base = m_new == -INFINITY ? 0.f : m_new;   // the slice has seen no key yet: weights 0
                const float alpha = m_run[h] == -INFINITY ? 0.f : ex2_approx(m_run[h] - base);
                m_run[h] = m_new;
                l_run[h] *= alpha;
                zero_sum[h] *= alpha;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[h][u] = ex2_approx(s[h][u] - base);
                    l_run[h] += s[h][u];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][e] = mul2(acc[h][e], make_float2(alpha, alpha));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 e[4];
                centred8(vcode[u], e);
                const float zero = fmaf(8.f, vp[u].x, vp[u].y);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float w = s[h][u] * vp[u].x;
                    zero_sum[h] = fmaf(s[h][u], zero, zero_sum[h]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[h][i] = fma2(make_float2(w, w), e[i], acc[h][i]);
                }
            }
        }
    }
    // the slices' states, lanes j of every slice
#pragma unroll
    for (int h = 0; h < H; ++h) {
        float M = m_run[h];
#pragma unroll
        for (int sh = W; sh < 32; sh <<= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, sh));
        const float f = m_run[h] == -INFINITY ? 0.f : exp2f(m_run[h] - M);
        float L = l_run[h] * f, z = zero_sum[h] * f;
#pragma unroll
        for (int sh = W; sh < 32; sh <<= 1) {
            L += __shfl_xor_sync(kFull, L, sh);
            z += __shfl_xor_sync(kFull, z, sh);
        }
        const size_t bi = bi0 + h;
        float *dst = nc == 1 ? p.out + bi * d : p.ws_o + (bi * p.splits + split) * d;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 y = mul2(acc[h][e], make_float2(f, f));
#pragma unroll
            for (int sh = W; sh < 32; sh <<= 1)
                y = add2(y, make_float2(__shfl_xor_sync(kFull, y.x, sh), __shfl_xor_sync(kFull, y.y, sh)));
            if (mine && slice == 0 && h < heads) {
                dst[j * 8 + e] = fmaf(y.x, 0x1p9f, z) / L;
                dst[j * 8 + e + 4] = fmaf(y.y, 0x1p9f, z) / L;
            }
        }
        if (lane == 0 && h < heads) {
            const float lse2 = M + log2f(L);
            if (nc > 1) p.ws_lse[bi * p.splits + split] = lse2;
            else if (p.lse != nullptr) p.lse[bi] = lse2 * kDecLn2;
        }
    }
}


template <template <int, int, int> class Rows>
cudaError_t launch_mma(const AttendQ4Params &P, int d, int bs, int G, dim3 grid, cudaStream_t stream) {
#define PKV_Q4_MMA(DD, BB, GG) launch_mma_as<DD, BB, GG, Rows<DD, BB, GG>>(P, grid, stream)
    if (bs == 16) {
        if (d == 64) return G == 1 ? PKV_Q4_MMA(64, 16, 1) : PKV_Q4_MMA(64, 16, 2);
        return G == 1 ? PKV_Q4_MMA(128, 16, 1) : G == 2 ? PKV_Q4_MMA(128, 16, 2) : PKV_Q4_MMA(128, 16, 4);
    }
    if (d == 64) return G == 1 ? PKV_Q4_MMA(64, 32, 1) : PKV_Q4_MMA(64, 32, 2);
    return G == 1 ? PKV_Q4_MMA(128, 32, 1) : G == 2 ? PKV_Q4_MMA(128, 32, 2) : PKV_Q4_MMA(128, 32, 4);
#undef PKV_Q4_MMA
}

template <int H>
cudaError_t launch_simt_as(const AttendQ4Args &a, const DecodeKParams &kp, cudaStream_t stream) {
    const long long units = static_cast<long long>(a.rows) * a.Hkv * ((kp.m + H - 1) / H);
    const dim3 grid(static_cast<unsigned>((units + 3) / 4), static_cast<unsigned>(kp.splits));
    const int words = a.d / 8, lanes = a.group / 8;
#define PKV_Q4_SIMT(WW) attend_q4_simt_kernel<WW, H><<<grid, 128, 0, stream>>>(a.k_cache, a.v_cache, kp, a.d, a.bs, lanes, a.rows)
    if (words <= 4) PKV_Q4_SIMT(4);
    else if (words <= 8) PKV_Q4_SIMT(8);
    else if (words <= 16) PKV_Q4_SIMT(16);
    else PKV_Q4_SIMT(32);
#undef PKV_Q4_SIMT
    return cudaGetLastError();
}

cudaError_t launch_simt(const AttendQ4Args &a, const DecodeKParams &kp, cudaStream_t stream) {
    const int heads = simt_heads(kp.m);
    return heads == 1 ? launch_simt_as<1>(a, kp, stream) : heads == 2 ? launch_simt_as<2>(a, kp, stream) : launch_simt_as<4>(a, kp, stream);
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
// (Query row, head) pairs of a sequence and KV head that go to the warp-MMA kernel, which takes eight at a
// time; the tcgen05 kernel's time hardly depends on them.  Measured, one scale group a row: 24 pairs over
// 4 x 65536 tokens 38.5 us, tcgen05 (32 pairs) 34.5; over 64 x 2048 tokens of four KV heads 69 and 77.  Two
// groups: 32 pairs 49.8 us, 40 pairs 58.7, tcgen05 (40 pairs) 48.3; over 64 x 2048 89, 105 and 102.  So the
// border lies lower for few long sequences than for many short ones, and one number is a compromise: at 24
// pairs and one group the long case gives up 4 us for 8 us of the short one.
int q4_mma_slots(int G) { return G == 1 ? 24 : 32; }

// Rows of partial results of a balanced launch: two units for every warp or block.
size_t balanced_rows(const Q4Plan &plan) {
    return static_cast<size_t>(plan.blocks) * 2 * (plan.umma ? kQ4UmmaSlots : kMmaWarps * plan.mma_rows);
}
}  // namespace

Q4Plan plan_attend_q4(int B, int rows, int max_q, int Hq, int Hkv, int d, int group, int bs, int pages,
                      int num_splits, int sm_count, bool aligned) {
    Q4Plan plan{};
    const int m = Hq / Hkv, sms = std::max(sm_count, 1);
    const long long slots = static_cast<long long>(max_q) * m;
    plan.umma = q4_umma_shape(d, group, bs) && aligned && slots > q4_mma_slots(d / group) && slots < (1 << 20);
    plan.mma = !plan.umma && (d == 64 || d == 128 || q4_wide_shape(d, group)) && (bs == 8 || bs == 16 || bs == 32) && aligned &&
               slots < (1 << 20);
    plan.mma_rows = slots <= 4 ? 4 : 8;
    const int per_tile = plan.umma ? kQ4UmmaSlots : plan.mma_rows;
    plan.tiles = plan.umma || plan.mma ? static_cast<int>((slots + per_tile - 1) / per_tile) : 1;
    const long long units = plan.umma || plan.mma ? static_cast<long long>(B) * Hkv * plan.tiles
                                                      : static_cast<long long>(rows) * Hkv * ((m + simt_heads(m) - 1) / simt_heads(m));
    int chunk = pages;
    if (num_splits > 1) {
        chunk = (pages + num_splits - 1) / num_splits;
    } else if (num_splits == 0 && (plan.umma || plan.mma)) {
        // An equal share for every warp (umma: block) the device holds at once, or equal chunks, at most
        // one wave of blocks.  Chunks where the units are so few that one would be left to merge parts
        // from many, with more sequences than a block scans, and for warp MMAs where the shares are
        // short, because a chunk's warps merge in shared memory: below 16 steps of 32 keys a warp (256
        // units of four rows: 512 tokens 16.3 us in equal shares, 10.6 in chunks, 2048 33.5 and 26.9, 4096,
        // 13.5 steps, 46.9 and 44.2; eight rows, 4096, 18 steps: 53.5 and 62.7), or 8 where one wave does
        // not hold the units (1024 of four rows: 256 tokens 21.6 and 16.7; 512 of eight: 19.4 and 18.0, 1024
        // tokens, 9 steps, 34.5 and 38.6).
        // All these go by the tokens that the table has room for: the lengths are on the device.  The figures
        // are those of tables as wide as the longest sequence.  Much wider ones get chunks and shares for sequences
        // that are not there: 4 x 8192 tokens, 64 heads on 8 of 128, 26.6 us, with a table for 131072 120.8; 32 x 512,
        // 32 heads on 8, 14.4 and 20.5; 64 x 2048, 64 heads on 8, 57.3 both.
        const int step = plan.umma ? 128 / (d / group) : kStageKeys;
        plan.blocks = sms * (plan.umma ? 1 : mma_blocks_per_sm(plan.mma_rows, d));
        const long long per_unit = std::max(1ll, plan.blocks / std::max(units, 1ll));
        // Tokens of a chunk: 512 where units fill the device (256 units of 2048: 26.9 us, in more chunks 31),
        // else 256, and down to 128 while at most eight chunks merge in place (two sequences of 512, four
        // units: four chunks 7.3 us, two 8.3; eight units of 1000: 7.8 in eight, 8.5 in four; 300 tokens: 6.0 in one
        // chunk, 6.5 in three).
        const long long tokens = static_cast<long long>(pages) * bs;
        const int least = (!plan.mma ? 256 : per_unit <= 8 || tokens <= 384 ? 512 : tokens <= 1024 ? 128 : 256) / bs;
        chunk = static_cast<int>(std::max<long long>(least, (pages + per_unit - 1) / per_unit));
        const long long share = units * (tokens / step) / (static_cast<long long>(plan.blocks) * kMmaWarps);
        const bool few = plan.umma ? plan.blocks > 8 * units : plan.blocks > 6 * units;
        const bool brief = plan.mma && (share < 8 ? units <= 2 * plan.blocks : share < 16 && units <= plan.blocks);
        plan.balanced = B <= kMaxBalanced && !few && !brief &&
                        units * (static_cast<long long>(pages) * bs / step + 1 + kUnitCost) < (1ll << 30);
    } else if (num_splits == 0) {
        // one warp per (row, heads, chunk): several warps for each scheduler, no chunk shorter
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
    kp.rows = a.rows;
    kp.max_q = a.max_q;
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
        P.q_sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
        kp.scale_log2 = a.scale == 0.f ? 1.f : std::fabs(kp.scale_log2);
        P.k = kp;
        P.kc = const_cast<uint8_t *>(a.k_cache);   // written only for a step's new tokens
        P.vc = const_cast<uint8_t *>(a.v_cache);
        P.balanced = plan.balanced;
        const dim3 grid = plan.balanced ? dim3(plan.blocks) : dim3(static_cast<unsigned>(plan.splits) * plan.tiles, a.Hkv, a.B);
        e = plan.umma ? launch_attend_q4_umma(P, a.d, a.bs, a.d / a.group, grid, stream)
            : a.bs == 8 ? launch_attend_q4_bs8(P, plan.mma_rows, a.d, a.d / a.group, grid, stream)
            : q4_wide_shape(a.d, a.group) ? launch_attend_q4_wide(P, plan.mma_rows, a.d, a.bs, a.d / a.group, grid, stream)
            : plan.mma_rows == 4 ? launch_mma<FourRows>(P, a.d, a.bs, a.d / a.group, grid, stream)
                                 : launch_mma<EightRows>(P, a.d, a.bs, a.d / a.group, grid, stream);
    } else {
        e = launch_simt(a, kp, stream);
    }
    if (e != cudaSuccess || plan.splits == 1 || plan.fused_merge) return e;
    return launch_decode_merge(kp, a.d, a.bs, static_cast<unsigned>(a.rows * a.Hq), stream);
}

}  // namespace pkv
