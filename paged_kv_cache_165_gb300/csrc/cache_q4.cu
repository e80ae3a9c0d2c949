// cache_q4.cu -- writes into and reads out of the 4-bit paged cache.
//
// kv_append_q4: each new token's K and V rows, quantised as q4_codes.cuh says, into the slot
//   slot_mapping[t] names (limoncc.com "大语言模型研究15——注意力机制优化之KV缓存" §2; the
//   low-bit trade-off of zwjcode.cn "KV Cache 的增量解码" §14).
// kv_gather_q4: the values of the rows in given slots, as bf16 or fp32 rows.
//
// Append: a thread owns sixteen consecutive elements (two 32-bit words of codes), so a group is 2, 4
// or 8 neighbouring lanes whatever the head size: groups never straddle a warp because its 512
// elements are a multiple of each group size.  Bound by its instructions (about 17 an element: extremes,
// an exactly rounded quotient, the pack; 15 us of them for the case below) and by its loads, which a
// thread waits for before its arithmetic with none of the next turn in flight (issue 64%, most stalls
// on loads).  The scale's and the address's share counts: with eight elements a thread 17153 tokens of 8 heads x 128 (bf16) took 35.9 us, with
// sixteen 25.9 (3.5 TB/s; 13.3 at the copy rate), with 32 (two blocks per SM) 29.  Both rows are loaded
// before either's arithmetic, which costs a few spilled registers at four blocks per SM (three: 26.9).
// Gather: a thread owns eight; its stores bound it (32768 tokens, 34 us, 5.0 TB/s).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "q4_codes.cuh"

namespace pkv {
namespace {

// n / d for 0 <= n < 2^31 by a multiplication: mul = ceil(2^(31 + s) / d), s = ceil(log2 d), is off
// by less than d <= 2^s over 2^(31 + s), which n < 2^31 cannot make visible.
struct FastDiv {
    uint32_t d, mul;
    int shift;   // s - 1; -1: d is 1
};
FastDiv fast_div(uint32_t d) {
    int s = 0;
    while ((1ull << s) < d) ++s;
    return {d, static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), s - 1};
}
__device__ __forceinline__ int div_by(int n, const FastDiv &f) {
    return f.shift < 0 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), f.mul) >> f.shift);
}

// 64-bit divisions would cost as much as the rest: words are numbered in 32 bits (a launch takes
// fewer than 2^31), and slots too unless the cache holds more than 2^31 of them.
struct Q4Rows {
    const int64_t *slots;
    int words;           // a thread's parts of K (and as many of V): T * Hkv * d / per
    int Hkv, row_words;  // d / per
    int lanes;           // threads that share a group: group / per
    int bs, page_bytes;  // bs * row bytes
    FastDiv by_row, by_head, by_bs;
    long long n_slots;
    unsigned *err;
};

// Where word w of the new rows lives: its page's byte offset, its row in the page and its
// position in the row; slot < 0 when the token is padding or its slot is out of range.
struct Q4Place {
    long long slot, page;
    int off, j;
};
__device__ __forceinline__ Q4Place q4_place(const Q4Rows &r, int w) {
    Q4Place a;
    const int th = div_by(w, r.by_row);   // t * Hkv + h
    a.j = w - th * r.row_words;
    const int t = div_by(th, r.by_head), h = th - t * r.Hkv;
    a.slot = __ldg(r.slots + t);
    if (a.slot >= r.n_slots) {
        if (h == 0 && a.j == 0) raise_error(r.err, PKV_DEVERR_SLOT);
        a.slot = -1;
    }
    const long long blk = r.n_slots <= 0x7fffffffll ? div_by(static_cast<int>(max(a.slot, 0ll)), r.by_bs) : max(a.slot, 0ll) / r.bs;
    a.off = static_cast<int>(a.slot - blk * r.bs);
    a.page = (blk * r.Hkv + h) * r.page_bytes;
    return a;
}

constexpr int kAppendWords = 2;   // of codes, for each thread of an append

template <typename T, bool VEC, int LANES>
__global__ void __launch_bounds__(256, 4)
    kv_append_q4_kernel(const T *__restrict__ k_new, const T *__restrict__ v_new, uint8_t *__restrict__ kc,
                        uint8_t *__restrict__ vc, const Q4Rows r) {
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
    constexpr int W = kAppendWords;
    // whole warps run each turn: the group's lanes exchange their extremes
    for (long long w0 = blockIdx.x * static_cast<long long>(blockDim.x) + (threadIdx.x & ~31); w0 < r.words;
         w0 += stride) {
        const int w = static_cast<int>(w0) + static_cast<int>(threadIdx.x & 31);
        const Q4Place a = q4_place(r, min(w, r.words - 1));
        const bool live = w < r.words && a.slot >= 0;
        Q4Loaded<T, W> x[2];   // both rows' loads before either's arithmetic
        q4_load<VEC, W>(live ? k_new + static_cast<size_t>(w) * (8 * W) : nullptr, x[0].v);
        q4_load<VEC, W>(live ? v_new + static_cast<size_t>(w) * (8 * W) : nullptr, x[1].v);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            __half2 par;
            uint32_t code[W];
            q4_quantise_loaded<LANES, W>(x[side].v, par, code);
            if (!live) continue;
            uint8_t *page = (side ? vc : kc) + a.page;
            uint32_t *dst = reinterpret_cast<uint32_t *>(page) + (a.off * r.row_words + a.j) * W;
#pragma unroll
            for (int i = 0; i < W; ++i) dst[i] = code[i];
            if (a.j % LANES == 0)
                reinterpret_cast<__half2 *>(page + r.bs * r.row_words * (4 * W))[a.off * (r.row_words / LANES) + a.j / LANES] = par;
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
    kv_gather_q4_kernel(T *__restrict__ k_out, T *__restrict__ v_out, const uint8_t *__restrict__ kc,
                        const uint8_t *__restrict__ vc, const Q4Rows r) {
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long w0 = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; w0 < r.words; w0 += stride) {
        const int w = static_cast<int>(w0);
        const Q4Place a = q4_place(r, w);
        uint32_t code[2] = {0, 0};
        __half2 par[2];
        par[0] = par[1] = __floats2half2_rn(0.f, 0.f);
        if (a.slot >= 0) {
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const uint8_t *page = (side ? vc : kc) + a.page;
                code[side] = __ldg(reinterpret_cast<const uint32_t *>(page) + a.off * r.row_words + a.j);
                par[side] = __ldg(reinterpret_cast<const __half2 *>(page + r.bs * r.row_words * 4) +
                                  a.off * (r.row_words / r.lanes) + a.j / r.lanes);
            }
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            // A code in the low bits of an f16 is the subnormal code * 2^-24, four bits further up
            // code * 2^-20: widened to fp32 exactly, the power of two goes into the scale.
            const float2 p = __half22float2(par[side]);
            const float s0 = p.x * 0x1p24f, s1 = p.x * 0x1p20f;
            float x[8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // elements 2i, 2i + 4 and 2i + 1, 2i + 5
                const uint32_t u = code[side] >> (8 * i), lo = u & 0x000f000fu, hi = u & 0x00f000f0u;
                const float2 a0 = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                const float2 a1 = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                x[2 * i] = fmaf(s0, a0.x, p.y);
                x[2 * i + 4] = fmaf(s0, a0.y, p.y);
                x[2 * i + 1] = fmaf(s1, a1.x, p.y);
                x[2 * i + 5] = fmaf(s1, a1.y, p.y);
            }
            T *dst = (side ? v_out : k_out) + static_cast<size_t>(w) * 8;
            if constexpr (sizeof(T) == 2) {
                // the fp32 value (one rounding of zero + scale * code) rounded to bf16
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
                if constexpr (VEC) {
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint16_t *>(dst)[i] = static_cast<uint16_t>(u[i / 2] >> (16 * (i & 1)));
                }
            } else if constexpr (VEC) {
                reinterpret_cast<float4 *>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i] = x[i];
            }
        }
    }
}

Q4Rows rows_of(const int64_t *slots, int T, int Hkv, int d, int group, int bs, int NB, int per, unsigned *err) {
    Q4Rows r;
    r.slots = slots;
    r.words = T * Hkv * (d / per);
    r.by_row = fast_div(d / per);
    r.by_head = fast_div(Hkv);
    r.by_bs = fast_div(bs);
    r.Hkv = Hkv;
    r.row_words = d / per;
    r.lanes = group / per;
    r.bs = bs;
    r.page_bytes = bs * q4_row_bytes(d, group);
    r.n_slots = static_cast<long long>(NB) * bs;
    r.err = err;
    return r;
}

// Tokens of one launch: fewer than 2^31 words (Hkv * d / 8 is below 2^21).
int tokens_per_launch(int Hkv, int d) { return std::max(1, (0x7fffffff - 256) / (Hkv * (d / 8))); }

unsigned grid_of(long long words, int sm_count) {
    return static_cast<unsigned>(std::min<long long>((words + 255) / 256, 8ll * sm_count));
}

bool aligned(const void *a, const void *b, unsigned n) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & (n - 1)) == 0;
}

}  // namespace

cudaError_t launch_kv_append_q4(const void *k_new, const void *v_new, pkv_dtype new_dt, uint8_t *k_cache,
                                uint8_t *v_cache, const int64_t *slot_mapping, int T, int Hkv, int d, int group,
                                int bs, int NB, int sm_count, unsigned *err, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    if (const int most = tokens_per_launch(Hkv, d); T > most) {
        const size_t skip = static_cast<size_t>(most) * Hkv * d * (new_dt == PKV_BF16 ? 2 : 4);
        const cudaError_t e = launch_kv_append_q4(k_new, v_new, new_dt, k_cache, v_cache, slot_mapping, most, Hkv, d, group,
                                                  bs, NB, sm_count, err, stream);
        if (e != cudaSuccess) return e;
        return launch_kv_append_q4(static_cast<const uint8_t *>(k_new) + skip, static_cast<const uint8_t *>(v_new) + skip,
                                   new_dt, k_cache, v_cache, slot_mapping + most, T - most, Hkv, d, group, bs, NB, sm_count,
                                   err, stream);
    }
    const Q4Rows r = rows_of(slot_mapping, T, Hkv, d, group, bs, NB, 8 * kAppendWords, err);
    const unsigned grid = grid_of(r.words, sm_count);
    const bool vec = aligned(k_new, v_new, 16);
#define PKV_Q4_APPEND(TT, VV, LL)                                                                     \
    kv_append_q4_kernel<TT, VV, LL><<<grid, 256, 0, stream>>>(static_cast<const TT *>(k_new),         \
                                                              static_cast<const TT *>(v_new), k_cache, v_cache, r)
#define PKV_Q4_APPEND_L(TT, VV)                       \
    switch (r.lanes) {                                \
        case 2: PKV_Q4_APPEND(TT, VV, 2); break;      \
        case 4: PKV_Q4_APPEND(TT, VV, 4); break;      \
        default: PKV_Q4_APPEND(TT, VV, 8); break;     \
    }
    if (new_dt == PKV_BF16) {
        if (vec) PKV_Q4_APPEND_L(__nv_bfloat16, true)
        else PKV_Q4_APPEND_L(__nv_bfloat16, false)
    } else {
        if (vec) PKV_Q4_APPEND_L(float, true)
        else PKV_Q4_APPEND_L(float, false)
    }
#undef PKV_Q4_APPEND_L
#undef PKV_Q4_APPEND
    return cudaGetLastError();
}

cudaError_t launch_kv_gather_q4(void *k_out, void *v_out, pkv_dtype out_dt, const uint8_t *k_cache,
                                const uint8_t *v_cache, const int64_t *slot_mapping, int T, int Hkv, int d,
                                int group, int bs, int NB, int sm_count, unsigned *err, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    if (const int most = tokens_per_launch(Hkv, d); T > most) {
        const size_t skip = static_cast<size_t>(most) * Hkv * d * (out_dt == PKV_BF16 ? 2 : 4);
        const cudaError_t e = launch_kv_gather_q4(k_out, v_out, out_dt, k_cache, v_cache, slot_mapping, most, Hkv, d, group,
                                                  bs, NB, sm_count, err, stream);
        if (e != cudaSuccess) return e;
        return launch_kv_gather_q4(static_cast<uint8_t *>(k_out) + skip, static_cast<uint8_t *>(v_out) + skip, out_dt,
                                   k_cache, v_cache, slot_mapping + most, T - most, Hkv, d, group, bs, NB, sm_count, err,
                                   stream);
    }
    const Q4Rows r = rows_of(slot_mapping, T, Hkv, d, group, bs, NB, 8, err);
    const unsigned grid = grid_of(r.words, sm_count);
    const bool vec = aligned(k_out, v_out, 16);
#define PKV_Q4_GATHER(TT, VV)                                                                     \
    kv_gather_q4_kernel<TT, VV><<<grid, 256, 0, stream>>>(static_cast<TT *>(k_out),               \
                                                          static_cast<TT *>(v_out), k_cache, v_cache, r)
    if (out_dt == PKV_BF16) {
        if (vec) PKV_Q4_GATHER(__nv_bfloat16, true);
        else PKV_Q4_GATHER(__nv_bfloat16, false);
    } else {
        if (vec) PKV_Q4_GATHER(float, true);
        else PKV_Q4_GATHER(float, false);
    }
#undef PKV_Q4_GATHER
    return cudaGetLastError();
}

}  // namespace pkv
