// decode_sinks.cuh -- what the kernels of paged attention with a window and first tokens that stay visible
// (sinks) share: the work of a block, numbers in three bf16 parts, and the end of a block (not part of the ABI).
#pragma once

#include <math.h>

#include "common.cuh"
#include "decode_kparams.cuh"
#include "internal.h"

namespace pkv {

constexpr int kSinksFusedChunks = 8;   // chunks of a sequence merged by its last block; more of them by the merge kernel

// x0, x1 as three bf16 parts each, packed in pairs.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x1), "f"(x0));
    const float r0 = x0 - __uint_as_float(hi << 16), r1 = x1 - __uint_as_float(hi & 0xffff0000u);
    split_bf16x2(r0, r1, mid, lo);
}

// What a block attends: pairs slot0 .. slot0 + npairs - 1 of sequence b's (row, head) slots (row = slot / m) for one
// KV head, over pages pg0 .. pg1 - 1 (numbered without the gap).  Its rows see the tokens [0, S) and [lo, hi)
// between them, and each of them all of [.., S) and [all_lo, all_hi).
struct SinksWork {
    int b, kvh, group, split, nc;   // nc: chunks of the sequence
    int slot0, npairs, c0, P0;      // c0: the sequence's first query row; P0: its position
    int pg0, pg1, lo, hi, all_lo, all_hi, shift;
    SeqSpan sp;

    __device__ __forceinline__ size_t row_of(const DecodeKParams &p, int pair) const {   // of out, lse, q
        const int slot = slot0 + pair;
        return static_cast<size_t>(c0 + slot / p.m) * p.Hq + kvh * p.m + slot % p.m;
    }
    __device__ __forceinline__ int position(const DecodeKParams &p, int pair) const { return P0 + (slot0 + pair) / p.m; }
    // the first token of its window, and one past its last token, of the row at a position
    __device__ __forceinline__ int lo_of(const DecodeKParams &p, int pos) const { return max(0, pos + 1 - p.window) - shift; }
    __device__ __forceinline__ int hi_of(int pos) const { return pos + 1 - shift; }
};

// The block's work: grid x = (chunk, group of pairs) with the group fastest, y = KV head, z = sequence.  False: none
// (rows that the sequence may not own, or of an empty one, have been written).
template <int D, int BS, int PAIRS>
__device__ __forceinline__ bool sinks_work(const DecodeKParams &p, int groups, SinksWork &w) {
    w.group = blockIdx.x % groups;
    w.split = blockIdx.x / groups;
    w.kvh = blockIdx.y;
    w.b = blockIdx.z;
    const bool report = threadIdx.x == 0 && blockIdx.x == 0 && w.kvh == 0;
    const int L = checked_len(p, w.b, BS, report);
    int nq = 1;
    w.c0 = w.b;
    if (p.cu_q != nullptr) {
        w.c0 = __ldg(p.cu_q + w.b);
        const int c1 = __ldg(p.cu_q + w.b + 1);
        nq = c1 - w.c0;
        if (!query_rows_ok(p, w.c0, c1, L)) {   // those of its rows that the call has: out = 0, lse = -inf
            if (report) raise_error(p.err, PKV_DEVERR_CU_SEQLENS);
            if (blockIdx.x != 0) return false;
            for (int r = max(w.c0, 0); r < min(c1, p.rows); ++r) {
                const size_t at = static_cast<size_t>(r) * p.Hq + w.kvh * p.m;
                for (int i = threadIdx.x; i < p.m * D; i += blockDim.x) p.out[at * D + i] = 0.f;
                if (p.lse != nullptr)
                    for (int i = threadIdx.x; i < p.m; i += blockDim.x) p.lse[at + i] = -INFINITY;
            }
            return false;
        }
    }
    w.slot0 = w.group * PAIRS;
    w.npairs = min(PAIRS, nq * p.m - w.slot0);
    if (w.npairs <= 0) return false;
    if (L == 0) {
        if (w.split != 0) return false;
        for (int i = threadIdx.x; i < w.npairs * D; i += blockDim.x) p.out[w.row_of(p, i / D) * D + i % D] = 0.f;
        if (p.lse != nullptr)
            for (int i = threadIdx.x; i < w.npairs; i += blockDim.x) p.lse[w.row_of(p, i)] = -INFINITY;
        return false;
    }
    w.P0 = L - nq;
    w.sp = sinks_span(p, w.b, L, max(0, w.P0 + 1 - p.window), BS);
    w.shift = w.sp.gap * BS;
    const int first = w.position(p, 0), last = w.position(p, w.npairs - 1);
    w.lo = w.lo_of(p, first);
    w.hi = w.hi_of(last);
    w.all_lo = w.lo_of(p, last);
    w.all_hi = w.hi_of(first);
    w.nc = (w.sp.npages + p.chunk_pages - 1) / p.chunk_pages;
    const int cp0 = w.split * p.chunk_pages, cp1 = min(w.sp.npages, cp0 + p.chunk_pages);
    w.pg0 = cp0 < w.sp.spages ? cp0 : max(cp0, w.lo / BS);
    w.pg1 = min(cp1, (w.hi + BS - 1) / BS);
    return cp0 < cp1;
}

// The end of a block: shared memory holds, from `smem`, the pairs' log-sum-exp (base 2) and NV parts of their
// normalised outputs, [NV][PAIRS][D], which only remain to be added; the block has synchronised.  A sequence of one
// chunk writes out and lse; otherwise the chunk's partial goes to the workspace, and where that has arrival
// counters the block that completes a group of pairs merges its chunks (nobody waits).  s_last: a number in shared
// memory, apart.
template <int D, int PAIRS, int NV>
__device__ __forceinline__ void finish_sinks(uint8_t *smem, int *s_last, const DecodeKParams &p, const SinksWork &w, int groups) {
    const float *lse2 = reinterpret_cast<const float *>(smem), *ow = lse2 + PAIRS;
    const bool vec = reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
    auto put = [&](float *dst, float4 x) {
        if (vec) {
            *reinterpret_cast<float4 *>(dst) = x;
        } else {
            dst[0] = x.x;
            dst[1] = x.y;
            dst[2] = x.z;
            dst[3] = x.w;
        }
    };
    for (int i = threadIdx.x; i < w.npairs * (D / 4); i += blockDim.x) {
        const int pair = i / (D / 4), c = i % (D / 4) * 4;
        float4 x = *reinterpret_cast<const float4 *>(ow + pair * D + c);
#pragma unroll
        for (int v = 1; v < NV; ++v) {
            const float4 y = *reinterpret_cast<const float4 *>(ow + (v * PAIRS + pair) * D + c);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
        }
        const size_t row = w.row_of(p, pair);
        if (w.nc == 1) {
            put(p.out + row * D + c, x);
            if (c == 0 && p.lse != nullptr) p.lse[row] = lse2[pair] * kDecLn2;
        } else {
            *reinterpret_cast<float4 *>(p.ws_o + (row * p.splits + w.split) * D + c) = x;
            if (c == 0) p.ws_lse[row * p.splits + w.split] = lse2[pair];
        }
    }
    if (w.nc == 1 || p.counters == nullptr) return;

    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned *ctr = p.counters + (static_cast<size_t>(w.b) * p.Hkv + w.kvh) * groups + w.group;
        *s_last = atomicAdd(ctr, 1u) + 1 == static_cast<unsigned>(w.nc);
        if (*s_last) *ctr = 0u;   // every chunk of this call has arrived
    }
    __syncthreads();
    if (!*s_last) return;
    __threadfence();
    float *wt = reinterpret_cast<float *>(smem);   // [pairs][chunks] the chunks' weights
    if (threadIdx.x < w.npairs) {
        const size_t row = w.row_of(p, threadIdx.x);
        float x[kSinksFusedChunks], M = -INFINITY, l = 0.f;
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) {
            x[c] = c < w.nc ? __ldcg(p.ws_lse + row * p.splits + c) : -INFINITY;
            M = fmaxf(M, x[c]);
        }
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) {
            x[c] = ex2_approx(x[c] - M);
            l += x[c];
        }
        const float il = 1.f / l;
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) wt[threadIdx.x * kSinksFusedChunks + c] = x[c] * il;
        if (p.lse != nullptr) p.lse[row] = (M + log2f(l)) * kDecLn2;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < w.npairs * (D / 4); i += blockDim.x) {
        const int pair = i / (D / 4), c4 = i % (D / 4) * 4;
        const size_t row = w.row_of(p, pair);
        const float *po = p.ws_o + row * p.splits * D + c4;
        float4 y[kSinksFusedChunks], acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c)
            y[c] = c < w.nc ? __ldcg(reinterpret_cast<const float4 *>(po + static_cast<size_t>(c) * D)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) {
            const float f = wt[pair * kSinksFusedChunks + c];
            acc.x += f * y[c].x;
            acc.y += f * y[c].y;
            acc.z += f * y[c].z;
            acc.w += f * y[c].w;
        }
        put(p.out + row * D + c4, acc);
    }
}

// The kernel on tcgen05 (decode_sinks_umma.cu): d in {64, 128}, kSinksUmmaPairs pairs a block, two blocks an SM; 16-byte
// aligned shared memory aside, what the caller of launch_decode_sinks checks.
constexpr int kSinksUmmaPairs = 32, kSinksUmmaKeys = 64;
constexpr int kSinksMmaPairs = 8;   // up to here the warp-MMA kernel
cudaError_t launch_decode_sinks_umma(const DecodeKParams &kp, const CUtensorMap &tk, const CUtensorMap &tv, int d, int bs, int groups,
                                     cudaStream_t stream);

// The kernel on CUDA cores (decode_sinks_simt.cu): every type, size and alignment.
void plan_sinks_simt(SinksPlan &plan, int rows, int Hq, int Hkv, int d, int bs, int pages, int num_splits, int sm_count);
cudaError_t launch_decode_sinks_simt(const DecodeKParams &kp, const void *k_cache, const void *v_cache, pkv_dtype dt, int d, int bs,
                                     int block_heads, cudaStream_t stream);

}  // namespace pkv
