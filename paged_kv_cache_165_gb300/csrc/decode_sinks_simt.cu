// decode_sinks_simt.cu -- paged attention with a window and first tokens that stay visible (sinks) on CUDA cores:
// fp32 caches, and bf16 ones of the sizes that the tensor-core kernels do not take.  What is computed and how the gap
// between the sinks and the window is left out stand in decode_sinks.cu.
//
// A block of four warps has one query row, up to kHeads heads of one KV head and a chunk of the row's pages.  Of a chunk
// a row sees at most two runs of tokens, which are numbered through, so that nothing unseen is read or masked.  The warps
// take batches of tokens in turn: a batch's K and V rows (lanes own elements lane + 32 j) are loaded together, its scores
// reduced together -- halves of the batch are exchanged between halves of the warp, so that eight sums take nine
// shuffles -- and the running maximum and sum move once a batch.  The warps' states meet in shared memory; where a row has
// several chunks, the block that completes them merges their partials.
//
// Small calls are bound by this chain's latency, larger ones by loads in flight (12 warps of 145 registers an SM).  2 sequences
// of 18 to 41 tokens, 8 heads on 2 of 64 in fp32: 6.3 us (a warp a head and one token at a time: 10.4); 32 of 4000 to 8000,
// window 2048 + 4, of 128 in fp32: 8 heads on 8 114 us (299), 4.7 TB/s, 32 on 8 149 (566): K and V come again for each four heads
// and each row.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "decode_kparams.cuh"
#include "decode_sinks.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kHeads = 4;          // of a block at most: registers of q and of the outputs (two above d = 128)

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// A lane owns elements V (lane + 32 j) .. + V - 1 of a head, j < J.
template <int V, int J>
struct SimtCfg {
    static constexpr int kOwn = V * J;                          // elements of a lane
    static constexpr int kBatch = kOwn <= 4 ? 8 : 4;            // tokens
    static constexpr int kMasks = kOwn <= 4 ? 3 : 2;            // log2 of it
    static constexpr int kMost = kOwn <= 4 ? kHeads : kHeads / 2;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece { T x[V]; };

// Sums of x[0 .. N) over the warp, N = 2^M: the lane whose upper M bits (of 5) are k gets that of x[k].
template <int N, int M>
__device__ __forceinline__ float sum_each(float (&x)[N], int lane) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int mask = 16 >> m, half = N >> (m + 1);
        const bool upper = lane & mask;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = upper ? x[half + i] : x[i], give = upper ? x[i] : x[half + i];
            x[i] = keep + __shfl_xor_sync(kFull, give, mask);
        }
    }
#pragma unroll
    for (int mask = 16 >> M; mask > 0; mask >>= 1) x[0] += __shfl_xor_sync(kFull, x[0], mask);
    return x[0];
}

template <typename T, int V, int J>
__global__ void __launch_bounds__(kThreads)
    decode_sinks_simt_kernel(const T *__restrict__ kc, const T *__restrict__ vc, const DecodeKParams p, const int d, const int bs,
                             const int block_heads) {
    using C = SimtCfg<V, J>;
    constexpr int KB = C::kBatch, M = C::kMasks, H = C::kMost, E = C::kOwn;
    __shared__ float s_o[kWarps][H][32 * E];
    __shared__ float2 s_ml[kWarps][H];      // running maximum (base 2) and sum
    __shared__ float s_w[H][kSinksFusedChunks];
    __shared__ int s_last;
    pdl_launch_dependents();   // a merge kernel after this one waits for the whole grid
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x, split = blockIdx.z, tiles = (p.m + block_heads - 1) / block_heads;
    const int kvh = blockIdx.y / tiles, tile = blockIdx.y % tiles, nh = min(block_heads, p.m - tile * block_heads);
    if (p.cu_q != nullptr) {   // rows behind the last sequence's (a padded batch) are left as they are
        const int end = __ldg(p.cu_q + p.B);
        if (row >= end && end >= max(0, __ldg(p.cu_q + p.B - 1))) return;
    }
    const SeqSpan sp = row_span<true>(p, row, bs, threadIdx.x == 0 && blockIdx.y == 0 && split == 0);
    const int nc = (sp.cnpages + p.chunk_pages - 1) / p.chunk_pages;   // the sequence's chunks
    const int c0 = split * p.chunk_pages, c1 = min(sp.cnpages, c0 + p.chunk_pages);
    const size_t bi = static_cast<size_t>(row) * p.Hq + kvh * p.m + tile * block_heads;   // the first head's row of out
    if (c0 >= c1) {
        if (split == 0) {   // an empty sequence: out = 0, lse = -inf
            for (int i = threadIdx.x; i < nh * d; i += kThreads) p.out[bi * d + i] = 0.f;
            if (threadIdx.x < nh && p.lse != nullptr) p.lse[bi + threadIdx.x] = -INFINITY;
        }
        return;
    }
    // the row's tokens of this chunk: n1 from `begin` on (sinks), then n2 from `from` on (its window)
    const int begin = c0 * bs, end = min(c1 * bs, sp.len);
    const int n1 = max(0, min(p.sinks, end) - begin), from = max(begin, max(sp.lo, p.sinks));
    const int n = n1 + max(0, end - from);

    float qv[H][E], acc[H][E], m_run[H], l_run[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        m_run[h] = -INFINITY;
        l_run[h] = 0.f;
#pragma unroll
        for (int x = 0; x < E; ++x) {
            const int e = V * (lane + 32 * (x / V)) + x % V;
            qv[h][x] = h < nh && e < d ? __ldg(p.q + (bi + h) * d + e) : 0.f;
            acc[h][x] = 0.f;
        }
    }
    bool own[J];   // only a head's last elements may be missing, V at a time
#pragma unroll
    for (int j = 0; j < J; ++j) own[j] = j < J - 1 || V * (lane + 32 * j) < d;
    // where the row of token i of the chunk starts (-1: past them, or in no block; such a block reads as zeros)
    auto row_at = [&](int i) {
        if (i >= n) return -1ll;
        const int v = i < n1 ? begin + i : from + (i - n1), page = v / bs;
        const int phys = __ldg(p.block_table + static_cast<size_t>(sp.b) * p.MBS + page_entry(sp, page));
        if (phys < 0 || phys >= p.NB) {
            raise_error(p.err, PKV_DEVERR_BLOCK);
            return -1ll;
        }
        return ((static_cast<long long>(phys) * p.Hkv + kvh) * bs + (v - page * bs)) * d;
    };
    const int mine = lane >> (5 - M);   // the token of a batch whose score this lane gets
    long long at = row_at(warp * KB + lane % KB);
    for (int i0 = warp * KB; i0 < n; i0 += kWarps * KB) {
        Piece<T, V> k[KB][J], v[KB][J];
#pragma unroll
        for (int i = 0; i < KB; ++i) {
            const long long r = __shfl_sync(kFull, at, i);
            const T *pk = kc + r + V * lane, *pv = vc + r + V * lane;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                k[i][j] = v[i][j] = Piece<T, V>{};
                if (r >= 0 && own[j]) {
                    k[i][j] = *reinterpret_cast<const Piece<T, V> *>(pk + 32 * V * j);
                    v[i][j] = *reinterpret_cast<const Piece<T, V> *>(pv + 32 * V * j);
                }
            }
        }
        at = row_at(i0 + kWarps * KB + lane % KB);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (h >= nh) break;
            float dot[KB];
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                dot[i] = 0.f;
#pragma unroll
                for (int x = 0; x < E; ++x) dot[i] += qv[h][x] * widen(k[i][x / V].x[x % V]);
            }
            const float sum_of_mine = sum_each<KB, M>(dot, lane);   // shuffles of the whole warp, past its last token too
            const float s = i0 + mine < n ? sum_of_mine * p.scale_log2 : -INFINITY;
            float mx = s;
#pragma unroll
            for (int m = 0; m < M; ++m) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16 >> m));
            const float m_new = fmaxf(m_run[h], mx), alpha = exp2f(m_run[h] - m_new), w = exp2f(s - m_new);
            float sum = w;
#pragma unroll
            for (int m = 0; m < M; ++m) sum += __shfl_xor_sync(kFull, sum, 16 >> m);
            l_run[h] = l_run[h] * alpha + sum;
            m_run[h] = m_new;
#pragma unroll
            for (int x = 0; x < E; ++x) acc[h][x] *= alpha;
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                const float wi = __shfl_sync(kFull, w, i << (5 - M));
#pragma unroll
                for (int x = 0; x < E; ++x) acc[h][x] += wi * widen(v[i][x / V].x[x % V]);
            }
        }
    }
    // ---- the warps' states to the block's
#pragma unroll
    for (int h = 0; h < H; ++h) {
        if (h >= nh) break;
        if (lane == 0) s_ml[warp][h] = make_float2(m_run[h], l_run[h]);
#pragma unroll
        for (int x = 0; x < E; ++x) s_o[warp][h][V * (lane + 32 * (x / V)) + x % V] = acc[h][x];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * 32 * E; i += kThreads) {
        const int h = i / (32 * E), e = i % (32 * E);
        float mw[kWarps], mx = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mw[w] = s_ml[w][h].x;
            mx = fmaxf(mx, mw[w]);
        }
        const float ref = mx == -INFINITY ? 0.f : mx;   // the chunk may hold keys of the sequence's other rows alone
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(mw[w] - ref);
            l += s_ml[w][h].y * f;
            o += s_o[w][h][e] * f;
        }
        o = l == 0.f ? 0.f : o / l;
        if (e < d) {
            if (nc == 1) p.out[(bi + h) * d + e] = o;
            else p.ws_o[((bi + h) * p.splits + split) * d + e] = o;
        }
        if (e == 0) {
            const float lse2 = mx + log2f(l);
            if (nc > 1) p.ws_lse[(bi + h) * p.splits + split] = lse2;
            else if (p.lse != nullptr) p.lse[bi + h] = lse2 * kDecLn2;
        }
    }
    if (nc == 1 || p.counters == nullptr) return;
    // ---- the last chunk to arrive merges them
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned *ctr = p.counters + static_cast<size_t>(row) * gridDim.y + blockIdx.y;
        s_last = atomicAdd(ctr, 1u) + 1 == static_cast<unsigned>(nc);
        if (s_last) *ctr = 0u;   // every chunk of this call has arrived
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    if (threadIdx.x < nh) {
        float x[kSinksFusedChunks], mx = -INFINITY, l = 0.f;
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) {
            x[c] = c < nc ? __ldcg(p.ws_lse + (bi + threadIdx.x) * p.splits + c) : -INFINITY;
            mx = fmaxf(mx, x[c]);
        }
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) {
            x[c] = exp2f(x[c] - mx);
            l += x[c];
        }
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) s_w[threadIdx.x][c] = x[c] / l;
        if (p.lse != nullptr) p.lse[bi + threadIdx.x] = (mx + log2f(l)) * kDecLn2;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nh * d; i += kThreads) {
        const int h = i / d, e = i % d;
        float y[kSinksFusedChunks], o = 0.f;
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c)
            y[c] = c < nc ? __ldcg(p.ws_o + ((bi + h) * p.splits + c) * d + e) : 0.f;
#pragma unroll
        for (int c = 0; c < kSinksFusedChunks; ++c) o += s_w[h][c] * y[c];
        p.out[(bi + h) * d + e] = o;
    }
}

template <typename T>
cudaError_t launch(const T *kc, const T *vc, const DecodeKParams &kp, dim3 grid, int d, int bs, int block_heads, cudaStream_t stream) {
    // four elements side by side where a warp has work for them (two up to d = 64), else one
    const int wide = d > 64 ? 4 : 2;
    const bool pieces = d % wide == 0 && (reinterpret_cast<uintptr_t>(kc) | reinterpret_cast<uintptr_t>(vc)) % (wide * sizeof(T)) == 0;
#define PKV_SINKS_SIMT(V, J) decode_sinks_simt_kernel<T, V, J><<<grid, kThreads, 0, stream>>>(kc, vc, kp, d, bs, block_heads)
    if (pieces && d > 128) {
        PKV_SINKS_SIMT(4, 2);
    } else if (pieces && d > 64) {
        PKV_SINKS_SIMT(4, 1);
    } else if (pieces) {
        PKV_SINKS_SIMT(2, 1);
    } else {
        switch ((d + 31) / 32) {
            case 1: PKV_SINKS_SIMT(1, 1); break;
            case 2: PKV_SINKS_SIMT(1, 2); break;
            case 3: PKV_SINKS_SIMT(1, 3); break;
            case 4: PKV_SINKS_SIMT(1, 4); break;
            case 5: PKV_SINKS_SIMT(1, 5); break;
            case 6: PKV_SINKS_SIMT(1, 6); break;
            case 7: PKV_SINKS_SIMT(1, 7); break;
            default: PKV_SINKS_SIMT(1, 8);
        }
    }
#undef PKV_SINKS_SIMT
    return cudaGetLastError();
}

}  // namespace

// Heads of a block and chunks of a sequence on CUDA cores, by a model of the time in tokens of one head: a block costs its
// tokens and 128 more, each further head of a block 0.24 of that, a wave of blocks (five an SM up to d = 64, three
// above) as much as a block, an incomplete one between its share and a whole one, a merge 64, and more chunks than a
// block merges 256.  (512 rows x KV heads of four heads of 64, window 1024: one chunk 72 us, two 53, three 60, with two
// heads a block 63, 67 and 70; 256 of 128, window 2048: 211, 223, 164 and, two heads a block, 315, 254, 233.)  No chunk is
// longer than 8192 tokens.
void plan_sinks_simt(SinksPlan &plan, int rows, int Hq, int Hkv, int d, int bs, int pages, int num_splits, int sm_count) {
    const int m = Hq / Hkv;
    const long long tokens = static_cast<long long>(pages) * bs, slots = static_cast<long long>(d <= 64 ? 5 : 3) * std::max(sm_count, 1);
    const long long most = std::min<long long>(pages, kDecodeMaxChunks);
    // at least one, so that no count of rows divides by zero
    auto units = [&](int heads) { return std::max(1ll, static_cast<long long>(rows) * Hkv * ((m + heads - 1) / heads)); };
    double best = -1;
    long long splits = 1;
    auto consider = [&](int heads, long long k) {
        if (k < 1 || k > most) return;
        const double waves = static_cast<double>(units(heads) * k) / slots;
        const double cost = (waves <= 1 ? 1 : (waves + std::ceil(waves)) / 2) * (128.0 + static_cast<double>(tokens) / k) *
                                (0.76 + 0.24 * heads) + (k > kSinksFusedChunks ? 256.0 : k > 1 ? 64.0 : 0.0);
        if (best >= 0 && cost >= best) return;
        best = cost;
        splits = k;
        plan.block_heads = heads;
    };
    const long long least = std::min((tokens + 8191) / 8192, most);
    for (int heads = 1; heads <= std::min(m, d <= 128 ? kHeads : kHeads / 2); heads = heads < m ? std::min(2 * heads, m) : m + 1) {
        if (num_splits > 0) {
            consider(heads, std::min<long long>(num_splits, most));
            continue;
        }
        for (long long k = least; k <= kSinksFusedChunks; ++k) consider(heads, k);
        consider(heads, least);
        if (slots / units(heads) > std::max<long long>(kSinksFusedChunks, least))
            consider(heads, std::min(slots / units(heads), std::max(least, tokens / 256)));
    }
    plan.chunk_pages = static_cast<int>((pages + splits - 1) / splits);
    plan.splits = (pages + plan.chunk_pages - 1) / plan.chunk_pages;
    plan.fused_merge = plan.splits > 1 && plan.splits <= kSinksFusedChunks &&
                       units(plan.block_heads) <= static_cast<long long>(PKV_DECODE_COUNTER_BYTES / sizeof(unsigned));
}

cudaError_t launch_decode_sinks_simt(const DecodeKParams &kp, const void *k_cache, const void *v_cache, pkv_dtype dt, int d, int bs,
                                     int block_heads, cudaStream_t stream) {
    const int tiles = (kp.m + block_heads - 1) / block_heads;
    const dim3 grid(kp.rows, kp.Hkv * tiles, kp.splits);
    if (dt == PKV_F32)
        return launch(static_cast<const float *>(k_cache), static_cast<const float *>(v_cache), kp, grid, d, bs, block_heads, stream);
    return launch(static_cast<const __nv_bfloat16 *>(k_cache), static_cast<const __nv_bfloat16 *>(v_cache), kp, grid, d, bs, block_heads,
                  stream);
}

}  // namespace pkv
