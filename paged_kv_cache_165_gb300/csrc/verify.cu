// verify.cu -- drafted tokens against the target's probabilities, from given random numbers.
//
// Sequence b has k drafts x_0 .. x_{k-1}, rows p_0 .. p_k of the target and q_0 .. q_{k-1} of the draft, and
// numbers u_0 .. u_k in [0, 1).  Draft i is accepted while u_i q_i(x_i) < p_i(x_i); with a accepted, the next
// token is drawn from r = max(p_a - q_a, 0) (a < k) or r = p_k (a = k): the lowest v with
//   r_0 + .. + r_v > u_k (r_0 + .. + r_{V-1}),
// so that what comes out is distributed as the target alone (rejection sampling).
//
// The sums are over whole numbers: a probability becomes the nearest multiple of 2^-46, so that sums do not depend
// on their order -- which token comes out does not depend on how a row is cut into pieces.  The number is kept as
// H 2^23 + L: 1 + p rounds to 1 + H 2^-23 (H are the lower bits of that fp32 number), and what is left of p,
// times 2^46, onto 1.5 * 2^23 rounds to L likewise: five fp32 operations, where fp64 sums would be this GPU's
// bottleneck and 64-bit shifts of the mantissa took twice the instructions.  max(p - q, 0) = max(p, q) - q, so a
// rest is the difference of two such numbers, and the constants of the bit patterns cancel.  u times the total
// is compared exactly.  Products u q are exact in fp64.
//
// One cluster per sequence: each block sums its share of the row (a contiguous run for each warp), the totals
// meet in distributed shared memory, and the warp whose run holds the border reads it once more, from L2.
// One row of p, and one of q where a draft was rejected, is all that is read of the V-long rows.  64 sequences of
// 131072 tokens: 18.6 us (56 MB from HBM, a floor of 8.2; 15.9 with the rows in L2), of which the chain offsets - drafts - their
// probabilities before the first load of a row and the border's search after the last take about half; one of 50001 tokens
// 7.0 us.  (Mantissas
// shifted in 64 bits instead of fp32: 33 us; the border sought 32 elements at a time: 48.)
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;
constexpr u64 kMost = 1ull << 63;   // sums of more than 2^17 (no distribution) stay there

__device__ __forceinline__ u64 capped(u64 a, u64 b) {   // a, b <= 2^63: associative whatever the order
    const u64 s = a + b;
    return s < a || s > kMost ? kMost : s;
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Sums of elements' H and L (units of 2^-23 and 2^-46), for at most 128 elements: |H| <= 2^23, |L| <= 2^23 each.
struct Parts {
    unsigned h = 0, l = 0;   // modulo 2^32
    __device__ __forceinline__ void add(float p) {   // p in [0, 1]
        const float t = p + 1.f;
        h += __float_as_uint(t);
        l += __float_as_uint(__fmaf_rn(p - (t - 1.f), 0x1p46f, 0x1.8p23f));
    }
    __device__ __forceinline__ void sub(float p) {
        const float t = p + 1.f;
        h -= __float_as_uint(t);
        l -= __float_as_uint(__fmaf_rn(p - (t - 1.f), 0x1p46f, 0x1.8p23f));
    }
    // n: elements added less elements subtracted
    __device__ __forceinline__ u64 units(int n) const {
        const long long H = static_cast<int>(h - static_cast<unsigned>(n) * 0x3f800000u);
        const long long L = static_cast<int>(l - static_cast<unsigned>(n) * 0x4b400000u);
        return static_cast<u64>((H << 23) + L);
    }
};

// u * total rounded down, from the exact product (24 bits times 64): what a sum of whole numbers has to exceed.  u of 1
// and more counts as just below it, and one below 0 or NaN as 0.
__device__ __forceinline__ u64 border_of(float u, u64 total) {
    if (!(u > 0.f)) return 0;
    if (u >= 1.f) return total - 1;
    const unsigned b = __float_as_uint(u), e = b >> 23;   // u = m 2^-n
    const u64 m = (b & 0x7fffffu) | (e > 0 ? 0x800000u : 0u);
    const int n = 150 - static_cast<int>(max(e, 1u));     // 24 .. 149
    const u64 hi = __umul64hi(m, total), lo = m * total;
    return n < 64 ? lo >> n | hi << (64 - n) : n < 128 ? hi >> (n - 64) : 0;
}

template <typename T>
struct Row {       // what is drawn from
    const T *p, *q;   // q: nullptr, or taken away from p
    int not_this;     // an element that counts as 0, or -1
};

// Elements v .. v + N - 1, in units.  Q: q is taken away; else one element may not count.  Saturation makes a
// probability at most 1, and 0 of a negative one and of NaN.
template <bool Q, typename T, int N>
__device__ __forceinline__ u64 rest_of(const Row<T> &r, const T (&p)[N], const T (&q)[N], int v) {
    Parts s;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float x = __saturatef(as_float(p[j]));
        if constexpr (Q) {
            const float y = __saturatef(as_float(q[j]));
            s.add(fmaxf(x, y));
            s.sub(y);
        } else {
            s.add(v + j == r.not_this ? 0.f : x);
        }
    }
    return s.units(Q ? 0 : N);
}

// Elements v .. v + N - 1 of the row, those from hi on 0.
template <typename T, int N>
struct alignas(sizeof(T) * N) Piece { T x[N]; };

template <bool Q, typename T, int N>
__device__ __forceinline__ void load_pieces(const Row<T> &r, int v, int hi, Piece<T, N> &p, Piece<T, N> &q) {
    if (v + N <= hi) {
        p = *reinterpret_cast<const Piece<T, N> *>(r.p + v);
        if constexpr (Q) q = *reinterpret_cast<const Piece<T, N> *>(r.q + v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            p.x[j] = v + j < hi ? r.p[v + j] : T(0.f);
            if constexpr (Q) q.x[j] = v + j < hi ? r.q[v + j] : T(0.f);
        }
    }
}

// The sum over elements [lo, hi) of the row by one warp; N elements a lane side by side, a few such pieces loaded
// before the first is used.
template <bool Q, typename T, int N>
__device__ __forceinline__ u64 warp_sum(const Row<T> &r, int lo, int hi, int lane) {
    constexpr int kAhead = N == 1 ? 8 : 4, span = 32 * N;
    u64 sum = 0;
    for (int v0 = lo; v0 < hi; v0 += kAhead * span) {
        Piece<T, N> p[kAhead], q[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_pieces<Q, T, N>(r, v0 + lane * N + i * span, hi, p[i], q[i]);
        u64 s = 0;   // at most 32 elements of 2^46
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += rest_of<Q, T, N>(r, p[i].x, q[i].x, v0 + lane * N + i * span);
        sum = capped(sum, s);
    }
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) sum = capped(sum, __shfl_xor_sync(kFull, sum, sh));
    return sum;
}

// Whole-warp: the first lane whose inclusive sum over the lanes (of `mine`, after `before`) exceeds `left`, and the
// sum before it; -1 where none does.
__device__ __forceinline__ int first_over(u64 mine, u64 left, int lane, u64 &before) {
    u64 s = mine;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const u64 y = __shfl_up_sync(kFull, s, sh);
        if (lane >= sh) s = capped(s, y);
    }
    const unsigned over = __ballot_sync(kFull, capped(before, s) > left);
    if (over == 0) {
        before = capped(before, __shfl_sync(kFull, s, 31));
        return -1;
    }
    const int first = __ffs(over) - 1;
    const u64 lower = __shfl_sync(kFull, s, max(first - 1, 0));
    if (first > 0) before = capped(before, lower);
    return first;
}

// The lowest v of [lo, hi) whose sum from lo on exceeds `left` (which the whole run's does): the 32 consecutive
// shares of the run first, then the one that holds it, so that two rounds of loads and scans do.
template <bool Q, typename T>
__device__ __forceinline__ int find(const Row<T> &r, int lo, int hi, u64 left, int lane) {
    const int share = (hi - lo + 31) / 32, a = min(hi, lo + lane * share), b = min(hi, a + share);
    u64 sum = 0, before = 0;
    for (int v0 = a; v0 < b; v0 += 8) {
        T p[8], q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = v0 + j < b ? r.p[v0 + j] : T(0.f);
            if constexpr (Q) q[j] = v0 + j < b ? r.q[v0 + j] : T(0.f);
        }
        sum = capped(sum, rest_of<Q, T, 8>(r, p, q, v0));
    }
    const int holder = first_over(sum, left, lane, before);
    if (holder < 0) return hi - 1;
    const int from = lo + holder * share, to = min(hi, from + share);
    for (int v0 = from; v0 < to; v0 += 32) {
        const int v = v0 + lane;
        const T p[1] = {v < to ? r.p[v] : T(0.f)}, q[1] = {Q && v < to ? r.q[v] : T(0.f)};
        const int first = first_over(rest_of<Q, T, 1>(r, p, q, v), left, lane, before);
        if (first >= 0) return v0 + first;
    }
    return to - 1;
}

// Whether draft i (of the sequence) is accepted.
template <typename T>
__device__ __forceinline__ bool accepts(const VerifyArgs &a, long long target_row, long long draft_row, int x, float u) {
    if (x < 0 || x >= a.V) return false;
    const float p = as_float(static_cast<const T *>(a.target)[target_row * a.target_stride + x]);
    const float q = a.draft != nullptr ? as_float(static_cast<const T *>(a.draft)[draft_row * a.draft_stride + x]) : 1.f;
    return isfinite(p) && isfinite(q) && static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a) {
    __shared__ u64 s_warp[kWarps], s_block;   // sums of the warps' runs; of the block's
    __shared__ int s_accepted;
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
    const int b = blockIdx.x / blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool lead = rank == 0 && threadIdx.x == 0;
    const int c0 = a.cu_drafts[b], c1 = a.cu_drafts[b + 1];
    if (c0 < 0 || c1 < c0 || c1 > a.D) {   // the whole cluster leaves: nothing is written but what refuses
        if (lead) {
            raise_error(a.err, PKV_DEVERR_CU_SEQLENS);
            a.accepted[b] = 0;
            if (a.lens_out != nullptr) a.lens_out[b] = a.lens[b];
        }
        return;
    }
    const int k = c1 - c0;
    const long long row0 = static_cast<long long>(c0) + b;   // of the target's rows, numbers and tokens
    if (warp == 0) {
        int acc = k;
        for (int i0 = 0; i0 < k; i0 += 32) {
            const int i = i0 + lane;
            bool yes = true;
            if (i < k) {
                const int x = a.draft_tokens[c0 + i];
                yes = accepts<T>(a, row0 + i, c0 + static_cast<long long>(i), x, a.uniforms[row0 + i]);
                if (!yes && (x < 0 || x >= a.V) && rank == 0) raise_error(a.err, PKV_DEVERR_PROBS);
            }
            const unsigned no = __ballot_sync(kFull, !yes);
            if (no != 0) {
                acc = i0 + __ffs(no) - 1;
                break;
            }
        }
        if (lane == 0) s_accepted = acc;
    }
    __syncthreads();
    const int acc = s_accepted;
    Row<T> r;
    r.p = static_cast<const T *>(a.target) + (row0 + acc) * a.target_stride;
    r.q = acc < k && a.draft != nullptr ? static_cast<const T *>(a.draft) + (c0 + static_cast<long long>(acc)) * a.draft_stride
                                        : nullptr;
    r.not_this = acc < k && a.draft == nullptr ? a.draft_tokens[c0 + acc] : -1;

    // runs of whole pieces, one for each warp of the cluster
    const int runs = blocks * kWarps;
    const int run = ((a.V + runs - 1) / runs + 32 * N - 1) / (32 * N) * (32 * N);
    const long long at = static_cast<long long>(rank * kWarps + warp) * run;
    const int lo = static_cast<int>(min(at, static_cast<long long>(a.V))), hi = static_cast<int>(min(at + run, static_cast<long long>(a.V)));
    const float u = a.uniforms[row0 + k];
    int token = -1;
    bool mine = false;   // this warp holds the border
    for (int pass = 0;; ++pass) {
        const bool has_q = r.q != nullptr;
        const u64 sum = has_q ? warp_sum<true, T, N>(r, lo, hi, lane) : warp_sum<false, T, N>(r, lo, hi, lane);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 t = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) t = capped(t, s_warp[w]);
            s_block = t;
        }
        cluster.sync();
        // lane c holds block c's sum; before: of the blocks before this one, and of its warps before this one
        const u64 theirs = lane < blocks ? *cluster.map_shared_rank(&s_block, lane) : 0;
        u64 total = theirs, before = lane < rank ? theirs : (lane >= 16 && lane - 16 < warp ? s_warp[lane - 16] : 0);
#pragma unroll
        for (int sh = 16; sh > 0; sh >>= 1) {
            total = capped(total, __shfl_xor_sync(kFull, total, sh));
            before = capped(before, __shfl_xor_sync(kFull, before, sh));
        }
        cluster.barrier_arrive();   // every block has read the sums once all have arrived
        if (total > 0) {
            const u64 border = border_of(u, total);   // the sum has to exceed it; below the total
            if (before <= border && capped(before, sum) > border) {
                mine = true;
                token = has_q ? find<true, T>(r, lo, hi, border - before, lane) : find<false, T>(r, lo, hi, border - before, lane);
            }
        }
        cluster.barrier_wait();
        if (total > 0) break;
        if (pass == 1 || (r.q == nullptr && r.not_this < 0)) {   // no mass at all: no token
            mine = rank == 0 && warp == 0;
            if (lead) raise_error(a.err, PKV_DEVERR_PROBS);
            break;
        }
        r.q = nullptr;   // p <= q everywhere, though a draft was rejected: from p itself
        r.not_this = -1;
    }
    if (mine && lane == 0) a.tokens[row0 + acc] = token;
    if (rank == 0) {
        for (int i = threadIdx.x; i <= k; i += kThreads)
            if (i != acc) a.tokens[row0 + i] = i < acc ? a.draft_tokens[c0 + i] : -1;
        if (threadIdx.x == 0) {
            a.accepted[b] = acc;
            if (a.lens_out != nullptr) a.lens_out[b] = a.lens[b] - (k - acc);
        }
    }
}

template <typename T, int N>
cudaError_t launch(const VerifyArgs &a, int blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // as launch_dependent
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T, N>, a);
}

template <typename T>
cudaError_t launch_type(const VerifyArgs &a, int sm_count, cudaStream_t stream) {
    // blocks of a sequence: the GPU filled about twice, and at least 2048 elements a block
    int blocks = 1;
    while (blocks < 8 && static_cast<long long>(a.B) * blocks < 2ll * std::max(sm_count, 1) && a.V > blocks * 2048) blocks *= 2;
    constexpr int kWide = 16 / sizeof(T);
    auto fits = [](const void *p, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % kWide == 0;
    };
    if (fits(a.target, a.target_stride) && (a.draft == nullptr || fits(a.draft, a.draft_stride)))
        return launch<T, kWide>(a, blocks, stream);
    return launch<T, 1>(a, blocks, stream);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, pkv_dtype dt, int sm_count, cudaStream_t stream) {
    return dt == PKV_BF16 ? launch_type<__nv_bfloat16>(a, sm_count, stream) : launch_type<float>(a, sm_count, stream);
}

}  // namespace pkv
