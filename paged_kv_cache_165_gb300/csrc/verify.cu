// verify.cu -- drafted tokens against the target's probabilities, from given random numbers.
//
// Sequence b has k drafts x_0 .. x_{k-1}, rows p_0 .. p_k of the target and q_0 .. q_{k-1} of the draft, and
// numbers u_0 .. u_k in [0, 1).  Draft i is accepted while u_i q_i(x_i) < p_i(x_i); with a accepted, the next
// token is drawn from r = max(p_a - q_a, 0) (a < k) or r = p_k (a = k): the lowest v with
//   r_0 + .. + r_v > u_k (r_0 + .. + r_{V-1}),
// so that what comes out is distributed as the target alone (rejection sampling).
//
// The sums are over whole numbers: a probability becomes its value in units of 2^-58, exactly where it is at
// least 2^-34 and rounded down below, so that sums do not depend on their order -- which token comes out does
// not depend on how a row is cut into pieces -- and cost two integer additions where fp64 would be the
// bottleneck of this GPU.  u times the total is compared exactly.  Products u q are exact in fp64.
//
// One cluster per sequence: each block sums its share of the row (a contiguous run for each warp), the totals
// meet in distributed shared memory, and the warp whose run holds the border reads it once more, from L2.
// One row of p, and one of q where a draft was rejected, is all that is read of the V-long rows: bound by HBM
// for a large batch, by latency for a few sequences.
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
constexpr u64 kMost = 1ull << 63;   // sums of more than 32 (no distribution) stay there

__device__ __forceinline__ u64 capped(u64 a, u64 b) {   // a, b <= 2^63: associative whatever the order
    const u64 s = a + b;
    return s < a || s > kMost ? kMost : s;
}

__device__ __forceinline__ unsigned bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ unsigned bits_of(__nv_bfloat16 x) {
    return static_cast<unsigned>(__bfloat16_as_ushort(x)) << 16;
}

// A probability in units of 2^-58: 0 for a negative one or NaN, 2^58 from 1 on.  Below 1 it is
// 2^(e - 127) (1 + m 2^-23), e <= 126: (2^23 + m) 2^34 shifted right by 126 - e, whose upper word is
// (2^23 + m) 2^2 and whose lower word is 0; PTX shifts by 32 and more give 0.
__device__ __forceinline__ u64 units(unsigned b) {
    if (b >= 0x3f800000u) return b <= 0x7f800000u ? 1ull << 58 : 0ull;
    const unsigned e = b >> 23, top = ((b & 0x7fffffu) | 0x800000u) << 2;
    unsigned hi, lo, lo2;
    asm("shr.u32 %0, %1, %2;" : "=r"(hi) : "r"(top), "r"(126u - e));
    asm("shl.b32 %0, %1, %2;" : "=r"(lo) : "r"(top), "r"(e - 94u));    // less than 32 to the right
    asm("shr.u32 %0, %1, %2;" : "=r"(lo2) : "r"(top), "r"(94u - e));   // more
    return static_cast<u64>(hi) << 32 | (lo | lo2);
}

// u in [0, 1) in units of 2^-64 (rounded down).
__device__ __forceinline__ u64 share_of_turn(float u) {
    if (!(u > 0.f)) return 0;
    if (u >= 1.f) return ~0ull;
    const unsigned b = __float_as_uint(u);
    const int s = static_cast<int>(b >> 23) - 86;
    const u64 m = (b & 0x7fffffu) | 0x800000u;
    return s >= 0 ? m << s : (s > -24 ? m >> -s : 0ull);
}

template <typename T>
struct Row {       // what is drawn from
    const T *p, *q;   // q: nullptr, or taken away from p
    int not_this;     // an element that counts as 0, or -1
};

template <typename T>
__device__ __forceinline__ float as_float(T x) { return __uint_as_float(bits_of(x)); }

template <typename T>
__device__ __forceinline__ u64 rest_of(const Row<T> &r, T p, T q, int v) {
    const u64 x = units(bits_of(p)), y = r.q != nullptr ? units(bits_of(q)) : 0;
    return v == r.not_this || x <= y ? 0 : x - y;
}

// Elements v .. v + N - 1 of the row (those from hi on count as 0): their sum, in units.
template <typename T, int N>
struct alignas(sizeof(T) * N) Piece { T x[N]; };

template <typename T, int N>
__device__ __forceinline__ void load_pieces(const Row<T> &r, int v, int hi, Piece<T, N> &p, Piece<T, N> &q) {
    if (v + N <= hi) {
        p = *reinterpret_cast<const Piece<T, N> *>(r.p + v);
        if (r.q != nullptr) q = *reinterpret_cast<const Piece<T, N> *>(r.q + v);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            p.x[j] = v + j < hi ? r.p[v + j] : T(0.f);
            q.x[j] = v + j < hi && r.q != nullptr ? r.q[v + j] : T(0.f);
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ u64 sum_piece(const Row<T> &r, int v, const Piece<T, N> &p, const Piece<T, N> &q) {
    u64 s = 0;      // at most 8 elements of 2^58
#pragma unroll
    for (int j = 0; j < N; ++j) s += rest_of(r, p.x[j], q.x[j], v + j);
    return s;
}

// Pieces a lane loads before it uses the first; a step of a warp covers 32 * N * kAhead elements.
template <int N>
constexpr int ahead() { return N == 1 ? 8 : 2; }

// The sum over elements [lo, hi) of the row by one warp; N elements a lane side by side.
template <typename T, int N>
__device__ __forceinline__ u64 warp_sum(const Row<T> &r, int lo, int hi, int lane) {
    constexpr int kAhead = ahead<N>(), span = 32 * N;
    u64 sum = 0;
    for (int v0 = lo + lane * N; v0 - lane * N < hi; v0 += kAhead * span) {
        Piece<T, N> p[kAhead], q[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_pieces<T, N>(r, v0 + i * span, hi, p[i], q[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) sum = capped(sum, sum_piece<T, N>(r, v0 + i * span, p[i], q[i]));
    }
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) sum = capped(sum, __shfl_xor_sync(kFull, sum, sh));
    return sum;
}

// The lowest v of [lo, hi) whose sum from lo on exceeds `left` (which the whole run's does).
template <typename T, int N>
__device__ __forceinline__ int find(const Row<T> &r, int lo, int hi, u64 left, int lane) {
    constexpr int kAhead = ahead<N>(), span = 32 * N;
    u64 before = 0;
    for (int w0 = lo; w0 < hi; w0 += kAhead * span) {
        Piece<T, N> p[kAhead], q[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_pieces<T, N>(r, w0 + lane * N + i * span, hi, p[i], q[i]);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int v = w0 + lane * N + i * span;
            const u64 mine = sum_piece<T, N>(r, v, p[i], q[i]);
            u64 s = mine;
#pragma unroll
            for (int sh = 1; sh < 32; sh <<= 1) {
                const u64 y = __shfl_up_sync(kFull, s, sh);
                if (lane >= sh) s = capped(s, y);
            }
            const unsigned over = __ballot_sync(kFull, capped(before, s) > left);
            if (over != 0) {
                const int first = __ffs(over) - 1;
                const u64 others = __shfl_up_sync(kFull, s, 1);
                u64 run = lane > 0 ? capped(before, others) : before;
                int at = v + N - 1;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    run = capped(run, rest_of(r, p[i].x[j], q[i].x[j], v + j));
                    if (run > left) at = min(at, v + j);
                }
                return __shfl_sync(kFull, at, first);
            }
            before = capped(before, __shfl_sync(kFull, s, 31));
        }
    }
    return hi - 1;
}

// Whether draft i (of the sequence) is accepted.
template <typename T>
__device__ __forceinline__ bool accepts(const VerifyArgs &a, long long target_row, long long draft_row, int x, float u) {
    if (x < 0 || x >= a.V) return false;
    const float p = as_float(static_cast<const T *>(a.target)[target_row * a.target_stride + x]);
    const float q = a.draft != nullptr ? as_float(static_cast<const T *>(a.draft)[draft_row * a.draft_stride + x]) : 1.f;
    return static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a) {
    __shared__ u64 s_warp[kWarps], s_block;   // sums of the warps' runs; of the block's
    __shared__ int s_accepted;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), blocks = static_cast<int>(cluster.num_blocks());
    const int b = blockIdx.x / blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool lead = rank == 0 && threadIdx.x == 0;
    const int c0 = __ldg(a.cu_drafts + b), c1 = __ldg(a.cu_drafts + b + 1);
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
                const int x = __ldg(a.draft_tokens + c0 + i);
                yes = accepts<T>(a, row0 + i, c0 + static_cast<long long>(i), x, __ldg(a.uniforms + row0 + i));
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
    r.not_this = acc < k && a.draft == nullptr ? __ldg(a.draft_tokens + c0 + acc) : -1;

    // runs of whole pieces, one for each warp of the cluster
    const int runs = blocks * kWarps;
    const int run = ((a.V + runs - 1) / runs + 32 * N - 1) / (32 * N) * (32 * N);
    const long long at = static_cast<long long>(rank * kWarps + warp) * run;
    const int lo = static_cast<int>(min(at, static_cast<long long>(a.V))), hi = static_cast<int>(min(at + run, static_cast<long long>(a.V)));
    const u64 u = share_of_turn(__ldg(a.uniforms + row0 + k));
    int token = -1;
    bool mine = false;   // this warp holds the border
    for (int pass = 0;; ++pass) {
        const u64 sum = warp_sum<T, N>(r, lo, hi, lane);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 t = 0;
            for (int w = 0; w < kWarps; ++w) t = capped(t, s_warp[w]);
            s_block = t;
        }
        cluster.sync();
        u64 total = 0, before = 0;
        for (int c = 0; c < blocks; ++c) {
            if (c == rank) before = total;
            total = capped(total, *cluster.map_shared_rank(&s_block, c));
        }
        cluster.sync();   // every block has read the sums
        if (total > 0) {
            const u64 border = __umul64hi(u, total);   // the sum has to exceed it; below the total
            for (int w = 0; w < warp; ++w) before = capped(before, s_warp[w]);
            if (before <= border && capped(before, sum) > border) {
                mine = true;
                token = find<T, N>(r, lo, hi, border - before, lane);
            }
            break;
        }
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
            if (i != acc) a.tokens[row0 + i] = i < acc ? __ldg(a.draft_tokens + c0 + i) : -1;
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
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
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
