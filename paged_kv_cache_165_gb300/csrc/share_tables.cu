// share_tables.cu -- blocks shared by several rows, kept on the GPU: forking rows, compacting the pool, and
// the block copies that both ask for (what BlockManager.fork and its reference counts do on the host:
// plumephp.com "KV Cache 优化与注意力机制加速" §4.3, 0539edu.com "从KV cache共享到批量调度…" §3.2).
//
// References are not carried from call to call but counted anew from the tables: a block that no row (and no
// `held` mark) names is free.  A finished row, a shorter one after rejected drafts and a beam that nobody
// continued need no bookkeeping of their own, and no count can go stale.  Counts are integer atomics and
// every rank comes from a scan in index order, so the results do not depend on the order of execution.
//
// fork: row b takes the sequence of row parents[b].  Blocks that are full (or follow nothing that will be
//   written) are shared; a last block that is only partly filled will be written by its row, so one row keeps
//   it -- the lowest of those that end in it, if no row has it inside -- and each of the others gets a copy in
//   a fresh block (the pair list).  Fresh blocks are the lowest free ids, in row order.
// compact: with n blocks in use, the i-th used block from id n on moves to the i-th free id below n.
//
// Both run as one cluster of 8 x 1024 threads, whose phases (clear, count, scan, write) are separated by
// hardware cluster barriers, in place of four launches: tables of a serving batch are some 10^4 to 10^5
// entries, bound by the latency of the phases.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kBlocks = 8;
constexpr unsigned kAll = kThreads * kBlocks;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kNobody = 0x7fffffff;

// Exclusive ranks of N flags counted over a block's threads; totals[i]: the block's.  All threads call it.
template <int N>
__device__ __forceinline__ void block_ranks(int (&x)[N], int (&s_warp)[N][32], int (&totals)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int in[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        in[i] = x[i];
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int y = __shfl_up_sync(kFull, x[i], sh);
            if (lane >= sh) x[i] += y;
        }
    }
    __syncthreads();   // the sums of an earlier call have been read
    if (lane == 31) {
#pragma unroll
        for (int i = 0; i < N; ++i) s_warp[i][warp] = x[i];
    }
    __syncthreads();
    if (warp < N) {
        int w = s_warp[warp][lane];
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int y = __shfl_up_sync(kFull, w, sh);
            if (lane >= sh) w += y;
        }
        s_warp[warp][lane] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (warp > 0) x[i] += s_warp[i][warp - 1];
        x[i] -= in[i];
        totals[i] = s_warp[i][31];
    }
}

// The block's part of n items, as [begin, end).
__device__ __forceinline__ uint2 part_of(unsigned n, unsigned rank) {
    const unsigned each = (n + kBlocks - 1) / kBlocks;
    return make_uint2(min(n, rank * each), min(n, (rank + 1) * each));
}

// Counts of N kinds of items in the block's part [begin, end): every block learns the sums before its part
// (before) and over all parts (all).
template <int N, typename Flags>
__device__ __forceinline__ void count_parts(cg::cluster_group &cluster, uint2 part, Flags flags, int (&s_warp)[N][32],
                                            int (&s_part)[N], int (&before)[N], int (&all)[N]) {
    int mine[N] = {};
    for (unsigned i = part.x + threadIdx.x; i < part.y; i += kThreads) {
        int f[N];
        flags(i, f);
#pragma unroll
        for (int k = 0; k < N; ++k) mine[k] += f[k];
    }
    int total[N];
    block_ranks<N>(mine, s_warp, total);
    if (threadIdx.x == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) s_part[k] = total[k];
    }
    cluster.sync();
#pragma unroll
    for (int k = 0; k < N; ++k) before[k] = all[k] = 0;
    for (unsigned c = 0; c < kBlocks; ++c) {
        const int *theirs = cluster.map_shared_rank(&s_part[0], c);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (c == cluster.block_rank()) before[k] = all[k];
            all[k] += theirs[k];
        }
    }
    cluster.sync();   // the sums have been read
}

// What row b of the result holds.
struct Source {
    int row, len;   // the row whose sequence it takes (-1: none), and its tokens
};

__device__ __forceinline__ Source source_of(const ShareArgs &a, int b, bool report) {
    Source s{a.parents != nullptr ? __ldg(a.parents + b) : b, 0};
    if (s.row < -1 || s.row >= a.B) {
        if (report) raise_error(a.err, PKV_DEVERR_PAIR);
        s.row = -1;
    }
    if (s.row >= 0) {
        s.len = a.lens[s.row];
        if (s.len < 0 || static_cast<long long>(s.len) > static_cast<long long>(a.MBS) * a.bs) {
            if (report) raise_error(a.err, PKV_DEVERR_LEN);
            s.len = 0;
        }
    }
    return s;
}

// A table entry, -1 where it names no block (-1: given back before; anything else is flagged).
__device__ __forceinline__ int entry_of(const ShareArgs &a, size_t at) {
    const int x = a.table[at];
    if (x >= 0 && x < a.NB) return x;
    if (x != -1) raise_error(a.err, PKV_DEVERR_BLOCK);
    return -1;
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads) fork_kernel(const ShareArgs a) {
    __shared__ int s_warp[1][32], s_part[1];
    cg::cluster_group cluster = cg::this_cluster();
    const unsigned rank = cluster.block_rank(), tid = rank * kThreads + threadIdx.x;
    const unsigned NB = a.NB, B = a.B;
    const unsigned warp = tid >> 5, lane = tid & 31, warps = kAll / 32;
    int *first = a.first;     // [NB] the lowest row that ends, partly filled, in a block
    for (unsigned i = tid; i < NB; i += kAll) {
        a.refs[i] = a.held != nullptr && __ldg(a.held + i) != 0 ? 1 : 0;
        first[i] = kNobody;
    }
    cluster.sync();
    // rows of the result: their entries, and the references of blocks that will not be written
    int32_t *rows = a.rows;   // [B][MBS], the table itself where the parents' rows are read no more
    for (unsigned b = warp; b < B; b += warps) {
        const Source s = source_of(a, b, lane == 0);
        const int n = static_cast<int>((static_cast<long long>(s.len) + a.bs - 1) / a.bs);
        const bool partly = s.len % a.bs != 0;
        const size_t to = static_cast<size_t>(b) * a.MBS, from = static_cast<size_t>(max(s.row, 0)) * a.MBS;
        for (unsigned j = lane; j < static_cast<unsigned>(a.MBS); j += 32) {
            int x = -1;
            if (j < static_cast<unsigned>(n)) {
                x = entry_of(a, from + j);
                if (x >= 0) {
                    if (partly && j == static_cast<unsigned>(n) - 1) atomicMin(first + x, static_cast<int>(b));
                    else atomicAdd(a.refs + x, 1);
                }
            }
            rows[to + j] = x;
        }
    }
    cluster.sync();
    // rows that get a copy of their last block
    auto copied = [&](unsigned b) -> int2 {   // (its block, its place in the row), or (-1, 0)
        const Source s = source_of(a, b, false);
        if (s.len % a.bs == 0) return make_int2(-1, 0);
        const int j = s.len / a.bs, x = rows[static_cast<size_t>(b) * a.MBS + j];
        if (x < 0 || (a.refs[x] == 0 && first[x] == static_cast<int>(b))) return make_int2(-1, 0);
        return make_int2(x, j);
    };
    const uint2 row_part = part_of(B, rank), block_part = part_of(NB, rank);
    int copies_before[1], copies[1], free_before[1], free_all[1];
    count_parts<1>(cluster, row_part, [&](unsigned b, int (&f)[1]) { f[0] = copied(b).x >= 0; }, s_warp, s_part,
                   copies_before, copies);
    count_parts<1>(cluster, block_part, [&](unsigned i, int (&f)[1]) { f[0] = a.refs[i] == 0 && first[i] == kNobody; }, s_warp,
                   s_part, free_before, free_all);
    // which row gets which fresh block, before the references change
    int at = copies_before[0];
    for (unsigned b0 = row_part.x; b0 < row_part.y; b0 += kThreads) {
        const unsigned b = b0 + threadIdx.x;
        const int2 c = b < row_part.y ? copied(b) : make_int2(-1, 0);
        int r[1] = {c.x >= 0}, total[1];
        block_ranks<1>(r, s_warp, total);
        if (b < row_part.y) a.place[b] = c.x >= 0 ? at + r[0] : -1;
        at += total[0];
    }
    cluster.sync();
    const int served = min(copies[0], free_all[0]), left = free_all[0] - served;
    at = free_before[0];
    for (unsigned i0 = block_part.x; i0 < block_part.y; i0 += kThreads) {
        const unsigned i = i0 + threadIdx.x;
        bool free = false, kept = false;
        if (i < block_part.y) {
            kept = a.refs[i] == 0 && first[i] != kNobody;
            free = a.refs[i] == 0 && !kept;
        }
        int r[1] = {free}, total[1];
        block_ranks<1>(r, s_warp, total);
        const int nth = at + r[0];
        if (free && nth < served) a.fresh[nth] = static_cast<int>(i);
        if (free && nth >= served) a.free_list[free_all[0] - 1 - nth] = static_cast<int>(i);
        if (kept || (free && nth < served)) a.refs[i] = 1;
        at += total[0];
    }
    for (unsigned i = tid; i < NB; i += kAll)
        if (i >= static_cast<unsigned>(left)) a.free_list[i] = -1;
    if (tid == 0) {
        *a.free_count = left;
        *a.pair_count = served;
        if (served < copies[0]) raise_error(a.err, PKV_DEVERR_POOL);
    }
    for (unsigned i = tid; i < B; i += kAll)
        if (i >= static_cast<unsigned>(served)) reinterpret_cast<int2 *>(a.pairs)[i] = make_int2(-1, -1);
    cluster.sync();
    // the rows themselves: a row of B a thread for what changes, then the whole table where it was built aside
    for (unsigned b = tid; b < B; b += kAll) {
        Source s = source_of(a, b, false);
        const int nth = a.place[b];
        const size_t last = static_cast<size_t>(b) * a.MBS + s.len / a.bs;
        if (nth >= 0 && nth < served) {
            reinterpret_cast<int2 *>(a.pairs)[nth] = make_int2(rows[last], a.fresh[nth]);
            rows[last] = a.fresh[nth];
        }
        a.place[b] = nth >= served ? 0 : s.len;   // its length: none for a row that the pool was too small for
    }
    cluster.sync();
    for (unsigned b = tid; b < B; b += kAll) a.lens_out[b] = a.place[b];
    for (unsigned b = warp; b < B; b += warps) {
        const bool none = a.place[b] == 0;
        if (rows == a.table_out && !none) continue;
        const size_t to = static_cast<size_t>(b) * a.MBS;
        for (unsigned j = lane; j < static_cast<unsigned>(a.MBS); j += 32) a.table_out[to + j] = none ? -1 : rows[to + j];
    }
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads) compact_kernel(const ShareArgs a) {
    __shared__ int s_warp[3][32], s_part[3], s_warp1[1][32], s_part1[1];
    cg::cluster_group cluster = cg::this_cluster();
    const unsigned rank = cluster.block_rank(), tid = rank * kThreads + threadIdx.x;
    const unsigned NB = a.NB, B = a.B;
    const unsigned warp = tid >> 5, lane = tid & 31, warps = kAll / 32;
    int *moved = a.first;     // [NB] where a block goes
    auto held = [&](unsigned i) { return a.held != nullptr && __ldg(a.held + i) != 0; };
    for (unsigned i = tid; i < NB; i += kAll) a.refs[i] = held(i) ? 1 : 0;
    cluster.sync();
    for (unsigned b = warp; b < B; b += warps) {
        const Source s = source_of(a, b, lane == 0);
        const int n = static_cast<int>((static_cast<long long>(s.len) + a.bs - 1) / a.bs);
        const size_t row = static_cast<size_t>(b) * a.MBS;
        for (int j = lane; j < n; j += 32) {
            const int x = entry_of(a, row + j);
            if (x >= 0) atomicAdd(a.refs + x, 1);
        }
    }
    cluster.sync();
    const uint2 part = part_of(NB, rank);
    int before1[1], used_[1];
    count_parts<1>(cluster, part, [&](unsigned i, int (&f)[1]) { f[0] = a.refs[i] != 0; }, s_warp1, s_part1, before1, used_);
    const unsigned used = used_[0];
    // blocks that move (in use, not held, from `used` on), free ids below, free or vacated ids from there on
    auto kinds = [&](unsigned i, int (&f)[3]) {
        const bool in_use = a.refs[i] != 0, high = i >= used, fixed = held(i);
        f[0] = in_use && high && !fixed;
        f[1] = !in_use && !high;
        f[2] = high && !fixed;
    };
    int before[3], all[3];
    count_parts<3>(cluster, part, kinds, s_warp, s_part, before, all);
    // as many ids are free below `used` as are taken from there on, so every mover has a place
    const int moves = all[0], spare = all[1] - moves, free_all = spare + all[2];
    for (unsigned i0 = part.x; i0 < part.y; i0 += kThreads) {
        const unsigned i = i0 + threadIdx.x;
        int f[3] = {0, 0, 0};
        if (i < part.y) kinds(i, f);
        int r[3] = {f[0], f[1], f[2]}, total[3];
        block_ranks<3>(r, s_warp, total);
        if (i < part.y) moved[i] = static_cast<int>(i);
        if (f[0]) reinterpret_cast<int2 *>(a.pairs)[before[0] + r[0]].x = static_cast<int>(i);
        if (f[1]) {
            const int nth = before[1] + r[1];
            if (nth < moves) reinterpret_cast<int2 *>(a.pairs)[nth].y = static_cast<int>(i);
            else a.free_list[free_all - 1 - (nth - moves)] = static_cast<int>(i);
        }
        if (f[2]) a.free_list[free_all - 1 - (spare + before[2] + r[2])] = static_cast<int>(i);
#pragma unroll
        for (int k = 0; k < 3; ++k) before[k] += total[k];
    }
    for (unsigned i = tid; i < NB; i += kAll)
        if (i >= static_cast<unsigned>(free_all)) a.free_list[i] = -1;
    for (unsigned i = tid; i < NB / 2; i += kAll)
        if (i >= static_cast<unsigned>(moves)) reinterpret_cast<int2 *>(a.pairs)[i] = make_int2(-1, -1);
    if (tid == 0) {
        *a.free_count = free_all;
        *a.pair_count = moves;
    }
    cluster.sync();
    for (unsigned i = tid; i < static_cast<unsigned>(moves); i += kAll) {
        const int2 p = reinterpret_cast<const int2 *>(a.pairs)[i];
        moved[p.x] = p.y;
        a.refs[p.y] = a.refs[p.x];
        a.refs[p.x] = 0;
    }
    cluster.sync();
    for (unsigned b = warp; b < B; b += warps) {
        const Source s = source_of(a, b, false);
        const unsigned n = static_cast<unsigned>((static_cast<long long>(s.len) + a.bs - 1) / a.bs);
        const size_t row = static_cast<size_t>(b) * a.MBS;
        for (unsigned j = lane; j < static_cast<unsigned>(a.MBS); j += 32) {
            int x = j < n ? a.table[row + j] : -1;
            x = x >= 0 && x < a.NB ? moved[x] : -1;
            a.table_out[row + j] = x;
        }
    }
}

// ---------------------------------------------------------------- copies of a list that the GPU counted

constexpr int kCopyThreads = 256, kCopyAhead = 4;

template <typename U>
__global__ void __launch_bounds__(kCopyThreads)
    kv_block_copy_counted_kernel(U *__restrict__ kc, U *__restrict__ vc, const int32_t *__restrict__ pairs, int n,
                                 const int32_t *__restrict__ count, long long block_units, int NB, unsigned *err) {
    int live = __ldg(count);
    if (live < 0 || live > n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(err, PKV_DEVERR_PAIR);
        live = max(0, min(live, n));
    }
    // pieces of kCopyThreads * kCopyAhead units: of K, then of V, of one pair after the other
    const long long span = kCopyThreads * kCopyAhead;
    const long long per = (block_units + span - 1) / span, pieces = 2 * per * live;
    for (long long w = blockIdx.x; w < pieces; w += gridDim.x) {
        const long long pair = w / (2 * per), rest = w - pair * 2 * per;
        const int src = __ldg(pairs + 2 * pair), dst = __ldg(pairs + 2 * pair + 1);
        if (src < 0 || src >= NB || dst < 0 || dst >= NB) {
            if (rest == 0 && threadIdx.x == 0) raise_error(err, PKV_DEVERR_PAIR);
            continue;
        }
        U *c = rest < per ? kc : vc;
        const long long u0 = (rest < per ? rest : rest - per) * span + threadIdx.x;
        const U *s = c + src * block_units;
        U *d = c + dst * block_units;
        U x[kCopyAhead];
#pragma unroll
        for (int i = 0; i < kCopyAhead; ++i)
            if (u0 + i * kCopyThreads < block_units) x[i] = s[u0 + i * kCopyThreads];
#pragma unroll
        for (int i = 0; i < kCopyAhead; ++i)
            if (u0 + i * kCopyThreads < block_units) d[u0 + i * kCopyThreads] = x[i];
    }
}

}  // namespace

// Scratch behind a call: a row's length or place [B], fresh blocks [B], one number a block [NB], and the
// table when it replaces the one that it is built from ([B][MBS]).
size_t share_workspace_bytes(int B, int MBS, int NB) {
    return (2 * static_cast<size_t>(B) + static_cast<size_t>(NB) + static_cast<size_t>(B) * MBS) * sizeof(int32_t);
}

cudaError_t launch_fork(ShareArgs a, void *workspace, bool aside, cudaStream_t stream) {
    int32_t *ws = static_cast<int32_t *>(workspace);
    a.first = ws;
    a.place = ws + a.NB;
    a.fresh = a.place + a.B;
    a.rows = aside ? a.fresh + a.B : a.table_out;
    fork_kernel<<<kBlocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_compact(ShareArgs a, void *workspace, cudaStream_t stream) {
    a.first = static_cast<int32_t *>(workspace);
    compact_kernel<<<kBlocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_block_copy_counted(void *k_cache, void *v_cache, int elem_bytes, const int32_t *pairs, int n,
                                         const int32_t *count, int Hkv, int d, int bs, int NB, int sm_count, unsigned *err,
                                         cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    const size_t bytes = static_cast<size_t>(Hkv) * bs * d * elem_bytes;
    size_t at = bytes | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
    const int u = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : at % 2 == 0 ? 2 : 1;
    const long long units = static_cast<long long>(bytes / u), span = kCopyThreads * kCopyAhead;
    const unsigned grid = static_cast<unsigned>(std::min(2ll * n * ((units + span - 1) / span), 8ll * std::max(sm_count, 1)));
#define PKV_COPY(UT)                                                                                                     \
    kv_block_copy_counted_kernel<UT><<<grid, kCopyThreads, 0, stream>>>(static_cast<UT *>(k_cache),                     \
                                                                        static_cast<UT *>(v_cache), pairs, n, count, units, NB, err)
    switch (u) {
        case 16: PKV_COPY(uint4); break;
        case 4: PKV_COPY(uint32_t); break;
        case 2: PKV_COPY(uint16_t); break;
        default: PKV_COPY(uint8_t); break;
    }
#undef PKV_COPY
    return cudaGetLastError();
}

}  // namespace pkv
