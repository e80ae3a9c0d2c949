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
// Both are one launch and bound by the latency of their phases (clear, count, scan, write): tables of a serving
// batch are some 10^2 to 10^5 entries.  Small ones run as one block of 1024 threads that keeps the counts in
// shared memory, where a phase ends with __syncthreads.  Larger ones run as a cluster of eight such blocks with
// the counts in global memory and hardware cluster barriers (about 0.6 us each, and what the blocks wait for one
// another); counts spread over the cluster's shared memories measured no faster.  Loads of a phase are issued without
// branches, so that they overlap; ids are ranked by ballots over bits kept from the first look at them (by scans over
// the block and a second look, 256 rows took 18.1 us and the pool of 25234 ids 85.4).  Device time, copies of the pairs
// included: eight rows of 20 blocks forked 8.4 us, 256 of 129 15.0 (one block: 31.5 without copies); six rows of 55
// compacted 7.4 us, 64 of 509 in a pool of 25234 81.  The counted copies move 6254 pairs of 64 KB at 6.48 TB/s (95% of
// the measured copy rate; four loads ahead instead of eight: 5.9).
#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kBlocks = 8;                // of the cluster
constexpr unsigned kFull = 0xffffffffu;
constexpr int kNobody = 0x7fffffff;
constexpr int kRowsEach = 8;                               // rows of a thread, at most: 65536 of a call
// what one block takes: two numbers an id and two a row in shared memory, four entries a thread
constexpr int kOneIds = 24576, kOneRows = 2048, kOneEntries = 4096;

// Of N counts of a warp each: their sums over the block's earlier warps (base) and over all (total).  All threads call
// it, once for an s_warp.
template <int N>
__device__ __forceinline__ void warp_bases(const int (&mine)[N], int (&s_warp)[N][32], int (&base)[N], int (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) s_warp[n][warp] = mine[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int x = s_warp[n][lane];
        base[n] = __reduce_add_sync(kFull, lane < warp ? x : 0);
        total[n] = __reduce_add_sync(kFull, x);
    }
}

// Items [begin, end) of a block, dealt to its warps in runs of 32 * rounds: a lane has first + 32 r, r < rounds.
struct Run {
    unsigned first, end, rounds;
    __device__ __forceinline__ explicit Run(uint2 part) : end(part.y), rounds((part.y - part.x + kThreads - 1) / kThreads) {
        first = part.x + (threadIdx.x >> 5) * 32 * rounds + (threadIdx.x & 31);
    }
    __device__ __forceinline__ unsigned at(unsigned r) const { return first + 32 * r; }
};

// flag(i) of a lane's items, kept as bits for the first 32 of them; its warp's count.  Four at a time, without branches
// (items past the end look at item 0 in vain), so that their loads overlap.
struct Flags {
    unsigned bits = 0;
    int count = 0;
    template <typename Flag>
    __device__ __forceinline__ Flags(const Run &run, Flag flag) {
        for (unsigned r0 = 0; r0 < run.rounds; r0 += 4) {
            bool f[4];
#pragma unroll
            for (unsigned k = 0; k < 4; ++k) {
                const bool there = (r0 + k < run.rounds) & (run.at(r0 + k) < run.end);
                f[k] = flag(there ? run.at(r0 + k) : 0u) & there;
            }
#pragma unroll
            for (unsigned k = 0; k < 4; ++k) {
                if (r0 + k < 32) bits |= static_cast<unsigned>(f[k]) << (r0 + k);
                count += __popc(__ballot_sync(kFull, f[k]));
            }
        }
    }
    template <typename Flag>
    __device__ __forceinline__ bool of(const Run &run, unsigned r, Flag flag) const {
        return r < 32 ? bits >> r & 1 : run.at(r) < run.end && flag(run.at(r));
    }
};

// A lane's rank among its warp's flags, counted on from `base`, which moves past them.
__device__ __forceinline__ int rank_of(bool f, int &base) {
    const unsigned b = __ballot_sync(kFull, f);
    const int rank = base + __popc(b & ((1u << (threadIdx.x & 31)) - 1u));
    base += __popc(b);
    return rank;
}

// The blocks of a launch: one, or the cluster.
template <bool ONE>
struct Team {
    static constexpr unsigned kTeam = ONE ? 1 : kBlocks, kAll = kTeam * kThreads;
    unsigned rank;
    __device__ __forceinline__ Team() : rank(ONE ? 0u : cg::this_cluster().block_rank()) {}
    __device__ __forceinline__ unsigned tid() const { return rank * kThreads + threadIdx.x; }
    __device__ __forceinline__ void sync() const {
        if constexpr (ONE) __syncthreads();
        else cg::this_cluster().sync();
    }
    // this block's part of n items
    __device__ __forceinline__ uint2 part(unsigned n) const {
        const unsigned each = (n + kTeam - 1) / kTeam;
        return make_uint2(min(n, rank * each), min(n, (rank + 1) * each));
    }
};

// The sums of N counts over the blocks before this one (before) and over all (all), by way of s_part, which
// is not written again.  Ends with a barrier of the team.
template <bool ONE, int N>
__device__ __forceinline__ void share_counts(const Team<ONE> &team, const int (&mine)[N], int (&s_part)[N], int (&before)[N],
                                             int (&all)[N]) {
    if constexpr (ONE) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            before[n] = 0;
            all[n] = mine[n];
        }
    } else {
        cg::cluster_group cluster = cg::this_cluster();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) s_part[n] = mine[n];
        }
        cluster.sync();
        // lane c reads block c's
        const int lane = threadIdx.x & 31;
        int theirs[N];
#pragma unroll
        for (int n = 0; n < N; ++n) theirs[n] = lane < kBlocks ? cluster.map_shared_rank(&s_part[0], lane)[n] : 0;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            before[n] = __reduce_add_sync(kFull, lane < static_cast<int>(team.rank) ? theirs[n] : 0);
            all[n] = __reduce_add_sync(kFull, theirs[n]);
        }
    }
}

// What row b of the result holds.
struct Source {
    int row, len;   // the row whose sequence it takes (-1: none), and its tokens
};

__device__ __forceinline__ Source source_of(const ShareArgs &a, int b, bool report) {
    Source s{a.parents != nullptr ? a.parents[b] : b, 0};
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
__device__ __forceinline__ int checked(const ShareArgs &a, int x) {
    if (x >= 0 && x < a.NB) return x;
    if (x != -1) raise_error(a.err, PKV_DEVERR_BLOCK);
    return -1;
}

__device__ __forceinline__ unsigned blocks_of(const ShareArgs &a, int len) {
    return (static_cast<unsigned>(len) + a.bs - 1u) / static_cast<unsigned>(a.bs);   // below 2^31: MBS * bs <= 2^31 - 1 - bs
}

// Every entry of the B rows, eight a thread at a time: first all are loaded (x = load(source, b, j, whether there is one),
// without branches), then all looked up (x = map(x)), then all put to use (use(source, b, j, x)), so that a thread's loads
// overlap.
// ONE: entries one after the other, their rows' sources (s_rows) at hand; else 256 entries of a row to a warp.
// The first pass (FIRST) starts with the team's barrier, past the loads of the cluster's first entries, which
// `held` keeps for the second pass.
constexpr int kAhead = 8, kSegment = 32 * kAhead;

struct Held {
    Source s;
    int x[kAhead];
};

template <bool FIRST, bool ONE, typename Load, typename Map, typename Use>
__device__ __forceinline__ void for_entries(const ShareArgs &a, const Team<ONE> &team, const Source *s_rows, Held &held, Load load,
                                            Map map, Use use) {
    const unsigned MBS = a.MBS;
    if constexpr (ONE) {
        if constexpr (FIRST) team.sync();
        // i / MBS for i, MBS <= 65536 (i < 2^16 where MBS > 1): the rounding of 2^32 / MBS upwards adds less than 1 / MBS
        const unsigned total = a.B * MBS, inv = MBS > 1 ? 0xffffffffu / MBS + 1 : 0;
        for (unsigned i0 = threadIdx.x; i0 < total; i0 += kAhead * kThreads) {
            int x[kAhead];
            unsigned row[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const unsigned i = i0 + k * kThreads;
                row[k] = MBS > 1 ? __umulhi(i, inv) : i;
                x[k] = i < total ? load(s_rows[row[k]], row[k], i - row[k] * MBS, true) : -1;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) x[k] = map(x[k]);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const unsigned i = i0 + k * kThreads;
                if (i < total) use(s_rows[row[k]], row[k], i - row[k] * MBS, x[k]);
            }
        }
    } else {
        const unsigned warp = team.tid() >> 5, lane = threadIdx.x & 31, segments = (MBS + kSegment - 1) / kSegment;
        const unsigned long long items = static_cast<unsigned long long>(a.B) * segments;
        unsigned long long i = warp;
        do {
            const unsigned b = static_cast<unsigned>(segments == 1 ? i : i / segments);
            const unsigned j0 = static_cast<unsigned>(i - static_cast<unsigned long long>(b) * segments) * kSegment + lane;
            Source s{-1, 0};
            int x[kAhead];
            if (FIRST || i != warp) {
                if (i < items) s = source_of(a, b, FIRST && j0 == 0);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) x[k] = load(s, b, j0 + 32 * k, (i < items) & (j0 + 32 * k < MBS));
            } else {
                s = held.s;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) x[k] = held.x[k];
            }
            if (FIRST && i == warp) {
                held.s = s;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) held.x[k] = x[k];
                team.sync();
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) x[k] = map(x[k]);
            if (i < items) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (j0 + 32 * k < MBS) use(s, b, j0 + 32 * k, x[k]);
            }
            i += Team<ONE>::kAll / 32;
        } while (i < items);
    }
}

// The start of both kernels: the ids' two numbers (in shared memory for one block) cleared to (held, second), and one
// block's rows' sources.  No barrier yet.
template <bool ONE>
__device__ __forceinline__ void clear(const ShareArgs &a, const Team<ONE> &team, int *refs, int *other, int second, Source *s_rows) {
    for (unsigned i = team.tid(); i < static_cast<unsigned>(a.NB); i += Team<ONE>::kAll) {
        refs[i] = a.held != nullptr && a.held[i] != 0 ? 1 : 0;
        other[i] = second;
    }
    if constexpr (ONE)
        for (unsigned b = threadIdx.x; b < static_cast<unsigned>(a.B); b += kThreads) s_rows[b] = source_of(a, b, true);
}

template <bool ONE>
__global__ void __launch_bounds__(kThreads) fork_kernel(const ShareArgs a) {
    extern __shared__ int s_ids[];
    __shared__ int s_warp[2][32], s_part[2];
    pdl_wait();
    const Team<ONE> team;
    const unsigned tid = team.tid(), NB = a.NB, B = a.B;
    int *refs = ONE ? s_ids : a.refs;              // entries that name a block inside a row, or hold it
    int *first = ONE ? s_ids + NB : a.first;       // the lowest row that ends, partly filled, in it
    Source *s_rows = reinterpret_cast<Source *>(s_ids + 2 * static_cast<size_t>(NB));
    clear(a, team, refs, first, kNobody, s_rows);
    const int32_t *table = a.B > 0 ? a.table : a.refs;   // an address to read in vain
    int32_t *rows = a.rows;   // [B][MBS] of the result: the table itself where nothing reads the parents' rows any more
    Held held;
    for_entries<true>(a, team, s_rows, held,
                [&](const Source &s, unsigned, unsigned j, bool there) {
                    there = there & (j < blocks_of(a, s.len));
                    const int x = table[there ? static_cast<size_t>(s.row) * a.MBS + j : 0];
                    return there ? x : -1;
                }, [](int x) { return x; },
                [&](const Source &s, unsigned b, unsigned j, int x) {
                    x = checked(a, x);
                    const bool last = s.len % a.bs != 0 && j == static_cast<unsigned>(s.len / a.bs);   // partly filled
                    if (x >= 0) {
                        if (last) atomicMin(first + x, static_cast<int>(b));
                        else atomicAdd(refs + x, 1);
                    }
                    if (last) a.last[b] = x;
                    if (j == 0) a.place[b] = s.len;
                    rows[static_cast<size_t>(b) * a.MBS + j] = x;
                });
    team.sync();
    // rows that get a copy of their last block, and free blocks; a thread keeps its rows to the end
    const Run my_rows(team.part(B)), my_ids(team.part(NB));
    int len[kRowsEach], old[kRowsEach], mine[2] = {0, 0}, base[2], total[2], before[2], all[2];
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
        const unsigned b = my_rows.at(k);
        const bool there = k < static_cast<int>(my_rows.rounds) && b < my_rows.end;
        len[k] = there ? a.place[b] : 0;
        const int last = there ? a.last[b] : -1;
        old[k] = len[k] % a.bs != 0 ? last : -1;   // of other rows this call has written none: whatever the workspace held
    }
    auto unused = [&](unsigned i) {
        const int inside = refs[i], ends = first[i];   // both loads at once
        return (inside == 0) & (ends == kNobody);
    };
    const Flags spare(my_ids, unused);
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
        const int b = static_cast<int>(my_rows.at(k));
        const int x = max(old[k], 0), inside = refs[x], ends = first[x];
        if (inside == 0 && ends == b) old[k] = -1;   // it keeps its block (old[k] of -1 stays)
        mine[0] += __popc(__ballot_sync(kFull, old[k] >= 0));
    }
    mine[1] = spare.count;
    warp_bases(mine, s_warp, base, total);
    share_counts(team, total, s_part, before, all);
    const int served = min(all[0], all[1]), left = all[1] - served;
    int row_base = before[0] + base[0], id_base = before[1] + base[1], nth[kRowsEach];
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) nth[k] = rank_of(old[k] >= 0, row_base);
    for (unsigned r = 0; r < my_ids.rounds; ++r) {
        const unsigned i = my_ids.at(r);
        const bool f = spare.of(my_ids, r, unused);
        const int at = rank_of(f, id_base);
        if (i >= my_ids.end) continue;
        const bool handed = f && at < served;
        if (handed) a.fresh[at] = static_cast<int>(i);
        else if (f) a.free_list[all[1] - 1 - at] = static_cast<int>(i);
        const int inside = f ? 0 : refs[i];   // of the rows that end in a block one at most still names it
        a.refs[i] = inside != 0 ? inside : handed || !f;
    }
    for (unsigned i = left + tid; i < NB; i += team.kAll) a.free_list[i] = -1;
    for (unsigned i = served + tid; i < B; i += team.kAll) reinterpret_cast<int2 *>(a.pairs)[i] = make_int2(-1, -1);
    if (tid == 0) {
        *a.free_count = left;
        *a.pair_count = served;
        if (served < all[0]) raise_error(a.err, PKV_DEVERR_POOL);
    }
    team.sync();
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
        const unsigned b = my_rows.at(k);
        if (k >= static_cast<int>(my_rows.rounds) || b >= my_rows.end) break;
        if (old[k] >= 0 && nth[k] < served) {
            const int to = a.fresh[nth[k]];
            reinterpret_cast<int2 *>(a.pairs)[nth[k]] = make_int2(old[k], to);
            rows[static_cast<size_t>(b) * a.MBS + len[k] / a.bs] = to;
        } else if (old[k] >= 0) {
            len[k] = 0;   // the pool was too small for this row: it is empty
        }
        a.lens_out[b] = a.place[b] = len[k];
    }
    if (rows == a.table_out && served == all[0]) return;
    team.sync();
    // the rows built aside go into the table; rows that the pool was too small for are empty
    for (unsigned b = tid >> 5; b < B; b += team.kAll / 32) {
        const bool none = a.place[b] == 0;
        if (rows == a.table_out && !none) continue;
#pragma unroll 8
        for (unsigned j = threadIdx.x & 31; j < static_cast<unsigned>(a.MBS); j += 32) {
            const size_t at = static_cast<size_t>(b) * a.MBS + j;
            a.table_out[at] = none ? -1 : __ldcg(rows + at);
        }
    }
}

template <bool ONE>
__global__ void __launch_bounds__(kThreads) compact_kernel(const ShareArgs a) {
    extern __shared__ int s_ids[];
    __shared__ int s_warp[3][32], s_part[3], s_warp1[1][32], s_part1[1];
    pdl_wait();
    const Team<ONE> team;
    const unsigned tid = team.tid(), NB = a.NB;
    int *refs = ONE ? s_ids : a.refs;              // entries that name a block
    int *moved = ONE ? s_ids + NB : a.first;       // where it goes; for now, of one that moves, its rank: -1 - rank
    Source *s_rows = reinterpret_cast<Source *>(s_ids + 2 * static_cast<size_t>(NB));
    auto held = [&](unsigned i) { return a.held != nullptr && a.held[i] != 0; };
    clear(a, team, refs, moved, 0, s_rows);
    const int32_t *table = a.B > 0 ? a.table : a.refs;   // an address to read in vain
    auto entry = [&](const Source &s, unsigned b, unsigned j, bool there) {
        there = there & (j < blocks_of(a, s.len));
        const int x = table[there ? static_cast<size_t>(b) * a.MBS + j : 0];
        return there ? x : -1;
    };
    Held first;
    for_entries<true>(a, team, s_rows, first, entry, [](int x) { return x; }, [&](const Source &, unsigned, unsigned, int x) {
        x = checked(a, x);
        if (x >= 0) atomicAdd(refs + x, 1);
    });
    team.sync();
    const Run ids(team.part(NB));
    auto in_use = [&](unsigned i) { return refs[i] != 0; };
    const Flags using_it(ids, in_use), holding(a.held != nullptr ? ids : Run(make_uint2(0, 0)), held);
    int base1[1], total1[1], before1[1], all1[1];
    {
        const int mine[1] = {using_it.count};
        warp_bases(mine, s_warp1, base1, total1);
    }
    share_counts(team, total1, s_part1, before1, all1);
    const unsigned used = all1[0];
    // blocks that move (in use, not held, from `used` on), free ids below, free or vacated ids from there on
    auto kinds = [&](unsigned r, bool (&f)[3]) {
        const unsigned i = ids.at(r);
        const bool there = i < ids.end, busy = using_it.of(ids, r, in_use), high = there && i >= used;
        const bool fixed = high && a.held != nullptr && holding.of(ids, r, held);
        f[0] = busy && high && !fixed;
        f[1] = there && !busy && !high;
        f[2] = high && !fixed;
    };
    int count[3] = {0, 0, 0}, base[3], total[3], before[3], all[3];
    for (unsigned r = 0; r < ids.rounds; ++r) {
        bool f[3];
        kinds(r, f);
#pragma unroll
        for (int n = 0; n < 3; ++n) count[n] += __popc(__ballot_sync(kFull, f[n]));
    }
    warp_bases(count, s_warp, base, total);
    share_counts(team, total, s_part, before, all);
#pragma unroll
    for (int n = 0; n < 3; ++n) base[n] += before[n];
    // as many ids are free below `used` as are taken from there on, so every mover has a place
    const int moves = all[0], spare = all[1] - moves, free_all = spare + all[2];
    for (unsigned r = 0; r < ids.rounds; ++r) {
        const unsigned i = ids.at(r);
        bool f[3];
        int at[3];
        kinds(r, f);
#pragma unroll
        for (int n = 0; n < 3; ++n) at[n] = rank_of(f[n], base[n]);
        if (i >= ids.end) continue;
        moved[i] = f[0] ? -1 - at[0] : static_cast<int>(i);
        if (f[1]) {
            if (at[1] < moves) a.fresh[at[1]] = static_cast<int>(i);
            else a.free_list[free_all - 1 - (at[1] - moves)] = static_cast<int>(i);
        }
        if (f[2]) a.free_list[free_all - 1 - (spare + at[2])] = static_cast<int>(i);
        // what stays; blocks that move write both ends below
        if (ONE && !f[0] && !(f[1] && at[1] < moves)) a.refs[i] = refs[i];
    }
    for (unsigned i = free_all + tid; i < NB; i += team.kAll) a.free_list[i] = -1;
    for (unsigned i = moves + tid; i < NB / 2; i += team.kAll) reinterpret_cast<int2 *>(a.pairs)[i] = make_int2(-1, -1);
    if (tid == 0) {
        *a.free_count = free_all;
        *a.pair_count = moves;
    }
    team.sync();
    const uint2 part = team.part(NB);
    for (unsigned i0 = max(part.x, used) + threadIdx.x; i0 < part.y; i0 += 4 * kThreads) {   // four a thread: their loads overlap
        int nth[4], n[4], to[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned i = i0 + k * kThreads;
            nth[k] = i < part.y ? -1 - moved[i] : -1;
            n[k] = i < part.y ? refs[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = nth[k] >= 0 ? a.fresh[nth[k]] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned i = i0 + k * kThreads;
            if (nth[k] >= 0) {
                moved[i] = to[k];
                reinterpret_cast<int2 *>(a.pairs)[nth[k]] = make_int2(static_cast<int>(i), to[k]);
                a.refs[to[k]] = n[k];
                a.refs[i] = 0;
            }
        }
    }
    team.sync();
    for_entries<false>(a, team, s_rows, first, entry,
                [&](int x) {
                    const bool there = (x >= 0) & (x < a.NB);
                    const int to = moved[there ? x : 0];
                    return there ? to : -1;
                },
                [&](const Source &, unsigned b, unsigned j, int x) { a.table_out[static_cast<size_t>(b) * a.MBS + j] = x; });
}

// ---------------------------------------------------------------- copies of a list that the GPU counted

constexpr int kCopyThreads = 256, kCopyAhead = 8;

template <typename U>
__global__ void __launch_bounds__(kCopyThreads, 5)
    kv_block_copy_counted_kernel(U *kc, U *vc, const int32_t *pairs, int n, const int32_t *count, long long block_units, int NB,
                                 unsigned *err) {
    pdl_wait();
    int live = *count;
    if (live < 0 || live > n) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(err, PKV_DEVERR_PAIR);
        live = max(0, min(live, n));
    }
    // pieces of kCopyThreads * kCopyAhead units: of K, then of V, of one pair after the other
    const long long span = kCopyThreads * kCopyAhead;
    const long long per = (block_units + span - 1) / span, pieces = 2 * per * live;
    for (long long w = blockIdx.x; w < pieces; w += gridDim.x) {
        const long long pair = w / (2 * per), rest = w - pair * 2 * per;
        const int src = pairs[2 * pair], dst = pairs[2 * pair + 1];
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

// Scratch behind a call: one number a block [NB], a row's length and last block [B] each, fresh blocks [B] or
// ids that blocks move to [NB / 2], and the table where it replaces the one that it is built from ([B][MBS]).
size_t share_workspace_bytes(int B, int MBS, int NB) {
    return (static_cast<size_t>(NB) + 2 * static_cast<size_t>(B) + std::max(static_cast<size_t>(B), static_cast<size_t>(NB) / 2) +
            static_cast<size_t>(B) * MBS) *
           sizeof(int32_t);
}

namespace {

template <typename Kernel>
cudaError_t launch_team(Kernel one, Kernel cluster, const ShareArgs &a, std::atomic<unsigned long long> &ready, cudaStream_t stream) {
    if (a.NB > kOneIds || a.B > kOneRows || static_cast<long long>(a.B) * a.MBS > kOneEntries) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(kBlocks);
        cfg.blockDim = dim3(kThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kBlocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // as launch_dependent
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, cluster, a);
    }
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {   // shared memory opted in, once a device
        e = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * (kOneIds + kOneRows));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit);
    }
    return launch_dependent(one, dim3(1), dim3(kThreads), 8 * (static_cast<size_t>(a.NB) + a.B), stream, a);
}

}  // namespace

cudaError_t launch_fork(ShareArgs a, void *workspace, bool aside, cudaStream_t stream) {
    static std::atomic<unsigned long long> ready{0};
    int32_t *ws = static_cast<int32_t *>(workspace);
    a.first = ws;
    a.place = ws + a.NB;
    a.last = a.place + a.B;
    a.fresh = a.last + a.B;
    a.rows = aside ? a.fresh + std::max(a.B, a.NB / 2) : a.table_out;
    return launch_team(fork_kernel<true>, fork_kernel<false>, a, ready, stream);
}

cudaError_t launch_compact(ShareArgs a, void *workspace, cudaStream_t stream) {
    static std::atomic<unsigned long long> ready{0};
    int32_t *ws = static_cast<int32_t *>(workspace);
    a.first = ws;
    a.fresh = ws + a.NB + 2 * static_cast<size_t>(a.B);
    return launch_team(compact_kernel<true>, compact_kernel<false>, a, ready, stream);
}

cudaError_t launch_kv_block_copy_counted(void *k_cache, void *v_cache, int elem_bytes, const int32_t *pairs, int n,
                                         const int32_t *count, int Hkv, int d, int bs, int NB, int sm_count, unsigned *err,
                                         cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    const size_t bytes = static_cast<size_t>(Hkv) * bs * d * elem_bytes;
    size_t at = bytes | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
    const int u = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : at % 2 == 0 ? 2 : 1;
    const long long units = static_cast<long long>(bytes / u), span = kCopyThreads * kCopyAhead;
    // fifteen blocks an SM, three times what it holds, so that none of few long ones ends alone (6254 pairs: eight 64.7 us,
    // fifteen 63.3; forty 61.7, but a list without pairs then costs their start)
    const unsigned grid = static_cast<unsigned>(std::min(2ll * n * ((units + span - 1) / span), 15ll * std::max(sm_count, 1)));
#define PKV_COPY(UT)                                                                                                     \
    return launch_dependent(kv_block_copy_counted_kernel<UT>, dim3(grid), dim3(kCopyThreads), 0, stream,                 \
                            static_cast<UT *>(k_cache), static_cast<UT *>(v_cache), pairs, n, count, units, NB, err)
    switch (u) {
        case 16: PKV_COPY(uint4);
        case 4: PKV_COPY(uint32_t);
        case 2: PKV_COPY(uint16_t);
        default: PKV_COPY(uint8_t);
    }
#undef PKV_COPY
}

}  // namespace pkv
