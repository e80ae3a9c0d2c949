// block_tables.cu -- block tables, slot maps and the free list of physical blocks, kept on the
// GPU: what BlockManager does on the host for sequences that own their blocks (plumephp.com
// "KV Cache 优化与注意力机制加速" §4.2-§4.3, BlockTable.allocate / get_kv: ceil(n / bs) blocks,
// position pos in slot table[pos / bs] * bs + pos % bs), so that a captured decode loop needs
// no host round trip between steps.
//
// extend: rows in order; row b holding L tokens and getting n more owns have = ceil(L / bs)
//   blocks and needs want - have, want = ceil((L + n) / bs).  With prefix sums over the rows of
//   the blocks needed (D) and the tokens (C), the i-th block needed is free_list[count - 1 - i]
//   and token t of the packed new tokens belongs to the row whose C holds it.  The sums are a
//   block-wide scan over 1024 rows at a time; tokens and table entries are then dealt to the
//   threads by number and find their row by binary search in shared memory, so one row with a
//   whole prompt and a thousand rows with one token each cost the same.  Every thread block
//   scans all rows (12 bytes each, from L2) and takes a share of tokens and entries; what may
//   alias an input (the lengths, the free count) is written by the last block to arrive.
// release: the blocks of logical range [first, end) of every row go back on top of the list in
//   reverse order, so that giving back what one extend took restores the list exactly.
//
// Both move a few bytes per row and block: they are bound by launch and memory latency.  A row's blocks
// are given back by one warp, 32 at a time, one turn after the other: four rows of 256 take 8 us, four
// of 8192 68 us, one of 65536 639 us.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kRows = 1024;   // rows per scan, and threads per block
constexpr unsigned kFull = 0xffffffffu;

// Rows, tokens and blocks number up to 2^31 - 1; loops over them count in unsigned, whose next step
// (at most a grid of threads further) does not wrap.

// Inclusive sums of N numbers over the block's threads; totals[i] are the block's sums.
template <int N>
__device__ __forceinline__ void block_scan(unsigned long long (&x)[N], unsigned long long (&warp_sums)[N][32],
                                           unsigned long long (&totals)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const unsigned long long y = __shfl_up_sync(kFull, x[i], sh);
            if (lane >= sh) x[i] += y;
        }
    }
    __syncthreads();   // the sums of an earlier scan have been read
    if (lane == 31) {
#pragma unroll
        for (int i = 0; i < N; ++i) warp_sums[i][warp] = x[i];
    }
    __syncthreads();
    if (warp < N) {   // warp i sums the warps' number i
        unsigned long long w = warp_sums[warp][lane];
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const unsigned long long y = __shfl_up_sync(kFull, w, sh);
            if (lane >= sh) w += y;
        }
        warp_sums[warp][lane] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (warp > 0) x[i] += warp_sums[i][warp - 1];
        totals[i] = warp_sums[i][31];
    }
}

// The row r of the scan with ends[r] <= i < ends[r + 1] (ends non-decreasing, ends[0] = 0).
__device__ __forceinline__ int row_of(const int *ends, int i) {
    int lo = 0;
#pragma unroll
    for (int step = kRows / 2; step > 0; step >>= 1)
        if (ends[lo + step] <= i) lo += step;
    return lo;
}

__global__ void __launch_bounds__(kRows) block_tables_extend_kernel(const ExtendArgs a) {
    __shared__ unsigned long long warp_sums[2][32];
    __shared__ int s_cu[kRows + 1], s_need[kRows + 1], s_len[kRows];
    __shared__ int s_last;
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    const long long capacity = static_cast<long long>(a.MBS) * a.bs;
    const int given = *a.free_count;   // plain loads of what the call may write at its end (*_out)
    int count = given;
    if (count < 0 || count > a.NB) {
        if (lead && tid == 0) raise_error(a.err, PKV_DEVERR_POOL);
        count = 0;
    }
    if (lead && tid == 0) a.cu_new[0] = 0;
    // tokens asked for, tokens placed, blocks asked for and blocks handed out by earlier scans
    unsigned long long asked = 0, wanted = 0;
    int placed = 0, taken = 0;
    const unsigned B = a.B;
    for (unsigned r0 = 0; r0 < B; r0 += kRows) {
        const unsigned row = r0 + tid;
        int L = 0, n = 0;
        if (row < B) {
            L = a.context_lens[row];
            n = __ldg(a.new_tokens + row);
            if (L < 0 || n < 0 || static_cast<long long>(L) + n > capacity) {
                if (lead) raise_error(a.err, PKV_DEVERR_LEN);
                n = 0;       // the row stays as it was
            }
        }
        const int have = n > 0 ? (L + a.bs - 1) / a.bs : 0;
        int need = n > 0 ? static_cast<int>((static_cast<long long>(L) + n + a.bs - 1) / a.bs) - have : 0;
        unsigned long long sum[2] = {static_cast<unsigned>(need), static_cast<unsigned>(n)}, total[2];
        block_scan(sum, warp_sums, total);
        const bool ok = n == 0 || ((need == 0 || wanted + sum[0] <= static_cast<unsigned>(count)) &&
                                   asked + sum[1] <= static_cast<unsigned>(a.T));
        asked += total[1];
        wanted += total[0];
        if (!ok) {
            if (lead) raise_error(a.err, PKV_DEVERR_POOL);
            n = need = 0;    // the row stays as it was
        }
        if (__syncthreads_or(!ok)) {   // the sums over the rows that are served
            sum[0] = static_cast<unsigned>(need);
            sum[1] = static_cast<unsigned>(n);
            block_scan(sum, warp_sums, total);
        }
        s_need[tid + 1] = static_cast<int>(sum[0]);
        s_cu[tid + 1] = static_cast<int>(sum[1]);
        s_len[tid] = L;
        if (tid == 0) s_cu[0] = s_need[0] = 0;
        __syncthreads();
        const unsigned tokens = s_cu[kRows], blocks = s_need[kRows];
        if (lead && row < B) {
            a.cu_new[row + 1] = placed + s_cu[tid + 1];
            if (a.step_slots != nullptr && n == 0) a.step_slots[row] = -1;
        }
        const unsigned at = blockIdx.x * kRows + tid, step = gridDim.x * kRows;
        const int top = count - 1 - taken;
        for (unsigned k = at; k < blocks; k += step) {
            const int i = k, r = row_of(s_need, i), j = (s_len[r] + a.bs - 1) / a.bs + i - s_need[r];
            int blk = __ldg(a.free_list + top - i);
            if (blk < 0 || blk >= a.NB) {
                raise_error(a.err, PKV_DEVERR_BLOCK);
                blk = -1;
            }
            a.block_table[static_cast<size_t>(r0 + r) * a.MBS + j] = blk;
        }
        for (unsigned k = at; k < tokens; k += step) {
            const int t = k, r = row_of(s_cu, t), pos = s_len[r] + t - s_cu[r], j = pos / a.bs;
            const int owned = (s_len[r] + a.bs - 1) / a.bs;
            const int blk = j < owned ? a.block_table[static_cast<size_t>(r0 + r) * a.MBS + j]
                                      : __ldg(a.free_list + top - (s_need[r] + j - owned));
            long long slot = -1;   // padding, skipped by the cache writes
            if (blk < 0 || blk >= a.NB) raise_error(a.err, PKV_DEVERR_BLOCK);
            else slot = static_cast<long long>(blk) * a.bs + (pos - j * a.bs);
            a.slot_mapping[placed + t] = slot;
            if (a.step_slots != nullptr && t + 1 == s_cu[r + 1]) a.step_slots[r0 + r] = slot;   // the row's last
        }
        placed += static_cast<int>(tokens);
        taken += static_cast<int>(blocks);
        __syncthreads();   // the scan's arrays are read before the next one writes them
    }
    for (long long t = placed + static_cast<long long>(blockIdx.x) * kRows + tid; t < a.T;
         t += static_cast<long long>(gridDim.x) * kRows)
        a.slot_mapping[t] = -1;
    if (gridDim.x > 1) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            s_last = atomicAdd(a.arrivals, 1u) + 1 == gridDim.x;
            if (s_last) *a.arrivals = 0u;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
    } else {
        __syncthreads();
    }
    for (unsigned row = tid; row < B; row += kRows)
        a.context_lens_out[row] = a.context_lens[row] + (__ldcg(a.cu_new + row + 1) - __ldcg(a.cu_new + row));
    if (tid == 0) a.free_count_out[0] = given - taken;
}

// The row's range of table entries, empty when it is out of bounds (flagged once, by `report`).
__device__ __forceinline__ int2 range_of(const ReleaseArgs &a, int row, bool report) {
    const int first = a.first_block != nullptr ? __ldg(a.first_block + row) : 0, end = __ldg(a.end_block + row);
    if (first < 0 || end > a.MBS) {
        if (report) raise_error(a.err, PKV_DEVERR_LEN);
        return make_int2(0, 0);
    }
    return make_int2(first, max(first, end));
}

// Entries of the row that name a block (one warp; -1: given back before).
__device__ __forceinline__ int count_row(const ReleaseArgs &a, int row, int lane) {
    const int2 rg = range_of(a, row, lane == 0);
    const int32_t *t = a.block_table + static_cast<size_t>(row) * a.MBS;
    int n = 0;
    bool bad = false;
    for (int j = rg.x + lane; j < rg.y; j += 32) {
        const int blk = t[j];
        n += blk >= 0 && blk < a.NB;
        bad |= blk < -1 || blk >= a.NB;
    }
    if (bad) raise_error(a.err, PKV_DEVERR_BLOCK);
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) n += __shfl_xor_sync(kFull, n, sh);
    return n;
}

// The row's blocks onto the list, its first one at list[top], the next below it (one warp).
__device__ __forceinline__ void give_back_row(const ReleaseArgs &a, int row, int top, int lane) {
    const int2 rg = range_of(a, row, false);
    int32_t *t = a.block_table + static_cast<size_t>(row) * a.MBS;
    for (int j0 = rg.x; j0 < rg.y; j0 += 32) {
        const int j = j0 + lane;
        const int blk = j < rg.y ? t[j] : -1;
        const bool give = blk >= 0 && blk < a.NB;
        const unsigned all = __ballot_sync(kFull, give);
        if (give) {
            a.free_list[top - __popc(all & ((1u << lane) - 1))] = blk;
            t[j] = -1;
        }
        top -= __popc(all);
    }
}

// ONE: a single block counts and writes; otherwise the counts come from the kernel before.
template <bool ONE>
__global__ void __launch_bounds__(kRows) block_tables_release_kernel(const ReleaseArgs a) {
    __shared__ unsigned long long warp_sums[1][32];
    __shared__ int s_off[kRows];
    __shared__ int s_count[ONE ? kRows : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int count = ONE ? *a.free_count : a.counts[a.B];
    if (ONE) {
        for (int row = warp; row < a.B; row += 32) {
            const int n = count_row(a, row, lane);
            if (lane == 0) s_count[row] = n;
        }
        __syncthreads();
    }
    // every row's count first: the first row's first block goes on top of the list
    unsigned long long all = 0;
    const unsigned B = a.B;
    for (unsigned r0 = 0; r0 < B; r0 += kRows) {
        const unsigned row = r0 + tid;
        const int n = row < B ? (ONE ? s_count[row] : a.counts[row]) : 0;
        unsigned long long end[1] = {static_cast<unsigned>(n)}, total[1];
        block_scan(end, warp_sums, total);
        if (ONE) s_off[tid] = static_cast<int>(end[0]) - n;
        all += total[0];
    }
    // more blocks than the list can hold: some were given back twice
    if (count < 0 || count > a.NB || all > static_cast<unsigned long long>(a.NB - count)) {
        if (blockIdx.x == 0 && tid == 0) {
            raise_error(a.err, PKV_DEVERR_POOL);
            a.free_count_out[0] = count;
        }
        return;
    }
    const int top = count + static_cast<int>(all) - 1;
    __syncthreads();
    if (ONE) {
        for (int row = warp; row < a.B; row += 32) give_back_row(a, row, top - s_off[row], lane);
    } else {
        int before = 0;
        for (unsigned r0 = 0; r0 < B; r0 += kRows) {
            const unsigned row = r0 + tid;
            const int n = row < B ? a.counts[row] : 0;
            unsigned long long end[1] = {static_cast<unsigned>(n)}, total[1];
            block_scan(end, warp_sums, total);
            s_off[tid] = before + static_cast<int>(end[0]) - n;
            __syncthreads();
            for (unsigned r = r0 + blockIdx.x * 32 + warp; r < min(B, r0 + kRows); r += gridDim.x * 32)
                give_back_row(a, r, top - s_off[r - r0], lane);
            before += static_cast<int>(total[0]);
            __syncthreads();
        }
    }
    if (blockIdx.x == 0 && tid == 0) a.free_count_out[0] = count + static_cast<int>(all);
}

__global__ void __launch_bounds__(256) block_tables_count_kernel(const ReleaseArgs a) {
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.counts[a.B] = __ldg(a.free_count);
    for (unsigned row = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; row < static_cast<unsigned>(a.B);
         row += (gridDim.x * blockDim.x) >> 5) {
        const int n = count_row(a, row, lane);
        if (lane == 0) a.counts[row] = n;
    }
}

}  // namespace

// Up to two tokens a thread from one block (no arrival to wait for), then one: 17153 tokens of
// eight prompts 5.8 us with one token a thread, 7.9 with four; 512 of them either way 5.8 to 6.1.
int extend_blocks(int T, int sm_count) {
    if (T <= 2 * kRows) return 1;
    return static_cast<int>(std::min<long long>((static_cast<long long>(T) + kRows - 1) / kRows, std::max(sm_count, 1)));
}

cudaError_t launch_block_tables_extend(const ExtendArgs &a, int sm_count, cudaStream_t stream) {
    block_tables_extend_kernel<<<extend_blocks(a.T, sm_count), kRows, 0, stream>>>(a);
    return cudaGetLastError();
}

// One block of 32 warps up to 64 K table entries, else a counting launch over many blocks first.  One
// block: 8 rows of 256 entries 8 us, 300 of 64 20, 16 of 4096 49, 8 of 8192 90, 1024 of 64 63; counted
// first: 17 of 4096 45, 9 of 8192 80, 1025 of 64 14.  With many rows the border lies too high.
bool release_in_one_block(int B, int MBS) {
    return B <= kRows && static_cast<long long>(B) * MBS <= (64 << 10);
}

cudaError_t launch_block_tables_release(const ReleaseArgs &a, int sm_count, cudaStream_t stream) {
    if (release_in_one_block(a.B, a.MBS)) {
        block_tables_release_kernel<true><<<1, kRows, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const int counting = static_cast<int>(std::min<long long>((a.B + 7ll) / 8, 8ll * std::max(sm_count, 1)));
    block_tables_count_kernel<<<counting, 256, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int writing = std::min((std::min(a.B, kRows) + 31) / 32, std::max(sm_count, 1));
    block_tables_release_kernel<false><<<writing, kRows, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
