// internal.h -- declarations shared by the library's translation units (not the ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

// ------------------------------------------------------------- host helpers

// Encode a 2-D / 3-D bf16 tiled tensor map with 128-byte swizzle.  dims[0] is the
// innermost (contiguous) dimension; strides are the byte strides of dims 1.. .
bool encode_map_bf16(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                     const uint64_t *strides_bytes, const uint32_t *box);
// The same for a byte array (FP8 codes).
bool encode_map_u8(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                   const uint64_t *strides_bytes, const uint32_t *box);

// Per-device state of the current device (SM count, device error word), set up on
// first use; and recording of the calling thread's pkv_last_error() message.
pkv_status current_device_info(int *sm_count, unsigned **err);
pkv_status record_error(pkv_status status, const char *message);

// ---------------------------------------------------------------- cache ops

cudaError_t launch_kv_append(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                             int elem_bytes, const int64_t *slot_mapping, int T, int Hkv, int d,
                             int bs, int NB, unsigned *err, cudaStream_t stream);

// FP8 append: new rows (dt PKV_BF16 or PKV_F32) quantised to E4M3 codes + fp32 row scales.
cudaError_t launch_kv_append_fp8(const void *k_new, const void *v_new, pkv_dtype new_dt, uint8_t *k_codes,
                                 uint8_t *v_codes, float *k_scale, float *v_scale,
                                 const int64_t *slot_mapping, int T, int Hkv, int d, int bs, int NB,
                                 unsigned *err, cudaStream_t stream);

cudaError_t launch_kv_block_copy(void *k_cache, void *v_cache, int elem_bytes,
                                 const int32_t *pairs, int n, int Hkv, int d, int bs, int NB,
                                 unsigned *err, cudaStream_t stream);

// 4-bit caches (cache_q4.cu): rows quantised into slots, and the values of slots read out.
// Sizes checked by the caller: d % group == 0, group 32, 64 or 128, caches 4-byte aligned.
cudaError_t launch_kv_append_q4(const void *k_new, const void *v_new, pkv_dtype new_dt, uint8_t *k_cache,
                                uint8_t *v_cache, const int64_t *slot_mapping, int T, int Hkv, int d, int group,
                                int bs, int NB, int sm_count, unsigned *err, cudaStream_t stream);
cudaError_t launch_kv_gather_q4(void *k_out, void *v_out, pkv_dtype out_dt, const uint8_t *k_cache,
                                const uint8_t *v_cache, const int64_t *slot_mapping, int T, int Hkv, int d,
                                int group, int bs, int NB, int sm_count, unsigned *err, cudaStream_t stream);

// ------------------------------------------------------------------ decode

struct DecodePlan {
    bool tensor_core;   // bf16 TMA + mma path; otherwise the CUDA-core path
    bool group;         // tensor-core path with 9..64 query heads per KV head: all head
                        // tiles of a KV head in one CTA sharing each page
    bool umma;          // the large-group case on tcgen05 (d in {64, 128})
    int splits;         // chunks per sequence at most (1: one pass, no workspace)
    int chunk_pages;    // blocks per chunk
    bool fused_merge;   // the last chunk of each unit merges (counters in the workspace)
    size_t counter_bytes = 0;  // bytes of arrival counters a call uses (from the start)
    int sm_count = 0;          // the device's SMs the plan was made for
    size_t workspace_bytes;
    int q_per_tile = 1; // tcgen05 kernel: query rows per block (several queries per sequence)
    int qtiles = 1;     // tcgen05 kernel: query tiles per sequence
    bool paged_prefill = false;   // many query rows per sequence: the chunked-prefill kernel
                                  // (128 rows of one head per block, all keys, no split)
};

// caches_aligned: both cache bases 16-byte aligned; q_aligned: q 16-byte aligned (the
// tcgen05 large-group kernel copies the group's queries in one bulk copy).
DecodePlan plan_decode(int B, int Hq, int Hkv, int d, int bs, int MBS, int NB, pkv_dtype dt,
                       int num_splits, int sm_count, bool caches_aligned, bool q_aligned);

// Several query rows per sequence (pkv_paged_attention with cu_q): Tq rows, at most max_q
// per sequence.  bf16 caches with d in {64, 128}, bs in {16, 32}, aligned caches and q:
// without a window and with at least kPagedPrefillMinRows rows in some sequence, the
// chunked-prefill kernel (paged_prefill.cu); otherwise, with up to 64 heads per KV head,
// the tcgen05 kernel with tiles of floor(64 / m) query rows; other shapes the CUDA-core
// path.  MBS: the blocks any row can see.
constexpr int kPagedPrefillMinRows = 64;
DecodePlan plan_attention_rows(int B, int Tq, int max_q, int Hq, int Hkv, int d, int bs, int MBS, int NB,
                               pkv_dtype dt, int window, int num_splits, int sm_count, bool caches_aligned,
                               bool q_aligned);

// Workspace that covers every plan these shapes can take (element type and alignment
// unknown).
size_t decode_workspace_upper_bound(int B, int Hq, int Hkv, int d, int bs, int MBS,
                                    int num_splits, int sm_count);

struct DecodeArgs {
    float *out;
    float *lse;
    const float *q;
    const void *k_cache;
    const void *v_cache;
    const int32_t *block_table;
    const int32_t *context_lens;
    int B, Hq, Hkv, d, bs, MBS, NB;
    float scale;
    void *workspace;
    unsigned *err;
    int window = 0;                  // > 0: sliding window of this many tokens
    int sinks = 0;                   // > 0 (with a window): as many first tokens stay visible
    const float *k_scale = nullptr;  // FP8 caches: per-row scales [NB][Hkv][bs]
    const float *v_scale = nullptr;
    const int32_t *cu_q = nullptr;   // query rows per sequence; nullptr: one per sequence
    int rows = -1;                   // query rows (B when cu_q is nullptr)
    int max_q = 1;                   // query rows of a sequence at most
    // the step's new tokens, appended inside the decode launch (decode_fuses_append)
    const void *k_new = nullptr, *v_new = nullptr;   // [B][Hkv][d], bf16
    const int64_t *new_slots = nullptr;              // [B]; < 0: no new token
    const int32_t *kv_start = nullptr;               // [B]: keys read from this token on (a shared
                                                     // prefix attended elsewhere); nullptr: 0
};

// Whether launch_decode can write the step's new tokens (one per sequence, at its last
// position; rows of type new_dt) inside the decode launch for this plan over a cache of
// type dt; otherwise kv_append (kv_append_fp8) runs first.
bool decode_fuses_append(const DecodePlan &plan, pkv_dtype dt, pkv_dtype new_dt, int Hq, int Hkv,
                         const void *k_new, const void *v_new);

// Blocks a query row can see: all of MBS, or with a window of W tokens at most
// ceil(W / bs) + 1 (the window may start inside a block).
inline int visible_blocks(int MBS, int bs, int window) {
    if (window <= 0) return MBS;
    const long long w = (static_cast<long long>(window) + bs - 1) / bs + 1;
    return static_cast<int>(w < MBS ? w : MBS);
}

// Blocks that the rows of a sequence, max_q at most, can see together.
inline int visible_blocks_of_rows(int MBS, int bs, int window, int max_q) {
    const long long w = window > 0 ? static_cast<long long>(window) + max_q - 1 : 0;
    return visible_blocks(MBS, bs, static_cast<int>(w < 0x7fffffff ? w : 0x7fffffff));
}

// The same with the first `sinks` tokens visible too: their blocks beside the windows'.
inline int visible_blocks_with_sinks(int MBS, int bs, int window, int sinks, int max_q) {
    const long long n = visible_blocks_of_rows(MBS, bs, window, max_q) + (static_cast<long long>(sinks) + bs - 1) / bs;
    return static_cast<int>(n < MBS ? n : MBS);
}

cudaError_t launch_decode(const DecodeArgs &a, const DecodePlan &plan, pkv_dtype dt,
                          cudaStream_t stream);

// Windows with first tokens that stay visible (decode_sinks.cu).
struct SinksPlan {
    bool mma;            // on tensor cores (else CUDA cores): warp MMAs, or
    bool umma;           // tcgen05
    int tiles, groups;   // tiles of 8 (query row, head) pairs of a block, blocks for the pairs of a KV head
    int block_heads;     // on CUDA cores: heads of a block
    int splits, chunk_pages;
    bool fused_merge;
    size_t workspace_bytes;
};

// pages: the blocks any row can see; aligned: caches on 16-byte boundaries (q on 8).
SinksPlan plan_sinks(int B, int rows, int max_q, int Hq, int Hkv, int d, int bs, int pages, int NB, pkv_dtype dt, int num_splits,
                     int sm_count, bool aligned);
cudaError_t launch_decode_sinks(const DecodeArgs &a, const SinksPlan &plan, pkv_dtype dt, cudaStream_t stream);

// ------------------------------------------------- attention over a 4-bit cache

struct Q4Plan {
    bool umma;           // many (query row, head) pairs per sequence and KV head: the tcgen05 kernel
    bool mma;            // most d and group sizes with bs 8, 16 or 32, aligned: the warp-MMA kernel; else CUDA cores
    int mma_rows;        // mma: pairs of a tile, 4 or 8
    int tiles;           // tiles of 64 (umma) or mma_rows pairs per sequence and KV head
    bool balanced;       // even shares of all sequences' keys for `blocks` thread blocks
    int blocks;
    bool fused_merge;    // the last chunk of a unit merges (counters in the workspace)
    int splits;          // chunks per sequence at most (1: one pass, no workspace)
    int chunk_pages;     // blocks per chunk
    size_t workspace_bytes;
};

// pages: the blocks any row can see; aligned: caches and q on 16-byte boundaries.
Q4Plan plan_attend_q4(int B, int rows, int max_q, int Hq, int Hkv, int d, int group, int bs, int pages,
                      int num_splits, int sm_count, bool aligned);

struct AttendQ4Args {
    float *out;
    float *lse;
    const float *q;
    const uint8_t *k_cache;
    const uint8_t *v_cache;
    const int32_t *block_table;
    const int32_t *context_lens;
    const int32_t *cu_q;   // query rows per sequence; nullptr: one per sequence
    int B, rows, max_q, Hq, Hkv, d, group, bs, MBS, NB;
    float scale;
    int window;
    void *workspace;
    unsigned *err;
    // a step's new tokens, written inside the attention launch (q4_fuses_append)
    const void *k_new, *v_new;
    pkv_dtype new_dt;
    const int64_t *new_slots;
};

// Whether the attention launch writes a step's new tokens itself: exactly one thread block reads
// the page that holds a sequence's last position for each KV head.
bool q4_fuses_append(const Q4Plan &plan);

cudaError_t launch_attend_q4(const AttendQ4Args &a, const Q4Plan &plan, cudaStream_t stream);

// ------------------------------------------------------------------ block tables

struct ExtendArgs {
    int32_t *block_table;
    const int32_t *context_lens, *new_tokens, *free_list, *free_count;
    int32_t *context_lens_out, *cu_new;
    int64_t *slot_mapping;
    int64_t *step_slots;   // nullptr: not wanted
    int32_t *free_count_out;
    int B, T, MBS, bs, NB;
    unsigned *arrivals;    // workspace (more than one block): zero before and after
    unsigned *err;
};

struct ReleaseArgs {
    int32_t *block_table;
    const int32_t *first_block, *end_block;
    int32_t *free_list;
    const int32_t *free_count;
    int32_t *free_count_out;
    int B, MBS, NB;
    int32_t *counts;       // workspace [B + 1]: entries given back per row, the count before
    unsigned *err;
};

int extend_blocks(int T, int sm_count);                  // thread blocks of an extend launch
bool release_in_one_block(int B, int MBS);
cudaError_t launch_block_tables_extend(const ExtendArgs &a, int sm_count, cudaStream_t stream);
cudaError_t launch_block_tables_release(const ReleaseArgs &a, int sm_count, cudaStream_t stream);

// Block tables with shared blocks (share_tables.cu).
struct ShareArgs {
    const int32_t *table;        // [B][MBS]
    const int32_t *lens;         // [B]
    const int32_t *parents;      // [B]; nullptr: every row its own
    const int32_t *held;         // [NB] blocks in use beside the tables; nullptr: none
    int32_t *table_out;          // may be `table`
    int32_t *lens_out;           // fork; may be `lens`
    int32_t *refs, *free_list;   // [NB]
    int32_t *free_count, *pair_count;
    int32_t *pairs;              // [B][2] (fork), [NB / 2][2] (compact)
    int B, MBS, bs, NB;
    int32_t *first, *place, *last, *fresh, *rows;   // scratch, set by the launch
    unsigned *err;
};

size_t share_workspace_bytes(int B, int MBS, int NB);
// aside: the rows are built in the workspace (table_out replaces the table that other rows still read)
cudaError_t launch_fork(ShareArgs a, void *workspace, bool aside, cudaStream_t stream);
cudaError_t launch_compact(ShareArgs a, void *workspace, cudaStream_t stream);
cudaError_t launch_kv_block_copy_counted(void *k_cache, void *v_cache, int elem_bytes, const int32_t *pairs, int n,
                                         const int32_t *count, int Hkv, int d, int bs, int NB, int sm_count, unsigned *err,
                                         cudaStream_t stream);

// ------------------------------------------------------------------- rotary positions

struct RopeArgs {
    void *q_out;                 // [T][Hq][d]
    const void *q, *k, *v;       // [T][heads][d], rows of a token at the strides (elements); k, v may be nullptr
    long long q_stride, k_stride, v_stride;
    void *k_dst, *v_dst;         // caches (with slots), or k_dst [T][Hkv][d]
    const int32_t *positions;
    const unsigned long long *turns;   // [rot / 2]
    const int64_t *slots;        // nullptr: rows
    int T, Hq, Hkv, d, rot, bs;
    long long n_slots;
    float mscale;
    bool inverse;
    int block_tokens;            // set by the launch
    unsigned *err;
};

cudaError_t launch_rope(const RopeArgs &a, pkv_dtype dt, pkv_dtype q_out_dt, bool interleaved, int sm_count,
                        cudaStream_t stream);
bool rope_turns(uint64_t *turns, int rot, double base, int scaling, double factor, double original, double low, double high);

// ------------------------------------------------------------------- drafted tokens

struct VerifyArgs {
    int32_t *accepted, *tokens;  // [B], [D + B]
    const void *target, *draft;  // [D + B][V], [D][V] or nullptr, rows at the strides (elements)
    long long target_stride, draft_stride;
    const int32_t *draft_tokens, *cu_drafts;
    const float *uniforms;       // [D + B]
    const int32_t *lens;
    int32_t *lens_out;           // nullptr: not wanted
    int B, D, V;
    unsigned *err;
};

cudaError_t launch_verify(const VerifyArgs &a, pkv_dtype dt, int sm_count, cudaStream_t stream);

// ----------------------------------------------------------------- prefill

struct PrefillArgs {
    float *out;
    float *lse;
    const void *q, *k, *v;
    const int32_t *cu_seqlens;
    int B, T, max_seqlen, Hq, Hkv, d;
    float scale;
    unsigned *err;
};

bool prefill_tensor_core_ok(pkv_dtype dt, int d, const void *q, const void *k, const void *v,
                            int T, int Hq, int Hkv);

cudaError_t launch_prefill(const PrefillArgs &a, pkv_dtype dt, cudaStream_t stream);

}  // namespace pkv
