// api_q4.cu -- the extern "C" entry points of the 4-bit cache and of the block tables kept on
// the GPU: host-side checks as in api.cu, then the launches.
#include <cstdarg>
#include <cstdio>

#include "common.cuh"
#include "internal.h"
#include "q4_codes.cuh"

namespace pkv {
namespace {

pkv_status fail(pkv_status s, const char *fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return record_error(s, text);
}

pkv_status cuda_fail(cudaError_t e, const char *where) {
    return fail(PKV_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned_to(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool new_dtype(pkv_dtype dt) { return dt == PKV_F32 || dt == PKV_BF16; }

bool q4_sizes(int d, int group) {
    return (group == 32 || group == 64 || group == 128) && d >= group && d <= 256 && d % group == 0;
}

constexpr int kMaxBlockSize = 1 << 16;

pkv_status check_rows(const char *what, pkv_dtype dt, int T, int Hkv, int d, int group, int bs, int NB) {
    if (!new_dtype(dt)) return fail(PKV_ERR_UNSUPPORTED, "%s: element type %d", what, dt);
    if (T < 0 || Hkv < 1 || Hkv > 65535 || bs < 1 || bs > kMaxBlockSize || NB < 1 || !q4_sizes(d, group))
        return fail(PKV_ERR_INVALID_ARG,
                    "%s: T=%d Hkv=%d d=%d group=%d bs=%d NB=%d (need group 32, 64 or 128, d a multiple of it, d <= 256)",
                    what, T, Hkv, d, group, bs, NB);
    return PKV_OK;
}

pkv_status check_attend(const char *what, int B, int Tq, int max_q, int Hq, int Hkv, int d, int group, int bs,
                        int MBS, int NB, int window, int num_splits) {
    if (B < 0 || B > 65535 || Hq < 1 || Hq > 65535 || Hkv < 1 || Hq % Hkv != 0 || bs < 1 || bs > kMaxBlockSize ||
        MBS < 1 || static_cast<long long>(MBS) * bs > 0x7fffffffll - bs || NB < 1 || window < 0 || num_splits < 0 ||
        !q4_sizes(d, group))
        return fail(PKV_ERR_INVALID_ARG,
                    "%s: B=%d Hq=%d Hkv=%d d=%d group=%d bs=%d MBS=%d NB=%d window=%d num_splits=%d (need Hq %% Hkv == 0, "
                    "group 32, 64 or 128, d a multiple of it, d <= 256)",
                    what, B, Hq, Hkv, d, group, bs, MBS, NB, window, num_splits);
    if (Tq < 0 || max_q < 0 || static_cast<long long>(Tq) > static_cast<long long>(B) * max_q ||
        static_cast<long long>(Tq) * Hq > 0x7fffffffll)
        return fail(PKV_ERR_INVALID_ARG, "%s: B=%d Tq=%d max_q=%d", what, B, Tq, max_q);
    return PKV_OK;
}

size_t workspace_bound(int B, int Tq, int max_q, int Hq, int Hkv, int d, int group, int bs, int MBS, int window,
                       int num_splits, int sm_count) {
    const int pages = visible_blocks_of_rows(MBS, bs, window, max_q);
    size_t most = 0;   // whatever the pointers' alignment
    for (bool aligned : {false, true}) {
        const size_t n = plan_attend_q4(B, Tq, max_q, Hq, Hkv, d, group, bs, pages, num_splits, sm_count, aligned)
                             .workspace_bytes;
        most = n > most ? n : most;
    }
    return most;
}

struct StepRows {   // a decode step's new tokens (null: none)
    const void *k_new = nullptr, *v_new = nullptr;
    pkv_dtype new_dt = PKV_BF16;
    const int64_t *slots = nullptr;
};

pkv_status attend(const char *what, float *out, float *lse, const float *q, const StepRows &step, const uint8_t *k_cache,
                  const uint8_t *v_cache, const int32_t *block_table, const int32_t *context_lens, const int32_t *cu_q,
                  int B, int Tq, int max_q, int Hq, int Hkv, int d, int group, int bs, int MBS, int NB, float scale,
                  int window, int num_splits, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!aligned_to(q, 8)) return fail(PKV_ERR_INVALID_ARG, "%s: q must be 8-byte aligned", what);
    if (!aligned_to(k_cache, 4) || !aligned_to(v_cache, 4))
        return fail(PKV_ERR_INVALID_ARG, "%s: the caches must be 4-byte aligned", what);
    int sm_count = 0;
    unsigned *err = nullptr;
    const pkv_status s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    const bool aligned = aligned_to(k_cache, 16) && aligned_to(v_cache, 16) && aligned_to(q, 16) && aligned_to(out, 16);
    const Q4Plan plan = plan_attend_q4(B, Tq, max_q, Hq, Hkv, d, group, bs, visible_blocks_of_rows(MBS, bs, window, max_q),
                                       num_splits, sm_count, aligned);
    if (plan.workspace_bytes > 0 &&
        (workspace == nullptr || workspace_bytes < plan.workspace_bytes || !aligned_to(workspace, 16)))
        return fail(PKV_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace, got %zu", what,
                    plan.workspace_bytes, workspace == nullptr ? size_t(0) : workspace_bytes);
    AttendQ4Args a{};
    a.out = out;
    a.lse = lse;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_table = block_table;
    a.context_lens = context_lens;
    a.cu_q = cu_q;
    a.B = B;
    a.rows = Tq;
    a.max_q = max_q;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.group = group;
    a.bs = bs;
    a.MBS = MBS;
    a.NB = NB;
    a.scale = scale;
    a.window = window;
    a.workspace = workspace;
    a.err = err;
    cudaError_t e = cudaSuccess;
    if (step.slots != nullptr && q4_fuses_append(plan)) {
        a.k_new = step.k_new;
        a.v_new = step.v_new;
        a.new_dt = step.new_dt;
        a.new_slots = step.slots;
    } else if (step.slots != nullptr) {
        e = launch_kv_append_q4(step.k_new, step.v_new, step.new_dt, const_cast<uint8_t *>(k_cache),
                                const_cast<uint8_t *>(v_cache), step.slots, B, Hkv, d, group, bs, NB, sm_count, err,
                                stream);
        if (e != cudaSuccess) return cuda_fail(e, what);
    }
    e = launch_attend_q4(a, plan, stream);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, what);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_q4_row_bytes(int d, int group) { return q4_sizes(d, group) ? q4_row_bytes(d, group) : -1; }

pkv_status pkv_kv_append_q4(const void *k_new, const void *v_new, pkv_dtype new_dt, uint8_t *k_cache,
                            uint8_t *v_cache, const int64_t *slot_mapping, int T, int Hkv, int d, int group,
                            int bs, int NB, pkv_stream_t stream) {
    pkv_status s = check_rows("kv_append_q4", new_dt, T, Hkv, d, group, bs, NB);
    if (s != PKV_OK) return s;
    if (T == 0) return PKV_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !slot_mapping)
        return fail(PKV_ERR_INVALID_ARG, "kv_append_q4: null pointer");
    if (!aligned_to(k_cache, 4) || !aligned_to(v_cache, 4))
        return fail(PKV_ERR_INVALID_ARG, "kv_append_q4: the caches must be 4-byte aligned");
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    const cudaError_t e = launch_kv_append_q4(k_new, v_new, new_dt, k_cache, v_cache, slot_mapping, T, Hkv, d, group, bs,
                                              NB, sm_count, err, stream);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, "kv_append_q4 launch");
}

pkv_status pkv_kv_gather_q4(void *k_out, void *v_out, pkv_dtype out_dt, const uint8_t *k_cache,
                            const uint8_t *v_cache, const int64_t *slot_mapping, int T, int Hkv, int d, int group,
                            int bs, int NB, pkv_stream_t stream) {
    pkv_status s = check_rows("kv_gather_q4", out_dt, T, Hkv, d, group, bs, NB);
    if (s != PKV_OK) return s;
    if (T == 0) return PKV_OK;
    if (!k_out || !v_out || !k_cache || !v_cache || !slot_mapping)
        return fail(PKV_ERR_INVALID_ARG, "kv_gather_q4: null pointer");
    if (!aligned_to(k_cache, 4) || !aligned_to(v_cache, 4))
        return fail(PKV_ERR_INVALID_ARG, "kv_gather_q4: the caches must be 4-byte aligned");
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    const cudaError_t e = launch_kv_gather_q4(k_out, v_out, out_dt, k_cache, v_cache, slot_mapping, T, Hkv, d, group, bs,
                                              NB, sm_count, err, stream);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, "kv_gather_q4 launch");
}

size_t pkv_paged_attention_q4_workspace_bytes(int B, int Tq, int max_q, int Hq, int Hkv, int d, int group, int bs,
                                              int MBS, int window, int num_splits) {
    if (check_attend("paged_attention_q4", B, Tq, max_q, Hq, Hkv, d, group, bs, MBS, 1, window, num_splits) != PKV_OK)
        return 0;
    int sm_count = 0;
    unsigned *err = nullptr;
    if (current_device_info(&sm_count, &err) != PKV_OK || B == 0 || Tq == 0) return 0;
    return workspace_bound(B, Tq, max_q, Hq, Hkv, d, group, bs, MBS, window, num_splits, sm_count);
}

pkv_status pkv_paged_attention_q4(float *out, float *lse, const float *q, const uint8_t *k_cache,
                                  const uint8_t *v_cache, const int32_t *block_table, const int32_t *context_lens,
                                  const int32_t *cu_q, int B, int Tq, int max_q, int Hq, int Hkv, int d, int group,
                                  int bs, int MBS, int NB, float scale, int window, int num_splits, void *workspace,
                                  size_t workspace_bytes, pkv_stream_t stream) {
    const pkv_status s =
        check_attend("paged_attention_q4", B, Tq, max_q, Hq, Hkv, d, group, bs, MBS, NB, window, num_splits);
    if (s != PKV_OK) return s;
    if (B == 0 || Tq == 0) return PKV_OK;
    const bool one_per_seq = Tq == B && max_q == 1;
    if (!out || !q || !k_cache || !v_cache || !block_table || !context_lens || (!one_per_seq && !cu_q))
        return fail(PKV_ERR_INVALID_ARG, "paged_attention_q4: null pointer");
    return attend("paged_attention_q4", out, lse, q, StepRows{}, k_cache, v_cache, block_table, context_lens,
                  one_per_seq ? nullptr : cu_q, B, Tq, max_q, Hq, Hkv, d, group, bs, MBS, NB, scale, window, num_splits,
                  workspace, workspace_bytes, stream);
}

pkv_status pkv_decode_step_q4(float *out, float *lse, const float *q, const void *k_new, const void *v_new,
                              pkv_dtype new_dt, const int64_t *slot_mapping, uint8_t *k_cache, uint8_t *v_cache,
                              const int32_t *block_table, const int32_t *context_lens, int B, int Hq, int Hkv, int d,
                              int group, int bs, int MBS, int NB, float scale, int window, int num_splits,
                              void *workspace, size_t workspace_bytes, pkv_stream_t stream) {
    if (!new_dtype(new_dt)) return fail(PKV_ERR_UNSUPPORTED, "decode_step_q4: input type %d", new_dt);
    const pkv_status s = check_attend("decode_step_q4", B, B, 1, Hq, Hkv, d, group, bs, MBS, NB, window, num_splits);
    if (s != PKV_OK) return s;
    if (B == 0) return PKV_OK;
    if (!out || !q || !k_new || !v_new || !slot_mapping || !k_cache || !v_cache || !block_table || !context_lens)
        return fail(PKV_ERR_INVALID_ARG, "decode_step_q4: null pointer");
    StepRows step;
    step.k_new = k_new;
    step.v_new = v_new;
    step.new_dt = new_dt;
    step.slots = slot_mapping;
    return attend("decode_step_q4", out, lse, q, step, k_cache, v_cache, block_table, context_lens, nullptr, B, B, 1, Hq,
                  Hkv, d, group, bs, MBS, NB, scale, window, num_splits, workspace, workspace_bytes, stream);
}

static pkv_status check_tables(const char *what, int B, int T, int MBS, int bs, int NB) {
    if (B < 0 || T < 0 || MBS < 1 || bs < 1 || NB < 1 || static_cast<long long>(MBS) * bs > 0x7fffffffll - bs)
        return fail(PKV_ERR_INVALID_ARG, "%s: B=%d T=%d MBS=%d bs=%d NB=%d", what, B, T, MBS, bs, NB);
    return PKV_OK;
}

size_t pkv_block_tables_extend_workspace_bytes(int B, int T) {
    int sm_count = 0;
    unsigned *err = nullptr;
    if (B < 0 || T < 0 || current_device_info(&sm_count, &err) != PKV_OK) return 0;
    return extend_blocks(T, sm_count) > 1 ? 16 : 0;
}

static pkv_status extend_tables(const char *what, ExtendArgs a, void *workspace, size_t workspace_bytes, pkv_stream_t stream) {
    pkv_status s = check_tables(what, a.B, a.T, a.MBS, a.bs, a.NB);
    if (s != PKV_OK) return s;
    if (!a.free_list || !a.free_count || !a.free_count_out || !a.cu_new ||
        (a.B > 0 && (!a.block_table || !a.context_lens || !a.new_tokens || !a.context_lens_out)) || (a.T > 0 && !a.slot_mapping))
        return fail(PKV_ERR_INVALID_ARG, "%s: null pointer", what);
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    if (extend_blocks(a.T, sm_count) > 1 && (workspace == nullptr || workspace_bytes < 16 || !aligned_to(workspace, 16)))
        return fail(PKV_ERR_WORKSPACE, "%s: needs 16 bytes of 16-byte aligned workspace, got %zu", what,
                    workspace == nullptr ? size_t(0) : workspace_bytes);
    a.arrivals = static_cast<unsigned *>(workspace);
    a.err = err;
    const cudaError_t e = launch_block_tables_extend(a, sm_count, stream);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, what);
}

pkv_status pkv_block_tables_extend(int32_t *block_table, const int32_t *context_lens, const int32_t *new_tokens,
                                   const int32_t *free_list, const int32_t *free_count, int32_t *context_lens_out,
                                   int32_t *cu_new, int64_t *slot_mapping, int32_t *free_count_out, int B, int T,
                                   int MBS, int bs, int NB, void *workspace, size_t workspace_bytes,
                                   pkv_stream_t stream) {
    return extend_tables("block_tables_extend",
                         ExtendArgs{block_table, context_lens, new_tokens, free_list, free_count, context_lens_out, cu_new,
                                    slot_mapping, nullptr, free_count_out, B, T, MBS, bs, NB, nullptr, nullptr},
                         workspace, workspace_bytes, stream);
}

pkv_status pkv_block_tables_extend_step(int32_t *block_table, const int32_t *context_lens, const int32_t *new_tokens,
                                        const int32_t *free_list, const int32_t *free_count, int32_t *context_lens_out,
                                        int32_t *cu_new, int64_t *slot_mapping, int64_t *step_slots,
                                        int32_t *free_count_out, int B, int T, int MBS, int bs, int NB, void *workspace,
                                        size_t workspace_bytes, pkv_stream_t stream) {
    if (B > 0 && !step_slots) return fail(PKV_ERR_INVALID_ARG, "block_tables_extend_step: null pointer");
    return extend_tables("block_tables_extend_step",
                         ExtendArgs{block_table, context_lens, new_tokens, free_list, free_count, context_lens_out, cu_new,
                                    slot_mapping, step_slots, free_count_out, B, T, MBS, bs, NB, nullptr, nullptr},
                         workspace, workspace_bytes, stream);
}

size_t pkv_block_tables_release_workspace_bytes(int B) { return B < 0 ? 0 : (static_cast<size_t>(B) + 1) * sizeof(int32_t); }

pkv_status pkv_block_tables_release(int32_t *block_table, const int32_t *first_block, const int32_t *end_block,
                                    int32_t *free_list, const int32_t *free_count, int32_t *free_count_out, int B,
                                    int MBS, int NB, void *workspace, size_t workspace_bytes, pkv_stream_t stream) {
    pkv_status s = check_tables("block_tables_release", B, 0, MBS, 1, NB);
    if (s != PKV_OK) return s;
    if (!free_list || !free_count || !free_count_out || (B > 0 && (!block_table || !end_block)))
        return fail(PKV_ERR_INVALID_ARG, "block_tables_release: null pointer");
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    if (!release_in_one_block(B, MBS) &&
        (workspace == nullptr || workspace_bytes < pkv_block_tables_release_workspace_bytes(B) || !aligned_to(workspace, 4)))
        return fail(PKV_ERR_WORKSPACE, "block_tables_release: needs %zu bytes of 4-byte aligned workspace, got %zu",
                    pkv_block_tables_release_workspace_bytes(B), workspace == nullptr ? size_t(0) : workspace_bytes);
    const ReleaseArgs a{block_table, first_block, end_block, free_list, free_count, free_count_out, B, MBS, NB,
                        static_cast<int32_t *>(workspace), err};
    const cudaError_t e = launch_block_tables_release(a, sm_count, stream);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, "block_tables_release launch");
}

}  // extern "C"
