// api_serve.cu -- the extern "C" entry points around the attention of a serving loop: rotary positions,
// drafted tokens, and block tables with shared blocks.  Host-side checks as in api.cu, then the launches.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "common.cuh"
#include "internal.h"

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

pkv_status done(cudaError_t e, const char *what) {
    return e == cudaSuccess ? PKV_OK : fail(PKV_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

bool aligned_to(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool value_type(pkv_dtype dt) { return dt == PKV_F32 || dt == PKV_BF16; }

unsigned value_bytes(pkv_dtype dt) { return dt == PKV_F32 ? 4 : 2; }

bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a != nullptr && b != nullptr && x < y + b_bytes && y < x + a_bytes;
}

// Bytes from the first to the last element of T rows of `row` elements, `stride` apart.
size_t span_bytes(int T, long long stride, long long row, unsigned elem) {
    return (static_cast<size_t>(T - 1) * static_cast<size_t>(stride) + static_cast<size_t>(row)) * elem;
}

pkv_status check_rope(const char *what, pkv_dtype dt, pkv_dtype q_out_dt, int rot, float mscale, int T, int Hq, int Hkv,
                      int d, long long q_stride, long long k_stride, long long v_stride, bool has_k) {
    if (!value_type(dt) || !value_type(q_out_dt))
        return fail(PKV_ERR_UNSUPPORTED, "%s: element types %d and %d", what, dt, q_out_dt);
    if (T < 0 || Hq < 1 || Hq > 65535 || Hkv < 1 || Hkv > 65535 || d < 1 || d > 256 || rot < 2 || rot % 2 != 0 || rot > d)
        return fail(PKV_ERR_INVALID_ARG, "%s: T=%d Hq=%d Hkv=%d d=%d rot=%d (need d <= 256, rot even, 2 <= rot <= d)", what, T,
                    Hq, Hkv, d, rot);
    const long long most = 1ll << 40;   // elements from a token to the next
    if (q_stride < static_cast<long long>(Hq) * d || q_stride > most ||
        (has_k && (k_stride < static_cast<long long>(Hkv) * d || k_stride > most || v_stride < static_cast<long long>(Hkv) * d ||
                   v_stride > most)))
        return fail(PKV_ERR_INVALID_ARG, "%s: strides %lld %lld %lld of tokens with %d and %d heads of %d", what, q_stride, k_stride,
                    v_stride, Hq, Hkv, d);
    if (!std::isfinite(mscale)) return fail(PKV_ERR_INVALID_ARG, "%s: mscale is not finite", what);
    return PKV_OK;
}

// out may be `in` where both have one type and layout, and share no bytes with it otherwise.
pkv_status check_in_place(const char *what, const char *name, const void *out, unsigned out_elem, const void *in, unsigned elem,
                          long long stride, int T, long long row) {
    if (out == in && out_elem == elem && stride == row) return PKV_OK;
    if (overlap(out, span_bytes(T, row, row, out_elem), in, span_bytes(T, stride, row, elem)))
        return fail(PKV_ERR_INVALID_ARG, "%s: %s overlaps its input (it may be the input where type and layout are the same)", what,
                    name);
    return PKV_OK;
}

pkv_status check_share(const char *what, int B, int MBS, int bs, int NB, const void *table, const void *lens, const void *table_out,
                       const void *held, const void *refs, const void *free_list, const void *free_count, const void *pairs,
                       const void *pair_count, bool want_pairs, const void *workspace, size_t workspace_bytes) {
    if (B < 0 || B > 65536 || MBS < 1 || bs < 1 || NB < 1 || static_cast<long long>(MBS) * bs > 0x7fffffffll - bs)
        return fail(PKV_ERR_INVALID_ARG, "%s: B=%d MBS=%d bs=%d NB=%d (need B <= 65536)", what, B, MBS, bs, NB);
    if (!refs || !free_list || !free_count || !pair_count || (want_pairs && !pairs) || (B > 0 && (!table || !lens || !table_out)))
        return fail(PKV_ERR_INVALID_ARG, "%s: null pointer", what);
    if (want_pairs && !aligned_to(pairs, 8)) return fail(PKV_ERR_INVALID_ARG, "%s: pairs must be 8-byte aligned", what);
    const size_t ids = static_cast<size_t>(NB) * sizeof(int32_t);   // held is still read when the others are written
    if (overlap(held, ids, refs, ids) || overlap(held, ids, free_list, ids))
        return fail(PKV_ERR_INVALID_ARG, "%s: held overlaps refs or free_list", what);
    const size_t need = share_workspace_bytes(B, MBS, NB);
    if (workspace == nullptr || workspace_bytes < need || !aligned_to(workspace, 4))
        return fail(PKV_ERR_WORKSPACE, "%s: needs %zu bytes of 4-byte aligned workspace, got %zu", what, need,
                    workspace == nullptr ? size_t(0) : workspace_bytes);
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_rope_turns(uint64_t *turns, int rot, double base, pkv_rope_scaling scaling, double factor, double original,
                          double low, double high) {
    if (!turns) return fail(PKV_ERR_INVALID_ARG, "rope_turns: null pointer");
    if (scaling < PKV_ROPE_NONE || scaling > PKV_ROPE_PARTS) return fail(PKV_ERR_UNSUPPORTED, "rope_turns: scaling %d", scaling);
    if (rot < 2 || rot > 256 || rot % 2 != 0 || !(base > 0) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor) ||
        (scaling == PKV_ROPE_BASE && rot < 4) ||
        (scaling == PKV_ROPE_PARTS && (!(original > 0) || !std::isfinite(original) || !(low < high) || !std::isfinite(high - low))))
        return fail(PKV_ERR_INVALID_ARG, "rope_turns: rot=%d base=%g factor=%g original=%g low=%g high=%g", rot, base, factor,
                    original, low, high);
    if (!rope_turns(turns, rot, base, scaling, factor, original, low, high))
        return fail(PKV_ERR_INVALID_ARG, "rope_turns: base=%g factor=%g: an angle is not finite", base, factor);
    return PKV_OK;
}

pkv_status pkv_rope_append(void *q_out, pkv_dtype q_out_dt, const void *q, const void *k_new, const void *v_new, pkv_dtype dt,
                           long long q_stride, long long k_stride, long long v_stride, const int32_t *positions,
                           const uint64_t *turns, int rot, int interleaved, float mscale, void *k_cache, void *v_cache,
                           const int64_t *slot_mapping, int T, int Hq, int Hkv, int d, int bs, int NB, pkv_stream_t stream) {
    pkv_status s = check_rope("rope_append", dt, q_out_dt, rot, mscale, T, Hq, Hkv, d, q_stride, k_stride, v_stride, true);
    if (s != PKV_OK) return s;
    if (bs < 1 || NB < 1) return fail(PKV_ERR_INVALID_ARG, "rope_append: bs=%d NB=%d", bs, NB);
    if (T == 0) return PKV_OK;
    if (!q_out || !q || !k_new || !v_new || !positions || !turns || !k_cache || !v_cache || !slot_mapping)
        return fail(PKV_ERR_INVALID_ARG, "rope_append: null pointer");
    const unsigned e = value_bytes(dt);
    s = check_in_place("rope_append", "q_out", q_out, value_bytes(q_out_dt), q, e, q_stride, T, static_cast<long long>(Hq) * d);
    if (s != PKV_OK) return s;
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    RopeArgs a{};
    a.q_out = q_out;
    a.q = q;
    a.k = k_new;
    a.v = v_new;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.k_dst = k_cache;
    a.v_dst = v_cache;
    a.positions = positions;
    a.turns = reinterpret_cast<const unsigned long long *>(turns);
    a.slots = slot_mapping;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.rot = rot;
    a.bs = bs;
    a.n_slots = static_cast<long long>(NB) * bs;
    a.mscale = mscale;
    a.err = err;
    return done(launch_rope(a, dt, q_out_dt, interleaved != 0, sm_count, stream), "rope_append");
}

pkv_status pkv_rope(void *q_out, pkv_dtype q_out_dt, void *k_out, const void *q, const void *k, pkv_dtype dt, long long q_stride,
                    long long k_stride, const int32_t *positions, const uint64_t *turns, int rot, int interleaved, float mscale,
                    int inverse, int T, int Hq, int Hkv, int d, pkv_stream_t stream) {
    if ((k == nullptr) != (k_out == nullptr)) return fail(PKV_ERR_INVALID_ARG, "rope: k and k_out go together");
    pkv_status s = check_rope("rope", dt, q_out_dt, rot, mscale, T, Hq, Hkv, d, q_stride, k_stride, k_stride, k != nullptr);
    if (s != PKV_OK) return s;
    if (T == 0) return PKV_OK;
    if (!q_out || !q || !positions || !turns) return fail(PKV_ERR_INVALID_ARG, "rope: null pointer");
    const unsigned e = value_bytes(dt);
    s = check_in_place("rope", "q_out", q_out, value_bytes(q_out_dt), q, e, q_stride, T, static_cast<long long>(Hq) * d);
    if (s == PKV_OK && k != nullptr)
        s = check_in_place("rope", "k_out", k_out, e, k, e, k_stride, T, static_cast<long long>(Hkv) * d);
    if (s != PKV_OK) return s;
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    RopeArgs a{};
    a.q_out = q_out;
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k != nullptr ? k_stride : 0;
    a.k_dst = k_out;
    a.positions = positions;
    a.turns = reinterpret_cast<const unsigned long long *>(turns);
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.rot = rot;
    a.bs = 1;
    a.mscale = mscale;
    a.inverse = inverse != 0;
    a.err = err;
    return done(launch_rope(a, dt, q_out_dt, interleaved != 0, sm_count, stream), "rope");
}

pkv_status pkv_verify_drafts(int32_t *accepted, int32_t *tokens, const void *target_probs, const void *draft_probs, pkv_dtype dt,
                             long long target_stride, long long draft_stride, const int32_t *draft_tokens,
                             const int32_t *cu_drafts, const float *uniforms, const int32_t *context_lens,
                             int32_t *context_lens_out, int B, int D, int V, pkv_stream_t stream) {
    if (!value_type(dt)) return fail(PKV_ERR_UNSUPPORTED, "verify_drafts: element type %d", dt);
    const long long most = 1ll << 40;
    if (B < 0 || B > 65535 || D < 0 || D > 0x7fffffff - 65535 || V < 1 || V >= 1 << 30 || target_stride < V || target_stride > most ||
        (draft_probs != nullptr && (draft_stride < V || draft_stride > most)))
        return fail(PKV_ERR_INVALID_ARG, "verify_drafts: B=%d D=%d V=%d, rows %lld and %lld apart", B, D, V, target_stride,
                    draft_stride);
    if ((context_lens == nullptr) != (context_lens_out == nullptr))
        return fail(PKV_ERR_INVALID_ARG, "verify_drafts: context_lens and context_lens_out go together");
    if (B == 0) return PKV_OK;
    if (!accepted || !tokens || !target_probs || !cu_drafts || !uniforms || (D > 0 && !draft_tokens))
        return fail(PKV_ERR_INVALID_ARG, "verify_drafts: null pointer");
    if (overlap(tokens, (static_cast<size_t>(D) + B) * 4, draft_tokens, static_cast<size_t>(D) * 4))
        return fail(PKV_ERR_INVALID_ARG, "verify_drafts: tokens overlaps draft_tokens");
    const size_t row_bytes = static_cast<size_t>(B) * 4;
    if (context_lens != context_lens_out && overlap(context_lens, row_bytes, context_lens_out, row_bytes))
        return fail(PKV_ERR_INVALID_ARG, "verify_drafts: context_lens_out overlaps context_lens");
    int sm_count = 0;
    unsigned *err = nullptr;
    const pkv_status s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    const VerifyArgs a{accepted, tokens, target_probs, draft_probs, target_stride, draft_stride, draft_tokens, cu_drafts, uniforms,
                       context_lens, context_lens_out, B, D, V, err};
    return done(launch_verify(a, dt, sm_count, stream), "verify_drafts");
}

size_t pkv_block_tables_share_workspace_bytes(int B, int MBS, int NB) {
    return B < 0 || MBS < 1 || NB < 1 ? 0 : share_workspace_bytes(B, MBS, NB);
}

pkv_status pkv_block_tables_fork(const int32_t *block_table, const int32_t *context_lens, const int32_t *parents,
                                 const int32_t *held, int32_t *block_table_out, int32_t *context_lens_out, int32_t *refs,
                                 int32_t *free_list, int32_t *free_count, int32_t *pairs, int32_t *pair_count, int B, int MBS,
                                 int bs, int NB, void *workspace, size_t workspace_bytes, pkv_stream_t stream) {
    pkv_status s = check_share("block_tables_fork", B, MBS, bs, NB, block_table, context_lens, block_table_out, held, refs,
                               free_list, free_count, pairs, pair_count, B > 0, workspace, workspace_bytes);
    if (s != PKV_OK) return s;
    if (B > 0 && !context_lens_out) return fail(PKV_ERR_INVALID_ARG, "block_tables_fork: null pointer");
    const size_t bytes = static_cast<size_t>(B) * MBS * sizeof(int32_t);
    const bool same = block_table == block_table_out, over = overlap(block_table, bytes, block_table_out, bytes);
    if (over && !same) return fail(PKV_ERR_INVALID_ARG, "block_tables_fork: block_table_out overlaps block_table");
    if (context_lens != context_lens_out && overlap(context_lens, B * sizeof(int32_t), context_lens_out, B * sizeof(int32_t)))
        return fail(PKV_ERR_INVALID_ARG, "block_tables_fork: context_lens_out overlaps context_lens");
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    ShareArgs a{block_table, context_lens, parents, held, block_table_out, context_lens_out, refs, free_list, free_count,
                pair_count, pairs, B, MBS, bs, NB, nullptr, nullptr, nullptr, nullptr, nullptr, err};
    return done(launch_fork(a, workspace, same && parents != nullptr, stream), "block_tables_fork");
}

pkv_status pkv_block_tables_compact(const int32_t *block_table, const int32_t *context_lens, const int32_t *held,
                                    int32_t *block_table_out, int32_t *refs, int32_t *free_list, int32_t *free_count,
                                    int32_t *pairs, int32_t *pair_count, int B, int MBS, int bs, int NB, void *workspace,
                                    size_t workspace_bytes, pkv_stream_t stream) {
    pkv_status s = check_share("block_tables_compact", B, MBS, bs, NB, block_table, context_lens, block_table_out, held, refs,
                               free_list, free_count, pairs, pair_count, NB > 1, workspace, workspace_bytes);
    if (s != PKV_OK) return s;
    const size_t bytes = static_cast<size_t>(B) * MBS * sizeof(int32_t);
    if (block_table != block_table_out && overlap(block_table, bytes, block_table_out, bytes))
        return fail(PKV_ERR_INVALID_ARG, "block_tables_compact: block_table_out overlaps block_table");
    int sm_count = 0;
    unsigned *err = nullptr;
    s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    ShareArgs a{block_table, context_lens, nullptr, held, block_table_out, nullptr, refs, free_list, free_count,
                pair_count, pairs, B, MBS, bs, NB, nullptr, nullptr, nullptr, nullptr, nullptr, err};
    return done(launch_compact(a, workspace, stream), "block_tables_compact");
}

pkv_status pkv_kv_block_copy_counted(void *k_cache, void *v_cache, pkv_dtype dt, const int32_t *pairs, int n, const int32_t *count,
                                     int Hkv, int d, int bs, int NB, pkv_stream_t stream) {
    if (!value_type(dt) && dt != PKV_FP8_E4M3) return fail(PKV_ERR_UNSUPPORTED, "kv_block_copy_counted: element type %d", dt);
    if (n < 0 || Hkv < 1 || d < 1 || bs < 1 || NB < 1)
        return fail(PKV_ERR_INVALID_ARG, "kv_block_copy_counted: n=%d Hkv=%d d=%d bs=%d NB=%d", n, Hkv, d, bs, NB);
    if (n == 0) return PKV_OK;
    if (!k_cache || !v_cache || !pairs || !count) return fail(PKV_ERR_INVALID_ARG, "kv_block_copy_counted: null pointer");
    int sm_count = 0;
    unsigned *err = nullptr;
    const pkv_status s = current_device_info(&sm_count, &err);
    if (s != PKV_OK) return s;
    return done(launch_kv_block_copy_counted(k_cache, v_cache, dt == PKV_FP8_E4M3 ? 1 : value_bytes(dt) , pairs, n, count, Hkv, d,
                                             bs, NB, sm_count, err, stream),
                "kv_block_copy_counted");
}

}  // extern "C"
