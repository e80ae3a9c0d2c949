"""pkv_paged_attention_sinks on the GPU against the 64-bit definition: every path, windows and first tokens that
meet, miss and share a block, several rows, NaN in keys that nobody sees, blocks given back between the two."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_165_gb300 as pkv
from oracle import serve
from paged_kv_cache_165_gb300 import _build
from workloads import gen

from helpers import assert_attn_close, assert_bits_equal, dev

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    pkv.lib()
    pkv.get_device_error()


def make_case(seed, lens, nqs, hq, hkv, d, bs, dtype, window, sinks):
    """Caches in which everything that no row of a sequence sees is NaN, and blocks that hold nothing else gone (-1)."""
    g = gen.generator(seed)
    per = [gen.blocks_needed(n, bs) for n in lens]
    nb = sum(per) + 3
    table = gen.block_table_from_order(gen.permutation(g, nb), per)
    kc, vc = (gen.randn(g, (nb, hkv, bs, d), dtype) for _ in range(2))
    q = gen.randn(g, (sum(nqs), hq, d), F32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(nqs)]), dtype=torch.int32)
    seen_slots = torch.zeros(nb * bs, dtype=torch.bool)
    for b, (L, nq) in enumerate(zip(lens, nqs)):
        for t in range(L):
            if nq and (window == 0 or t < sinks or t > L - nq - window):
                seen_slots[int(table[b, t // bs]) * bs + t % bs] = True
    seen = seen_slots.view(nb, bs)
    kp, vp = (torch.where(seen[:, None, :, None], x, torch.full_like(x, float("nan"))) for x in (kc, vc))
    tp = table.clone()
    for b, L in enumerate(lens):
        for j in range(per[b]):
            if not seen[int(table[b, j])].any():
                tp[b, j] = -1
    return q, kc, vc, kp, vp, table, tp, torch.tensor(lens, dtype=torch.int32), cu


def run(q, kc, vc, table, lens, cu, window, sinks, splits=0, scale=None, max_q=None, bare=False):
    Tq, Hq, d = q.shape
    NB, Hkv, bs, _ = kc.shape
    B = lens.numel()
    one = bool(((cu[1:] - cu[:-1]) == 1).all())
    max_q = int((cu[1:] - cu[:-1]).max()) if max_q is None else max_q
    out, lse = torch.full((Tq, Hq, d), float("nan"), device="cuda"), torch.full((Tq, Hq), float("nan"), device="cuda")
    n = pkv.paged_attention_sinks_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, bs, table.shape[1], window, sinks, splits)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    pkv.paged_attention_sinks(out, dev(q), dev(kc), dev(vc), dev(table), dev(lens), scale or 1 / math.sqrt(d), window, sinks,
                              cu_q=None if one else dev(cu), max_q=max_q, lse=lse, num_splits=splits, workspace=ws)
    torch.cuda.synchronize()
    assert not ws[:1024].any() or ws.numel() <= 16        # the counters are zero again
    return out, lse


PATHS = [
    (8, 8, 128, BF16, 16),      # one head a KV head
    (16, 2, 128, BF16, 32),     # eight heads a KV head
    (12, 4, 64, BF16, 16),
    (64, 1, 128, BF16, 16),     # many heads a KV head
    (32, 2, 64, BF16, 32),
    (32, 2, 256, BF16, 16),
    (4, 2, 256, BF16, 32),
    (8, 2, 96, BF16, 24),       # CUDA cores
    (8, 2, 64, F32, 16),
    (80, 1, 64, BF16, 16),      # more than 64 heads a KV head
]
# Three bf16 parts hold an fp32 number, so what is left are sums: the tensor core adds 16 products at a time, d / 16 times
# a score, each addition off by at most 2^-23 of sum |q k| scale (some 0.64 sqrt(d), below 15 for d = 128 and 20 for
# 256), the lower parts adding 2^-8 of that: 1.5e-5 a score, 4e-5 for d = 256.  An output is off by at most that, and
# 2^-22 for the weight itself, times the spread of V (below 6): 1e-4, and 3e-4.  CUDA cores, fp32 sums of at most 256 terms and
# 700 keys: 2e-5 for fp32 caches, and no more for bf16 ones.
def atol(dtype, d):
    return 2e-5 if dtype is F32 else 1e-4 if d <= 128 else 3e-4


@pytest.mark.parametrize("hq,hkv,d,dtype,bs", PATHS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 4), (16, 16), (33, 3), (100, 17), (64, 70), (1000, 4)])
def test_one_row_on_every_path(hq, hkv, d, dtype, bs, window, sinks):
    lens = [1, 15, 16, 17, 100, 257, 700, 33, 2]
    q, kc, vc, kp, vp, table, tp, clens, cu = make_case(hq + d + window, lens, [1] * len(lens), hq, hkv, d, bs, dtype, window, sinks)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / math.sqrt(d), window, sinks)
    tol = atol(dtype, d)
    for splits in (1, 3, 0):
        out, lse = run(q, kp, vp, tp, clens, cu, window, sinks, splits)
        assert pkv.get_device_error() == 0
        assert_attn_close(out, ref, f"splits {splits} out", tol)
        assert_attn_close(lse, ref_lse, f"splits {splits} lse", tol)


@pytest.mark.parametrize("hq,hkv,d,dtype,bs", PATHS)
@pytest.mark.parametrize("window,sinks", [(1, 1), (7, 4), (40, 20), (64, 3)])
def test_several_rows(hq, hkv, d, dtype, bs, window, sinks):
    lens = [50, 300, 17, 9, 400, 64, 1]
    nqs = [4, 1, 0, 9, 33, 5, 1]
    q, kc, vc, kp, vp, table, tp, clens, cu = make_case(hq * 3 + window, lens, nqs, hq, hkv, d, bs, dtype, window, sinks)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / math.sqrt(d), window, sinks)
    tol = atol(dtype, d)
    for splits in (1, 2, 0):
        out, lse = run(q, kp, vp, tp, clens, cu, window, sinks, splits)
        assert pkv.get_device_error() == 0
        assert_attn_close(out, ref, f"splits {splits} out", tol)
        assert_attn_close(lse, ref_lse, f"splits {splits} lse", tol)


@pytest.mark.parametrize("hq,hkv,d,dtype,bs", [
    (5, 1, 33, F32, 8), (3, 3, 7, BF16, 3), (6, 2, 100, F32, 16), (10, 2, 160, BF16, 16), (4, 2, 250, F32, 24), (9, 3, 130, F32, 16),
    (14, 2, 128, F32, 32), (2, 1, 1, F32, 1), (4, 4, 256, F32, 16), (7, 1, 64, BF16, 16)])
@pytest.mark.parametrize("window,sinks", [(3, 2), (150, 20)])
@pytest.mark.parametrize("unaligned", [False, True])
def test_sizes_on_cuda_cores(hq, hkv, d, dtype, bs, window, sinks, unaligned):
    # heads of every width, blocks of one head to four, and caches that start at an odd element
    lens, nqs = [700, 1, 90, 300, 64], [2, 1, 5, 0, 1]
    q, kc, vc, kp, vp, table, tp, clens, cu = make_case(d + window, lens, nqs, hq, hkv, d, bs, dtype, window, sinks)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / math.sqrt(d), window, sinks)
    if unaligned:
        kp, vp = (torch.cat([torch.zeros(1, dtype=dtype), x.flatten()]).cuda()[1:].view(x.shape) for x in (kp, vp))
    for splits in (0, 1, 2, 5, 11):
        out, lse = run(q, kp, vp, tp, clens, cu, window, sinks, splits)
        assert pkv.get_device_error() == 0
        assert_attn_close(out, ref, f"splits {splits} out", atol(dtype, d))
        assert_attn_close(lse, ref_lse, f"splits {splits} lse", atol(dtype, d))


def test_many_rows_and_a_long_sequence():
    # a chunk of new tokens on a cached prefix, and contexts many times the window
    lens, nqs = [900, 130, 3000], [70, 130, 2]
    q, kc, vc, kp, vp, table, tp, clens, cu = make_case(1, lens, nqs, 8, 2, 128, 16, BF16, 200, 10)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / math.sqrt(128), 200, 10)
    out, lse = run(q, kp, vp, tp, clens, cu, 200, 10)
    assert pkv.get_device_error() == 0
    assert_attn_close(out, ref, "out")
    assert_attn_close(lse, ref_lse, "lse")


@pytest.mark.parametrize("window,sinks", [(0, 4), (50, 0)])
@pytest.mark.parametrize("nq", [1, 3])
def test_what_needs_no_sinks_is_the_plain_attention(window, sinks, nq):
    lens = [600, 17, 320]
    q, kc, vc, _, _, table, _, clens, cu = make_case(5, lens, [nq] * 3, 16, 2, 128, 16, BF16, 0, 0)
    out, lse = run(q, kc, vc, table, clens, cu, window, sinks)
    plain = window if sinks == 0 else 0
    want, want_lse = torch.empty_like(out), torch.empty_like(lse)
    n = pkv.paged_attention_workspace_bytes(3, 3 * nq, nq, 16, 2, 128, 16, table.shape[1], plain)
    pkv.paged_attention(want, dev(q), dev(kc), dev(vc), dev(table), dev(clens), 1 / math.sqrt(128), cu_q=dev(cu) if nq > 1 else None,
                        max_q=nq, window=plain, lse=want_lse, workspace=torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda"))
    assert_bits_equal(out, want)
    assert_bits_equal(lse, want_lse)


@pytest.mark.parametrize("window,sinks", [(400, 300), (2 ** 31 - 1, 2 ** 31 - 1), (700, 5), (1, 2 ** 31 - 1)])
@pytest.mark.parametrize("nq,hq,dtype", [(1, 16, BF16), (3, 16, BF16), (70, 8, BF16), (3, 16, F32)])
def test_windows_that_cover_the_tables(window, sinks, nq, hq, dtype):
    lens = [600, 70, 320]
    q, kc, vc, _, _, table, _, clens, cu = make_case(5, lens, [nq] * 3, hq, 2, 128, 16, dtype, 0, 0)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / math.sqrt(128), 0, 0)
    out, lse = run(q, kc, vc, table, clens, cu, window, sinks)
    assert pkv.get_device_error() == 0
    assert_attn_close(out, ref, "out", atol(dtype, 128))
    assert_attn_close(lse, ref_lse, "lse", atol(dtype, 128))


def test_empty_sequences_and_bad_lengths_and_blocks():
    lens = [100, 0, 60]
    q, kc, vc, _, _, table, _, clens, cu = make_case(8, [100, 16, 60], [1, 1, 1], 8, 2, 64, 16, BF16, 20, 4)
    out, lse = run(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32), cu, 20, 4)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all() and torch.isfinite(out[[0, 2]]).all()
    assert pkv.get_device_error() == 0
    out, lse = run(q, kc, vc, table, torch.tensor([100, -3, 10000], dtype=torch.int32), cu, 20, 4)
    assert (out[1:] == 0).all() and (lse[1:] == -math.inf).all()
    assert pkv.get_device_error() == pkv.DEVERR["len"]
    bad = table.clone()
    bad[0, 0], bad[2, 3] = 10 ** 6, -5
    out, _ = run(q, kc, vc, bad, clens, cu, 20, 4)
    assert pkv.get_device_error() == pkv.DEVERR["block"] and torch.isfinite(out).all()


@pytest.mark.parametrize("dtype,hq", [(BF16, 16), (F32, 16)])
def test_rows_that_a_sequence_may_not_own(dtype, hq):
    lens, nqs = [40, 90, 30], [3, 2, 4]
    q, kc, vc, _, _, table, _, clens, cu = make_case(8, lens, nqs, hq, 2, 64, 16, dtype, 20, 4)
    ref, _ = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / 8, 20, 4)
    out, lse = run(q, kc, vc, table, clens, cu, 20, 4, max_q=3)      # the last sequence's four rows are one too many
    assert pkv.get_device_error() == pkv.DEVERR["cu_seqlens"]
    assert_attn_close(out[:5], ref[:5], "served rows")
    assert (out[5:] == 0).all() and (lse[5:] == -math.inf).all()


@pytest.mark.parametrize("window", [300, 1000, 2 ** 31 - 1])      # the last two cover the tables
@pytest.mark.parametrize("dtype,hq,splits", [(BF16, 16, 1), (BF16, 4, 0), (F32, 4, 1), (F32, 4, 3), (BF16, 4, 12), (BF16, 130, 0)])
def test_rows_behind_the_last_sequence_stay_as_they_are(dtype, hq, splits, window):
    lens, nqs = [40, 900, 30], [3, 2, 4]
    q, kc, vc, _, _, table, _, clens, cu = make_case(8, lens, nqs, hq, 2, 64, 16, dtype, window, 4)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / 8, window, 4)
    tol = atol(dtype, 64)
    padded = torch.cat([q, torch.full((3, hq, 64), float("nan"))])
    n = pkv.paged_attention_sinks_workspace_bytes(3, 12, 4, hq, 2, 64, 16, table.shape[1], window, 4, splits)
    out, lse = torch.full((12, hq, 64), 7.0, device="cuda"), torch.full((12, hq), 7.0, device="cuda")
    pkv.paged_attention_sinks(out, dev(padded), dev(kc), dev(vc), dev(table), dev(clens), 1 / 8, window, 4, cu_q=dev(cu), max_q=4, lse=lse,
                              num_splits=splits, workspace=torch.zeros(max(16, n), dtype=torch.uint8, device="cuda"))
    assert pkv.get_device_error() == 0
    assert_attn_close(out[:9], ref, "rows", tol)
    assert_attn_close(lse[:9], ref_lse, "lse", tol)
    assert (out[9:] == 7).all() and (lse[9:] == 7).all()


@pytest.mark.parametrize("window", [5, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype,hq", [(BF16, 4), (BF16, 32), (F32, 4)])
@pytest.mark.parametrize("splits", [0, 3])
def test_a_padded_batch_of_as_many_rows_as_sequences(dtype, hq, splits, window):
    # four sequences, two of them idle, and four rows: two to serve and two of padding
    lens, nqs = [40, 90, 300, 30], [1, 0, 1, 0]
    q, kc, vc, _, _, table, _, clens, cu = make_case(9, lens, nqs, hq, 2, 64, 16, dtype, window, 4)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / 8, window, 4)
    tol = atol(dtype, 64)
    padded = torch.cat([q, torch.full((2, hq, 64), float("nan"))])
    n = pkv.paged_attention_sinks_workspace_bytes(4, 4, 1, hq, 2, 64, 16, table.shape[1], window, 4, splits)
    out, lse = torch.full((4, hq, 64), 7.0, device="cuda"), torch.full((4, hq), 7.0, device="cuda")
    pkv.paged_attention_sinks(out, dev(padded), dev(kc), dev(vc), dev(table), dev(clens), 1 / 8, window, 4, cu_q=dev(cu), max_q=1, lse=lse,
                              num_splits=splits, workspace=torch.zeros(max(16, n), dtype=torch.uint8, device="cuda"))
    assert pkv.get_device_error() == 0
    assert_attn_close(out[:2], ref, "rows", tol)
    assert_attn_close(lse[:2], ref_lse, "lse", tol)
    assert (out[2:] == 7).all() and (lse[2:] == 7).all()


def test_streams_and_a_graph_over_growing_lengths():
    lens = [70, 200]
    q, kc, vc, _, _, table, _, clens, cu = make_case(8, lens, [1, 1], 16, 2, 128, 16, BF16, 32, 5)
    qd, kd, vd, td, ld = dev(q), dev(kc), dev(vc), dev(table), dev(clens) - 20
    out, lse = torch.empty_like(qd), torch.empty(2, 16, device="cuda")
    n = pkv.paged_attention_sinks_workspace_bytes(2, 2, 1, 16, 2, 128, 16, table.shape[1], 32, 5)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    step = lambda **kw: pkv.paged_attention_sinks(out, qd, kd, vd, td, ld, 0.1, 32, 5, lse=lse, workspace=ws, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in range(20):
        ld += 1
        g.replay()
        torch.cuda.synchronize()
        ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, ld.cpu(), cu, 0.1, 32, 5)
        assert_attn_close(out, ref, f"step {n}")
        assert_attn_close(lse, ref_lse, f"step {n}")


def test_two_calls_at_once():
    # one path each, chunks merged by their last block, on two streams with a workspace each
    cases = []
    for hq, dtype, nqs, splits in ((16, BF16, [1, 1], 4), (64, BF16, [3, 2], 3), (4, F32, [1, 2], 5)):
        q, kc, vc, _, _, table, _, clens, cu = make_case(hq, [700, 900], nqs, hq, 2, 128, 16, dtype, 300, 20)
        ref, _ = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 0.1, 300, 20)
        Tq, mq = sum(nqs), max(nqs)
        n = pkv.paged_attention_sinks_workspace_bytes(2, Tq, mq, hq, 2, 128, 16, table.shape[1], 300, 20, splits)
        t = [dev(x) for x in (q, kc, vc, table, clens, cu)]
        for _ in range(2):
            cases.append((t, mq, splits, torch.zeros(max(16, n), dtype=torch.uint8, device="cuda"), torch.empty_like(t[0]), ref, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(30):
        for (q, kc, vc, table, clens, cu), mq, splits, ws, out, _, s in cases:
            pkv.paged_attention_sinks(out, q, kc, vc, table, clens, 0.1, 300, 20, cu_q=cu, max_q=mq, num_splits=splits, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for t, _, _, _, out, ref, _ in cases:
        assert_attn_close(out, ref, "out", 1e-4)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("dtype,d,bs", [(F32, 64, 16), (BF16, 128, 16), (BF16, 256, 32), (BF16, 96, 24)])
@pytest.mark.parametrize("B", [0, 3])
def test_batches_without_rows(B, dtype, d, bs):
    for max_q in (0, 1, 4):
        assert pkv.paged_attention_sinks_workspace_bytes(B, 0, max_q, 8, 2, d, bs, 64, 100, 4) == 0
    t = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
    cache = t(5, 2, bs, d, dt=dtype)
    pkv.paged_attention_sinks(t(0, 8, d, dt=F32), t(0, 8, d, dt=F32), cache, cache, t(B, 64), t(B), 1.0, 100, 4, cu_q=t(B + 1), max_q=4)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype,bs", [(4, 2, 64, F32, 16), (4, 1, 128, F32, 16), (2, 2, 256, F32, 16), (6, 2, 33, BF16, 8)])
def test_the_last_batch_of_tokens_of_every_size(hq, hkv, d, dtype, bs):
    # 1 to 40 visible tokens: a warp's last batch of four or eight holds every number of them, none included
    lens = list(range(1, 41))
    q, kc, vc, kp, vp, table, tp, clens, cu = make_case(d, lens, [1] * 40, hq, hkv, d, bs, dtype, 29, 11)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / math.sqrt(d), 29, 11)
    for splits in (1, 2):
        out, lse = run(q, kp, vp, tp, clens, cu, 29, 11, splits)
        assert pkv.get_device_error() == 0
        assert_attn_close(out, ref, f"splits {splits} out", atol(dtype, d))
        assert_attn_close(lse, ref_lse, f"splits {splits} lse", atol(dtype, d))


@pytest.mark.parametrize("nq", [1, 2])
def test_sequences_that_fill_the_sms_once_are_not_split(nq):
    # heads of 256 in pages of 32: one block an SM fits, so a second chunk would only be a second wave
    B, nb, width = torch.cuda.get_device_properties(0).multi_processor_count, 70, 64
    g = gen.generator(3)
    kc, vc = (gen.randn(g, (nb, 1, 32, 256), BF16) for _ in range(2))
    q = gen.randn(g, (B * nq, 8, 256), F32)
    table = torch.randint(0, nb, (B, width), generator=g, dtype=torch.int32)
    lens = torch.full((B,), width * 32, dtype=torch.int32)
    cu = torch.arange(0, B * nq + 1, nq, dtype=torch.int32)
    ref, _ = serve.paged_attention_sinks(q[:nq], kc, vc, table[:1], lens[:1], cu[:2], 1 / 16, 2000, 8)
    out = torch.empty(B * nq, 8, 256, device="cuda")
    pkv.paged_attention_sinks(out, dev(q), dev(kc), dev(vc), dev(table), dev(lens), 1 / 16, 2000, 8, cu_q=dev(cu), max_q=nq)   # no workspace
    assert pkv.get_device_error() == 0
    assert_attn_close(out[:nq], ref, "out", atol(BF16, 256))


@pytest.mark.parametrize("hq,hkv,d,dtype,bs", PATHS)
def test_any_bound_of_the_rows_of_a_sequence(hq, hkv, d, dtype, bs):
    # max_q says how many rows a sequence may have, not how many it has
    lens, nqs = [300, 17, 90], [3, 0, 2]
    q, kc, vc, kp, vp, table, tp, clens, cu = make_case(hq, lens, nqs, hq, hkv, d, bs, dtype, 40, 6)
    ref, ref_lse = serve.paged_attention_sinks(q, kc, vc, table, clens, cu, 1 / math.sqrt(d), 40, 6)
    for max_q in (3, 5, 1000, 10 ** 6, 2 ** 31 - 1):
        for splits in (0, 1, 3):
            out, lse = run(q, kp, vp, tp, clens, cu, 40, 6, splits, max_q=max_q)
            assert pkv.get_device_error() == 0
            assert_attn_close(out, ref, f"max_q {max_q} out", atol(dtype, d))
            assert_attn_close(lse, ref_lse, f"max_q {max_q} lse", atol(dtype, d))
