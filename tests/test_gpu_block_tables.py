"""Block tables built on the GPU against the oracle's row-by-row form, and the 4-bit decode loop
over them: tables, slots, appends, attention and blocks given back, captured into a graph."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_165_gb300 as pkv
from oracle import oracle as orc
from paged_kv_cache_165_gb300 import _build
from workloads import gen

from helpers import assert_attn_close, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    pkv.lib()
    pkv.get_device_error()


def pool(rng, lens, bs, mbs, spare):
    """A table whose rows own their blocks, and the free list of the rest."""
    have = [-(-n // bs) for n in lens]
    nb = sum(have) + spare
    order = rng.permutation(nb).astype(np.int32)
    table = np.full((len(lens), mbs), -1, np.int32)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = order[at:at + n]
        at += n
    free = np.full(nb, -7, np.int32)
    free[:nb - at] = order[at:]
    return table, free, nb - at


def extend(table, lens, new, free, count, bs, T, in_place=False):
    t, l, n, f = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in
                  (table, np.array(lens, np.int32), np.array(new, np.int32), free))
    c = torch.tensor([count], dtype=torch.int32, device="cuda")
    lo = l if in_place else torch.full_like(l, -9)
    co = c if in_place else torch.full_like(c, -9)
    cu = torch.full((len(lens) + 1,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -9, dtype=torch.int64, device="cuda")
    ws = torch.zeros(max(16, pkv.block_tables_extend_workspace_bytes(len(lens), T)), dtype=torch.uint8, device="cuda")
    pkv.block_tables_extend(t, l, n, f, c, lo, cu, slots, co, bs, workspace=ws)
    assert not ws.any()
    return [x.cpu().numpy() for x in (t, lo, cu, slots)] + [int(co)]


def check_extend(lens, new, bs, mbs, spare, T=None, in_place=False, count=None, flags=0):
    rng = np.random.default_rng(len(lens) + bs)
    table, free, n = pool(rng, [max(0, min(x, mbs * bs)) for x in lens], bs, mbs, spare)
    count = n if count is None else count
    T = sum(max(x, 0) for x in new) if T is None else T
    got = extend(table, lens, new, free, count, bs, T, in_place)
    want = table.copy()
    olens, cu, slots, left = orc.block_tables_extend(want, lens, new, free, count, bs, T)
    assert pkv.get_device_error() == flags
    assert np.array_equal(got[0], want)
    assert np.array_equal(got[1], olens)
    assert np.array_equal(got[2], cu)
    assert np.array_equal(got[3], slots)
    assert got[4] == left


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,bs,hi,nhi", [(1, 16, 40, 1), (5, 16, 40, 1), (33, 8, 300, 20), (8, 16, 0, 4096),
                                         (256, 16, 2000, 1), (1024, 32, 100, 3), (1025, 16, 64, 2), (3000, 24, 50, 9)])
def test_extend_matches_the_row_by_row_form(B, bs, hi, nhi, in_place):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, hi + 1, B).tolist()
    new = rng.integers(0, nhi + 1, B).tolist()
    check_extend(lens, new, bs, (hi + nhi) // bs + 2, sum(new) + 5, in_place=in_place)
    check_extend(lens, new, bs, (hi + nhi) // bs + 2, sum(new) + 5, T=sum(new) + 2000, in_place=in_place)


def test_extend_lengths_at_block_ends_and_no_new_tokens():
    check_extend([0, 16, 15, 17, 32, 0], [0, 1, 1, 15, 16, 16], 16, 4, 10)
    check_extend([3, 16, 0], [0, 0, 0], 16, 4, 2)
    check_extend([7], [0], 1, 9, 1)
    check_extend([7], [2], 1, 9, 2)


def test_extend_leaves_rows_that_do_not_fit_as_they_were():
    pool_bit, len_bit = pkv.DEVERR["pool"], pkv.DEVERR["len"]
    # four free blocks: rows 0 and 1 take three, row 2 needs two, row 3 none, row 4 one
    check_extend([16, 16, 0, 5, 16], [20, 1, 20, 2, 1], 16, 8, 4, flags=pool_bit)
    check_extend([0, 0, 0], [5, 6, 7], 16, 8, 9, T=12, flags=pool_bit)              # the slot map ends in row 2
    check_extend([60, 3, 10], [5, 2, 1 << 30], 16, 4, 9, flags=len_bit, T=100)      # past the table
    check_extend([5, -3, 10], [5, 2, -1], 16, 4, 9, flags=len_bit, T=100)
    check_extend([0] * 1500, [16] * 1500, 16, 2, 1300, flags=pool_bit)               # refused in the second scan
    check_extend([0, 4], [5, 6], 16, 8, 5, count=0, flags=pool_bit)


def test_extend_flags_bad_block_ids_and_counts():
    table = np.full((2, 4), -1, np.int32)
    table[1, 0] = 99                                   # a partial block with an id outside the pool
    free = np.array([0, 1, 7, -2], np.int32)
    got = extend(table, [0, 3], [17, 2], free, 4, 16, 19)
    assert pkv.get_device_error() == pkv.DEVERR["block"]
    assert got[0][0].tolist() == [-1, -1, -1, -1] and got[3].tolist() == [-1] * 19 and got[4] == 2
    got = extend(table[:1], [0], [17], free, 5, 16, 17)      # more free blocks than the list holds
    assert pkv.get_device_error() & pkv.DEVERR["pool"]
    assert got[1].tolist() == [0]
    for count in (5, -3):                                    # passed on; rows that need no block are served
        got = extend(np.array([[2, -1]], np.int32), [3], [4], free, count, 16, 4)
        assert pkv.get_device_error() == pkv.DEVERR["pool"]
        assert got[1].tolist() == [7] and got[3].tolist() == [35, 36, 37, 38] and got[4] == count


def release(table, first, end, free, count):
    t, f = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (table, free))
    c = torch.tensor([count], dtype=torch.int32, device="cuda")
    fi = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
    en = torch.tensor(end, dtype=torch.int32, device="cuda")
    ws = torch.full((pkv.block_tables_release_workspace_bytes(len(end)),), 0xEE, dtype=torch.uint8, device="cuda")
    pkv.block_tables_release(t, fi, en, f, c, c, workspace=ws)
    return t.cpu().numpy(), f.cpu().numpy(), int(c)


@pytest.mark.parametrize("B,mbs", [(1, 3), (7, 40), (300, 100), (1024, 70), (1500, 9), (4, 20000)])
def test_release_gives_back_ranges_in_reverse_order(B, mbs):
    rng = np.random.default_rng(B)
    bs = 16
    lens = rng.integers(0, min(mbs, 3000) * bs + 1, B)
    table, free, count = pool(rng, lens.tolist(), bs, mbs, 3)
    have = -(-lens // bs)
    first = rng.integers(0, mbs + 1, B)
    end = rng.integers(0, mbs + 1, B)
    want, blocks = table.copy(), []
    for b in range(B):
        for j in range(first[b], end[b]):
            if j < have[b]:
                blocks.append(table[b, j])
                want[b, j] = -1
    t, f, c = release(table, first.tolist(), end.tolist(), free, count)
    assert pkv.get_device_error() == 0
    assert np.array_equal(t, want) and c == count + len(blocks)
    assert f[:c].tolist() == free[:count].tolist() + blocks[::-1]
    # the rest: everything back, and every block in the list once
    t, f, c = release(t, None, [mbs] * B, f, c)
    assert (t == -1).all() and c == len(free) and sorted(f.tolist()) == list(range(len(free)))
    t, f2, c = release(t, None, [mbs] * B, f, c)       # again: nothing left to give
    assert c == len(free) and np.array_equal(f, f2) and pkv.get_device_error() == 0


def test_release_restores_what_extend_took():
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 200, 50)
    new = rng.integers(0, 90, 50)
    table, free, count = pool(rng, lens.tolist(), 16, 20, 400)
    t, out, _, _, left = extend(table, lens, new, free, count, 16, int(new.sum()))
    t2, f2, c2 = release(t, (-(-lens // 16)).tolist(), (-(-out // 16)).tolist(), free, left)
    assert np.array_equal(t2, table) and np.array_equal(f2, free) and c2 == count
    assert pkv.get_device_error() == 0


def test_release_flags_bad_ranges_entries_and_double_returns():
    table = np.array([[0, 1, -1], [2, 77, 3]], np.int32)
    free = np.full(5, -7, np.int32)
    t, f, c = release(table, [0, 0], [4, 3], free, 0)         # row 0's range passes the table
    assert pkv.get_device_error() == pkv.DEVERR["len"] | pkv.DEVERR["block"]
    assert t.tolist() == [[0, 1, -1], [-1, 77, -1]] and f[:c].tolist() == [3, 2]
    t, f, c = release(np.array([[0, 1], [0, 1]], np.int32), None, [2, 2], np.array([2, -7, -7], np.int32), 1)
    assert pkv.get_device_error() == pkv.DEVERR["pool"]        # four blocks for two places
    assert t.tolist() == [[0, 1], [0, 1]] and c == 1 and f.tolist() == [2, -7, -7]


@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop_over_a_4_bit_cache(graph):
    """Prompts admitted, decode steps (eager, or one captured graph replayed), a finished row's blocks
    given back and taken by a new prompt: against the oracle after every step."""
    rows, hq, hkv, d, group, bs, mbs = 4, 8, 2, 128, 64, 16, 8
    nb = 24
    g = gen.generator(21)
    blocks = pkv.DeviceBlocks(nb, bs, rows, mbs, 128, order=gen.permutation(g, nb))
    kc = torch.zeros((nb, hkv, bs, pkv.q4_row_bytes(d, group)), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    scale = 1 / math.sqrt(d)
    held = [[torch.zeros(0, hkv, d)] * 2 for _ in range(rows)]   # the values every row should hold
    ws = torch.zeros(max(16, pkv.paged_attention_q4_workspace_bytes(rows, rows, 1, hq, hkv, d, group, bs, mbs)),
                     dtype=torch.uint8, device="cuda")

    def values(x):
        codes, params = orc.quantize_rows_q4(x, group)
        p = np.repeat(params.astype(np.float64), group, axis=-2)
        return torch.from_numpy(p[..., 1] + p[..., 0] * codes)

    def admit(lens):
        n = torch.tensor(lens, dtype=torch.int32)
        k, v = gen.randn(g, (128, hkv, d), torch.bfloat16), gen.randn(g, (128, hkv, d), torch.bfloat16)
        slots = blocks.extend(dev(n))
        pkv.kv_append_q4(dev(k), dev(v), kc, vc, slots, group)
        at = 0
        for b, m in enumerate(lens):
            held[b] = [torch.cat([h.double(), values(x[at:at + m])]) for h, x in zip(held[b], (k, v))]
            at += m

    q = torch.zeros((rows, hq, d), device="cuda")
    kn = torch.zeros((rows, hkv, d), dtype=torch.bfloat16, device="cuda")
    vn = torch.zeros_like(kn)
    one = torch.ones(rows, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((rows, hq), device="cuda")

    def step():
        slots = blocks.extend(one, rows)
        pkv.decode_step_q4(out, q, kn, vn, slots, kc, vc, blocks.block_table, blocks.context_lens, scale, group, lse=lse,
                           workspace=ws)

    admit([5, 31, 16, 40])
    captured = None
    for i in range(20):
        if i == 9:      # row 1 is done; a new prompt takes its place
            blocks.finish(torch.tensor([False, True, False, False], device="cuda"))
            held[1] = [torch.zeros(0, hkv, d)] * 2
            admit([0, 50, 0, 0])
        hq_, hk, hv = gen.randn(g, q.shape), gen.randn(g, kn.shape, torch.bfloat16), gen.randn(g, vn.shape, torch.bfloat16)
        q.copy_(hq_)
        kn.copy_(hk)
        vn.copy_(hv)
        if graph and i >= 1:
            if captured is None:
                captured = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(captured):
                    step()
            captured.replay()
        else:
            step()
        assert pkv.get_device_error() == 0
        for b in range(rows):
            held[b] = [torch.cat([h, values(x[b:b + 1])]) for h, x in zip(held[b], (hk, hv))]
            ref, ref_lse = oracle.attend_contiguous(hq_[b].numpy(), held[b][0].numpy(), held[b][1].numpy(), scale)
            assert_attn_close(out[b], ref, f"step {i} row {b} out", 2e-4)
            assert_attn_close(lse[b], ref_lse, f"step {i} row {b} lse", 2e-4)
    lens = blocks.context_lens.cpu()
    assert lens.tolist() == [25, 61, 36, 60]
    # the cached prefix as a bf16 cache, through the chunked entry
    slots = torch.tensor([oracle.slot_of(blocks.block_table[3].cpu(), p, bs) for p in range(60)])
    ko = torch.zeros((60, hkv, d), device="cuda")
    vo = torch.zeros_like(ko)
    pkv.kv_gather_q4(ko, vo, kc, vc, dev(slots), group)
    assert np.allclose(ko.cpu().numpy(), held[3][0].numpy(), rtol=2.0 ** -23, atol=0)
    assert np.allclose(vo.cpu().numpy(), held[3][1].numpy(), rtol=2.0 ** -23, atol=0)
    blocks.finish(torch.ones(rows, dtype=torch.bool, device="cuda"))
    assert int(blocks.free_count) == nb and sorted(blocks.free_list.tolist()) == list(range(nb))
    assert pkv.get_device_error() == 0


# ------------------------------------------------------------------------ slots of a decode step

@pytest.mark.parametrize("B,nhi,T,spare", [(1, 1, None, 9), (40, 3, None, 200), (40, 3, 50, 200), (40, 3, None, 12), (40, 9, None, 3),
                                           (1500, 2, None, 900), (1500, 2, None, 40), (8, 2000, None, 1200)])
def test_step_slots_name_every_row_by_itself(B, nhi, T, spare):
    """Rows with none, one or many new tokens; too small a slot map (T) or pool (spare) refuses some."""
    rng = np.random.default_rng(B + spare)
    bs, mbs = 16, 140
    lens, new = rng.integers(0, 100, B), rng.integers(0, nhi + 1, B)
    table, free, count = pool(rng, lens.tolist(), bs, mbs, spare)
    t, l, n, f = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (table, lens, new, free))
    c = torch.tensor([count], dtype=torch.int32, device="cuda")
    T = int(new.sum()) if T is None else T
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    slots, steps = torch.empty(T, dtype=torch.int64, device="cuda"), torch.full((B,), -9, dtype=torch.int64, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    pkv.block_tables_extend(t, l, n, f, c, l, cu, slots, c, bs, workspace=ws, step_slots=steps)
    want = table.copy()
    olens, ocu, oslots, left = orc.block_tables_extend(want, lens.tolist(), new.tolist(), free, count, bs, T)
    refused = any(olens[b] != lens[b] + new[b] for b in range(B))
    assert refused == (spare in (3, 40) or T == 50) and pkv.get_device_error() == (pkv.DEVERR["pool"] if refused else 0)
    assert np.array_equal(t.cpu().numpy(), want) and np.array_equal(l.cpu().numpy(), olens) and int(c) == left
    assert np.array_equal(cu.cpu().numpy(), ocu) and np.array_equal(slots.cpu().numpy(), oslots)
    last = [oracle.slot_of(want[b], int(olens[b]) - 1, bs) if olens[b] > lens[b] else -1 for b in range(B)]
    assert steps.tolist() == last


def test_step_slots_of_bad_block_ids_are_padding():
    table = torch.tensor([[99, -1], [2, -1]], dtype=torch.int32, device="cuda")
    l = torch.tensor([3, 3], dtype=torch.int32, device="cuda")
    one = torch.ones_like(l)
    free, c = torch.tensor([0, 1, -7, -7], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    slots, steps = torch.empty(2, dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int64, device="cuda")
    pkv.block_tables_extend(table, l, one, free, c, l, torch.empty(3, dtype=torch.int32, device="cuda"), slots, c, 16,
                            step_slots=steps)
    assert pkv.get_device_error() == pkv.DEVERR["block"]
    assert slots.tolist() == [-1, 35] and steps.tolist() == [-1, 35]


@pytest.mark.parametrize("hq,bs", [(8, 16), (32, 16), (8, 24), (128, 16)])   # one launch; append and attention in two
@pytest.mark.parametrize("graph", [False, True])
def test_decode_loop_with_idle_and_refused_rows(hq, bs, graph):
    """Row 2 is idle, and row 1 finds the pool empty when its block is full: the rows behind them keep
    writing their own slots, and nobody else's."""
    rows, hkv, d, group, mbs = 4, 2, 128, 64, 6
    g = gen.generator(83)
    start = [5, 3 * bs - 1, bs, 2 * bs - 6]
    nb = sum(-(-n // bs) for n in start)
    blocks = pkv.DeviceBlocks(nb, bs, rows, mbs, 160, order=gen.permutation(g, nb))
    caches = [torch.zeros((nb, hkv, bs, pkv.q4_row_bytes(d, group)), dtype=torch.uint8) for _ in range(2)]
    gk, gv = (dev(t) for t in caches)
    prompt = [gen.randn(g, (sum(start), hkv, d), torch.bfloat16) for _ in range(2)]
    slots = blocks.extend(torch.tensor(start, dtype=torch.int32, device="cuda"), sum(start))
    pkv.kv_append_q4(*(dev(t) for t in prompt), gk, gv, slots, group)
    orc.kv_append_q4(*caches, *prompt, slots.cpu(), group)
    new = torch.tensor([1, 1, 0, 1], dtype=torch.int32, device="cuda")
    q, kn, vn = (torch.zeros((rows, h, d), dtype=t, device="cuda") for h, t in
                 ((hq, torch.float32), (hkv, torch.bfloat16), (hkv, torch.bfloat16)))
    out, lse = torch.zeros_like(q), torch.zeros((rows, hq), device="cuda")
    ws = torch.zeros(max(16, pkv.paged_attention_q4_workspace_bytes(rows, rows, 1, hq, hkv, d, group, bs, mbs)),
                     dtype=torch.uint8, device="cuda")

    def step():
        blocks.extend(new, rows)
        pkv.decode_step_q4(out, q, kn, vn, blocks.step_slots, gk, gv, blocks.block_table, blocks.context_lens, 0.1, group,
                           lse=lse, workspace=ws)

    held = list(start)
    captured = None
    for i in range(5):
        x = [gen.randn(g, t.shape).to(t.dtype) for t in (q, kn, vn)]
        for t, y in zip((q, kn, vn), x):
            t.copy_(y)
        if graph and i >= 1:
            if captured is None:
                captured = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(captured):
                    step()
            captured.replay()
        else:
            step()
        served = [True, held[1] < 3 * bs, False, True]
        assert pkv.get_device_error() == (0 if served[1] else pkv.DEVERR["pool"])
        held = [n + s for n, s in zip(held, served)]
        assert blocks.context_lens.tolist() == held
        table = blocks.block_table.cpu()
        mine = torch.tensor([oracle.slot_of(table[b], held[b] - 1, bs) if served[b] else -1 for b in range(rows)])
        assert blocks.step_slots.tolist() == mine.tolist()
        orc.kv_append_q4(*caches, x[1], x[2], mine, group)
        assert torch.equal(gk.cpu(), caches[0]) and torch.equal(gv.cpu(), caches[1])
        ref, ref_lse = oracle.paged_decode(x[0], *(orc.dequantize_q4(c, d, group) for c in caches), table,
                                           torch.tensor(held, dtype=torch.int32), 0.1)
        assert_attn_close(out, ref, f"step {i} out", 2e-4)
        assert_attn_close(lse, ref_lse, f"step {i} lse", 2e-4)


@pytest.mark.parametrize("raw", [False, True])
def test_a_loop_on_a_stream_of_its_own(raw):
    """extend and finish enqueued behind other work of a side stream, given as a Stream or as its handle."""
    blocks = pkv.DeviceBlocks(40, 16, 3, 20, 300)
    new = torch.tensor([100, 3, 60], dtype=torch.int32, device="cuda")
    done = torch.tensor([True, False, True], device="cuda")
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)         # a few milliseconds
    blocks.extend(new, 163, stream=stream)
    blocks.finish(done, stream=stream)
    blocks.extend(new, 163, stream=stream)
    side.synchronize()
    assert pkv.get_device_error() == 0
    assert blocks.context_lens.tolist() == [100, 6, 60] and int(blocks.free_count) == 40 - 7 - 1 - 4
    held = [x for row in blocks.block_table.tolist() for x in row if x >= 0]
    assert sorted(held + blocks.free_list[:28].tolist()) == list(range(40))


def test_extend_of_as_many_tokens_as_fit_32_bits():
    """2^31 - 1 tokens of two rows (a slot map of 17 GB): the last token's number plus a grid of threads passes 2^31."""
    bs, mbs, nb = 1 << 16, 1 << 14, 40000
    T = (1 << 31) - 1
    table = torch.full((2, mbs), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    new = torch.tensor([1 << 30, (1 << 30) - 1], dtype=torch.int32, device="cuda")
    free = torch.randperm(nb, dtype=torch.int32, device="cuda")
    count = torch.tensor([nb], dtype=torch.int32, device="cuda")
    cu, steps = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int64, device="cuda")
    slots = torch.full((T,), -9, dtype=torch.int64, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    pkv.block_tables_extend(table, lens, new, free, count, lens, cu, slots, count, bs, workspace=ws, step_slots=steps)
    assert pkv.get_device_error() == 0
    assert lens.tolist() == new.tolist() and cu.tolist() == [0, 1 << 30, T] and int(count) == nb - 2 * mbs
    assert torch.equal(table.flatten(), free.flip(0)[:2 * mbs])
    pos = torch.arange(bs, device="cuda")
    for lo in range(0, 2 * mbs, 1024):                        # block by block, in the rows' order
        want = (table.flatten()[lo:lo + 1024, None].long() * bs + pos).flatten()
        got = slots[lo * bs:(lo + 1024) * bs]
        assert torch.equal(got, want[:got.numel()])
    assert steps.tolist() == [int(slots[(1 << 30) - 1]), int(slots[-1])]
