"""Block tables that share blocks, on the GPU, entry by entry equal to the row-by-row form: forks, beams, shorter
rows, held blocks, pools that run out, compaction, and the copies that go with them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_165_gb300 as pkv
from oracle import serve
from paged_kv_cache_165_gb300 import DeviceBlocks, _build

from helpers import assert_bits_equal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    pkv.lib()
    pkv.get_device_error()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def tables(rng, B, bs, width, lens, share=0.5, spare=6, gone=0.1):
    """Rows of random ids, some with the leading blocks of an earlier row, some entries given back (-1)."""
    rows, used = [], 0
    for b in range(B):
        n = -(-int(lens[b]) // bs)
        lead = []
        if b and rng.random() < share:
            other = rows[int(rng.integers(0, b))]
            lead = other[:int(rng.integers(0, min(n, len(other)) + 1))]
        rows.append(lead + list(range(used, used + n - len(lead))))
        used += n - len(lead)
    nb = max(2, used + spare)
    order = rng.permutation(nb)
    table = rng.integers(-3, 5, (B, width))       # what lies behind a row's blocks is not looked at
    for b, t in enumerate(rows):
        table[b, :len(t)] = order[t] if t else []
        if len(t) > 1:
            hit = rng.random(len(t)) < gone
            table[b, :len(t)][hit] = -1
    return table, nb


def fork(table, lens, parents, bs, nb, held=None, in_place=False):
    B, width = table.shape
    t, l = dev(table), dev(lens)
    p = None if parents is None else dev(parents)
    h = None if held is None else dev(held)
    to, lo = (t, l) if in_place else (torch.full_like(t, -9), torch.full_like(l, -9))
    refs, free = (torch.full((nb,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    fc, pc = (torch.full((1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    pairs = torch.full((B, 2), -9, dtype=torch.int32, device="cuda")
    ws = torch.randint(-99, 99, (pkv.block_tables_share_workspace_bytes(B, width, nb) // 4,), dtype=torch.int32, device="cuda")
    pkv.block_tables_fork(t, l, p, to, lo, refs, free, fc, pairs, pc, bs, held=h, workspace=ws)
    return dict(table=to, lens=lo, refs=refs, free_list=free, free_count=fc, pairs=pairs, pair_count=pc)


def same(got, want):
    n = len(want["pairs"])
    assert int(got["pair_count"]) == n and int(got["free_count"]) == want["free_count"]
    pairs = got["pairs"].tolist()
    assert pairs == [list(p) for p in want["pairs"]] + [[-1, -1]] * (len(pairs) - n)
    for name in ("table", "lens", "refs", "free_list"):
        if name in want:
            assert got[name].tolist() == want[name], name


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,bs,hi", [(1, 16, 5), (2, 4, 40), (8, 16, 300), (33, 8, 100), (100, 1, 9), (1030, 16, 64), (5000, 4, 12), (3, 16, 20000)])
def test_fork_matches_the_row_by_row_form(B, bs, hi, in_place):
    for seed in range(3):
        rng = np.random.default_rng(seed * 1000 + B)
        lens = rng.integers(0, hi + 1, B)
        width = -(-hi // bs) + 2
        table, nb = tables(rng, B, bs, width, lens, spare=B + 3)
        for parents in (rng.integers(-1, B, B), np.zeros(B, int), np.arange(B), None):
            want = serve.block_tables_fork(table, lens, parents, bs, nb)
            got = fork(table, lens, parents, bs, nb, in_place=in_place)
            assert pkv.get_device_error() == 0
            same(got, want)


def test_fork_with_held_blocks_and_a_pool_that_runs_out():
    rng = np.random.default_rng(7)
    for seed in range(8):
        B, bs = 12, 4
        lens = rng.integers(0, 30, B)
        table, nb = tables(rng, B, bs, 9, lens, spare=3)
        held = (rng.random(nb) < 0.3).astype(int) * 5
        parents = rng.integers(-1, B, B)
        want = serve.block_tables_fork(table, lens, parents, bs, nb, held)
        got = fork(table, lens, parents, bs, nb, held, in_place=bool(seed % 2))
        short = any(L == 0 and p >= 0 and lens[p] > 0 for L, p in zip(want["lens"], parents))
        assert pkv.get_device_error() == (pkv.DEVERR["pool"] if short else 0)
        same(got, want)


def test_bad_parents_lengths_and_entries_are_flagged():
    table, lens = np.array([[0, 1, 2], [3, 99, 4], [5, -7, 6]]), np.array([12, 12, 9])
    want = serve.block_tables_fork(table, lens, [0, 1, 2], 4, 12)
    same(fork(table, lens, [0, 1, 2], 4, 12), want)
    assert pkv.get_device_error() == pkv.DEVERR["block"]
    same(fork(table, lens, [0, 5, -4], 4, 12), serve.block_tables_fork(table, lens, [0, -1, -1], 4, 12))
    assert pkv.get_device_error() == pkv.DEVERR["pair"]
    bad = np.array([12, -1, 13])
    same(fork(table, bad, None, 4, 12), serve.block_tables_fork(table, [12, 0, 0], None, 4, 12))
    assert pkv.get_device_error() == pkv.DEVERR["len"]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,bs,hi,spare", [(1, 16, 5, 0), (1, 4, 40, 100), (8, 16, 300, 30), (33, 8, 100, 1000), (1030, 16, 64, 1),
                                           (3, 16, 20000, 9000)])
def test_compact_matches_the_row_by_row_form(B, bs, hi, spare, in_place):
    for seed in range(3):
        rng = np.random.default_rng(seed + B)
        lens = rng.integers(0, hi + 1, B)
        table, nb = tables(rng, B, bs, -(-hi // bs) + 1, lens, spare=spare)
        for held in (None, (rng.random(nb) < 0.2).astype(int)):
            want = serve.block_tables_compact(table, lens, bs, nb, held)
            t = dev(table)
            to = t if in_place else torch.full_like(t, -9)
            refs, free = (torch.full((nb,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
            fc, pc = (torch.full((1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
            pairs = torch.full((nb // 2, 2), -9, dtype=torch.int32, device="cuda")
            ws = torch.randint(-99, 99, (pkv.block_tables_share_workspace_bytes(B, table.shape[1], nb) // 4,), dtype=torch.int32, device="cuda")
            pkv.block_tables_compact(t, dev(lens), to, refs, free, fc, pairs, pc, bs, held=None if held is None else dev(held), workspace=ws)
            assert pkv.get_device_error() == 0
            same(dict(table=to, refs=refs, free_list=free, free_count=fc, pairs=pairs, pair_count=pc), want)


@pytest.mark.parametrize("nb", [1, 9, 30000])
def test_no_rows_at_all(nb):
    i = lambda *n: torch.full(n, -9, dtype=torch.int32, device="cuda")
    ws = i(pkv.block_tables_share_workspace_bytes(0, 4, nb) // 4)
    for held in (None, [1] + [0] * (nb - 1)):
        refs, free, fc, pc = i(nb), i(nb), i(1), i(1)
        h = None if held is None else dev(held)
        for call in (lambda: pkv.block_tables_fork(i(0, 4), i(0), None, i(0, 4), i(0), refs, free, fc, i(0, 2), pc, 8, held=h, workspace=ws),
                     lambda: pkv.block_tables_compact(i(0, 4), i(0), i(0, 4), refs, free, fc, i(nb // 2, 2), pc, 8, held=h, workspace=ws)):
            call()
            n = nb - (held is not None)
            assert int(fc) == n and int(pc) == 0 and refs.tolist() == (held or [0] * nb)
            assert free.tolist() == list(range(nb - 1, nb - 1 - n, -1)) + [-1] * (nb - n)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("nb", [24576, 24577, 262144, 262145, 700001])
def test_pools_at_the_borders_of_the_ways_to_count(nb):
    # one block's shared memory, a lane's bits for 32 ids, and past them; blocks used at both ends of the pool
    rng = np.random.default_rng(nb)
    B, bs, width = 40, 8, 30
    lens = rng.integers(0, width * bs + 1, B)
    ids = np.concatenate([rng.permutation(600), nb - 1 - rng.permutation(600)])
    table = ids[:B * width].reshape(B, width)
    table[3] = table[2]
    held = np.zeros(nb, int)
    held[[5, 700, nb - 7, nb // 2]] = 1
    parents = rng.integers(-1, B, B)
    for h in (None, held):
        want = serve.block_tables_fork(table, lens, parents, bs, nb, h)
        same(fork(table, lens, parents, bs, nb, h), want)
        want = serve.block_tables_compact(table, lens, bs, nb, h)
        t, to = dev(table), torch.full((B, width), -9, dtype=torch.int32, device="cuda")
        refs, free = (torch.full((nb,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        fc, pc = (torch.full((1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        pairs = torch.full((nb // 2, 2), -9, dtype=torch.int32, device="cuda")
        ws = torch.randint(-99, 99, (pkv.block_tables_share_workspace_bytes(B, width, nb) // 4,), dtype=torch.int32, device="cuda")
        pkv.block_tables_compact(t, dev(lens), to, refs, free, fc, pairs, pc, bs, held=None if h is None else dev(h), workspace=ws)
        same(dict(table=to, refs=refs, free_list=free, free_count=fc, pairs=pairs, pair_count=pc), want)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("shape,dtype", [((9, 2, 16, 64), torch.bfloat16), ((9, 3, 5, 7), torch.float32), ((9, 1, 3, 5), torch.bfloat16),
                                         ((9, 8, 32, 128), torch.float32), ((9, 2, 16, 72), torch.uint8), ((9, 4, 16, 1), torch.float32)])
def test_counted_copies(shape, dtype):
    mk = lambda s: (torch.randn(shape, generator=torch.Generator().manual_seed(s)) * 50).to(dtype).cuda()
    pairs = torch.tensor([[0, 4], [1, 5], [0, 6], [2, 7]], dtype=torch.int32, device="cuda")
    for count, flags in ((0, 0), (2, 0), (4, 0), (5, pkv.DEVERR["pair"]), (-1, pkv.DEVERR["pair"])):
        k, v = mk(1), mk(2)
        wk, wv = k.clone(), v.clone()
        for s, d in pairs[:max(0, min(count, 4))].tolist():
            wk[d], wv[d] = k[s], v[s]
        pkv.kv_block_copy(k, v, pairs, count=torch.tensor([count], dtype=torch.int32, device="cuda"))
        assert pkv.get_device_error() == flags
        assert_bits_equal(k, wk)
        assert_bits_equal(v, wv)
    bad = torch.tensor([[0, 9], [-1, 3], [1, 8]], dtype=torch.int32, device="cuda")
    k, v = mk(1), mk(2)
    want = k.clone()
    want[8] = k[1]
    pkv.kv_block_copy(k, v, bad, count=torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert pkv.get_device_error() == pkv.DEVERR["pair"]
    assert_bits_equal(k, want)


def test_device_blocks_beams_grow_shrink_and_compact():
    """Beams over three sequences, each row's tokens known by their values: after any fork, extension, rejection,
    finish and compaction a row reads back what it should hold."""
    rng = np.random.default_rng(1)
    B, bs, nb = 6, 4, 64
    blocks = DeviceBlocks(nb, bs, B, 10, 64)
    k, v = (torch.zeros((nb, 1, bs, 1), device="cuda") for _ in range(2))
    held_tokens = [[] for _ in range(B)]
    serial = 0

    def check():
        t, lens = blocks.block_table.tolist(), blocks.context_lens.tolist()
        assert lens == [len(h) for h in held_tokens]
        flat = k.flatten().tolist()
        for b in range(B):
            assert [flat[t[b][p // bs] * bs + p % bs] for p in range(lens[b])] == held_tokens[b]
        assert torch.equal(k, -v)
        assert pkv.get_device_error() == 0

    for step in range(60):
        what = rng.choice(["extend", "extend", "extend", "fork", "reject", "finish", "compact"])
        if what == "extend":
            room = [min(4, 40 - len(h)) for h in held_tokens]
            new = [int(rng.integers(0, r + 1)) for r in room]
            slots = blocks.extend(dev(new)).tolist()
            at = 0
            vals = []
            for b in range(B):
                for _ in range(new[b]):
                    serial += 1
                    held_tokens[b] = held_tokens[b] + [float(serial)]
                    vals.append(float(serial))
            pad = vals + [0.0] * (len(slots) - len(vals))
            x = torch.tensor(pad, device="cuda").view(-1, 1, 1)
            pkv.kv_append(x, -x, k, v, blocks.slot_mapping)
        elif what == "fork":
            parents = rng.integers(-1 if step % 3 == 0 else 0, B, B)
            blocks.fork(dev(parents))
            blocks.copy(k, v)
            held_tokens = [list(held_tokens[p]) if p >= 0 else [] for p in parents]
        elif what in ("reject", "finish"):
            cut = [int(rng.integers(0, min(5, len(h)) + 1)) if what == "reject" else (len(h) if rng.random() < 0.3 else 0)
                   for h in held_tokens]
            blocks.context_lens.sub_(dev(cut))
            blocks.settle()
            blocks.copy(k, v)
            held_tokens = [h[:len(h) - c] for h, c in zip(held_tokens, cut)]
        else:
            blocks.compact()
            blocks.copy(k, v)
            used = nb - int(blocks.free_count)
            assert all(x < used for row in blocks.block_table.tolist() for x in row)
        check()


def test_fork_and_copies_in_a_graph():
    B, bs, nb = 4, 4, 40
    blocks = DeviceBlocks(nb, bs, B, 6, 32)
    k, v = (torch.arange(nb * bs, dtype=torch.float32, device="cuda").view(nb, 1, bs, 1).clone() for _ in range(2))
    blocks.extend(dev([6, 9, 0, 0]))
    parents = dev([0, 1, 0, 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        blocks.fork(parents)
        blocks.copy(k, v)
    row = lambda b: [k.flatten()[blocks.block_table[b, p // bs] * bs + p % bs].item() for p in range(int(blocks.context_lens[b]))]
    want = [row(0), row(1)]
    for swap in ([0, 1, 0, 1], [1, 1, 0, 0], [3, 2, 1, 0]):
        parents.copy_(dev(swap))
        before = [row(b) if b < 2 or swap != [0, 1, 0, 1] else [] for b in range(4)]
        g.replay()
        torch.cuda.synchronize()
        assert [row(b) for b in range(4)] == [before[p] for p in swap]
    assert pkv.get_device_error() == 0 and want[0]


def test_refusals_on_the_gpu():
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    n = pkv.block_tables_share_workspace_bytes(3, 5, 20)
    ok = dict(block_table=i(3, 5), context_lens=i(3), parents=i(3), block_table_out=i(3, 5), context_lens_out=i(3), refs=i(20),
              free_list=i(20), free_count=i(1), pairs=i(3, 2), pair_count=i(1), bs=4, workspace=i(n // 4))
    pkv.block_tables_fork(**ok)
    for bad in (dict(parents=i(4)), dict(block_table=i(15)), dict(refs=i(19)), dict(pairs=i(2, 2)), dict(free_count=i(2)), dict(held=i(19)),
                dict(context_lens_out=None), dict(block_table_out=None), dict(context_lens=torch.zeros(3, device="cuda")),
                dict(workspace=None), dict(workspace=i(n // 4 - 1)), dict(bs=0), dict(refs=i(20).cpu())):
        with pytest.raises((ValueError, TypeError, pkv.PkvError)):
            pkv.block_tables_fork(**{**ok, **bad})
    pkv.get_device_error()


@pytest.mark.parametrize("fill", ["largest", "lowest", "any"])
@pytest.mark.parametrize("B,bs,hi,spare", [(1, 16, 16, 3), (9, 16, 90, 9), (64, 4, 40, 70), (300, 16, 300, 300), (2100, 4, 12, 2100), (8, 16, 300, 25000)])
def test_workspaces_of_any_contents(B, bs, hi, spare, fill):
    """Rows without a partly filled last block (idle ones, and whole blocks) leave their scratch unwritten."""
    rng = np.random.default_rng(B)
    lens = np.where(rng.random(B) < 0.4, 0, np.where(rng.random(B) < 0.5, rng.integers(0, hi // bs + 1, B) * bs, rng.integers(0, hi + 1, B)))
    width = -(-hi // bs) + 1
    table, nb = tables(rng, B, bs, width, lens, spare=spare)
    n = pkv.block_tables_share_workspace_bytes(B, width, nb) // 4
    most = 2 ** 31 - 1
    lo, end = {"largest": (most, most + 1), "lowest": (-most - 1, -most), "any": (-most - 1, most + 1)}[fill]
    i = lambda *shape: torch.full(shape, -9, dtype=torch.int32, device="cuda")
    ws = lambda: torch.randint(lo, end, (n,), dtype=torch.int32, device="cuda")
    for parents in (None, rng.integers(-1, B, B)):
        want = serve.block_tables_fork(table, lens, parents, bs, nb)
        for in_place in (False, True):
            t, l = dev(table), dev(lens)
            got = dict(table=t if in_place else i(B, width), lens=l if in_place else i(B), refs=i(nb), free_list=i(nb), free_count=i(1),
                       pairs=i(B, 2), pair_count=i(1))
            pkv.block_tables_fork(t, l, None if parents is None else dev(parents), *got.values(), bs, workspace=ws())
            assert pkv.get_device_error() == 0
            same(got, want)
    got = dict(table=i(B, width), refs=i(nb), free_list=i(nb), free_count=i(1), pairs=i(nb // 2, 2), pair_count=i(1))
    pkv.block_tables_compact(dev(table), dev(lens), *got.values(), bs, workspace=ws())
    assert pkv.get_device_error() == 0
    same(got, serve.block_tables_compact(table, lens, bs, nb))


def test_device_blocks_over_recycled_memory():
    blocks = DeviceBlocks(40, 4, 6, 6, 32)
    blocks._share_ws.fill_(2 ** 31 - 1)   # what torch.empty may find
    blocks.extend(dev([6, 8, 0, 0, 9, 0]))
    before = blocks.block_table.tolist()
    blocks.settle()                       # idle rows and whole blocks: nothing to do
    assert int(blocks.pair_count) == 0 and int(blocks.free_count) == 40 - 2 - 2 - 3
    lens = blocks.context_lens.tolist()
    assert lens == [6, 8, 0, 0, 9, 0]
    assert [row[:-(-n // 4)] for row, n in zip(blocks.block_table.tolist(), lens)] == [row[:-(-n // 4)] for row, n in zip(before, lens)]
    assert pkv.get_device_error() == 0


def rows_of(blocks, k):
    bs, flat, table = blocks.block_size, k.flatten().tolist(), blocks.block_table.tolist()
    return [[flat[table[b][p // bs] * bs + p % bs] for p in range(n)] for b, n in enumerate(blocks.context_lens.tolist())]


def captured(call):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_copies_of_a_list_that_a_replayed_graph_wrote():
    B, bs, nb = 4, 4, 60
    k, v = (torch.arange(nb * bs, dtype=torch.float32, device="cuda").view(nb, 1, bs, 1).clone() for _ in range(2))
    blocks = DeviceBlocks(nb, bs, B, 6, 32, order=[int(i) for i in np.random.default_rng(4).permutation(nb)])
    parents = dev([0, 1, 0, 1])
    forking = captured(lambda: blocks.fork(parents))
    blocks.extend(dev([6, 9, 0, 0]))
    first = rows_of(blocks, k)
    blocks.compact()                    # the last call from Python
    blocks.copy(k, v)
    assert rows_of(blocks, k) == first
    forking.replay()                    # the last to run
    blocks.copy(k, v)
    assert rows_of(blocks, k) == [first[p] for p in (0, 1, 0, 1)] and rows_of(blocks, v) == rows_of(blocks, k)

    # and the other way round: a compaction in a graph, a fork called
    blocks.context_lens.copy_(dev([6, 0, 6, 0]))
    blocks.settle()
    blocks.copy(k, v)
    compacting = captured(blocks.compact)
    blocks.fork(dev([-1, 2, 2, 2]))
    blocks.copy(k, v)
    before = rows_of(blocks, k)
    assert before == [[], first[0], first[0], first[0]]
    blocks.extend(dev([20, 3, 3, 3]))
    blocks.context_lens.copy_(dev([0, 9, 9, 9]))
    blocks.settle()
    blocks.copy(k, v)
    before = rows_of(blocks, k)
    compacting.replay()
    blocks.copy(k, v)
    assert rows_of(blocks, k) == before and rows_of(blocks, v) == before
    used = nb - int(blocks.free_count)
    assert all(x < used for row in blocks.block_table.tolist() for x in row)
    assert pkv.get_device_error() == 0


def test_a_captured_copy_refuses_a_longer_list():
    nb = 40
    k, v = (torch.arange(nb, dtype=torch.float32, device="cuda").view(nb, 1, 1, 1).clone() for _ in range(2))
    blocks = DeviceBlocks(nb, 1, 1, 8, 8, order=list(range(nb - 1, -1, -1)))
    copying = captured(lambda: blocks.copy(k, v))
    blocks.extend(dev([5]))
    row = rows_of(blocks, k)
    blocks.compact()
    assert int(blocks.pair_count) == 5
    copying.replay()
    torch.cuda.synchronize()
    assert pkv.get_device_error() == pkv.DEVERR["pair"]
    blocks.copy(k, v)
    assert rows_of(blocks, k) == row and pkv.get_device_error() == 0
