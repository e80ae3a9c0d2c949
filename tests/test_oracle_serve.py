"""Pins of the oracle's serving operators (rotary positions, windows with first tokens, drafted tokens,
shared block tables) and the library's refusals of them, all on the CPU."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_165_gb300 as pkv
from oracle import serve
from paged_kv_cache_165_gb300 import BlockManager, _build
from workloads import gen

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    _build.build()
    return pkv.lib()


# ---------------------------------------------------------------- rotary positions

def test_rope_is_a_product_of_complex_numbers():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 12))
    pos = np.array([0, 1, -7, 100000, 3])
    f = serve.rope_frequencies(8)
    z = np.exp(1j * pos[:, None, None] * f)
    got = serve.rope_rows(x, pos, f, interleaved=True)
    want = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) * z
    assert np.allclose(got[..., 0:8:2], want.real, atol=1e-12) and np.allclose(got[..., 1:8:2], want.imag, atol=1e-12)
    assert np.array_equal(got[..., 8:], x[..., 8:])
    half = serve.rope_rows(np.concatenate([x[..., 0:8:2], x[..., 1:8:2], x[..., 8:]], -1), pos, f)
    assert np.allclose(half[..., :4], want.real, atol=1e-12) and np.allclose(half[..., 4:8], want.imag, atol=1e-12)
    back = serve.rope_rows(got, pos, f, interleaved=True, inverse=True)
    assert np.allclose(back, x, atol=1e-12)


def test_rope_scores_depend_on_the_distance():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 16))
    f = serve.rope_frequencies(16)
    dot = lambda i, j: float(np.sum(serve.rope_rows(q, [i], f) * serve.rope_rows(k, [j], f)))
    assert math.isclose(dot(17, 5), dot(1012, 1000), rel_tol=1e-10)


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
@pytest.mark.parametrize("rot", [4, 32, 128])
def test_rope_turns_are_the_frequencies(L, rot, scaling):
    kw = dict(scaling=scaling, factor=8.0, original=8192.0, low=1.0, high=4.0) if scaling != "none" else {}
    got = pkv.rope_turns(rot, base=500000.0, device="cpu", **kw).numpy().view(np.uint64)
    want = serve.rope_frequencies(rot, 500000.0, **kw) / (2 * np.pi)
    # fp64 on both sides: pow, two or three products and a quotient, a few 2^-53 each, and 2^-63 of a turn
    for g, w in zip(got.tolist(), want.tolist()):
        assert abs(Fraction(g, 2 ** 64) - Fraction(w)) <= Fraction(w) * 16 / 2 ** 53 + Fraction(1, 2 ** 62)


def test_rope_turns_refuses(L):
    buf = (ctypes.c_uint64 * 128)()
    call = lambda rot=8, base=1e4, kind=0, factor=1.0, orig=1.0, low=1.0, high=2.0: L.pkv_rope_turns(
        buf, rot, base, kind, factor, orig, low, high)
    assert call() == 0
    for kw in (dict(rot=7), dict(rot=0), dict(rot=258), dict(base=0.0), dict(base=math.inf), dict(base=math.nan),
               dict(factor=0.0), dict(factor=math.nan), dict(kind=2, rot=2), dict(kind=3, low=2.0), dict(kind=3, orig=0.0)):
        assert call(**kw) == INVALID, kw
    assert call(kind=4) == UNSUPPORTED
    assert L.pkv_rope_turns(None, 8, 1e4, 0, 1.0, 1.0, 1.0, 2.0) == INVALID
    with pytest.raises(ValueError, match="scaling"):
        pkv.rope_turns(8, scaling="other", device="cpu")


def test_rope_turns_that_are_not_finite(L):
    buf = (ctypes.c_uint64 * 128)()
    for base, kind, factor in ((1e-320, 0, 1.0), (1e4, 1, 1e-320), (1e4, 2, 1e-320), (1e4, 3, 1e-320)):
        assert L.pkv_rope_turns(buf, 256, base, kind, factor, 1.0, 1e9, 2e9) == INVALID, (base, kind, factor)
        assert b"finite" in L.pkv_last_error()
    assert L.pkv_rope_turns(buf, 256, 1e-300, 0, 1.0, 1.0, 1.0, 2.0) == 0


P = ctypes.c_void_p
NZ = P(1 << 20)   # never dereferenced: the call is refused first


def test_rope_calls_refuse(L):
    def append(q_out=NZ, qdt=0, q=P(1 << 24), dt=1, qs=1024, ks=256, vs=256, rot=64, m=1.0, T=4, Hq=8, Hkv=2, d=128, bs=16, NB=4,
               pos=NZ, slots=NZ):
        return L.pkv_rope_append(q_out, qdt, q, NZ, NZ, dt, qs, ks, vs, pos, NZ, rot, 0, m, NZ, NZ, slots, T, Hq, Hkv, d, bs, NB, None)
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(d=257), dict(rot=3), dict(rot=0), dict(rot=130), dict(qs=1023),
               dict(ks=255), dict(vs=255), dict(qs=1 << 41), dict(m=math.inf), dict(bs=0), dict(NB=0), dict(pos=None), dict(slots=None),
               dict(q_out=None)):
        assert append(**kw) == INVALID, kw
    assert append(dt=2) == UNSUPPORTED and append(qdt=2) == UNSUPPORTED
    assert append(T=0) == 0
    # the output over its input: another type, another layout, shifted
    assert append(q=NZ) == INVALID                                  # bf16 in, fp32 out
    assert append(q=NZ, qdt=1, qs=1536) == INVALID                  # rows further apart
    assert append(q=P((1 << 20) + 256), qdt=1) == INVALID
    assert b"overlaps" in L.pkv_last_error()

    def rope(k=NZ, k_out=NZ, qdt=0, ks=256, q=P(1 << 24)):
        return L.pkv_rope(NZ, qdt, k_out, q, k, 1, 1024, ks, NZ, NZ, 64, 0, 1.0, 0, 4, 8, 2, 128, None)
    assert rope(k=None) == INVALID and rope(k_out=None) == INVALID
    assert rope(ks=128) == INVALID
    assert rope(ks=512) == INVALID        # k_out is k, its rows further apart


# ------------------------------------------------------ windows with first tokens

@pytest.mark.parametrize("window,sinks", [(5, 0), (0, 3), (300, 4), (7, 300), (150, 140)])
def test_sinks_reduce_to_the_plain_attention(window, sinks):
    g = gen.generator(3)
    lens, nqs, bs = [40, 9, 1], [3, 2, 1], 8
    per = [gen.blocks_needed(n, bs) for n in lens]
    table = gen.block_table_from_order(gen.permutation(g, sum(per)), per)
    kc, vc = (gen.randn(g, (sum(per), 2, bs, 16), torch.float32) for _ in range(2))
    q = gen.randn(g, (sum(nqs), 4, 16), torch.float32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(nqs)]), dtype=torch.int32)
    plain_window = window if sinks == 0 else 0
    want, want_lse = oracle.paged_attention(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32), cu, 0.25, plain_window)
    got, lse = serve.paged_attention_sinks(q, kc, vc, table, torch.tensor(lens), cu, 0.25, window, sinks)
    assert np.allclose(got, want, atol=1e-12) and np.allclose(lse, want_lse, atol=1e-12)


def test_sinks_are_two_ranges_of_keys():
    # the log-sum-exp merge of the first tokens and of the window, by hand
    rng = np.random.default_rng(5)
    K, V, q = rng.standard_normal((30, 8)), rng.standard_normal((30, 8)), rng.standard_normal(8)
    table = np.arange(8)[None]
    cache = lambda x: np.concatenate([x, np.full((2, 8), np.nan)]).reshape(8, 1, 4, 8)
    out, lse = serve.paged_attention_sinks(q.reshape(1, 1, 8).astype(np.float64), cache(K), cache(V), table, [30], [0, 1], 1.0, 10, 3)
    w = np.exp(np.concatenate([K[:3], K[20:]]) @ q)
    assert np.allclose(out[0, 0], w @ np.concatenate([V[:3], V[20:]]) / w.sum()) and np.isclose(lse[0, 0], np.log(w.sum()))


def test_paged_attention_sinks_refuses(L):
    def call(B=2, Tq=2, max_q=1, Hq=8, Hkv=2, d=64, MBS=8, NB=8, window=16, sinks=4, dt=1, q=NZ, splits=0, bs=16):
        return L.pkv_paged_attention_sinks(NZ, None, q, NZ, NZ, dt, NZ, NZ, None, B, Tq, max_q, Hq, Hkv, d, bs, MBS, NB, 0.1, window,
                                           sinks, splits, None, 0, None)
    for kw in (dict(window=-1), dict(sinks=-1), dict(Hq=9), dict(d=300), dict(NB=0), dict(Tq=3), dict(splits=-1),
               dict(q=P((1 << 20) + 4)), dict(q=None), dict(MBS=1 << 27, bs=16), dict(MBS=(1 << 27) - 200, bs=16), dict(Tq=2, max_q=2)):
        assert call(**kw) == INVALID, kw
    assert call(dt=2) == UNSUPPORTED
    assert call(B=0, Tq=0) == 0


def test_block_manager_keeps_the_blocks_of_first_tokens():
    m = BlockManager(20, 4)
    m.add_sequence(0, 50)
    first = m.tables[0][:2]
    released = m.release_outside_window(0, 9, sinks=5)      # positions 41 .. 49 and 0 .. 4 stay: blocks 10 .. 12, 0 and 1
    assert len(released) == 8 and m.tables[0][:2] == first and m.tables[0][2:10] == [-1] * 8
    assert m.num_free == 20 - 13 + 8
    m.audit()
    assert m.release_outside_window(0, 9, sinks=5) == []


# ---------------------------------------------------------------- drafted tokens

def test_verified_tokens_are_distributed_as_the_target():
    # one draft, three tokens: the measure of (draft, u_0, u_1) that gives each token, summed over a grid
    p0, q0 = np.array([0.5, 0.25, 0.25]), np.array([0.125, 0.625, 0.25])
    n = 64
    u = (np.arange(n) + 0.5) / n
    mass = np.zeros(3)
    for x in range(3):
        for a in u:
            for b in u:
                acc, tok = serve.verify_drafts(np.array([p0, [1.0, 0, 0]]), q0[None], [x], [0, 1], [a, b])
                mass[tok[0]] += q0[x] / n ** 2
    assert np.allclose(mass, p0, atol=1.0 / n)


def test_verify_takes_the_lowest_token_past_the_border():
    p = np.array([[0.0, 0.25, 0.0, 0.5, 0.25, 0.0]])
    at = lambda u: serve.verify_drafts(p, None, [], [0, 0], [u])[1][0]
    assert [at(u) for u in (0.0, 0.24, 0.25, 0.74, 0.75, 1 - 2.0 ** -24)] == [1, 1, 3, 3, 4, 4]
    # without the draft's probabilities a rejected token is not drawn again
    two = np.array([[0.5, 0.5], [1.0, 0.0]])
    assert serve.verify_drafts(two, None, [0], [0, 1], [0.5, 0.0]) == ([0], [1, -1])
    assert serve.verify_drafts(two, None, [0], [0, 1], [0.499, 0.0]) == ([1], [0, 0])
    # nothing left over: from the target itself
    assert serve.verify_drafts(np.array([[0.25, 0.0], [1.0, 0]]), np.array([[0.5, 0.5]]), [1], [0, 1], [0.0, 0.9])[1] == [0, -1]
    assert serve.units([1.0, 2.0 ** -22 * (1 + 2.0 ** -23), 2.0 ** -47, 3 * 2.0 ** -47, 2.0 ** -48, math.nan, -1.0, math.inf]) == \
        [2 ** 46, 2 ** 24 + 2, 0, 2, 0, 0, 0, 2 ** 46]


def test_verify_drafts_refuses(L):
    def call(dt=0, ts=100, ds=100, B=2, D=3, V=100, draft=NZ, toks=P(1 << 22), lens=None, lens_out=None, tokens=NZ):
        return L.pkv_verify_drafts(NZ, tokens, NZ, draft, dt, ts, ds, toks, NZ, NZ, lens, lens_out, B, D, V, None)
    for kw in (dict(ts=99), dict(ds=99), dict(B=-1), dict(B=65536), dict(D=-1), dict(V=0), dict(V=1 << 30, ts=1 << 30, ds=1 << 30),
               dict(toks=None), dict(tokens=None), dict(lens=NZ), dict(lens_out=NZ), dict(ts=1 << 41)):
        assert call(**kw) == INVALID, kw
    assert call(dt=2) == UNSUPPORTED
    assert call(B=0) == 0
    assert call(toks=P((1 << 20) + 8)) == INVALID and b"overlaps" in L.pkv_last_error()


def test_verify_drafts_refuses_lengths_that_overlap(L):
    call = lambda lens, out: L.pkv_verify_drafts(NZ, NZ, NZ, NZ, 0, 100, 100, P(1 << 22), NZ, NZ, P(lens), P(out), 4, 3, 100, None)
    assert call(1 << 23, (1 << 23) + 4) == INVALID and b"overlaps" in L.pkv_last_error()
    assert call((1 << 23) + 12, 1 << 23) == INVALID


# --------------------------------------------------------- tables that share blocks

def host_and_fork(seed, bs=4, nb=64):
    """A BlockManager whose sequence 0 forks to 1 and 2, and the same through the oracle's fork."""
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 40))
    m = BlockManager(nb, bs)
    m.add_sequence(0, n)
    m.fork(0, 1)
    m.fork(0, 2)
    table = np.full((3, 16), -1)
    table[0, :len(m.tables[0])] = m.tables[0]
    return m, n, serve.block_tables_fork(table, [n, 0, 0], [0, 0, 0], bs, nb)


@pytest.mark.parametrize("seed", range(6))
def test_fork_shares_what_the_block_manager_shares(seed):
    m, n, got = host_and_fork(seed)
    full = n // 4
    for b in range(3):
        assert got["table"][b][:full] == m.tables[b][:full]
        assert got["lens"][b] == m.lengths[b]
    # the copies that a first write of each fork would make, made at once
    copies = [c for s in (1, 2) for c in [m.append_slot(s)[1]] if c is not None]
    assert len(got["pairs"]) == len(copies)
    refs = np.zeros(64, int)
    for t in got["table"]:
        for x in t:
            if x >= 0:
                refs[x] += 1
    assert refs.tolist() == got["refs"]
    assert sorted(got["free_list"][:got["free_count"]]) == [i for i in range(64) if refs[i] == 0]


def test_compact_keeps_contents():
    rng = np.random.default_rng(2)
    nb, bs = 40, 4
    order = rng.permutation(nb)
    table = np.full((3, 8), -1)
    table[0, :5], table[1, :3], table[2, :7] = order[:5], order[3:6], order[10:17]
    data = rng.standard_normal(nb)
    got = serve.block_tables_compact(table, [20, 10, 27], bs, nb)
    moved = data.copy()
    for s, d in got["pairs"]:
        moved[d] = data[s]
    for t, u in zip(table.tolist(), got["table"]):
        assert [data[x] for x in t if x >= 0] == [moved[x] for x in u if x >= 0]
    used = {x for t in got["table"] for x in t if x >= 0}
    assert used == set(range(len(used)))


def test_share_calls_refuse(L):
    ws = P(1 << 21)
    need = L.pkv_block_tables_share_workspace_bytes(4, 8, 32)
    assert need > 0 and L.pkv_block_tables_share_workspace_bytes(-1, 8, 32) == 0

    def fork(table=NZ, lens=NZ, out=P(1 << 23), lens_out=NZ, refs=NZ, free=NZ, pairs=NZ, B=4, MBS=8, bs=16, NB=32, ws=ws, n=need):
        return L.pkv_block_tables_fork(table, lens, None, None, out, lens_out, refs, free, NZ, pairs, NZ, B, MBS, bs, NB, ws, n, None)
    for kw in (dict(B=-1), dict(MBS=0), dict(bs=0), dict(NB=0), dict(MBS=1 << 27), dict(table=None), dict(lens=None), dict(out=None),
               dict(lens_out=None), dict(refs=None), dict(free=None), dict(pairs=None), dict(pairs=P((1 << 20) + 4)),
               dict(out=P((1 << 20) + 32))):
        assert fork(**{**kw, **({"n": 1 << 40} if kw.get("MBS") else {})}) == INVALID, kw
    assert b"overlaps" in L.pkv_last_error()
    assert fork(n=need - 1) == WORKSPACE and fork(ws=None) == WORKSPACE and fork(ws=P((1 << 21) + 2)) == WORKSPACE

    def compact(out=P(1 << 23), pairs=NZ, n=need):
        return L.pkv_block_tables_compact(NZ, NZ, None, out, NZ, NZ, NZ, pairs, NZ, 4, 8, 16, 32, ws, n, None)
    assert compact(out=None) == INVALID and compact(pairs=None) == INVALID and compact(out=P((1 << 20) + 4)) == INVALID
    assert compact(n=0) == WORKSPACE

    def copy(dt=1, n=3, pairs=NZ, count=NZ, NB=4):
        return L.pkv_kv_block_copy_counted(NZ, NZ, dt, pairs, n, count, 2, 64, 16, NB, None)
    assert copy(dt=9) == UNSUPPORTED and copy(n=0) == 0
    for kw in (dict(n=-1), dict(pairs=None), dict(count=None), dict(NB=0)):
        assert copy(**kw) == INVALID, kw


def test_share_calls_refuse_held_that_they_write(L):
    ws, n = P(1 << 21), 1 << 20
    refs, free = 1 << 23, 1 << 24
    for held in (refs, refs + 4, refs - 124, free, free + 64):
        assert L.pkv_block_tables_fork(NZ, NZ, None, P(held), NZ, NZ, P(refs), P(free), NZ, NZ, NZ, 4, 8, 16, 32, ws, n, None) == INVALID
        assert b"held" in L.pkv_last_error()
        assert L.pkv_block_tables_compact(NZ, NZ, P(held), NZ, P(refs), P(free), NZ, NZ, NZ, 4, 8, 16, 32, ws, n, None) == INVALID


def test_release_outside_window_refuses_negative_sinks():
    m = BlockManager(8, 4)
    m.add_sequence(0, 20)
    with pytest.raises(ValueError, match="sinks"):
        m.release_outside_window(0, 4, sinks=-4)
    assert -1 not in m.tables[0]


def test_python_calls_refuse_host_tensors(L):
    t = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)
    f = torch.float32
    with pytest.raises((ValueError, TypeError)):
        pkv.rope_append(t(2, 4, 8, dt=f), t(2, 4, 8, dt=f), t(2, 1, 8, dt=f), t(2, 1, 8, dt=f), t(3, 1, 4, 8, dt=f), t(3, 1, 4, 8, dt=f),
                        t(2), t(2, dt=torch.int64), t(4, dt=torch.int64))
    with pytest.raises(TypeError):
        pkv.rope(None, None, None, None, None, None)
    with pytest.raises((ValueError, TypeError)):
        pkv.paged_attention_sinks(t(1, 4, 8, dt=f), t(1, 4, 8, dt=f), t(3, 1, 4, 8, dt=f), t(3, 1, 4, 8, dt=f), t(1, 3), t(1), 1.0, 4, 1)
    with pytest.raises((ValueError, TypeError)):
        pkv.verify_drafts(t(1), t(1), t(1, 9, dt=f), t(0), t(2), t(1, dt=f))
    with pytest.raises((ValueError, TypeError)):
        pkv.block_tables_fork(t(1, 3), t(1), None, t(1, 3), t(1), t(4), t(4), t(1), t(1, 2), t(1), 4, workspace=t(40))
    with pytest.raises((ValueError, TypeError)):
        pkv.kv_block_copy(t(3, 1, 4, 8, dt=f), t(3, 1, 4, 8, dt=f), t(1, 2), count=t(1))


def test_the_binding_refuses_other_machines(L, monkeypatch):
    from paged_kv_cache_165_gb300 import _binding
    monkeypatch.setattr(_binding, "_lib", None)
    monkeypatch.setattr("platform.machine", lambda: "riscv64")
    with pytest.raises(RuntimeError, match="riscv64"):
        pkv.lib()
    monkeypatch.undo()
    assert pkv.lib() is L
