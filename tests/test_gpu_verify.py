"""pkv_verify_drafts on the GPU, token by token equal to the definition in whole numbers."""
import numpy as np
import pytest
import torch

import paged_kv_cache_165_gb300 as pkv
from oracle import serve
from paged_kv_cache_165_gb300 import _build

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    pkv.lib()
    pkv.get_device_error()


def rows(t, pitch):
    """The rows of t, `pitch` elements apart."""
    if t is None or pitch == 0:
        return t
    buf = torch.full((t.shape[0], t.shape[1] + pitch), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def run(target, draft, toks, cu, u, lens=None, D=None):
    B = len(cu) - 1
    dev = lambda x, dt: torch.as_tensor(np.asarray(x), dtype=dt).cuda()
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    out = torch.full((target.shape[0],), -2, dtype=torch.int32, device="cuda")
    ld = None if lens is None else dev(lens, torch.int32)
    pkv.verify_drafts(acc, out, target, dev(toks, torch.int32), dev(cu, torch.int32), dev(u, F32), draft_probs=draft,
                      context_lens=ld, context_lens_out=ld)
    return acc.tolist(), out.tolist(), None if ld is None else ld.tolist()


def case(seed, V, ks, dtype, sharp=2.0, near=0.7):
    g = torch.Generator().manual_seed(seed)
    B, D = len(ks), sum(ks)
    cu = np.concatenate([[0], np.cumsum(ks)])
    logits = torch.randn((D + B, V), generator=g) * sharp
    target = torch.softmax(logits, 1)
    seq = np.repeat(np.arange(B), ks)
    mine = torch.softmax(logits[torch.from_numpy(np.arange(D) + seq)] + near * torch.randn((D, V), generator=g), 1)
    toks = torch.multinomial(mine, 1, generator=g)[:, 0] if D else torch.zeros(0, dtype=torch.int64)
    u = torch.rand(D + B, generator=g)
    return target.to(dtype).cuda(), mine.to(dtype).cuda(), toks.tolist(), cu.tolist(), u.tolist()


@pytest.mark.parametrize("V", [1, 2, 31, 33, 128, 1000, 4099, 32768, 50001])
@pytest.mark.parametrize("dtype,pitch", [(F32, 0), (BF16, 0), (F32, 3), (BF16, 8)])
@pytest.mark.parametrize("drafted", [True, False])
def test_every_token_is_the_definition_s(V, dtype, pitch, drafted):
    ks = [0, 1, 4, 3, 0, 7, 2, 40] if V <= 4099 else [0, 2, 4]
    for seed in range(3):
        target, draft, toks, cu, u = case(seed + V, V, ks, dtype)
        draft = draft if drafted else None
        lens = [50 + 3 * b for b in range(len(ks))]
        want = serve.verify_drafts(target, draft, toks, cu, u)
        acc, out, after = run(rows(target, pitch), rows(draft, pitch), toks, cu, u, lens)
        assert pkv.get_device_error() == 0
        assert acc == want[0] and out == want[1]
        assert after == [n - k + a for n, k, a in zip(lens, ks, acc)]


def test_many_sequences_and_a_large_vocabulary():
    ks = [4] * 40
    target, draft, toks, cu, u = case(5, 131072, ks, F32)
    acc, out, _ = run(target, draft, toks, cu, u)
    for b in range(0, 40, 7):
        c = cu[b]
        want = serve.verify_drafts(target[c + b:c + b + 5], draft[c:c + 4], toks[c:c + 4], [0, 4], u[c + b:c + b + 5])
        assert acc[b] == want[0][0] and out[c + b:c + b + 5] == want[1]
    ks = [k % 3 for k in range(700)]
    target, draft, toks, cu, u = case(6, 257, ks, F32)
    assert run(target, draft, toks, cu, u)[:2] == serve.verify_drafts(target, draft, toks, cu, u)


def test_borders_ties_and_extreme_numbers():
    p = torch.tensor([[0.0, 0.25, 0.0, 0.5, 0.25, 0.0]], device="cuda")
    for u, want in ((0.0, 1), (0.25, 3), (0.75, 4), (1 - 2.0 ** -24, 4), (2.0 ** -60, 1), (1e-45, 1), (1.0, 4), (-1.0, 1), (float("nan"), 1)):
        assert run(p, None, [], [0, 0], [u])[:2] == ([0], [want]), u
    # equal products are not below: u q = p is a rejection
    t = torch.tensor([[0.25, 0.75], [0.5, 0.5]], device="cuda")
    q = torch.tensor([[0.5, 0.5]], device="cuda")
    assert run(t, q, [0], [0, 1], [0.5, 0.0])[0] == [0]
    assert run(t, q, [0], [0, 1], [0.5 - 2.0 ** -25, 0.0])[0] == [1]
    # probabilities of 2^-40 and below still count, in order
    t = torch.full((1, 5000), 2.0 ** -40, device="cuda")
    for u in (0.0, 0.1, 0.99999):
        assert run(t, None, [], [0, 0], [u])[:2] == serve.verify_drafts(t, None, [], [0, 0], torch.tensor([u]))
    # no distribution: everything 1
    t = torch.ones((1, 4000), device="cuda")
    acc, out, _ = run(t, None, [], [0, 0], [0.5])
    assert 0 <= out[0] < 4000
    assert pkv.get_device_error() == 0


def test_small_numbers_are_multiplied_exactly():
    # u with bits far below 2^-64, at borders between tokens of a few units of 2^-46: u * total is just above a whole
    # number, at it, and just below
    t = torch.full((1, 64), 3 * 2.0 ** -46, device="cuda")
    t[0, 63] = 1 - 63 * 3 * 2.0 ** -46
    t = t.double().float()
    total = sum(serve.units(t[0].cpu()))
    for border in (3, 6, 9, 30, 60, 186):
        at = np.float32(border / total)
        for u in (np.nextafter(at, np.float32(0)), at, np.nextafter(at, np.float32(1))):
            assert run(t, None, [], [0, 0], [float(u)])[:2] == serve.verify_drafts(t, None, [], [0, 0], [float(u)]), (border, u)
    g = np.random.default_rng(4)
    for u in np.ldexp(g.random(200), -g.integers(30, 150, 200)).astype(np.float32):
        assert run(t, None, [], [0, 0], [float(u)])[:2] == serve.verify_drafts(t, None, [], [0, 0], [float(u)]), u


def test_infinite_probabilities_reject_a_draft():
    inf = float("inf")
    for p, q in ((inf, 0.5), (0.5, inf), (inf, inf), (0.5, -inf), (-inf, 0.5), (float("nan"), 0.5), (0.5, float("nan"))):
        t = torch.tensor([[p, 0.25, 0.25], [0.0, 0.0, 1.0]], device="cuda")
        d = torch.tensor([[q, 0.25, 0.25]], device="cuda")
        for drafted in (d, None):
            want = serve.verify_drafts(t, drafted, [0], [0, 1], [0.25, 0.5])
            assert run(t, drafted, [0], [0, 1], [0.25, 0.5])[:2] == want and (want[0] == [0]) == (drafted is not None or p != 0.5), (p, q)
    pkv.get_device_error()


def test_nothing_left_and_no_mass():
    flags = pkv.DEVERR["probs"]
    t = torch.tensor([[0.25, 0.0, 0.0], [1.0, 0.0, 0.0]], device="cuda")
    q = torch.tensor([[0.5, 0.25, 0.25]], device="cuda")
    assert run(t, q, [1], [0, 1], [0.0, 0.9])[:2] == ([0], [0, -1])        # p <= q everywhere: from p
    assert pkv.get_device_error() == 0
    for bad in (0.0, -1.0, float("nan")):
        z = torch.full((1, 300), bad, device="cuda")
        assert run(z, None, [], [0, 0], [0.5])[:2] == ([0], [-1])
        assert pkv.get_device_error() == flags
    # NaN among probabilities counts as 0; a NaN for a drafted token rejects it
    t = torch.tensor([[float("nan"), 0.5, 0.5], [1.0, 0.0, 0.0]], device="cuda")
    assert run(t, q, [0], [0, 1], [0.0, 0.0])[:2] == ([0], [1, -1])
    assert pkv.get_device_error() == 0


def test_drafts_outside_the_vocabulary_and_bad_offsets():
    target, draft, toks, cu, u = case(3, 100, [2, 3, 1], F32)
    for x in (-1, 100, 2 ** 31 - 1):
        for d in (draft, None):
            bad = list(toks)
            bad[0] = x
            acc, out, _ = run(target, d, bad, cu, u)
            assert pkv.get_device_error() == pkv.DEVERR["probs"]
            assert (acc, out) == serve.verify_drafts(target, d, bad, cu, u) and acc[0] == 0
    for wrong in ([0, 2, 1, 6], [0, 2, 9, 6], [0, -1, 5, 6]):
        acc, out, after = run(target, draft, toks, wrong, u, [10, 20, 30])
        assert pkv.get_device_error() == pkv.DEVERR["cu_seqlens"]
        refused = [not 0 <= a <= b <= 6 for a, b in zip(wrong, wrong[1:])]
        for b in range(3):
            if refused[b]:
                assert acc[b] == 0 and after[b] == 10 * (b + 1)


def test_stream_graph_and_two_calls_at_once():
    a, b = case(1, 9000, [3, 0, 5], F32), case(2, 9000, [3, 0, 5], BF16)
    wants = [serve.verify_drafts(*x) for x in (a, b)]
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for x, s in zip((a, b), streams):
        t = [x[0], x[1]] + [torch.tensor(v, dtype=dt, device="cuda") for v, dt in zip(x[2:], (torch.int32, torch.int32, F32))]
        outs.append((torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(11, dtype=torch.int32, device="cuda"), t, s))
    torch.cuda.synchronize()
    for _ in range(20):
        for acc, tok, t, s in outs:
            pkv.verify_drafts(acc, tok, t[0], t[2], t[3], t[4], draft_probs=t[1], stream=s)
    torch.cuda.synchronize()
    for (acc, tok, _, _), want in zip(outs, wants):
        assert (acc.tolist(), tok.tolist()) == want
    acc, tok, t, _ = outs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.verify_drafts(acc, tok, t[0], t[2], t[3], t[4], draft_probs=t[1])
    acc.zero_()
    tok.zero_()
    g.replay()
    assert (acc.tolist(), tok.tolist()) == wants[0]


def test_refusals_on_the_gpu():
    target, draft, toks, cu, u = case(3, 100, [2, 1], F32)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ok = dict(accepted=i([0, 0]), tokens=i([0] * 5), target_probs=target, draft_tokens=i(toks), cu_drafts=i(cu),
              uniforms=torch.tensor(u, device="cuda"), draft_probs=draft)
    pkv.verify_drafts(**ok)
    for bad in (dict(target_probs=target.half()), dict(target_probs=target.t()), dict(draft_probs=draft.to(BF16)), dict(draft_probs=draft[:2]),
                dict(tokens=i([0] * 4)), dict(uniforms=ok["uniforms"].double()), dict(cu_drafts=i([0, 3])), dict(context_lens=i([1, 2])),
                dict(context_lens_out=i([1, 2])), dict(draft_tokens=torch.tensor(toks)), dict(target_probs=target.cpu())):
        with pytest.raises((ValueError, TypeError, pkv.PkvError)):
            pkv.verify_drafts(**{**ok, **bad})


def test_sums_stay_at_two_to_the_seventeen():
    # no distribution: ones past 2^17 elements no longer add to the sums
    for V in (1 << 17, (1 << 18) + 5):
        t = torch.ones((1, V), device="cuda")
        for u, want in ((0.0, 0), (0.25, 1 << 15), (0.5, 1 << 16), (1 - 2.0 ** -24, (1 << 17) - 1)):
            assert run(t, None, [], [0, 0], [u])[:2] == ([0], [want]), (V, u)
    assert pkv.get_device_error() == 0
