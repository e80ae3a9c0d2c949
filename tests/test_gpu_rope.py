"""Rotary positions on the GPU against the 64-bit definition: layouts, part of the head, types, strides, far
positions, padding, bad slots, in place, and the inverse as the gradient."""
import numpy as np
import pytest
import torch

import paged_kv_cache_165_gb300 as pkv
from oracle import serve
from paged_kv_cache_165_gb300 import _build

from helpers import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    pkv.lib()
    pkv.get_device_error()


def bound(x, rot, interleaved, mscale, want, dtype):
    """Errors of a rotated row: cosine and sine are off by an ulp of the function (2^-24 at most 1), by the angle's
    own rounding (at most pi / 4 * 2^-24 after the quarter turns) and by the product with mscale (2^-24), so
    3 * 2^-24 * mscale; two products and a sum add 2 * 2^-24 of the same terms.  Then the output's rounding, half
    a step of the value (and of what it may be off by)."""
    x = np.abs(x.double().cpu().numpy())
    terms = np.zeros_like(x)
    half = rot // 2
    if interleaved:
        terms[..., 0:rot:2] = terms[..., 1:rot:2] = x[..., 0:rot:2] + x[..., 1:rot:2]
    else:
        terms[..., :half] = terms[..., half:rot] = x[..., :half] + x[..., half:rot]
    b = 6 * 2.0 ** -24 * mscale * terms
    return b + torch.finfo(dtype).eps / 2 * (np.abs(want) + b)


def close(got, want, b):
    g = got.double().cpu().numpy()
    bad = np.abs(g - want) > b
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.abs(g - want)[bad].max():.3e}"


def inputs(seed, T, hq, hkv, d, dtype, packed=False, far=5000):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, hq + 2 * hkv, d), generator=g).to(dtype).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
    return q, k, v, pos


@pytest.mark.parametrize("T,hq,hkv,d,rot,bs", [
    (1, 1, 1, 2, 2, 1), (3, 8, 2, 64, 64, 16), (64, 64, 8, 128, 128, 16), (37, 6, 3, 96, 32, 8), (5, 4, 4, 80, 40, 16),
    (700, 8, 1, 256, 128, 32), (2500, 4, 2, 64, 32, 16), (9, 3, 1, 33, 6, 4), (2, 5, 5, 7, 4, 3), (11, 2, 2, 24, 20, 5)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,qdt,packed", [(BF16, F32, True), (BF16, BF16, False), (F32, F32, False), (F32, BF16, True)])
def test_rope_append(T, hq, hkv, d, rot, bs, interleaved, dtype, qdt, packed):
    q, k, v, pos = inputs(T + d, T, hq, hkv, d, dtype, packed)
    kw = dict(base=10000.0, scaling="parts", factor=4.0, original=1000.0)
    turns, freq = pkv.rope_turns(rot, **kw), serve.rope_frequencies(rot, **kw)
    nb = -(-T // bs) + 2
    kc, vc = (torch.full((nb, hkv, bs, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    slots = torch.from_numpy(np.random.default_rng(T).permutation(nb * bs)[:T].astype(np.int64))
    slots[::4] = -1                                    # padding
    qo = torch.full((T, hq, d), float("nan"), dtype=qdt, device="cuda")
    pkv.rope_append(qo, q, k, v, kc, vc, pos, slots.cuda(), turns, interleaved=interleaved, mscale=1.25)
    assert pkv.get_device_error() == 0
    want = serve.rope_rows(q, pos.cpu(), freq, interleaved, 1.25)
    close(qo, want, bound(q, rot, interleaved, 1.25, want, qdt))
    want = serve.rope_rows(k, pos.cpu(), freq, interleaved, 1.25)
    b = bound(k, rot, interleaved, 1.25, want, dtype)
    got_k = kc.transpose(1, 2).reshape(nb * bs, hkv, d)
    got_v = vc.transpose(1, 2).reshape(nb * bs, hkv, d)
    kept = slots >= 0
    at = slots[kept].cuda()
    close(got_k[at], want[kept.numpy()], b[kept.numpy()])
    assert_bits_equal(got_v[at], v[kept.cuda()])
    assert_bits_equal(got_k[at][..., rot:], k[kept.cuda()][..., rot:])
    rest = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (got_k[rest] == 7).all() and (got_v[rest] == 7).all()      # nothing else is written


@pytest.mark.parametrize("base", [10000.0, 1.0, 5e6])
def test_far_positions_keep_their_angle(base):
    rot = 64
    pos = torch.tensor([0, 1, -1, 12345678, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7, 1000003], dtype=torch.int32)
    x = torch.randn((8, 2, rot), generator=torch.Generator().manual_seed(1)).cuda()
    turns = pkv.rope_turns(rot, base=base)
    # the angle in whole numbers from the turns that the kernel is given
    t = [int(v) % 2 ** 64 for v in turns.tolist()]
    want = np.zeros((8, 2, rot))
    xs = x.double().cpu().numpy()
    for i, p in enumerate(pos.tolist()):
        phi = np.array([(p * f % 2 ** 64) / 2 ** 64 for f in t]) * 2 * np.pi
        want[i] = np.concatenate([xs[i, :, :32] * np.cos(phi) - xs[i, :, 32:] * np.sin(phi),
                                  xs[i, :, :32] * np.sin(phi) + xs[i, :, 32:] * np.cos(phi)], -1)
    out = torch.empty_like(x)
    pkv.rope(out, x, None, None, pos.cuda(), turns)
    close(out, want, bound(x, rot, False, 1.0, want, F32))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (96, 32), (10, 6)])
def test_the_inverse_is_the_gradient(d, rot, interleaved):
    T, hq, hkv = 6, 3, 2
    q, k, _, pos = inputs(d, T, hq, hkv, d, F32)
    turns = pkv.rope_turns(rot)
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    pkv.rope(dq, gq, dk, gk, pos, turns, interleaved=interleaved, mscale=1.5, inverse=True)
    freq = serve.rope_frequencies(rot)
    for g, got in ((gq, dq), (gk, dk)):
        want = serve.rope_rows(g, pos.cpu(), freq, interleaved, 1.5, inverse=True)
        close(got, want, bound(g, rot, interleaved, 1.5, want, F32))
    # against differences of <g, rope(q)>: the map is linear, so a difference is the derivative; fp32 gradients
    # of some hundred terms
    fwd = lambda x: serve.rope_rows(x, pos.cpu(), freq, interleaved, 1.5)
    rng = np.random.default_rng(0)
    for _ in range(5):
        step = rng.standard_normal(q.shape)
        got = float((dq.double().cpu().numpy() * step).sum())
        want = float((gq.double().cpu().numpy() * (fwd(q.double().cpu().numpy() + step) - fwd(q.double().cpu().numpy()))).sum())
        assert abs(got - want) < 1e-4


def test_unaligned_rows_and_odd_strides():
    T, hq, hkv, d = 5, 2, 1, 16
    for dtype in (BF16, F32):
        for shift, pitch in ((1, 4 * d + 3), (3, 4 * d + 1), (8, 4 * d + 8)):
            buf = torch.randn(T * pitch + 64, generator=torch.Generator().manual_seed(shift)).to(dtype).cuda()
            row = lambda h0, h: torch.as_strided(buf, (T, h, d), (pitch, d, 1), shift + h0 * d)
            q, k, v = row(0, hq), row(hq, hkv), row(hq + hkv, hkv)
            pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37
            turns = pkv.rope_turns(d)
            for inter in (False, True):
                kc, vc = (torch.zeros(T + 1, hkv, 1, d, dtype=dtype, device="cuda") for _ in range(2))
                qo = torch.empty((T, hq, d), device="cuda")
                pkv.rope_append(qo, q, k, v, kc, vc, pos, torch.arange(T, device="cuda"), turns, interleaved=inter)
                ref_q, ref_k = torch.empty_like(qo), torch.empty((T, hkv, d), dtype=dtype, device="cuda")
                pkv.rope(ref_q, q.contiguous(), ref_k, k.contiguous(), pos, turns, interleaved=inter)
                assert_bits_equal(qo, ref_q)
                assert_bits_equal(kc[:T, :, 0], ref_k)
                assert_bits_equal(vc[:T, :, 0], v)
                want = serve.rope_rows(q, pos.cpu(), serve.rope_frequencies(d), inter)
                close(qo, want, bound(q, d, inter, 1.0, want, F32))


def test_bad_slots_are_flagged_and_skipped_and_v_keeps_its_bits():
    T, hq, hkv, d, bs, nb = 4, 2, 2, 32, 4, 3
    q, k, v, pos = inputs(9, T, hq, hkv, d, BF16)
    v.view(torch.int16)[1] = 0x7fc1    # a NaN with a payload
    kc, vc = (torch.zeros((nb, hkv, bs, d), dtype=BF16, device="cuda") for _ in range(2))
    slots = torch.tensor([0, 5, nb * bs, 2 ** 40], device="cuda")
    qo = torch.empty((T, hq, d), device="cuda")
    pkv.rope_append(qo, q, k, v, kc, vc, pos, slots, pkv.rope_turns(d))
    assert pkv.get_device_error() == pkv.DEVERR["slot"]
    assert_bits_equal(vc[1, :, 1], v[1])
    assert kc[2].abs().sum() == 0 and not torch.isnan(qo).any()


def test_in_place_and_on_another_stream_and_in_a_graph():
    T, hq, hkv, d = 300, 8, 2, 128
    q, k, _, pos = inputs(4, T, hq, hkv, d, BF16)
    turns = pkv.rope_turns(d)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.rope(qo, q, ko, k, pos, turns)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qi, ki = q.clone(), k.clone()
    s.wait_stream(torch.cuda.current_stream())
    pkv.rope(qi, qi, ki, ki, pos, turns, stream=s)
    s.synchronize()
    assert_bits_equal(qi, qo)
    assert_bits_equal(ki, ko)
    g = torch.cuda.CUDAGraph()
    q2, k2 = torch.zeros_like(q), torch.zeros_like(k)
    with torch.cuda.graph(g):
        pkv.rope(q2, q, k2, k, pos, turns)
    g.replay()
    torch.cuda.synchronize()
    assert_bits_equal(q2, qo)
    assert_bits_equal(k2, ko)


def test_refusals_on_the_gpu():
    T, hq, hkv, d = 2, 4, 2, 16
    q, k, v, pos = inputs(1, T, hq, hkv, d, F32)
    turns, slots = pkv.rope_turns(d), torch.zeros(T, dtype=torch.int64, device="cuda")
    kc = torch.zeros((2, hkv, 4, d), device="cuda")
    qo = torch.empty_like(q)
    ok = dict(q_out=qo, q=q, k_new=k, v_new=v, k_cache=kc, v_cache=kc.clone(), positions=pos, slot_mapping=slots, turns=turns)
    pkv.rope_append(**ok)
    for bad in (dict(q_out=qo[:1]), dict(q=q.transpose(0, 1)), dict(k_new=k[:, :1]), dict(k_new=k.to(BF16)), dict(positions=pos.long()),
                dict(slot_mapping=slots.int()), dict(turns=turns.int()), dict(turns=pkv.rope_turns(2 * d)), dict(k_cache=kc[0]),
                dict(k_cache=kc.transpose(1, 2)), dict(q=q.cpu()), dict(q_out=qo.half())):
        with pytest.raises((ValueError, TypeError, pkv.PkvError)):
            pkv.rope_append(**{**ok, **bad})
    with pytest.raises(pkv.PkvError, match="overlaps"):
        pkv.rope(q.view(-1)[:q.numel()].view(T, hq, d)[:1], q.view(-1)[8:8 + hq * d].view(1, hq, d), None, None, pos[:1], turns)
    assert pkv.get_device_error() == 0
