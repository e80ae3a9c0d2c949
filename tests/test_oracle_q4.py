"""The oracle of the 4-bit cache and of the GPU block tables against worked examples, error
bounds and the host block manager; refusals of the entry points before any launch.  No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_165_gb300 as pkv
from oracle import oracle as orc
from paged_kv_cache_165_gb300 import BlockManager, _binding, _build
from workloads import gen


@pytest.fixture(scope="module")
def L():
    _build.build()
    return pkv.lib()


def test_q4_worked_example():
    # group of 32: 0..30 and 45: zero 0, scale 3, codes rint(x / 3) with ties to even (1.5 -> 2 is no tie of thirds)
    x = np.concatenate([np.arange(31), [45.0]]).astype(np.float32)
    codes, params = orc.quantize_rows_q4(x[None], 32)
    assert params[0, 0].tolist() == [3.0, 0.0]
    assert codes[0].tolist() == [int(np.rint(v / 3)) for v in x]
    # exact ties: scale 2, odd x: x / 2 = k + 1/2 goes to the even code
    x = np.concatenate([np.arange(31), [30.0]]).astype(np.float32)
    codes, params = orc.quantize_rows_q4(x[None], 32)
    assert params[0, 0].tolist() == [2.0, 0.0]
    assert codes[0, 1] == 0 and codes[0, 3] == 2 and codes[0, 5] == 2 and codes[0, 7] == 4


@pytest.mark.parametrize("group", [32, 64, 128])
def test_q4_values_lie_within_half_a_step(group):
    g = gen.generator(group)
    x = gen.randn(g, (50, 256)) * torch.logspace(-3, 3, 50)[:, None] + 7 * gen.randn(g, (50, 1))
    codes, params = orc.quantize_rows_q4(x, group)
    p = np.repeat(params.astype(np.float64), group, axis=1)
    err = np.abs(p[..., 1] + p[..., 0] * codes - x.double().numpy())
    # half a step, and where the scale was rounded down up to 15 * 2^-11 of a step more at the top
    assert np.all(err <= p[..., 0] * (0.5 + 15 * 2.0 ** -11) + 1e-12)
    assert np.all(params[..., 1].astype(np.float64) <= x.double().numpy().reshape(50, -1, group).min(-1))


def test_q4_constant_nan_and_out_of_range_groups():
    x = np.zeros((4, 64), np.float32)
    x[0] = 0.5                       # exact in fp16: scale 0, codes 0
    x[1, 3] = np.nan
    x[2, 5], x[2, 6] = 1e30, -np.inf
    x[3, :32] = -1e-9                # below fp16's subnormals: zero is the first one under it
    codes, params = orc.quantize_rows_q4(x, 32)
    assert params[0, 0].tolist() == [0.0, 0.5] and not codes[0].any()
    assert np.isnan(params[1, 0, 1]) and params[1, 0, 0] == 0 and not codes[1, :32].any()
    assert params[1, 1].tolist() == [0.0, 0.0]
    assert params[2, 0, 1] == -65504 and codes[2, 5] == 15 and codes[2, 6] == 0
    assert params[3, 0, 1] == -(2.0 ** -24)


def test_q4_append_packs_pages_as_documented():
    nb, hkv, bs, d, group = 3, 2, 8, 64, 32
    row = d // 2 + 4 * (d // group)
    cache = np.full((nb, hkv, bs, row), 0xA5, np.uint8)
    kc, vc = cache.copy(), cache.copy()
    g = gen.generator(1)
    kn, vn = gen.randn(g, (2, hkv, d)), gen.randn(g, (2, hkv, d))
    orc.kv_append_q4(kc, vc, kn, vn, np.array([bs + 3, -1]), group)
    codes, params = orc.quantize_rows_q4(kn, group)
    page = kc[1, 1].reshape(-1)
    assert [int(b) for b in page[3 * 32:4 * 32]] == [int(codes[0, 1, 2 * j]) | int(codes[0, 1, 2 * j + 1]) << 4 for j in range(32)]
    assert np.array_equal(page[bs * 32:].view(np.float16).reshape(bs, 2, 2)[3], params[0, 1])
    changed = (kc != cache).reshape(nb, hkv, -1)
    assert not changed[0].any() and not changed[2].any() and changed[1].sum() <= 2 * (32 + 8)
    want = params[0, 1, :, 1].astype(np.float64).repeat(32) + params[0, 1, :, 0].astype(np.float64).repeat(32) * codes[0, 1]
    assert np.array_equal(orc.dequantize_q4(kc, d, group)[1, 1, 3], want)


def test_extend_oracle_agrees_with_the_host_block_manager():
    bs, nb = 16, 64
    order = gen.permutation(gen.generator(3), nb)
    bm = BlockManager(nb, bs, order=order)
    lens = [0, 5, 16, 31, 40]
    table = np.full((5, 12), -1, np.int32)
    free = np.array(order[::-1], np.int32)
    count = nb
    got = np.zeros(5, np.int32)
    for n in (lens, [1] * 5, [17, 0, 16, 1, 30]):
        for s, k in enumerate(n):                       # the manager takes tokens one by one, in the same order
            if s not in bm.tables:
                bm.add_sequence(s, 0)
            host = [bm.append_slot(s)[0] for _ in range(k)]
            bm_slots = host if s == 0 else bm_slots + host
        got, cu, slots, count = orc.block_tables_extend(table, got, np.array(n), free, count, bs, sum(n) + 2)
        assert slots.tolist() == bm_slots + [-1, -1]
        assert cu.tolist() == np.concatenate([[0], np.cumsum(n)]).tolist()
        assert got.tolist() == bm.context_lens(range(5)).tolist()
        assert count == bm.num_free
    assert np.array_equal(table, bm.block_table(range(5), 12).numpy())


P16 = ctypes.c_void_p(16)   # never dereferenced: validation fails first


def test_q4_calls_reject_bad_arguments_before_any_launch(L):
    def rows(fn, dt=1, T=3, Hkv=2, d=128, group=64, bs=16, NB=4, a=P16, cache=P16):
        return fn(a, P16, dt, cache, P16, P16, T, Hkv, d, group, bs, NB, None)
    for fn in (L.pkv_kv_append_q4, L.pkv_kv_gather_q4):
        assert rows(fn, dt=2) == _binding.PKV_ERR_UNSUPPORTED
        for bad in (dict(T=-1), dict(Hkv=0), dict(group=16), dict(group=48), dict(d=96, group=64), dict(d=288, group=32),
                    dict(d=0), dict(bs=0), dict(NB=0), dict(a=None), dict(cache=ctypes.c_void_p(18))):
            assert rows(fn, **bad) == _binding.PKV_ERR_INVALID_ARG, bad
        assert rows(fn, T=0) == _binding.PKV_OK

    def attend(B=2, Tq=2, max_q=1, Hq=8, Hkv=2, d=128, group=64, bs=16, MBS=4, NB=8, window=0, splits=0, out=P16, q=P16,
               cu=None):
        return L.pkv_paged_attention_q4(out, None, q, P16, P16, P16, P16, cu, B, Tq, max_q, Hq, Hkv, d, group, bs, MBS,
                                        NB, 0.1, window, splits, None, 0, None)
    for bad in (dict(Hq=9), dict(B=-1), dict(group=256), dict(d=96), dict(MBS=0), dict(NB=0), dict(window=-1),
                dict(splits=-1), dict(Tq=3), dict(out=None), dict(Tq=3, max_q=2), dict(q=ctypes.c_void_p(20)),
                dict(MBS=1 << 28)):
        assert attend(**bad) == _binding.PKV_ERR_INVALID_ARG, bad
    assert attend(B=0, Tq=0) == _binding.PKV_OK
    assert attend(Tq=0) == _binding.PKV_OK

    def step(new_dt=1, B=2, Hq=8, NB=8, k_new=P16, group=64):
        return L.pkv_decode_step_q4(P16, None, P16, k_new, P16, new_dt, P16, P16, P16, P16, P16, B, Hq, 2, 128, group, 16,
                                    4, NB, 0.1, 0, 0, None, 0, None)
    assert step(new_dt=2) == _binding.PKV_ERR_UNSUPPORTED
    for bad in (dict(Hq=9), dict(NB=0), dict(k_new=None), dict(group=33)):
        assert step(**bad) == _binding.PKV_ERR_INVALID_ARG, bad
    assert step(B=0) == _binding.PKV_OK
    assert L.pkv_q4_row_bytes(128, 64) == 72 and L.pkv_q4_row_bytes(96, 64) == -1
    assert L.pkv_paged_attention_q4_workspace_bytes(2, 2, 1, 9, 2, 128, 64, 16, 4, 0, 0) == 0


def test_block_table_calls_reject_bad_arguments_before_any_launch(L):
    def extend(B=2, T=2, MBS=4, bs=16, NB=8, lens=P16, slots=P16, cu=P16):
        return L.pkv_block_tables_extend(P16, lens, P16, P16, P16, P16, cu, slots, P16, B, T, MBS, bs, NB, None, 0, None)
    for bad in (dict(B=-1), dict(T=-1), dict(MBS=0), dict(bs=0), dict(NB=0), dict(lens=None), dict(slots=None),
                dict(cu=None), dict(MBS=1 << 28)):
        assert extend(**bad) == _binding.PKV_ERR_INVALID_ARG, bad

    def release(B=2, MBS=4, NB=8, end=P16, table=P16):
        return L.pkv_block_tables_release(table, None, end, P16, P16, P16, B, MBS, NB, None, 0, None)
    for bad in (dict(B=-1), dict(MBS=0), dict(NB=0), dict(end=None), dict(table=None)):
        assert release(**bad) == _binding.PKV_ERR_INVALID_ARG, bad


def test_q4_bindings_check_tensors():
    cpu = torch.zeros((2, 2, 128))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_append_q4(cpu, cpu, torch.zeros((1, 2, 16, 72), dtype=torch.uint8),
                         torch.zeros((1, 2, 16, 72), dtype=torch.uint8), torch.zeros(2, dtype=torch.int64), 64)
    for call in (lambda: pkv.kv_append_q4(None, cpu, cpu, cpu, cpu, 64), lambda: pkv.kv_gather_q4(cpu.numpy(), cpu, cpu, cpu, cpu, 64),
                 lambda: pkv.paged_attention_q4(cpu, None, cpu, cpu, cpu, cpu, 0.1, 64),
                 lambda: pkv.block_tables_release(None, None, cpu, cpu, cpu, cpu)):
        with pytest.raises((TypeError, ValueError), match="torch.Tensor|CUDA"):
            call()
    with pytest.raises(ValueError, match="q4_row_bytes"):
        pkv.q4_row_bytes(128, 48)
    with pytest.raises(ValueError, match="permutation"):
        pkv.DeviceBlocks(4, 16, 2, 2, 4, order=[0, 1, 1, 2], device="cpu")


def test_extend_step_rejects_bad_arguments_before_any_launch(L):
    def extend(B=2, T=2, MBS=4, bs=16, NB=8, lens=P16, steps=P16):
        return L.pkv_block_tables_extend_step(P16, lens, P16, P16, P16, P16, P16, P16, steps, P16, B, T, MBS, bs, NB, None, 0, None)
    for bad in (dict(B=-1), dict(T=-1), dict(MBS=0), dict(bs=0), dict(NB=0), dict(lens=None), dict(steps=None)):
        assert extend(**bad) == _binding.PKV_ERR_INVALID_ARG, bad


def test_device_blocks_refuse_more_tokens_than_their_slot_map_holds(L):
    blocks = pkv.DeviceBlocks(4, 16, 2, 2, 4, device="cpu")
    for n in (5, -1):
        with pytest.raises(ValueError, match="max_tokens"):
            blocks.extend(torch.ones(2, dtype=torch.int32), n)
    with pytest.raises(ValueError, match="CUDA"):
        blocks.extend(torch.ones(2, dtype=torch.int32), 4)
