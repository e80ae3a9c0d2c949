"""4-bit KV cache on the GPU against the fp64 oracle: quantising appends bit-exact, values read
back, and attention over the values on every kernel path."""
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

# out and lse in fp32, inputs ~ N(0, 1).  A score is a sum of d terms q * value and is off by at most
# ~(d / 8 + 16) * 2^-24 * scale * sum |q| (|zero| + 15 scale_g) (fp32 partial sums; the split of q into two
# f16 parts adds 2^-22 of the same sum): at d = 256, sum |q| * 5 = 1100 / 16, 48 * 6e-8 * 69 = 2e-4.  lse is
# off by as much; out by twice that times max |value| / 2 in the worst case, and rounding errors that do not
# all point one way stay well below: one bound for both.
ATOL = 2e-4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    pkv.lib()
    pkv.get_device_error()


def row_bytes(d, group):
    return d // 2 + 4 * (d // group)


def q4_cache(rows, group):
    """uint8 cache [NB][Hkv][bs][row] of rows [NB][Hkv][bs][d]."""
    nb, hkv, bs, d = rows.shape
    codes, params = orc.quantize_rows_q4(rows, group)
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(nb, hkv, -1)
    out = np.concatenate([packed, np.ascontiguousarray(params).view(np.uint8).reshape(nb, hkv, -1)], -1)
    return torch.from_numpy(out.reshape(nb, hkv, bs, row_bytes(d, group)))


# ------------------------------------------------------------------ append and gather

@pytest.mark.parametrize("dtype,d,group,bs,hkv", [
    (torch.bfloat16, 128, 64, 16, 4), (torch.bfloat16, 128, 128, 32, 1), (torch.float32, 64, 32, 16, 2),
    (torch.float32, 96, 32, 8, 3), (torch.bfloat16, 256, 128, 16, 2), (torch.bfloat16, 32, 32, 24, 5),
])
@pytest.mark.parametrize("T", [1, 37])
def test_append_q4_bit_exact_and_gather(dtype, d, group, bs, hkv, T):
    nb = 9
    g = gen.generator(d + T)
    kn = gen.randn(g, (T, hkv, d)) * torch.logspace(-6, 5, T)[:, None, None]
    vn = gen.randn(g, (T, hkv, d)) + 3.0
    kn[T // 2, 0] = 0.25                          # a constant group: scale 0
    vn[T - 1, hkv - 1, 1] = float("nan")
    kn[0, 0, 0], kn[0, 0, 1] = float("inf"), -1e6
    kn, vn = kn.to(dtype), vn.to(dtype)
    slots = torch.tensor(gen.permutation(g, nb * bs)[:T], dtype=torch.int64)
    if T > 4:
        slots[4] = -1
    kc = torch.full((nb, hkv, bs, row_bytes(d, group)), 0x5A, dtype=torch.uint8)
    vc = kc.clone()
    gk, gv = dev(kc), dev(vc)
    pkv.kv_append_q4(dev(kn), dev(vn), gk, gv, dev(slots), group)
    assert pkv.get_device_error() == 0
    orc.kv_append_q4(kc, vc, kn, vn, slots, group)
    # a NaN zero may carry any NaN bits: compare those values as values
    gkn, gvn = gk.cpu().numpy(), gv.cpu().numpy()
    assert np.array_equal(gkn, kc.numpy())
    diff = gvn != vc.numpy()
    dk, dv = orc.dequantize_q4(kc, d, group), orc.dequantize_q4(gvn, d, group)
    assert diff.sum() <= 2 and np.isnan(orc.dequantize_q4(vc, d, group)[np.isnan(dv)]).all()
    # the values read back: fp32 rounds zero + scale * code once (2^-24), bf16 once more (2^-8)
    for out_dt, tol in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8 * (1 + 2.0 ** -15))):
        ko = torch.full((T, hkv, d), 7.0, dtype=out_dt, device="cuda")
        vo = ko.clone()
        pkv.kv_gather_q4(ko, vo, gk, gv, dev(slots), group)
        assert pkv.get_device_error() == 0
        for got, want in ((ko, dk), (vo, dv)):
            w = np.stack([want[s // bs, :, s % bs] if s >= 0 else np.zeros((hkv, d)) for s in slots.tolist()])
            x = got.double().cpu().numpy()
            assert np.array_equal(np.isnan(x), np.isnan(w))
            ok = ~np.isnan(w)
            assert np.all(np.abs(x[ok] - w[ok]) <= tol * np.abs(w[ok]))


def test_append_q4_at_rounding_boundaries():
    """Rows whose quotients sit on or one fp32 step beside k + 1/2, and ranges whose fp16 scale does."""
    g = gen.generator(5)
    rows = []
    for i in range(400):
        s = float(np.float16(0.01 + 0.37 * i))
        z = float(np.float16(-1.7 * i - 0.3))
        k = torch.randint(0, 15, (64,), generator=g).double()
        x = (z + (k + 0.5) * s).float()
        x = torch.where(torch.arange(64) % 3 == 1, torch.nextafter(x, torch.tensor(1e9)), x)
        x = torch.where(torch.arange(64) % 3 == 2, torch.nextafter(x, torch.tensor(-1e9)), x)
        x[0], x[1] = z, z + 15 * s
        rows.append(x)
        h = np.float16(0.5 + 0.01 * i)
        mid = (float(h) + float(np.nextafter(h, np.float16(np.inf)))) / 2      # halfway between two scales
        y = torch.rand(64, generator=g) * 15 * mid
        y[0], y[1] = 0.0, 15 * mid
        if i % 3:
            y[1] = torch.nextafter(y[1], torch.tensor(1e9 if i % 3 == 1 else -1e9))
        rows.append(y)
    new = torch.stack(rows).view(-1, 1, 64)
    T = new.shape[0]
    kc = torch.zeros((T // 16, 1, 16, row_bytes(64, 64)), dtype=torch.uint8)
    vc = kc.clone()
    gk, gv = dev(kc), dev(vc)
    slots = torch.arange(T)
    pkv.kv_append_q4(dev(new), dev(-new), gk, gv, dev(slots), 64)
    orc.kv_append_q4(kc, vc, new, -new, slots, 64)
    assert torch.equal(gk.cpu(), kc) and torch.equal(gv.cpu(), vc)


def test_append_q4_unaligned_rows_and_out_of_range_slots():
    g = gen.generator(6)
    base = gen.randn(g, (3 * 2 * 64 + 1,), torch.bfloat16)
    new = dev(base)[1:].view(3, 2, 64)            # contiguous, two bytes off a 16-byte boundary
    kc = torch.zeros((2, 2, 16, row_bytes(64, 32)), dtype=torch.uint8)
    gk, gv = dev(kc), dev(kc)
    slots = torch.tensor([3, 32, 17])
    pkv.kv_append_q4(new, new, gk, gv, dev(slots), 32)
    assert pkv.get_device_error() & pkv.DEVERR["slot"]
    vc = kc.clone()
    orc.kv_append_q4(kc, vc, base[1:].view(3, 2, 64)[[0, 2]], base[1:].view(3, 2, 64)[[0, 2]], slots[[0, 2]], 32)
    assert torch.equal(gk.cpu(), kc) and torch.equal(gv.cpu(), vc)
    out = torch.full((3 * 2 * 64 + 1,), 9.0, device="cuda")
    ko = out[1:].view(3, 2, 64)
    pkv.kv_gather_q4(ko, torch.empty_like(ko), gk, gv, dev(slots), 32)
    assert pkv.get_device_error() & pkv.DEVERR["slot"]
    assert torch.all(ko[1] == 0) and torch.any(ko[0] != 0) and out[0] == 9.0


def test_q4_block_copy_moves_pages():
    g = gen.generator(8)
    kc = torch.randint(0, 255, (6, 2, 16, 72), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 255, (6, 2, 16, 72), generator=g, dtype=torch.uint8)
    pairs = torch.tensor([[1, 4], [2, 0]], dtype=torch.int32)
    gk, gv = dev(kc), dev(vc)
    pkv.kv_block_copy(gk, gv, dev(pairs))
    oracle.kv_block_copy(kc, vc, pairs)
    assert torch.equal(gk.cpu(), kc) and torch.equal(gv.cpu(), vc)


# ------------------------------------------------------------------------- attention

def q4_case(seed, lens, hq, hkv, d, group, bs, rows=None, spare=3, poison=True):
    """Caches, tables, lengths and queries; slots past a sequence's end hold NaN parameters."""
    g = gen.generator(seed)
    per_seq = [gen.blocks_needed(n, bs) for n in lens]
    nb = sum(per_seq) + spare
    table = gen.block_table_from_order(gen.permutation(g, nb), per_seq)
    k = gen.randn(g, (nb, hkv, bs, d)) + 0.5
    v = gen.randn(g, (nb, hkv, bs, d))
    if poison:
        for b, n in enumerate(lens):
            for pos in range(n, per_seq[b] * bs):
                s = oracle.slot_of(table[b], pos, bs)
                k[s // bs, :, s % bs] = float("nan")
                v[s // bs, :, s % bs] = float("nan")
    kc, vc = q4_cache(k, group), q4_cache(v, group)
    rows = rows or [1] * len(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32)
    q = gen.randn(g, (int(cu[-1]), hq, d))
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32), cu


def run_q4(case, group, scale, window=0, num_splits=0, decode=True, max_q=1, stream=None):
    q, kc, vc, table, lens, cu = case
    Tq, Hq, d = q.shape
    NB, Hkv, bs, _ = kc.shape
    B = lens.numel()
    out = torch.full((Tq, Hq, d), float("nan"), device="cuda")
    lse = torch.full((Tq, Hq), float("nan"), device="cuda")
    n = pkv.paged_attention_q4_workspace_bytes(B, Tq, max_q, Hq, Hkv, d, group, bs, table.shape[1], window, num_splits)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    pkv.paged_attention_q4(out, dev(q), dev(kc), dev(vc), dev(table), dev(lens), scale, group,
                           cu_q=None if decode else dev(cu), max_q=max_q, window=window, lse=lse, num_splits=num_splits,
                           workspace=ws)
    torch.cuda.synchronize()
    assert int(ws[:pkv_counter_bytes(n)].max()) == 0 if n else True
    return out, lse


def pkv_counter_bytes(n):
    return min(n, 256 << 10)


def expect(case, group, scale, window):
    q, kc, vc, table, lens, cu = case
    d = q.shape[2]
    live = [b for b in range(lens.numel()) if int(lens[b]) > 0 and int(cu[b + 1]) > int(cu[b])]
    rows = np.concatenate([np.arange(int(cu[b]), int(cu[b + 1])) for b in live])
    n = np.concatenate([[0], np.cumsum([int(cu[b + 1] - cu[b]) for b in live])]).astype(np.int32)
    kd, vd = (np.nan_to_num(orc.dequantize_q4(c, d, group)) for c in (kc, vc))   # unseen slots: anything finite
    out, lse = oracle.paged_attention(q[rows], kd, vd, table[live], lens[live], n, scale, window)
    return rows, out, lse


SHAPES = [  # hq, hkv, d, group, bs
    (8, 8, 128, 64, 16), (16, 4, 128, 128, 16), (64, 8, 128, 64, 16), (16, 2, 128, 32, 32), (8, 2, 64, 64, 16),
    (6, 2, 64, 32, 32), (7, 1, 128, 128, 32),                       # up to eight query heads per KV head
    (16, 1, 128, 64, 16), (64, 2, 128, 64, 16), (24, 2, 64, 32, 16), (64, 1, 128, 128, 32), (40, 1, 128, 32, 16),
    (8, 2, 96, 32, 16), (4, 2, 256, 128, 16), (4, 4, 128, 64, 8), (10, 2, 32, 32, 24), (2, 1, 160, 32, 16),
    (130, 1, 128, 64, 16),                                            # more heads than a tile
    (8, 1, 96, 32, 32), (24, 2, 192, 64, 16), (3, 1, 192, 32, 32), (16, 2, 256, 64, 16), (2, 2, 256, 64, 32),
    (12, 2, 160, 32, 32), (6, 2, 256, 32, 16), (5, 1, 224, 32, 16), (1, 1, 96, 32, 8), (3, 1, 32, 32, 16),
    (8, 1, 128, 32, 8), (5, 1, 256, 128, 8), (20, 1, 64, 32, 8), (6, 2, 128, 64, 24),
]


@pytest.mark.parametrize("hq,hkv,d,group,bs", SHAPES)
@pytest.mark.parametrize("window", [0, 50])
def test_q4_decode_matches_the_oracle(hq, hkv, d, group, bs, window):
    lens = [1, 15, 16, 17, 100, 0, 257, 1000, 33]
    case = q4_case(hq + d + bs + window, lens, hq, hkv, d, group, bs)
    scale = 1 / math.sqrt(d)
    live, ref, ref_lse = expect(case, group, scale, window)
    for splits in (1, 3, 0):
        out, lse = run_q4(case, group, scale, window, splits)
        assert pkv.get_device_error() == 0
        assert_attn_close(out[live], ref, f"splits {splits} out", ATOL)
        assert_attn_close(lse[live], ref_lse, f"splits {splits} lse", ATOL)
        assert torch.all(out[5] == 0) and torch.all(torch.isneginf(lse[5]))


@pytest.mark.parametrize("hq,hkv,d,group,bs", [(64, 8, 128, 64, 16), (8, 8, 128, 128, 16), (16, 1, 64, 32, 32),
                                               (4, 2, 96, 32, 16), (64, 1, 128, 64, 16)])
@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("max_q", [2, 4, 70])
def test_q4_query_rows_match_the_oracle(hq, hkv, d, group, bs, window, max_q):
    lens = [1, 16, 90, 17, 300, 0, 75, 1100]
    rows = [min(n, r) for n, r in zip(lens, [1, max_q, max_q, 1, max_q, 0, 0, max_q - 1])]
    case = q4_case(hq + d + max_q + window, lens, hq, hkv, d, group, bs, rows)
    scale = 1 / math.sqrt(d)
    live, ref, ref_lse = expect(case, group, scale, window)
    for splits in (1, 3, 0):
        out, lse = run_q4(case, group, scale, window, splits, decode=False, max_q=max_q)
        assert pkv.get_device_error() == 0
        assert_attn_close(out[live], ref, f"splits {splits} out", ATOL)
        assert_attn_close(lse[live], ref_lse, f"splits {splits} lse", ATOL)


def test_q4_rows_beyond_the_sequence_are_flagged():
    case = list(q4_case(3, [5, 40], 8, 1, 128, 64, 16, [6, 2]))
    out, lse = run_q4(case, 64, 0.1, decode=False, max_q=6)
    assert pkv.get_device_error() & pkv.DEVERR["cu_seqlens"]
    assert torch.all(out[:6] == 0) and torch.all(torch.isneginf(lse[:6]))
    live, ref, _ = expect((case[0][6:], case[1], case[2], case[3][1:], case[4][1:], torch.tensor([0, 2])), 64, 0.1, 0)
    assert_attn_close(out[6:], ref, "the good sequence", ATOL)


@pytest.mark.parametrize("hq,hkv,d,bs", [(16, 2, 128, 16), (64, 1, 128, 16), (4, 2, 96, 16)])
def test_q4_bad_block_reads_zeros_and_bad_length_is_empty(hq, hkv, d, bs):
    group = 32
    case = list(q4_case(5, [200, 300, 64], hq, hkv, d, group, bs, poison=False))
    q, kc, vc, table, lens, cu = case
    bad = table.clone()
    bad[1, 2], bad[1, 3] = kc.shape[0] + 9, -5
    wrong = lens.clone()
    wrong[2] = table.shape[1] * bs + 1
    out, lse = run_q4((q, kc, vc, bad, wrong, cu), group, 0.1)
    err = pkv.get_device_error()
    assert err & pkv.DEVERR["block"] and err & pkv.DEVERR["len"]
    assert torch.all(out[2] == 0) and torch.all(torch.isneginf(lse[2]))
    # the bad blocks as blocks of zeros: codes and parameters 0
    z = torch.zeros_like(kc[:1])
    good = table.clone()
    good[1, 2] = good[1, 3] = kc.shape[0]
    live, ref, ref_lse = expect((q[:2], torch.cat([kc, z]), torch.cat([vc, z]), good[:2], lens[:2], cu[:3]), group, 0.1, 0)
    assert_attn_close(out[:2], ref, "out", ATOL)
    assert_attn_close(lse[:2], ref_lse, "lse", ATOL)


@pytest.mark.parametrize("hq,hkv", [(8, 1), (64, 1)])
def test_q4_long_context_many_splits(hq, hkv):
    lens = [20011, 3, 9000]
    case = q4_case(11, lens, hq, hkv, 128, 64, 16)
    scale = 1 / math.sqrt(128)
    live, ref, ref_lse = expect(case, 64, scale, 0)
    for splits in (0, 7, 64):
        out, lse = run_q4(case, 64, scale, 0, splits)
        assert_attn_close(out[live], ref, f"splits {splits} out", ATOL)
        assert_attn_close(lse[live], ref_lse, f"splits {splits} lse", ATOL)
    assert pkv.get_device_error() == 0


# Equal weights over n keys: out is the mean of values zero + scale * code, |scale * (code - 8)| <= 2.4 for
# values ~ N(0, 1).  A weight times scale in two f16 parts is off by 2^-22; a tensor core's sum of 32 keys
# takes four additions cut off at 2^-23 of at most 32 * 2.4 (of 1024 keys: 128, of at most four standard
# deviations 4 * sqrt(1024) * 0.9 once the codes are centred); adding those in fp32 to a running sum of at most
# 4 * sqrt(n) * 0.9 costs 2^-24 of it n / 32 times; the zeros' running sums (mean 0.15) 5 * sqrt(n / 16) * 2^-24
# * 0.15.  Relative to n weights, n = 40003: 6e-7 + 1.2e-6 (1.8e-6) + 1.4e-6 + 2e-6 < 6e-6.  Sums whose
# error grows with n (uncentred codes added up by the tensor core) are off by 1e-5 and more.
ATOL_MEAN = 6e-6


@pytest.mark.parametrize("hq,d,group,bs", [(8, 128, 64, 16), (4, 128, 32, 32), (1, 64, 64, 16), (64, 128, 128, 16),
                                           (64, 128, 64, 32), (64, 64, 64, 16), (2, 96, 32, 16), (2, 96, 32, 8),
                                           (8, 256, 64, 16), (5, 224, 32, 16), (1, 128, 128, 24)])
def test_q4_errors_do_not_grow_with_the_context(hq, d, group, bs):
    case = q4_case(12, [40003], hq, 1, d, group, bs)
    case = (torch.zeros_like(case[0]), *case[1:])
    live, ref, _ = expect((case[0][:, :1], *case[1:]), group, 0.1, 0)
    for splits in (0, 1):
        out, lse = run_q4(case, group, 0.1, 0, splits)
        assert_attn_close(out, np.broadcast_to(ref, out.shape), f"splits {splits} out", ATOL_MEAN)
        assert_attn_close(lse, np.full(lse.shape, math.log(40003)), f"splits {splits} lse", 4e-6)   # 4 ulp of 10.6


@pytest.mark.parametrize("hq,hkv", [(8, 1), (32, 1)])
def test_q4_large_and_masked_values(hq, hkv):
    """Queries and caches far from 1: the scores' range, not their number format, decides."""
    case = list(q4_case(13, [130, 64], hq, hkv, 128, 64, 16))
    for f in (1e-20, 1e4, 0.0):
        q = case[0] * f
        scale = 0.0883 * (1e-4 if f == 1e4 else 1.0)
        live, ref, ref_lse = expect((q, *case[1:]), 64, scale, 0)
        out, lse = run_q4((q, *case[1:]), 64, scale)
        assert_attn_close(out[live], ref, f"q * {f} out", ATOL)
        assert_attn_close(lse[live], ref_lse, f"q * {f} lse", ATOL)


@pytest.mark.parametrize("hq,hkv,d,group,bs,rows,window", [
    (1, 1, 128, 64, 16, 4, 0), (2, 1, 64, 32, 32, 2, 20), (8, 2, 128, 64, 16, 2, 0), (4, 1, 128, 128, 16, 4, 30),
    (16, 1, 128, 64, 16, 4, 0), (16, 1, 64, 64, 32, 4, 70), (4, 2, 96, 32, 16, 3, 9), (4, 2, 96, 32, 8, 3, 9),
    (8, 1, 256, 128, 16, 2, 0)])
def test_q4_a_nan_reaches_only_the_rows_that_see_it(hq, hkv, d, group, bs, rows, window):
    """K and V of the last token, and of the token that only the first row's window reaches, are NaN."""
    n = 150
    case = q4_case(23, [n, 40], hq, hkv, d, group, bs, [rows, rows])
    q, kc, vc, table, lens, cu = case
    bad = [n - 1] + ([n - rows - window + 1] if window else [])
    pages = row_bytes(d, group) * bs
    for pos in bad:
        blk, off = int(table[0, pos // bs]), pos % bs
        for cache in (kc, vc):
            page = cache.view(cache.shape[0], hkv, pages)[blk]
            at = bs * d // 2 + off * 4 * (d // group)
            page[:, at:at + 4 * (d // group)] = torch.tensor([0, 0, 0xff, 0x7f] * (d // group), dtype=torch.uint8)
    out, lse = run_q4(case, group, 0.1, window, decode=False, max_q=rows)
    live, ref, ref_lse = expect(case, group, 0.1, window)   # NaN parameters read as 0 there
    clean = [i for i in range(2 * rows) if i != rows - 1 and not (window and i == 0)]
    assert_attn_close(out[clean], ref[clean], "rows that do not see it", ATOL)
    assert_attn_close(lse[clean], ref_lse[clean], "lse", ATOL)
    assert torch.isnan(out[rows - 1]).all()
    if window:
        assert torch.isnan(out[0]).all()


@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (8, 1, 128), (64, 1, 128), (2, 1, 96)])
@pytest.mark.parametrize("scale", [0.0, -0.1])
def test_q4_scales_that_are_not_positive(hq, hkv, d, scale):
    """Keys past the end and before the window stay masked whatever the sign of the scale."""
    case = q4_case(29, [150, 1, 40], hq, hkv, d, 32 if d == 96 else 64, 16, [3, 1, 2])
    live, ref, ref_lse = expect(case, 32 if d == 96 else 64, scale, 37)
    out, lse = run_q4(case, 32 if d == 96 else 64, scale, 37, decode=False, max_q=3)
    assert_attn_close(out[live], ref, "out", ATOL)
    assert_attn_close(lse[live], ref_lse, "lse", ATOL)


def test_q4_workspace_too_small_is_refused():
    case = q4_case(3, [4000], 8, 1, 128, 64, 16)
    q, kc, vc, table, lens, _ = [dev(t) for t in case]
    out = torch.zeros_like(q)
    with pytest.raises(pkv.PkvError) as e:
        pkv.paged_attention_q4(out, q, kc, vc, table, lens, 0.1, 64, num_splits=8)
    assert e.value.status == 3
    with pytest.raises(ValueError, match="row_bytes"):
        pkv.paged_attention_q4(out, q, kc, vc, table, lens, 0.1, 32)


@pytest.mark.parametrize("hq,hkv,d,group,bs,max_q", [(2, 1, 64, 64, 16, 1), (40, 1, 64, 64, 16, 1), (2, 1, 96, 32, 16, 1),
                                                     (4, 1, 64, 32, 32, 3)])
def test_q4_more_sequences_than_a_block_scans(hq, hkv, d, group, bs, max_q):
    g = gen.generator(31)
    lens = torch.randint(0, 41, (1100,), generator=g).tolist()
    rows = [min(n, b % (max_q + 1)) for b, n in enumerate(lens)] if max_q > 1 else None
    case = q4_case(31, lens, hq, hkv, d, group, bs, rows)
    live, ref, ref_lse = expect(case, group, 0.1, 0)
    out, lse = run_q4(case, group, 0.1, decode=max_q == 1, max_q=max_q)
    assert_attn_close(out[live], ref, "out", ATOL)
    assert_attn_close(lse[live], ref_lse, "lse", ATOL)
    if max_q == 1:
        empty = [b for b, n in enumerate(lens) if n == 0]
        assert empty and torch.all(out[empty] == 0) and torch.all(torch.isneginf(lse[empty]))
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv", [(16, 2), (40, 1)])
def test_q4_pointers_aligned_to_their_elements_only(hq, hkv):
    """Caches 4 bytes and queries 8 bytes past an aligned address: another kernel, the same results."""
    d, group, bs = 128, 64, 16
    case = q4_case(17, [300, 1, 64], hq, hkv, d, group, bs)
    q, kc, vc, table, lens, cu = case
    live, ref, ref_lse = expect(case, group, 0.1, 0)

    def shifted(t, by):
        room = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        view = room[by:by + t.numel()].view(t.shape)
        view.copy_(t)
        return view
    out = torch.empty(q.shape, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    ws = torch.zeros(pkv.paged_attention_q4_workspace_bytes(3, 3, 1, hq, hkv, d, group, bs, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    for kk, vv, qq in ((shifted(kc, 4), dev(vc), dev(q)), (dev(kc), dev(vc), shifted(q, 2)), (shifted(kc, 12), shifted(vc, 4), dev(q))):
        pkv.paged_attention_q4(out, qq, kk, vv, dev(table), dev(lens), 0.1, group, lse=lse, workspace=ws)
        assert_attn_close(out[live], ref, "out", ATOL)
        assert_attn_close(lse[live], ref_lse, "lse", ATOL)
    for kk, qq in ((shifted(kc, 1), dev(q)), (dev(kc), shifted(q, 1))):
        with pytest.raises(pkv.PkvError, match="aligned"):
            pkv.paged_attention_q4(out, qq, kk, dev(vc), dev(table), dev(lens), 0.1, group, lse=lse, workspace=ws)


@pytest.mark.parametrize("hq,hkv,d,group,bs,rows,window", [
    (16, 8, 128, 64, 16, 1, 0), (64, 8, 128, 64, 16, 1, 0), (8, 8, 256, 128, 16, 1, 0), (32, 8, 96, 32, 16, 1, 70), (8, 8, 64, 64, 8, 2, 0),
    (16, 4, 128, 32, 32, 4, 0), (40, 4, 64, 64, 16, 1, 0), (64, 4, 128, 64, 16, 3, 100)])
def test_q4_shares_of_many_sequences(hq, hkv, d, group, bs, rows, window):
    """Tables much longer than the sequences and many of those: equal shares for every warp or block, which
    begin and end inside units."""
    g = gen.generator(61)
    lens = torch.randint(0, 400, (70 if hkv == 8 else 150,), generator=g).tolist()
    lens[3], lens[10], lens[-1] = 1, 2500, 700
    case = list(q4_case(61, lens, hq, hkv, d, group, bs, [min(rows, n) for n in lens] if rows > 1 else None))
    case[3] = torch.cat([case[3], torch.full((len(lens), 8000 // bs - case[3].shape[1]), -1, dtype=torch.int32)], 1)
    live, ref, ref_lse = expect(case, group, 0.1, window)
    out, lse = run_q4(case, group, 0.1, window, decode=rows == 1, max_q=rows)
    assert_attn_close(out[live], ref, "out", ATOL)
    assert_attn_close(lse[live], ref_lse, "lse", ATOL)
    again = run_q4(case, group, 0.1, window, decode=rows == 1, max_q=rows)
    assert torch.equal(out[live], again[0][live]) and torch.equal(lse[live], again[1][live])
    assert pkv.get_device_error() == 0


def test_q4_streams_and_a_workspace_used_in_turn():
    """Two streams with workspaces of their own at once; calls of different shapes one after the other in one."""
    shapes = [(16, 2, 128, 64, 16), (64, 1, 128, 128, 16), (8, 2, 64, 32, 16), (4, 2, 96, 32, 16)]
    cases = [q4_case(41 + i, [3000, 7, 129], hq, hkv, d, group, bs) for i, (hq, hkv, d, group, bs) in enumerate(shapes)]
    alone = [run_q4(c, s[3], 0.1) for c, s in zip(cases, shapes)]
    on_gpu = [[dev(t) for t in c] for c in cases]
    n = max(pkv.paged_attention_q4_workspace_bytes(3, 3, 1, *s, c[3].shape[1]) for c, s in zip(cases, shapes))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    got = []
    for turn in range(4):
        for stream, ws in zip(streams, spaces):
            with torch.cuda.stream(stream):
                for i, (q, kc, vc, table, lens, _) in enumerate(on_gpu):
                    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
                    pkv.paged_attention_q4(out, q, kc, vc, table, lens, 0.1, shapes[i][3], lse=lse, workspace=ws)
                    got.append((i, out, lse))
    torch.cuda.synchronize()
    for i, out, lse in got:
        assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])
    assert pkv.get_device_error() == 0


def test_q4_tensors_of_the_wrong_kind_are_refused():
    case = q4_case(3, [40], 8, 1, 128, 64, 16)
    q, kc, vc, table, lens, _ = [dev(t) for t in case]
    out, rows = torch.empty_like(q), torch.zeros(1, 1, 128, device="cuda")
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    wide = torch.zeros(1, 8, 256, device="cuda")[:, :, ::2]
    for error, match, call in (
            (TypeError, "q must be", lambda: pkv.paged_attention_q4(out, q.double(), kc, vc, table, lens, 0.1, 64)),
            (ValueError, "q must be contiguous", lambda: pkv.paged_attention_q4(out, wide, kc, vc, table, lens, 0.1, 64)),
            (TypeError, "lse must be", lambda: pkv.paged_attention_q4(out, q, kc, vc, table, lens, 0.1, 64, lse=slots)),
            (TypeError, "v_cache must be", lambda: pkv.decode_step_q4(out, q, rows, rows, slots, kc, None, table, lens, 0.1, 64)),
            (TypeError, "v_new must be", lambda: pkv.decode_step_q4(out, q, rows, rows.bfloat16(), slots, kc, vc, table, lens, 0.1, 64)),
            (ValueError, "context_lens must be on", lambda: pkv.paged_attention_q4(out, q, kc, vc, table, lens.cpu(), 0.1, 64)),
            (TypeError, "element type", lambda: pkv.kv_append_q4(rows.double(), rows.double(), kc, vc, slots, 64)),
            (ValueError, "shapes", lambda: pkv.kv_append_q4(rows, rows, kc, vc, slots[:0], 64)),
            (ValueError, "shapes", lambda: pkv.paged_attention_q4(out[:, :4], q, kc, vc, table, lens, 0.1, 64)),
            (TypeError, "slot_mapping must be", lambda: pkv.kv_gather_q4(rows, rows, kc, vc, slots.int(), 64))):
        with pytest.raises(error, match=match):
            call()


def test_q4_tensors_of_another_device_are_refused(monkeypatch):
    """On the host, before any launch: the current device is not the tensors'."""
    case = q4_case(3, [40], 8, 1, 128, 64, 16)
    q, kc, vc, table, lens, _ = [dev(t) for t in case]
    rows, slots = torch.zeros(1, 1, 128, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setattr(pkv._binding, "_current_device", lambda: 1)
    for call in (lambda: pkv.paged_attention_q4(torch.empty_like(q), q, kc, vc, table, lens, 0.1, 64),
                 lambda: pkv.decode_step_q4(torch.empty_like(q), q, rows, rows, slots, kc, vc, table, lens, 0.1, 64),
                 lambda: pkv.kv_append_q4(rows, rows, kc, vc, slots, 64), lambda: pkv.kv_gather_q4(rows, rows, kc, vc, slots, 64),
                 lambda: pkv.block_tables_extend(table, lens, one, one, one, one, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                                 slots, one, 16),
                 lambda: pkv.block_tables_release(table, None, one, one, one, one)):
        with pytest.raises(ValueError, match="device"):
            call()


# ----------------------------------------------------------------------- decode step

def run_step(case, k_new, v_new, slots, group, scale, window, num_splits, fused):
    q, kc, vc, table, lens, _ = case
    B, Hq, d = q.shape
    NB, Hkv, bs, _ = kc.shape
    gk, gv = dev(kc), dev(vc)
    out = torch.full((B, Hq, d), float("nan"), device="cuda")
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    n = pkv.paged_attention_q4_workspace_bytes(B, B, 1, Hq, Hkv, d, group, bs, table.shape[1], window, num_splits)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    kw = dict(window=window, lse=lse, num_splits=num_splits, workspace=ws)
    if fused:
        pkv.decode_step_q4(out, dev(q), dev(k_new), dev(v_new), dev(slots), gk, gv, dev(table), dev(lens), scale, group, **kw)
    else:
        pkv.kv_append_q4(dev(k_new), dev(v_new), gk, gv, dev(slots), group)
        pkv.paged_attention_q4(out, dev(q), gk, gv, dev(table), dev(lens), scale, group, **kw)
    torch.cuda.synchronize()
    return out, lse, gk.cpu(), gv.cpu()


@pytest.mark.parametrize("hq,hkv,d,group,bs", [(64, 8, 128, 64, 16), (8, 8, 128, 128, 16), (16, 2, 128, 32, 32),
                                               (8, 2, 64, 32, 16), (32, 2, 128, 64, 16), (64, 1, 128, 128, 16),
                                               (4, 2, 96, 32, 8), (8, 2, 96, 32, 16), (4, 2, 256, 64, 16),
                                               (16, 2, 192, 64, 32), (16, 2, 256, 128, 16), (10, 2, 160, 32, 16),
                                               (8, 1, 128, 64, 8), (4, 2, 128, 64, 24)])
@pytest.mark.parametrize("new_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("num_splits,window", [(0, 0), (1, 0), (3, 40)])
def test_q4_decode_step_equals_append_then_attention(hq, hkv, d, group, bs, new_dtype, num_splits, window):
    lens = [1, 16, 17, 700, 2049, 33, 5, 1000]
    case = q4_case(hq + bs + num_splits, lens, hq, hkv, d, group, bs)
    g = gen.generator(77)
    k_new, v_new = gen.randn(g, (8, hkv, d), new_dtype), gen.randn(g, (8, hkv, d), new_dtype)
    slots = torch.tensor([oracle.slot_of(case[3][b], n - 1, bs) for b, n in enumerate(lens)])
    slots[2] = -1                                     # sequence 2 has no new token this step
    scale = 1 / math.sqrt(d)
    out, lse, kc, vc = run_step(case, k_new, v_new, slots, group, scale, window, num_splits, True)
    assert pkv.get_device_error() == 0
    out2, lse2, kc2, vc2 = run_step(case, k_new, v_new, slots, group, scale, window, num_splits, False)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    want_k, want_v = case[1].clone(), case[2].clone()
    orc.kv_append_q4(want_k, want_v, k_new, v_new, slots, group)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    live, ref, ref_lse = expect((case[0], want_k, want_v, *case[3:]), group, scale, window)
    assert_attn_close(out[live], ref, "out", ATOL)
    assert_attn_close(lse[live], ref_lse, "lse", ATOL)


@pytest.mark.parametrize("hq,fused", [(8, True), (16, False)])
def test_q4_decode_step_slots_that_are_not_the_last_position(hq, fused):
    """Quantised in the attention launch: only the last position's slot is taken.  Else kv_append_q4's rules."""
    lens = [40, 20, 0, 33]
    d, group, bs, hkv = 128, 64, 16, 1
    case = q4_case(19, lens, hq, hkv, d, group, bs, poison=False)
    g = gen.generator(5)
    k_new, v_new = gen.randn(g, (4, hkv, d)), gen.randn(g, (4, hkv, d))
    slots = torch.tensor([oracle.slot_of(case[3][b], max(n, 1) - 1, bs) if n else -1 for b, n in enumerate(lens)])
    right = slots.clone()
    slots[1] = oracle.slot_of(case[3][1], 3, bs)      # a position before the last
    out, _, kc, vc = run_step(case, k_new, v_new, slots, group, 0.1, 0, 0, True)
    err = pkv.get_device_error()
    if fused:
        assert err == pkv.DEVERR["slot"]
        right[1] = -1
    else:
        assert err == 0
        right[1] = slots[1]
    want_k, want_v = case[1].clone(), case[2].clone()
    orc.kv_append_q4(want_k, want_v, k_new, v_new, right, group)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    live, ref, _ = expect((case[0], want_k, want_v, *case[3:]), group, 0.1, 0)
    assert_attn_close(out[live], ref, "out", ATOL)
    assert torch.all(out[2] == 0)
    slots[1], slots[2] = -1, 0                        # a new token of an empty sequence
    if fused:
        _, _, kc, _ = run_step(case, k_new, v_new, slots, group, 0.1, 0, 0, True)
        assert pkv.get_device_error() == pkv.DEVERR["slot"]


# ------------------------------------------------------------------ rows that a call refuses

REFUSALS = [  # hq, hkv, d, group, bs, window, num_splits: the kernel that attends, and how its parts meet
    (4, 1, 128, 64, 24, 24, 1), (4, 1, 128, 64, 24, 24, 3), (4, 1, 128, 64, 24, 0, 0), (2, 2, 224, 32, 16, 100, 0),   # CUDA cores
    (8, 1, 128, 64, 16, 0, 20), (4, 2, 96, 32, 8, 0, 20), (8, 1, 128, 64, 16, 0, 3), (8, 1, 128, 64, 16, 50, 0),      # warp MMAs
    (64, 1, 128, 64, 16, 0, 5), (64, 2, 64, 64, 16, 40, 0), (64, 1, 128, 128, 32, 0, 1)]                             # tcgen05


@pytest.mark.parametrize("hq,hkv,d,group,bs,window,splits", REFUSALS)
def test_q4_more_rows_than_max_q_are_flagged_on_every_path(hq, hkv, d, group, bs, window, splits):
    """Five rows where max_q says two: refused whichever kernel attends and whichever one merges."""
    case = q4_case(71, [500, 2000, 70, 33], hq, hkv, d, group, bs, [5, 2, 1, 0])
    q, kc, vc, table, lens, cu = case
    out, lse = run_q4(case, group, 0.1, window, splits, decode=False, max_q=2)
    assert pkv.get_device_error() == pkv.DEVERR["cu_seqlens"]
    assert torch.all(out[:5] == 0) and torch.all(torch.isneginf(lse[:5]))
    live, ref, ref_lse = expect((q[5:], kc, vc, table[1:], lens[1:], cu[1:] - 5), group, 0.1, window)
    assert_attn_close(out[5:], ref, "the other sequences", ATOL)
    assert_attn_close(lse[5:], ref_lse, "the other sequences' lse", ATOL)


@pytest.mark.parametrize("hq,hkv,d,group,bs,window,splits", REFUSALS)
@pytest.mark.parametrize("bounds", [(0, 2, 9), (-3, 2, 4)])
def test_q4_rows_outside_the_call_are_flagged_on_every_path(hq, hkv, d, group, bs, window, splits, bounds):
    """Offsets that leave [0, Tq]: that sequence's rows within the call are refused, the other's are not."""
    case = list(q4_case(73, [700, 2000], hq, hkv, d, group, bs, [2, 2]))
    q, kc, vc, table, lens, _ = case
    case[5] = torch.tensor(bounds, dtype=torch.int32)
    out, lse = run_q4(case, group, 0.1, window, splits, decode=False, max_q=8)
    assert pkv.get_device_error() == pkv.DEVERR["cu_seqlens"]
    good, bad = (0, 1) if bounds[0] == 0 else (1, 0)
    assert torch.all(out[2 * bad:2 * bad + 2] == 0) and torch.all(torch.isneginf(lse[2 * bad:2 * bad + 2]))
    at = slice(2 * good, 2 * good + 2)
    live, ref, ref_lse = expect((q[at], kc, vc, table[good:good + 1], lens[good:good + 1], torch.tensor([0, 2], dtype=torch.int32)),
                                group, 0.1, window)
    assert_attn_close(out[at], ref, "the good sequence", ATOL)
    assert_attn_close(lse[at], ref_lse, "the good sequence's lse", ATOL)


# ------------------------------------------------------------------------ scores of NaN

def poison_tokens(cache, table_row, positions, d, group, heads=slice(None)):
    """NaN zeros (scale 0) in the rows at these positions, as an append of NaN writes them."""
    nb, hkv, bs, _ = cache.shape
    for pos in positions:
        page = cache.view(nb, hkv, -1)[int(table_row[pos // bs])]
        at = bs * d // 2 + pos % bs * 4 * (d // group)
        page[heads, at:at + 4 * (d // group)] = torch.tensor([0, 0, 0xff, 0x7f] * (d // group), dtype=torch.uint8)


@pytest.mark.parametrize("hq,hkv,d,group,bs", [(8, 1, 128, 64, 16), (4, 1, 128, 64, 16), (64, 1, 128, 64, 16), (40, 1, 64, 64, 32),
                                               (4, 2, 96, 32, 16), (8, 1, 128, 32, 8), (3, 1, 224, 32, 16), (4, 1, 128, 128, 24)])
@pytest.mark.parametrize("many", [False, True])   # many: equal shares of a table much longer than the sequences
def test_q4_lse_of_scores_that_are_nan(hq, hkv, d, group, bs, many):
    """A row's lse is NaN exactly where a key that it sees is, whatever the split, as its out is; NaN in V
    alone leaves the lse as it is."""
    lens = [1, 600, 70, 33, 2, 300] + ([40] * 150 if many else [])
    case = list(q4_case(91, lens, hq, hkv, d, group, bs))
    q, kc, vc, table, clens, cu = case
    if many:
        case[3] = torch.cat([table, torch.full((len(lens), 16000 // bs - table.shape[1]), -1, dtype=torch.int32)], 1)
    live, ref, ref_lse = expect(case, group, 0.1, 0)
    bad = {0: range(1), 1: range(256), 3: range(33), 4: range(1, 2)}
    for b, positions in bad.items():
        poison_tokens(kc, table[b], positions, d, group)
    poison_tokens(vc, table[5], range(300), d, group)
    clean = [b for b in range(len(lens)) if b not in bad and b != 5]
    for splits in ((0,) if many else (0, 1, 3, 20)):
        out, lse = run_q4(case, group, 0.1, 0, splits)
        assert torch.isnan(out[list(bad)]).all() and torch.isnan(lse[list(bad)]).all()
        assert torch.isnan(out[5]).all()
        assert_attn_close(lse[5], ref_lse[5], "lse of clean keys", ATOL)
        assert_attn_close(out[clean], ref[clean], "clean rows", ATOL)
        assert_attn_close(lse[clean], ref_lse[clean], "clean rows' lse", ATOL)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,group,bs", [(2, 1, 64, 64, 16), (8, 1, 128, 64, 32), (40, 1, 64, 64, 16)])
def test_q4_equal_shares_of_as_many_sequences_as_a_block_scans(hq, hkv, d, group, bs):
    """1024 sequences: the scan fills its part of the shared memory that the page copies then use."""
    g = gen.generator(67)
    lens = torch.randint(0, 60, (1024,), generator=g).tolist()
    case = list(q4_case(67, lens, hq, hkv, d, group, bs))
    case[3] = torch.cat([case[3], torch.full((1024, 4096 // bs - case[3].shape[1]), -1, dtype=torch.int32)], 1)
    live, ref, ref_lse = expect(case, group, 0.1, 0)
    first = run_q4(case, group, 0.1)
    assert_attn_close(first[0][live], ref, "out", ATOL)
    assert_attn_close(first[1][live], ref_lse, "lse", ATOL)
    for _ in range(5):
        out, lse = run_q4(case, group, 0.1)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,group,bs", [(8, 1, 128, 64, 16), (4, 1, 128, 32, 16), (1, 1, 64, 32, 8), (64, 1, 128, 64, 16),
                                               (64, 1, 128, 128, 32), (5, 1, 224, 32, 16), (4, 1, 256, 64, 16)])
@pytest.mark.parametrize("sign", [-1, 0])   # all scales negative, or of either sign
def test_q4_caches_with_negative_scales(hq, hkv, d, group, bs, sign):
    """A cache from elsewhere: zero + scale * code with scales below 0, the same values ~ N(0, 1)."""
    case = list(q4_case(37, [300, 1, 64, 77], hq, hkv, d, group, bs, poison=False))
    g = gen.generator(38)
    for i in (1, 2):
        cache = case[i]
        nb = cache.shape[0]
        page = cache.view(nb, hkv, -1)
        par = page[:, :, bs * d // 2:].clone().view(torch.float16).view(nb, hkv, bs, d // group, 2)
        codes = page[:, :, :bs * d // 2].view(nb, hkv, bs, d // group, group // 2)
        flip = torch.ones(par.shape[:-1], dtype=torch.bool) if sign else torch.rand(par.shape[:-1], generator=g) < 0.5
        s, z = par[..., 0].float(), par[..., 1].float()
        par[..., 1] = torch.where(flip, z + 15 * s, z).half()          # code c becomes 15 - c
        par[..., 0] = torch.where(flip, -s, s).half()
        codes.copy_(torch.where(flip[..., None], 255 - codes, codes))
        page[:, :, bs * d // 2:] = par.reshape(nb, hkv, -1).view(torch.uint8)
    live, ref, ref_lse = expect(case, group, 1 / math.sqrt(d), 0)
    for splits in (0, 1, 3):
        out, lse = run_q4(case, group, 1 / math.sqrt(d), 0, splits)
        assert_attn_close(out[live], ref, f"splits {splits} out", ATOL)
        assert_attn_close(lse[live], ref_lse, f"splits {splits} lse", ATOL)


# ------------------------------------------------------------------------ values far from 1 and mixed

def scaled_case(kind, lens, hq, hkv, d, group, bs):
    """q4_case's inputs with K and V scaled by `kind`, and a scale that keeps the scores ~ N(0, 1)."""
    g = gen.generator(97)
    per_seq = [gen.blocks_needed(n, bs) for n in lens]
    nb = sum(per_seq) + 2
    table = gen.block_table_from_order(gen.permutation(g, nb), per_seq)
    k, v = gen.randn(g, (nb, hkv, bs, d)) + 0.5, gen.randn(g, (nb, hkv, bs, d))
    q = gen.randn(g, (len(lens), hq, d))
    fk, fv = torch.ones((nb, 1, bs, d)), torch.ones((nb, 1, bs, d))
    if kind in ("tiny", "huge"):
        fk *= 1e-5 if kind == "tiny" else 1e4
        fv *= 1e-5 if kind == "tiny" else 1e4
    elif kind == "one group":
        fk[..., :group] = fv[..., :group] = 1e4
    else:                                            # V grows, or falls, by 2^10 three fifths into every sequence
        for b, n in enumerate(lens):
            for pos in range(3 * n // 5, n):
                fv[int(table[b, pos // bs]), :, pos % bs] = 2.0 ** (10 if kind == "growing" else -10)
    scale = {"tiny": 1e5, "huge": 1e-4, "one group": 1e-4}.get(kind, 1.0) / math.sqrt(d)
    cu = torch.arange(len(lens) + 1, dtype=torch.int32)
    return (q, q4_cache(k * fk, group), q4_cache(v * fv, group), table, torch.tensor(lens, dtype=torch.int32), cu), scale


def bounds(case, group, scale, ref_lse):
    """Error bounds of out, by row, head and group, and of lse, by row and head.

    A score is off by ds = (d / 8 + 20) * 2^-24 * scale * sum |q| (|zero| + 15 |scale_t|) at most, of the key
    where that is largest (as ATOL above).  That moves lse by ds and out by 2 ds times the largest |value| A of
    its group; sums, exponentials and divisions in fp32 by 8e-6 of A (ATOL_MEAN's account).  A weight times
    scale, in two f16 parts, is kept to 2^-22 of it and to no less than half of f16's least step, 2^-25, in units
    where 1 stands for a weight of at least 2^-7 / (2 max scale) (the tcgen05 kernel's reference; 2^-14 on warp
    MMAs): with centred codes of at most 8, n keys and sum p = exp(lse - max score) that is
    n / sum p * 8 * 2^-25 * 2^-7 * 2 max scale = n / sum p * 2^-28 max scale."""
    q, kc, vc, table, lens, _ = case
    B, hq, d = q.shape
    nb, hkv, bs, _ = kc.shape
    m, G = hq // hkv, d // group
    kd, vd = orc.dequantize_q4(kc, d, group), orc.dequantize_q4(vc, d, group)
    par = [c.view(nb, hkv, -1)[:, :, bs * d // 2:].contiguous().view(torch.float16).view(nb, hkv, bs, G, 2).double().numpy()
           for c in (kc, vc)]
    out, lse = np.zeros((B, hq, d)), np.zeros((B, hq))
    for b in range(B):
        L = int(lens[b])
        at = [(int(table[b, p // bs]), p % bs) for p in range(L)]
        blk, off = np.array([x[0] for x in at]), np.array([x[1] for x in at])
        for h in range(hq):
            j, x = h // m, q[b, h].double().numpy()
            K, V = kd[blk, j, off], vd[blk, j, off]
            reach = (np.abs(par[0][blk, j, off][..., 1]) + 15 * np.abs(par[0][blk, j, off][..., 0])).repeat(group, -1)
            ds = (d / 8 + 20) * 2.0 ** -24 * scale * (reach * np.abs(x)).sum(-1).max()
            n_by_p = L / math.exp(ref_lse[b, h] - (K @ x * scale).max())
            A = np.abs(V).reshape(L, G, group).max((0, 2)).repeat(group)
            out[b, h] = (2 * ds + 8e-6) * A + n_by_p * 2.0 ** -28 * np.abs(par[1][blk, j, off][..., 0]).max()
            lse[b, h] = ds + 4e-6
    return out, lse


@pytest.mark.parametrize("hq,hkv,d,group,bs", [(8, 1, 128, 64, 16), (4, 1, 128, 32, 16), (1, 1, 64, 32, 8), (64, 1, 128, 64, 16),
                                               (64, 1, 128, 128, 32), (5, 1, 224, 32, 16), (4, 2, 256, 64, 16), (16, 2, 128, 64, 24)])
@pytest.mark.parametrize("kind", ["tiny", "huge", "growing", "falling", "one group"])
def test_q4_values_far_from_1_and_mixed(hq, hkv, d, group, bs, kind):
    """Every group as exact as its own values allow, beside groups and keys of other sizes."""
    case, scale = scaled_case(kind, [700, 1, 90, 2000], hq, hkv, d, group, bs)
    live, ref, ref_lse = expect(case, group, scale, 0)
    tol, lse_tol = bounds(case, group, scale, ref_lse)
    for splits in (0, 1, 3):
        out, lse = run_q4(case, group, scale, 0, splits)
        worst = np.abs(out.double().cpu().numpy() - ref) / tol
        assert worst.max() <= 1, f"splits {splits}: {worst.max():.2f} of the bound"
        worst = np.abs(lse.double().cpu().numpy() - ref_lse) / lse_tol
        assert worst.max() <= 1, f"splits {splits} lse: {worst.max():.2f} of the bound"


@pytest.mark.parametrize("hq,hkv,d,group,bs", [(8, 1, 128, 64, 16), (4, 1, 128, 32, 16), (1, 1, 64, 32, 8), (64, 1, 128, 64, 16),
                                               (64, 1, 64, 64, 32), (5, 1, 224, 32, 16), (4, 2, 256, 64, 16), (3, 1, 96, 32, 16)])
def test_q4_scores_keep_their_bits(hq, hkv, d, group, bs):
    """Queries with one element each: a score is one product, whatever the kernel adds up besides zeros.  Of
    scale * |q| (|zero| + 15 scale_t) it may lose 2^-22 to the two parts of q, 2^-23 to each of three cut-off
    sums of a tensor core, and 2^-24 to each of six roundings (scale, zero, their sums, the base-2 factor): 16 * 2^-24."""
    case = list(q4_case(59, [700, 3, 90, 1100], hq, hkv, d, group, bs))
    q, kc, vc, table, lens, cu = case
    at = torch.arange(hq * 4).view(4, hq) * 37 % d
    x = torch.where(torch.arange(d) == at[..., None], torch.linspace(-3.7, 4.1, hq * 4).view(4, hq, 1), 0.0)
    case[0] = x
    live, ref, ref_lse = expect(case, group, 1.0, 0)
    kd, vd = (np.nan_to_num(orc.dequantize_q4(c, d, group)) for c in (kc, vc))
    ds = 16 * 2.0 ** -24 * x.abs().amax(-1).double().numpy() * 2 * np.abs(kd).max()     # |zero| + 15 scale_t: twice the largest
    for splits in (0, 1, 3):
        out, lse = run_q4(case, group, 1.0, 0, splits)
        assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse) <= ds + 4e-6)
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= (2 * ds[..., None] + 8e-6) * np.abs(vd).max())
