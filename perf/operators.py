"""What the operators of the 4-bit paged cache and of the GPU-built block tables cost: the cases that are
measured, their plain torch forms, and their values in 64 bits.

The 4-bit cache holds K and V as uint8 [NB][Hkv][bs][row], row = d/2 + 4*G bytes with G = d/group: the
bs*row bytes of one (block, head) page are the codes [bs][d/2] (byte j: element 2j in the low nibble, 2j+1
in the high one), then the parameters [bs][G][2] in fp16 (scale, zero).  A group of `group` elements x,
clamped to +-65504, is stored as
    zero = fp16 rounded down (min x),  scale = fp16 ((max x - zero) / 15),
    code = round half to even ((x - zero) / scale) clamped to 0..15  (0 where scale is 0),
each from the exact quotient with one rounding; the value it stands for is zero + scale * code.

Kinds of case:
  append   new rows quantised into their slots, then the same slots read back as values
  gather   the values of a cached prefix read out row by row
  attend   attention of the newest row(s) of every sequence over the cache (out and log-sum-exp)
  step     a decode step: the new token of every sequence quantised into its slot, then attended
  extend   blocks handed out, block tables, slot map and lengths of a step, from the request lengths
  cycle    extend, then the blocks of that step given back
"""
import math

import numpy as np
import torch

own = False

MAX = 65504.0
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # two short requests with fp32 rows, head size 64: the smallest step, launch latency
        dict(name="step_tiny", kind="step", B=2, hq=8, hkv=2, d=64, group=64, bs=16, lo=18, hi=41, window=0, new="fp32"),
        # a 70B-shaped grouped-query layer, ragged lengths: the ordinary decode step
        dict(name="step_gqa", kind="step", B=64, hq=64, hkv=8, d=128, group=64, bs=16, lo=513, hi=8193, window=0, new="bf16"),
        # a 7B-shaped layer with a KV head for every query head, one scale per row
        dict(name="step_mha", kind="step", B=32, hq=32, hkv=32, d=128, group=128, bs=16, lo=2049, hi=2049, window=0, new="bf16"),
        # sliding-window decode: 16384 tokens cached, the last 4096 seen, blocks of 32, the finest groups
        dict(name="attend_window", kind="attend", B=64, hq=32, hkv=8, d=128, group=32, bs=32, lo=16384, hi=16384, window=4096, rows=1),
        # very long contexts, few sequences: the split over keys
        dict(name="attend_long_gqa", kind="attend", B=4, hq=64, hkv=8, d=128, group=64, bs=16, lo=131072, hi=131072, window=0, rows=1),
        # one KV head for all 64 query heads
        dict(name="attend_long_mqa", kind="attend", B=4, hq=64, hkv=1, d=128, group=128, bs=16, lo=131072, hi=131072, window=0, rows=1),
        # up to four proposed tokens of each sequence checked at once
        dict(name="attend_verify", kind="attend", B=64, hq=64, hkv=8, d=128, group=64, bs=16, lo=512, hi=8192, window=0, rows=4),
        # eight prompts' rows into the cache and read back, 64-element groups
        dict(name="append_prompts", kind="append", T=17153, hkv=8, d=128, group=64, bs=16, new="bf16", skip=0),
        # a few fp32 rows of head size 96 with padding tokens among them
        dict(name="append_odd", kind="append", T=37, hkv=3, d=96, group=32, bs=8, new="fp32", skip=5),
        # a cached prefix of 8 x 4096 tokens read out in bf16
        dict(name="gather_prefix", kind="gather", T=32768, hkv=8, d=128, group=128, bs=16, new="bf16", skip=0),
        # one token more for each of 256 running requests
        dict(name="extend_decode", kind="extend", B=256, bs=16, lo=16, hi=32768, nlo=1, nhi=1),
        # prompts admitted and finished: their tables and slots, then the blocks given back
        dict(name="cycle_prompts", kind="cycle", B=8, bs=16, lo=0, hi=0, nlo=256, nhi=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "gather", "attend", "attend", "step", "step", "extend", "cycle"])
    if kind in ("extend", "cycle"):
        nhi = _log(rng, 1, 2048) if kind == "cycle" or rng.random() < 0.5 else 1
        B = _log(rng, 1, 1500 if nhi < 8 else 32)
        return dict(kind=kind, B=B, bs=rng.choice([8, 16, 32]), lo=0, hi=_log(rng, 1, 20000),
                    nlo=rng.choice([0, 1]) if B >= 8 else 1, nhi=nhi)
    fast = rng.random() < 0.8          # the head sizes that models have; else odd ones, on smaller problems
    d = rng.choice([64, 128, 128]) if fast else rng.choice([32, 96, 160, 256])
    group = rng.choice([g for g in (32, 64, 128) if d % g == 0])
    hkv = rng.choice([1, 2, 3, 8]) if fast else rng.choice([1, 2])
    bs = rng.choice([16, 32]) if fast else rng.choice([8, 16, 24])
    if kind in ("append", "gather"):
        return dict(kind=kind, T=_log(rng, 1, 16000 // hkv), hkv=hkv, d=d, group=group, bs=bs,
                    new=rng.choice(["bf16", "fp32"]), skip=rng.choice([0, 0, 3, 7]))
    m = rng.choice([1, 3, 4, 8, 16]) if fast else rng.choice([1, 2, 5])
    B = _log(rng, 1, 48 if fast else 6)
    hi = max(2, _log(rng, 8, 200000 // B if fast else 2000))
    case = dict(kind=kind, B=B, hq=m * hkv, hkv=hkv, d=d, group=group, bs=bs, lo=rng.randint(1, hi), hi=hi,
                window=rng.choice([0, 0, 0, rng.randint(1, 2 * hi)]))
    if kind == "step":
        case["new"] = rng.choice(["bf16", "bf16", "fp32"])
    else:
        case["rows"] = rng.choice([1, 1, 1, 2, 5])
    return case


# ------------------------------------------------------------------------------------------ the plain forms

def _parts(cache, d, group):
    """Views of the codes [NB][Hkv][bs][d/2] and the parameters [NB][Hkv][bs][G][2] of a cache."""
    nb, hkv, bs, row = cache.shape
    page = cache.view(nb, hkv, bs * row)
    codes = page[:, :, :bs * d // 2].unflatten(2, (bs, d // 2))
    par = page[:, :, bs * d // 2:].view(torch.float16).unflatten(2, (bs, d // group, 2))
    return codes, par


def _half_down(x):
    """fp16 at most x (x double, exact in fp32)."""
    h = x.to(torch.float16)
    bits = h.view(torch.int16).int()
    lower = torch.where(bits > 0, bits - 1, torch.where(bits == 0, torch.full_like(bits, -32767), bits + 1))
    return torch.where(h.double() > x, lower.to(torch.int16).view(torch.float16), h)


def _half_nearest(x):
    """fp16 nearest to x >= 0 (double), ties to even, one rounding."""
    e = torch.frexp(x)[1] - 1
    q = torch.exp2(torch.clamp(e, min=-14).double() - 10)
    return (torch.round(x / q) * q).to(torch.float16)


def _quantise(x, group):
    """Packed codes [..., d/2] and parameters [..., G, 2]; in 64 bits, as quotients next to a half decide codes."""
    x = x.double().clamp(-MAX, MAX).unflatten(-1, (-1, group))
    zero = _half_down(x.amin(-1))
    scale = _half_nearest((x.amax(-1) - zero.double()) / 15)
    s = scale.double()[..., None]
    t = torch.round((x - zero.double()[..., None]) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, 15)
    c = torch.where(s > 0, t, torch.zeros_like(t)).flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([scale, zero], -1)


def _values(codes, par):
    """The values (fp32) of packed codes [..., d/2] with parameters [..., G, 2]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    p = par.float()
    c = c.unflatten(-1, (p.shape[-2], -1))
    return (p[..., 1:] + p[..., :1] * c).flatten(-2)


def _scatter(cache, new, slots, d, group):
    codes, par = _parts(cache, d, group)
    c, p = _quantise(new, group)
    keep = slots >= 0
    s = slots[keep]
    bs = cache.shape[2]
    codes[s // bs, :, s % bs] = c[keep]
    par[s // bs, :, s % bs] = p[keep]


def _read(cache, slots, d, group, dtype):
    codes, par = _parts(cache, d, group)
    bs = cache.shape[2]
    s = slots.clamp(min=0)
    v = _values(codes[s // bs, :, s % bs], par[s // bs, :, s % bs])
    return torch.where(slots[:, None, None] >= 0, v, torch.zeros_like(v)).to(dtype)


def _plain_attention(s):
    c = s["case"]
    hq, hkv, d, group, bs, W = c["hq"], c["hkv"], c["d"], c["group"], c["bs"], c["window"]
    q = s["q"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device)
    kc, kp = _parts(s["k"], d, group)
    vc, vp = _parts(s["v"], d, group)
    for b, L in enumerate(s["lens_host"]):
        r0, r1 = s["cu_host"][b], s["cu_host"][b + 1]
        nq = r1 - r0
        if L == 0 or nq == 0:
            continue
        t0 = max(0, L - nq + 1 - W) if W > 0 else 0
        blk = s["table"][b, t0 // bs:(L + bs - 1) // bs].long()
        t0 = t0 // bs * bs
        K = _values(kc[blk], kp[blk]).transpose(0, 1).flatten(1, 2)[:, :L - t0]      # [Hkv][keys][d]
        V = _values(vc[blk], vp[blk]).transpose(0, 1).flatten(1, 2)[:, :L - t0]
        x = q[r0:r1].view(nq, hkv, hq // hkv, d).permute(1, 0, 2, 3).flatten(1, 2)    # [Hkv][nq*m][d]
        sc = torch.matmul(x, K.transpose(1, 2)) * s["scale"]
        if nq > 1 or W > 0:
            key = torch.arange(t0, L, device=q.device)
            pos = torch.arange(L - nq, L, device=q.device).repeat_interleave(hq // hkv)[:, None]
            seen = key <= pos
            if W > 0:
                seen &= key > pos - W
            sc = sc.masked_fill(~seen, -math.inf)
        top = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, V) / total
        out[r0:r1] = o.view(hkv, nq, hq // hkv, d).permute(1, 0, 2, 3).reshape(nq, hq, d)
        lse[r0:r1] = (top + torch.log(total)).view(hkv, nq, hq // hkv).permute(1, 0, 2).reshape(nq, hq)
    return out, lse


def _plain_extend(s):
    c = s["case"]
    bs, T = c["bs"], s["T"]
    L, n = s["lens"].long(), s["new_tokens"].long()
    have, want = (L + bs - 1) // bs, (L + n + bs - 1) // bs
    need = want - have
    end = torch.cumsum(need, 0)
    i = torch.arange(s["needed"], device=L.device)
    row = torch.searchsorted(end, i, right=True)
    table = s["table"]
    table[row, have[row] + i - (end - need)[row]] = s["free_list"][s["free_count"].long() - 1 - i]
    cu = torch.cat([torch.zeros_like(L[:1]), torch.cumsum(n, 0)])
    t = torch.arange(T, device=L.device)
    row = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = L[row] + t - cu[row]
    slots = table[row, pos // bs].long() * bs + pos % bs
    return table, (L + n).int(), cu.int(), slots, (s["free_count"] - end[-1]).int(), want


def _plain_release(s, count, first, end):
    table, bs = s["table"], s["case"]["bs"]
    col = torch.arange(table.shape[1], device=table.device)
    mine = (col >= first[:, None]) & (col < end[:, None])
    blocks = table[mine]
    new = (count + blocks.numel()).int()
    s["free_list"][new.long() - 1 - torch.arange(blocks.numel(), device=table.device)] = blocks
    table[mine] = -1
    return new


# ---------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    """N(0, 1) rows with some channels off centre, as keys have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    x += 0.5 * torch.randn(shape[-1:], generator=g, device="cuda").clamp(min=0)
    return x.to(dtype)


def _fill(g, cache, d, group):
    """Every slot of a cache holds a quantised random row."""
    codes, par = _parts(cache, d, group)
    step = max(1, (1 << 25) // (cache.shape[1] * cache.shape[2] * d))
    for b in range(0, cache.shape[0], step):
        n = min(step, cache.shape[0] - b)
        x = _randn(g, (n, cache.shape[1], cache.shape[2], d // group, group), torch.float32)
        zero = x.amin(-1).half() - 0.01
        scale = ((x.amax(-1) - zero.float()) / 15).half()
        c = torch.round((x - zero.float()[..., None]) / scale.float()[..., None]).clamp(0, 15).flatten(-2).to(torch.uint8)
        codes[b:b + n] = c[..., 0::2] | (c[..., 1::2] << 4)
        par[b:b + n] = torch.stack([scale, zero], -1)


def _cache(nb, c):
    row = c["d"] // 2 + 4 * (c["d"] // c["group"])
    return torch.zeros((nb, c["hkv"], c["bs"], row), dtype=torch.uint8, device="cuda")


def _sizes(case, r, *ranges):
    """One whole number from each (lo, hi) for every row: a case has the same ones for every seed, in another order."""
    base = np.random.default_rng(case["B"])
    drawn = [base.integers(lo, hi + 1, case["B"]) for lo, hi in ranges]
    order = r.permutation(case["B"])
    return [x[order] for x in drawn]


def prepare(case, seed):
    g = _gen(seed)
    r = np.random.default_rng(seed)
    s = {"case": case}
    bs = case["bs"]
    if case["kind"] in ("extend", "cycle"):
        B = case["B"]
        L, n = _sizes(case, r, (case["lo"], case["hi"]), (case["nlo"], case["nhi"]))
        have, want = -(-L // bs), -(-(L + n) // bs)
        nb = int(want.sum()) + 61
        order = r.permutation(nb).astype(np.int32)
        table = np.full((B, int(want.max(initial=1)) + 2), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :have[b]] = order[at:at + have[b]]
            at += int(have[b])
        free = np.zeros(nb, np.int32)
        free[:nb - at] = order[at:]
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        s.update(table=dev(table), lens=dev(L.astype(np.int32)), new_tokens=dev(n.astype(np.int32)), free_list=dev(free),
                 free_count=dev(np.array([nb - at], np.int32)), T=int(n.sum()), needed=int((want - have).sum()), nb=nb)
        if own:
            import paged_kv_cache_165_gb300 as pkv
            ws = max(pkv.block_tables_extend_workspace_bytes(B, s["T"]), pkv.block_tables_release_workspace_bytes(B))
            both = torch.stack([s["lens"], s["lens"]])   # the lengths before and after, next to each other
            blocks = torch.empty_like(both)
            s.update(both=both, lens=both[0], lens_out=both[1], blocks=blocks, first=blocks[0], end=blocks[1],
                     cu=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                     slots=torch.empty(s["T"], dtype=torch.int64, device="cuda"), count1=torch.empty_like(s["free_count"]),
                     count2=torch.empty_like(s["free_count"]), ws=torch.zeros(max(16, ws), dtype=torch.uint8, device="cuda"))
        return s
    d, group, hkv = case["d"], case["group"], case["hkv"]
    if case["kind"] in ("append", "gather"):
        T = case["T"]
        nb = -(-T // bs) + 2
        slots = (r.permutation(nb)[:-(-T // bs), None] * bs + np.arange(bs)).reshape(-1)[:T].astype(np.int64)
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1
        s.update(slots=torch.from_numpy(slots).cuda(), k=_cache(nb, case), v=_cache(nb, case))
        if case["kind"] == "append":
            s.update(k_new=_randn(g, (T, hkv, d), DT[case["new"]]), v_new=_randn(g, (T, hkv, d), DT[case["new"]]))
        else:
            _fill(g, s["k"], d, group)
            _fill(g, s["v"], d, group)
        s.update(k_out=torch.empty((T, hkv, d), dtype=DT[case["new"]], device="cuda"),
                 v_out=torch.empty((T, hkv, d), dtype=DT[case["new"]], device="cuda"))
        return s
    B, hq, W = case["B"], case["hq"], case["window"]
    rows = case.get("rows", 1)
    lens, nq = _sizes(case, r, (case["lo"], case["hi"]), (1, rows))
    nq = np.minimum(nq, lens)
    blocks = -(-lens // bs)
    nb = int(blocks.sum()) + 3
    order = r.permutation(nb).astype(np.int32)
    table = np.full((B, max(1, int(blocks.max()))), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = order[at:at + blocks[b]]
        at += int(blocks[b])
    cu = np.concatenate([[0], np.cumsum(nq)])
    s.update(k=_cache(nb, case), v=_cache(nb, case), table=torch.from_numpy(table).cuda(),
             lens=torch.from_numpy(lens.astype(np.int32)).cuda(), lens_host=lens.tolist(), cu_host=cu.tolist(),
             cu=torch.from_numpy(cu.astype(np.int32)).cuda(), scale=1 / math.sqrt(d), rows=rows,
             q=torch.randn((int(cu[-1]), hq, d), generator=g, device="cuda"))
    _fill(g, s["k"], d, group)
    _fill(g, s["v"], d, group)
    if case["kind"] == "step":
        last = lens - 1
        slots = table[np.arange(B), last // bs].astype(np.int64) * bs + last % bs
        s.update(slots=torch.from_numpy(slots).cuda(), k_new=_randn(g, (B, hkv, d), DT[case["new"]]),
                 v_new=_randn(g, (B, hkv, d), DT[case["new"]]))
        s.update(k_out=torch.empty_like(s["k_new"]), v_out=torch.empty_like(s["v_new"]))
    s.update(out=torch.empty_like(s["q"]), lse=torch.empty(s["q"].shape[:2], device="cuda"))
    if own:
        import paged_kv_cache_165_gb300 as pkv
        n = pkv.paged_attention_q4_workspace_bytes(B, int(cu[-1]), rows, hq, hkv, d, group, bs, table.shape[1], W)
        s["ws"] = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------- one pass

def _run_plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind in ("extend", "cycle"):
        table, lens, cu, slots, count, want = _plain_extend(s)
        got = dict(lens=lens, cu=cu, slots=slots, count=count)
        if kind == "cycle":
            have = (s["lens"].long() + c["bs"] - 1) // c["bs"]
            got["count_back"] = _plain_release(s, count, have, want)
            got["free_list"] = s["free_list"]
        got["table"] = table
        return got
    d, group = c["d"], c["group"]
    if kind in ("append", "step"):
        _scatter(s["k"], s["k_new"], s["slots"], d, group)
        _scatter(s["v"], s["v_new"], s["slots"], d, group)
    got = {}
    if kind in ("attend", "step"):
        got["out"], got["lse"] = _plain_attention(s)
    if kind != "attend":
        got["k"] = _read(s["k"], s["slots"], d, group, s["k_out"].dtype)
        got["v"] = _read(s["v"], s["slots"], d, group, s["v_out"].dtype)
    return got


def _run_own(s):
    import paged_kv_cache_165_gb300 as pkv
    c = s["case"]
    kind = c["kind"]
    if kind in ("extend", "cycle"):
        pkv.block_tables_extend(s["table"], s["lens"], s["new_tokens"], s["free_list"], s["free_count"], s["lens_out"],
                                s["cu"], s["slots"], s["count1"], c["bs"], workspace=s["ws"])
        got = dict(lens=s["lens_out"], cu=s["cu"], slots=s["slots"], count=s["count1"])
        if kind == "cycle":
            # the blocks that the tokens took: ceil(length / bs) before and after, of lengths that the GPU holds
            torch.add(s["both"], c["bs"] - 1, out=s["blocks"]).floor_divide_(c["bs"])
            pkv.block_tables_release(s["table"], s["first"], s["end"], s["free_list"], s["count1"], s["count2"],
                                     workspace=s["ws"])
            got["count_back"] = s["count2"]
            got["free_list"] = s["free_list"]
        got["table"] = s["table"]
        return got
    group = c["group"]
    got = {}
    if kind == "append":
        pkv.kv_append_q4(s["k_new"], s["v_new"], s["k"], s["v"], s["slots"], group)
    elif kind == "attend":
        pkv.paged_attention_q4(s["out"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], group,
                               cu_q=s["cu"] if s["rows"] > 1 else None, max_q=s["rows"], window=c["window"], lse=s["lse"],
                               workspace=s["ws"])
    elif kind == "step":
        pkv.decode_step_q4(s["out"], s["q"], s["k_new"], s["v_new"], s["slots"], s["k"], s["v"], s["table"], s["lens"],
                           s["scale"], group, window=c["window"], lse=s["lse"], workspace=s["ws"])
    if kind in ("attend", "step"):
        got["out"], got["lse"] = s["out"], s["lse"]
    if kind != "attend":
        pkv.kv_gather_q4(s["k_out"], s["v_out"], s["k"], s["v"], s["slots"], group)
        got["k"], got["v"] = s["k_out"], s["v_out"]
    return got


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------- the least work of a pass

def work(case):
    bs = case["bs"]
    if case["kind"] in ("extend", "cycle"):
        n = case["B"] * (case["nlo"] + case["nhi"]) / 2
        blocks = n / bs
        # lengths, counts and offsets of the rows; a slot for each token; a block id read and written for each block
        total = case["B"] * 16 + 8 * n + 8 * blocks * (2 if case["kind"] == "cycle" else 1)
        return {"bytes": int(total), "flops": 0}
    d, hkv = case["d"], case["hkv"]
    row = d // 2 + 4 * (d // case["group"])
    if case["kind"] in ("append", "gather"):
        e = 2 if case["new"] == "bf16" else 4
        once = 2 * hkv * case["T"] * (row + e * d)
        return {"bytes": int(once * (2 if case["kind"] == "append" else 1) + 8 * case["T"]),
                "flops": 2 * 6 * hkv * case["T"] * d}
    B, hq, W = case["B"], case["hq"], case["window"]
    rows = (1 + case.get("rows", 1)) / 2
    mean = (case["lo"] + case["hi"]) / 2
    seen = min(mean, W) if W > 0 else mean
    total = B * seen * hkv * 2 * row + B * seen / bs * 4 + B * rows * hq * (8 * d + 4)
    if case["kind"] == "step":
        total += 2 * B * hkv * 2 * d * (2 if case["new"] == "bf16" else 4)
    return {"bytes": int(total), "flops": int(4 * B * rows * hq * seen * d)}


# ------------------------------------------------------------------------------------------- values in 64 bits

def _exact_rows(x, group):
    """Codes, scales and zeros of rows [..., d] from their definition, in numpy's 64 bits."""
    x = np.clip(x.float().cpu().numpy().astype(np.float64), -MAX, MAX)
    x = x.reshape(*x.shape[:-1], -1, group)
    lo = x.min(-1)
    zero = lo.astype(np.float16)
    zero = np.where(zero.astype(np.float64) > lo, np.nextafter(zero, np.float16(-np.inf)), zero).astype(np.float64)
    scale = ((x.max(-1) - zero) / 15).astype(np.float16).astype(np.float64)
    s = np.where(scale > 0, scale, 1.0)[..., None]
    code = np.where(scale[..., None] > 0, np.clip(np.rint((x - zero[..., None]) / s), 0, 15), 0.0)
    return (zero[..., None] + scale[..., None] * code).reshape(*x.shape[:-2], -1)


def _exact_table(case, cache):
    """The values of a whole cache's pages, in 64 bits: a function from block ids to [n][Hkv][bs][d]."""
    nb, hkv, bs, row = cache.shape
    d, G = case["d"], case["d"] // case["group"]
    flat = cache.reshape(nb, hkv, bs * row)
    nibble = torch.tensor([[c % 16, c // 16] for c in range(256)], dtype=torch.float64, device=cache.device)

    def pages(ids):
        p = flat[ids]
        code = nibble[p[..., :bs * d // 2].int()].reshape(len(ids), hkv, bs, G, case["group"])
        par = p[..., bs * d // 2:].contiguous().view(torch.float16).double().reshape(len(ids), hkv, bs, G, 2)
        return (code * par[..., 0:1] + par[..., 1:2]).reshape(len(ids), hkv, bs, d)
    return pages


def _exact_attention(s, kv):
    """kv(b, head, t0, t1): K and V rows of a sequence's positions, in 64 bits."""
    c = s["case"]
    m = c["hq"] // c["hkv"]
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, L in enumerate(s["lens_host"]):
        r0, nq = s["cu_host"][b], s["cu_host"][b + 1] - s["cu_host"][b]
        if L == 0:
            continue
        for h in range(c["hkv"]):
            lowest = max(0, L - nq + 1 - c["window"]) if c["window"] else 0
            K, V = kv(b, h, lowest, L)
            for i in range(nq):
                end = L - nq + i + 1
                begin = max(0, end - c["window"]) if c["window"] else 0
                k, v = K[begin - lowest:end - lowest], V[begin - lowest:end - lowest]
                z = s["q"][r0 + i, h * m:(h + 1) * m].double() @ k.T * s["scale"]
                l = torch.logsumexp(z, 1)
                lse[r0 + i, h * m:(h + 1) * m] = l
                out[r0 + i, h * m:(h + 1) * m] = torch.exp(z - l[:, None]) @ v
    return out, lse


def _exact_extend(s):
    c, bs = s["case"], s["case"]["bs"]
    table, L, n = s["table"].cpu().numpy().astype(np.int64), s["lens"].tolist(), s["new_tokens"].tolist()
    free = s["free_list"].cpu().numpy().astype(np.int64)
    count = int(s["free_count"])
    taken, cu, slots = [], [0], []
    for b in range(c["B"]):
        for j in range(-(-L[b] // bs), -(-(L[b] + n[b]) // bs)):
            count -= 1
            table[b, j] = free[count]
            taken.append((b, j))
        for p in range(L[b], L[b] + n[b]):
            slots.append(table[b, p // bs] * bs + p % bs)
        cu.append(cu[-1] + n[b])
    got = dict(lens=np.array(L) + np.array(n), cu=np.array(cu), slots=np.array(slots, np.int64), count=np.array([count]))
    if c["kind"] == "cycle":
        for b, j in reversed(taken):
            free[count] = table[b, j]
            table[b, j] = -1
            count += 1
        got["count_back"], got["free_list"] = np.array([count]), free
    got["table"] = table
    return got


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("extend", "cycle"):
        return _exact_extend(s)
    keep = (s["slots"] >= 0).cpu().numpy()[:, None, None] if kind != "attend" else None
    if kind == "append":
        return {x: np.where(keep, _exact_rows(s[x + "_new"], case["group"]), 0.0) for x in ("k", "v")}
    if kind == "gather":
        slots = s["slots"].clamp(min=0)
        got = {}
        for x in ("k", "v"):
            v = _exact_table(case, s[x])(torch.arange(s[x].shape[0], device="cuda"))
            got[x] = np.where(keep, v[slots // case["bs"], :, slots % case["bs"]].cpu().numpy(), 0.0)
        return got
    if case["B"] * case["hkv"] * case.get("rows", 1) * 2 > 4096:
        return None
    pages = [_exact_table(case, s[x]) for x in ("k", "v")]
    new = {x: torch.from_numpy(_exact_rows(s[x + "_new"], case["group"])).cuda() for x in ("k", "v")} if kind == "step" else None
    held = [None, None]

    def kv(b, h, t0, t1):
        if held[0] != b:
            bs = case["bs"]
            rows = []
            for x, p in zip("kv", pages):
                v = p(s["table"][b, t0 // bs:-(-t1 // bs)].long()).transpose(0, 1).flatten(1, 2)
                v = v[:, t0 % bs:t0 % bs + t1 - t0].clone()
                if new is not None:
                    v[:, -1] = new[x][b]
                rows.append(v)
            held[:] = [b, rows]
        return held[1][0][h], held[1][1][h]

    out, lse = _exact_attention(s, kv)
    got = dict(out=out.cpu().numpy(), lse=lse.cpu().numpy())
    if kind == "step":
        got["k"], got["v"] = new["k"].cpu().numpy(), new["v"].cpu().numpy()
    return got
