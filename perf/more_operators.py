"""What the operators of a serving loop around the paged attention cost: the cases that are measured, their
plain torch forms, and their values in 64 bits.

Kinds of case:
  rope     rotary positions: q rotated into fp32 or bf16, K rotated and K, V written into their cache slots
           (to = "cache"), or q and K rotated into rows, forwards or backwards (to = "rows").  The pair (a, b) of
           dimension pair j at position p becomes mscale * (a cos - b sin, a sin + b cos) of the angle p * f_j;
           pairs are (2j, 2j + 1) (inter) or (j, j + rot/2); dimensions from rot on are left as they are.
  sinks    attention of the newest row(s) of every sequence: the row at position p sees the keys t <= p with
           t < sinks or t > p - window (out and log-sum-exp)
  verify   drafted tokens accepted while u * q(x) < p(x); at the first rejection a token from max(p - q, 0),
           after k acceptances one from p: the lowest v whose cumulative sum exceeds u * total
  fork     rows take the sequence of their parent row: whole blocks shared, a last block that is partly filled
           and shared copied, references counted, blocks without any free, lowest ids handed out first
  compact  the blocks in use moved to the lowest ids, tables and free list to match
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the decode step of a 70B-shaped grouped-query layer: one token of 64 sequences, packed q, k, v rows
        dict(name="rope_step", kind="rope", T=64, hq=64, hkv=8, d=128, rot=128, inter=False, new="bf16", qout="fp32", bs=16,
             far=8192, skip=0, packed=True, to="cache", scaling="none", inverse=False),
        # eight prompts of that layer, contexts extended eightfold by parts
        dict(name="rope_prompts", kind="rope", T=17153, hq=64, hkv=8, d=128, rot=128, inter=False, new="bf16", qout="bf16", bs=16,
             far=131072, skip=0, packed=True, to="cache", scaling="parts", inverse=False),
        # the gradient of fp32 rows with a third of the head rotated in neighbouring pairs, ragged count
        dict(name="rope_back_odd", kind="rope", T=1037, hq=12, hkv=3, d=96, rot=32, inter=True, new="fp32", qout="fp32", bs=8,
             far=4096, skip=0, packed=False, to="rows", scaling="linear", inverse=True),
        # two short requests in fp32, a window inside the sequence: launch latency
        dict(name="sinks_tiny", kind="sinks", B=2, hq=8, hkv=2, d=64, bs=16, new="fp32", lo=18, hi=41, window=12, sinks=3, rows=1),
        # sliding-window decode: 16384 tokens cached, the last 4096 and the first 4 seen
        dict(name="sinks_window", kind="sinks", B=64, hq=32, hkv=8, d=128, bs=16, new="bf16", lo=16385, hi=16385, window=4096, sinks=4, rows=1),
        # up to four drafted tokens of each sequence checked at once, ragged lengths around the window
        dict(name="sinks_verify", kind="sinks", B=64, hq=64, hkv=8, d=128, bs=16, new="bf16", lo=512, hi=8192, window=2048, sinks=16, rows=4),
        # one request, five drafts at most, an odd vocabulary: latency
        dict(name="verify_one", kind="verify", B=1, V=50001, k=5, new="fp32", drafted="probs"),
        # a batch of requests with four drafts at most
        dict(name="verify_batch", kind="verify", B=64, V=131072, k=4, new="fp32", drafted="probs"),
        # two beam searches of four beams: one step's reordering
        dict(name="fork_beams", kind="fork", B=8, beams=4, bs=16, hkv=8, d=128, new="bf16", lo=40, hi=400, child=False),
        # every one of 128 requests forked once for parallel sampling
        dict(name="fork_pairs", kind="fork", B=256, beams=2, bs=16, hkv=8, d=128, new="bf16", lo=64, hi=2048, child=True),
        # the pool of a handful of requests
        dict(name="compact_few", kind="compact", B=6, bs=16, hkv=2, d=64, new="bf16", lo=33, hi=900, fill=0.6),
        # a cache half of whose blocks have come free, over its whole length
        dict(name="compact_pool", kind="compact", B=64, bs=16, hkv=4, d=128, new="bf16", lo=512, hi=8192, fill=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "sinks", "sinks", "verify", "verify", "fork", "compact"])
    if kind == "rope":
        d = rng.choice([64, 128, 128, 96, 80, 256])
        m, hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 8])
        to = rng.choice(["cache", "cache", "rows"])
        rot = rng.choice([d, d, d // 2, 32])
        return dict(kind=kind, T=_log(rng, 1, 100000 // (m * hkv + 2 * hkv)), hq=m * hkv, hkv=hkv, d=d, rot=rot,
                    inter=rng.random() < 0.4, new=rng.choice(["bf16", "bf16", "fp32"]), qout=rng.choice(["fp32", "bf16"]),
                    bs=rng.choice([8, 16, 32]), far=_log(rng, 16, 1000000), skip=rng.choice([0, 0, 5]) if to == "cache" else 0,
                    packed=rng.random() < 0.5, to=to, scaling=rng.choice(["none", "linear", "base", "parts"]),
                    inverse=to == "rows" and rng.random() < 0.5)
    if kind == "sinks":
        fast = rng.random() < 0.8          # the head sizes that models have; else odd ones, on smaller problems
        d = rng.choice([64, 128, 128]) if fast else rng.choice([32, 96, 256])
        hkv = rng.choice([1, 2, 3, 8]) if fast else rng.choice([1, 2])
        m = rng.choice([1, 3, 4, 8, 16]) if fast else rng.choice([1, 2, 5])
        B = _log(rng, 1, 48 if fast else 6)
        hi = max(2, _log(rng, 8, 200000 // B if fast else 2000))
        return dict(kind=kind, B=B, hq=m * hkv, hkv=hkv, d=d, bs=rng.choice([16, 32]) if fast else rng.choice([8, 16, 24]),
                    new="bf16" if fast else rng.choice(["bf16", "fp32"]), lo=rng.randint(1, hi), hi=hi,
                    window=_log(rng, 1, 2 * hi), sinks=rng.choice([1, 4, 4, 16, 33, 128]), rows=rng.choice([1, 1, 1, 2, 5]))
    if kind == "verify":
        V = _log(rng, 500, 200000)
        return dict(kind=kind, B=_log(rng, 1, min(200, 8000000 // V)), V=V, k=rng.choice([0, 1, 3, 4, 8]),
                    new=rng.choice(["fp32", "fp32", "bf16"]), drafted=rng.choice(["probs", "probs", "tokens"]))
    hkv, d, bs = rng.choice([1, 2, 8]), rng.choice([64, 128]), rng.choice([8, 16, 32])
    new = rng.choice(["bf16", "bf16", "fp32"])
    B = _log(rng, 1, 128)
    hi = _log(rng, 4, min(8192, 100000 * 8 // (B * hkv)))
    if kind == "fork":
        return dict(kind=kind, B=B, beams=rng.choice([1, 2, 4, 5]), bs=bs, hkv=hkv, d=d, new=new, lo=rng.randint(1, hi), hi=hi,
                    child=rng.random() < 0.5)
    return dict(kind=kind, B=B, bs=bs, hkv=hkv, d=d, new=new, lo=rng.randint(1, hi), hi=hi, fill=rng.uniform(0.3, 0.95))


# --------------------------------------------------------------------------------------- frequencies of rotation

BASE, FACTOR, ORIGINAL, LOW, HIGH = 10000.0, 8.0, 16384, 1.0, 32.0


def _mscale(case):
    return 1.0 if case["scaling"] == "none" else 0.1 * math.log(FACTOR) + 1.0


def _frequencies(case):
    """Radians per position of every pair, in 64 bits."""
    rot, kind = case["rot"], case["scaling"]
    j = np.arange(rot // 2, dtype=np.float64)
    base = BASE * FACTOR ** (rot / (rot - 2)) if kind == "base" else BASE
    f = base ** (-2 * j / rot)
    if kind == "linear":
        f = f / FACTOR
    if kind == "parts":   # fast pairs as they are, slow ones slower, those between by their turns over the original context
        r = np.clip((ORIGINAL * f / (2 * np.pi) - LOW) / (HIGH - LOW), 0, 1)
        f = f * (r + (1 - r) / FACTOR)
    return f


# ------------------------------------------------------------------------------------------ the plain forms

def _rotate(x, s, dtype):
    """x [T][H][d] rotated: angles in 64 bits, products in 32."""
    c = s["case"]
    rot = c["rot"]
    angle = s["positions"].double()[:, None] * s["freq"]
    if c["inverse"]:
        angle = -angle
    cos = (torch.cos(angle) * s["mscale"]).float()[:, None]
    sin = (torch.sin(angle) * s["mscale"]).float()[:, None]
    x = x.float()
    y = x.clone()
    if c["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = a * sin + b * cos
    return y.to(dtype)


def _plain_rope(s):
    c = s["case"]
    q = _rotate(s["q"], s, DT[c["qout"]])
    k = _rotate(s["k_new"], s, DT[c["new"]])
    if c["to"] == "rows":
        return dict(q=q, k=k)
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    s["k"][at // c["bs"], :, at % c["bs"]] = k[keep]
    s["v"][at // c["bs"], :, at % c["bs"]] = s["v_new"][keep]
    return dict(q=q, k=s["k"], v=s["v"])


def _plain_sinks(s):
    c = s["case"]
    hq, hkv, d, bs, W, S = c["hq"], c["hkv"], c["d"], c["bs"], c["window"], c["sinks"]
    q = s["q"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, device=q.device)
    for b, L in enumerate(s["lens_host"]):
        r0, r1 = s["cu_host"][b], s["cu_host"][b + 1]
        nq = r1 - r0
        if nq == 0:
            continue
        t0 = max(0, L - nq + 1 - W) // bs          # the first block of the window, the blocks of the sinks before it
        pages = list(range(min(t0, -(-S // bs)))) + list(range(t0, -(-L // bs)))
        pages = torch.tensor(pages, device=q.device)
        blk = s["table"][b, pages].long()
        key = (pages[:, None] * bs + torch.arange(bs, device=q.device)).flatten()
        held = key < L
        key = key[held]
        K = s["k"][blk].transpose(0, 1).flatten(1, 2)[:, held].float()      # [Hkv][keys][d]
        V = s["v"][blk].transpose(0, 1).flatten(1, 2)[:, held].float()
        x = q[r0:r1].view(nq, hkv, hq // hkv, d).permute(1, 0, 2, 3).flatten(1, 2)    # [Hkv][nq*m][d]
        sc = torch.matmul(x, K.transpose(1, 2)) * s["scale"]
        pos = torch.arange(L - nq, L, device=q.device).repeat_interleave(hq // hkv)[:, None]
        sc = sc.masked_fill(~((key <= pos) & ((key < S) | (key > pos - W))), -math.inf)
        top = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, V) / total
        out[r0:r1] = o.view(hkv, nq, hq // hkv, d).permute(1, 0, 2, 3).reshape(nq, hq, d)
        lse[r0:r1] = (top + torch.log(total)).view(hkv, nq, hq // hkv).permute(1, 0, 2).reshape(nq, hq)
    return out, lse


def _plain_verify(s):
    c = s["case"]
    B, D = c["B"], s["draft_tokens"].numel()
    cu = s["cu"].long()
    k = cu[1:] - cu[:-1]
    accepted = torch.zeros(B, dtype=torch.int64, device="cuda")
    if D > 0:
        t = torch.arange(D, device="cuda")
        seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        x = s["draft_tokens"].long()
        p = s["target"][t + seq, x].double()
        q = s["draft"][t, x].double() if s["draft"] is not None else torch.ones_like(p)
        # tests passed up to each draft, counted within its sequence
        missed = torch.cumsum((s["uniforms"][t + seq].double() * q >= p).long(), 0)
        before = torch.where(cu[:-1] > 0, missed[(cu[:-1] - 1).clamp(min=0)], torch.zeros_like(k))
        accepted.index_add_(0, seq, (missed - before[seq] == 0).long())
    rows = torch.arange(B, device="cuda")
    at = cu[:-1] + rows + accepted
    r = s["target"][at].double()
    turned = accepted < k
    if D > 0:
        i = (cu[:-1] + accepted).clamp(max=D - 1)
        if s["draft"] is not None:
            rest = (r - s["draft"][i].double()).clamp(min=0)
        else:
            rest = r.scatter(1, s["draft_tokens"][i].long()[:, None], 0.0)
        r = torch.where((turned & (rest.sum(1) > 0))[:, None], rest, r)
    sums = torch.cumsum(r, 1)
    u = s["uniforms"][cu[1:] + rows].double()
    token = (sums <= u[:, None] * sums[:, -1:]).sum(1)
    tokens = torch.full((D + B,), -1, dtype=torch.int32, device="cuda")
    if D > 0:
        tokens[t + seq] = torch.where(t - cu[seq] < accepted[seq], s["draft_tokens"], -torch.ones_like(s["draft_tokens"]))
    tokens[at] = token.int()
    return dict(accepted=accepted.int(), tokens=tokens, lens=(s["lens"] - k + accepted).int())


def _references(s, table, mine):
    """Entries of the tables that name each block; those without any, the lowest id last."""
    nb = s["nb"]
    refs = torch.zeros(nb, dtype=torch.int64, device="cuda")
    named = table[mine].long()
    refs.index_add_(0, named, torch.ones_like(named))
    return refs, torch.nonzero(refs == 0).flatten().flip(0)


def _listed_after(s, free):
    out = torch.full((s["nb"],), -1, dtype=torch.int32, device="cuda")
    out[:free.numel()] = free.int()
    return out


def _copy(s, src, dst):
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]


def _plain_fork(s):
    c = s["case"]
    bs, B = c["bs"], c["B"]
    parent = s["parents"].long()
    col = torch.arange(s["table"].shape[1], device="cuda")
    taken = torch.where(parent >= 0, s["lens"][parent.clamp(min=0)].long(), torch.zeros_like(parent))
    table = torch.where(col < ((taken + bs - 1) // bs)[:, None], s["table"][parent.clamp(min=0)].long(), -torch.ones_like(col))
    refs, free = _references(s, table, table >= 0)
    row = torch.arange(B, device="cuda")
    part = taken % bs > 0
    last = (taken - 1).clamp(min=0) // bs
    blk = torch.where(part, table[row, last], torch.full_like(row, s["nb"]))      # nb: no such block
    partly = torch.zeros(s["nb"] + 1, dtype=torch.int64, device="cuda").index_add_(0, blk, part.long())
    first = torch.full((s["nb"] + 1,), B, dtype=torch.int64, device="cuda").scatter_reduce_(0, blk, row, "amin")
    refs1 = torch.cat([refs, refs[:1]])
    copied = part & ((refs1[blk] > partly[blk]) | (first[blk] != row))
    src = blk[copied]
    n = src.numel()
    dst = free[free.numel() - 1 - torch.arange(n, device="cuda")]
    table[row[copied], last[copied]] = dst
    refs.index_add_(0, src, -torch.ones_like(src))
    refs[dst] = 1
    _copy(s, src, dst)
    pairs = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    pairs[:n, 0], pairs[:n, 1] = src.int(), dst.int()
    count = torch.tensor([n], dtype=torch.int32, device="cuda")
    free = free[:free.numel() - n]
    return dict(table=table.int(), refs=refs.int(), free_list=_listed_after(s, free), free_count=torch.full_like(count, free.numel()),
                pairs=pairs, pair_count=count, k=s["k"], v=s["v"], lens=taken.int())


def _plain_compact(s):
    c = s["case"]
    bs, nb = c["bs"], s["nb"]
    col = torch.arange(s["table"].shape[1], device="cuda")
    mine = (col < ((s["lens"].long() + bs - 1) // bs)[:, None]) & (s["table"] >= 0)
    refs, free = _references(s, s["table"], mine)
    used = nb - free.numel()
    block = torch.arange(nb, device="cuda")
    src = torch.nonzero((refs > 0) & (block >= used)).flatten()
    dst = torch.nonzero((refs == 0) & (block < used)).flatten()[:src.numel()]
    to = block.clone()
    to[src] = dst
    table = torch.where(mine, to[s["table"].long().clamp(min=0)], torch.full_like(s["table"], -1).long())
    refs[dst] = refs[src]
    refs[src] = 0
    _copy(s, src, dst)
    n = src.numel()
    pairs = torch.full((nb // 2, 2), -1, dtype=torch.int32, device="cuda")
    pairs[:n, 0], pairs[:n, 1] = src.int(), dst.int()
    count = torch.tensor([n], dtype=torch.int32, device="cuda")
    return dict(table=table.int(), refs=refs.int(), free_list=_listed_after(s, torch.nonzero(refs == 0).flatten().flip(0)),
                free_count=torch.full_like(count, nb - used), pairs=pairs, pair_count=count, k=s["k"], v=s["v"])


# ---------------------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    """N(0, 1) rows with some channels off centre, as keys have them."""
    x = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)
    return x.add_((0.5 * torch.randn(shape[-1:], generator=g, device="cuda").clamp(min=0)).to(dtype))


def _sizes(case, r, *ranges):
    """One whole number from each (lo, hi) for every row: a case has the same ones for every seed, in another order."""
    base = np.random.default_rng(case["B"])
    drawn = [base.integers(lo, hi + 1, case["B"]) for lo, hi in ranges]
    order = r.permutation(case["B"])
    return [x[order] for x in drawn]


def _dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(dtype))).cuda()


def _prepare_rope(s, case, g, r):
    T, hq, hkv, d, bs = case["T"], case["hq"], case["hkv"], case["d"], case["bs"]
    dt = DT[case["new"]]
    if case["packed"]:      # one row of q, k and v heads a token, as a projection gives it
        x = _randn(g, (T, hq + 2 * hkv, d), dt)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (_randn(g, (T, h, d), dt) for h in (hq, hkv, hkv))
    start = r.integers(0, max(1, case["far"] - T), size=8)     # the tokens of a few sequences one after the other
    pos = np.concatenate([np.arange(a.size) + at for a, at in zip(np.array_split(np.arange(T), 8), start)])
    s.update(q=q, k_new=k, v_new=v, positions=_dev(pos), freq=torch.from_numpy(_frequencies(case)).cuda(),
             mscale=_mscale(case), q_out=torch.empty((T, hq, d), dtype=DT[case["qout"]], device="cuda"))
    if case["to"] == "cache":
        nb = -(-T // bs) + 2
        slots = (r.permutation(nb)[:-(-T // bs), None] * bs + np.arange(bs)).reshape(-1)[:T].astype(np.int64)
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1
        s.update(slots=_dev(slots, np.int64), k=torch.zeros((nb, hkv, bs, d), dtype=dt, device="cuda"),
                 v=torch.zeros((nb, hkv, bs, d), dtype=dt, device="cuda"))
    else:
        s.update(k_out=torch.empty((T, hkv, d), dtype=dt, device="cuda"))
    if own:
        import paged_kv_cache_165_gb300 as pkv
        kind = case["scaling"]
        s["turns"] = pkv.rope_turns(case["rot"], base=BASE, scaling=kind, factor=1.0 if kind == "none" else FACTOR,
                                    original=ORIGINAL, low=LOW, high=HIGH, device="cuda")


def _prepare_sinks(s, case, g, r):
    B, hq, hkv, d, bs, rows = case["B"], case["hq"], case["hkv"], case["d"], case["bs"], case["rows"]
    lens, nq = _sizes(case, r, (case["lo"], case["hi"]), (1, rows))
    nq = np.minimum(nq, lens)
    # blocks between the first tokens and the window have been given back
    blocks = -(-lens // bs)
    gone = np.maximum(0, np.maximum(0, lens - nq + 1 - case["window"]) // bs - (-(-case["sinks"] // bs)))
    nb = int((blocks - gone).sum()) + 3
    order = r.permutation(nb)
    table = np.full((B, int(blocks.max())), -1)
    at = 0
    for b in range(B):
        keep = np.ones(blocks[b], bool)
        keep[-(-case["sinks"] // bs):][:gone[b]] = False
        table[b, :blocks[b]][keep] = order[at:at + keep.sum()]
        at += int(keep.sum())
    cu = np.concatenate([[0], np.cumsum(nq)])
    s.update(k=_randn(g, (nb, hkv, bs, d), DT[case["new"]]), v=_randn(g, (nb, hkv, bs, d), DT[case["new"]]),
             table=_dev(table), lens=_dev(lens), lens_host=lens.tolist(), cu=_dev(cu), cu_host=cu.tolist(), scale=1 / math.sqrt(d),
             q=torch.randn((int(cu[-1]), hq, d), generator=g, device="cuda"))
    s.update(out=torch.empty_like(s["q"]), lse=torch.empty(s["q"].shape[:2], device="cuda"))
    if own:
        import paged_kv_cache_165_gb300 as pkv
        n = pkv.paged_attention_sinks_workspace_bytes(B, int(cu[-1]), rows, hq, hkv, d, bs, table.shape[1], case["window"],
                                                      case["sinks"])
        s["ws"] = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")


def _prepare_verify(s, case, g, r):
    B, V, dt = case["B"], case["V"], DT[case["new"]]
    k, lens = _sizes(case, r, (0 if B > 1 else case["k"], case["k"]), (100, 9000))
    cu = np.concatenate([[0], np.cumsum(k)])
    D = int(cu[-1])
    seq = np.repeat(np.arange(B), k)
    logits = torch.randn((D + B, V), generator=g, device="cuda") * 2.5
    target = torch.softmax(logits, 1).to(dt)
    draft, tokens = None, torch.zeros(0, dtype=torch.int32, device="cuda")
    if D > 0:
        mine = logits[_dev(np.arange(D) + seq, np.int64)]
        mine = torch.softmax(mine + 0.7 * torch.randn((D, V), generator=g, device="cuda"), 1)
        race = mine / torch.empty((D, V), device="cuda").exponential_(generator=g)      # a token drawn from each row
        tokens = race.argmax(1).int()
        draft = mine.to(dt) if case["drafted"] == "probs" else None
    elif case["drafted"] == "probs":
        draft = torch.zeros((0, V), dtype=dt, device="cuda")
    s.update(target=target, draft=draft, draft_tokens=tokens, cu=_dev(cu), lens=_dev(lens),
             uniforms=torch.rand(D + B, generator=g, device="cuda"), accepted=torch.empty(B, dtype=torch.int32, device="cuda"),
             tokens=torch.empty(D + B, dtype=torch.int32, device="cuda"), lens_out=torch.empty(B, dtype=torch.int32, device="cuda"))


def _prepare_blocks(s, case, g, r):
    B, bs = case["B"], case["bs"]
    lens = np.random.default_rng(B).integers(case["lo"], case["hi"] + 1, B)      # the same for every seed, and so the pool's size
    group = case.get("beams", 3)
    rows, used = [], 0
    for b in range(B):
        first = b - b % group
        if case["kind"] == "fork":
            lens[b] = lens[first]      # beams have the same length
            if case["child"] and b != first:
                lens[b] = 0
        n = -(-int(lens[b]) // bs)
        shared = rows[first][:min(n, int(lens[first]) // bs * 2 // 3)] if b != first else []     # with the group's first row
        rows.append(shared + list(range(used, used + n - len(shared))))
        used += n - len(shared)
    nb = used + B + 5 if case["kind"] == "fork" else max(2, int(used / case["fill"]))
    order = r.permutation(nb)
    table = np.full((B, max(1, max(map(len, rows)) + 1)), -1)
    for b, t in enumerate(rows):
        table[b, :len(t)] = order[t]
    shape = (nb, case["hkv"], bs, case["d"])
    s.update(nb=nb, table=_dev(table), lens=_dev(lens), k=_randn(g, shape, DT[case["new"]]), v=_randn(g, shape, DT[case["new"]]))
    if case["kind"] == "fork":
        first = np.arange(B) - np.arange(B) % group
        size = np.minimum(first + group, B) - first
        s["parents"] = _dev(first if case["child"] else first + r.integers(0, size))
    i32 = dict(dtype=torch.int32, device="cuda")
    s.update(table_out=torch.empty_like(s["table"]), lens_out=torch.empty_like(s["lens"]), refs=torch.empty(nb, **i32),
             free_list=torch.empty(nb, **i32), free_count=torch.empty(1, **i32), pair_count=torch.empty(1, **i32),
             pairs=torch.empty((B if case["kind"] == "fork" else nb // 2, 2), **i32))
    if own:
        import paged_kv_cache_165_gb300 as pkv
        s["ws"] = torch.zeros(max(16, pkv.block_tables_share_workspace_bytes(B, table.shape[1], nb)), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    s = {"case": case}
    make = {"rope": _prepare_rope, "sinks": _prepare_sinks, "verify": _prepare_verify}.get(case["kind"], _prepare_blocks)
    make(s, case, _gen(seed), np.random.default_rng(seed))
    return s


# ------------------------------------------------------------------------------------------------- one pass

def _run_plain(s):
    kind = s["case"]["kind"]
    if kind == "sinks":
        s["out"], s["lse"] = _plain_sinks(s)
        return dict(out=s["out"], lse=s["lse"])
    return {"rope": _plain_rope, "verify": _plain_verify, "fork": _plain_fork, "compact": _plain_compact}[kind](s)


def _run_own(s):
    import paged_kv_cache_165_gb300 as pkv
    c = s["case"]
    kind = c["kind"]
    if kind == "rope" and c["to"] == "cache":
        pkv.rope_append(s["q_out"], s["q"], s["k_new"], s["v_new"], s["k"], s["v"], s["positions"], s["slots"], s["turns"],
                        interleaved=c["inter"], mscale=s["mscale"])
        return dict(q=s["q_out"], k=s["k"], v=s["v"])
    if kind == "rope":
        pkv.rope(s["q_out"], s["q"], s["k_out"], s["k_new"], s["positions"], s["turns"], interleaved=c["inter"],
                 mscale=s["mscale"], inverse=c["inverse"])
        return dict(q=s["q_out"], k=s["k_out"])
    if kind == "sinks":
        pkv.paged_attention_sinks(s["out"], s["q"], s["k"], s["v"], s["table"], s["lens"], s["scale"], c["window"], c["sinks"],
                                  cu_q=s["cu"] if c["rows"] > 1 else None, max_q=c["rows"], lse=s["lse"], workspace=s["ws"])
        return dict(out=s["out"], lse=s["lse"])
    if kind == "verify":
        pkv.verify_drafts(s["accepted"], s["tokens"], s["target"], s["draft_tokens"], s["cu"], s["uniforms"],
                          draft_probs=s["draft"], context_lens=s["lens"], context_lens_out=s["lens_out"])
        return dict(accepted=s["accepted"], tokens=s["tokens"], lens=s["lens_out"])
    got = dict(table=s["table_out"], refs=s["refs"], free_list=s["free_list"], free_count=s["free_count"], pairs=s["pairs"],
               pair_count=s["pair_count"], k=s["k"], v=s["v"])
    if kind == "fork":
        pkv.block_tables_fork(s["table"], s["lens"], s["parents"], s["table_out"], s["lens_out"], s["refs"], s["free_list"],
                              s["free_count"], s["pairs"], s["pair_count"], c["bs"], workspace=s["ws"])
        got["lens"] = s["lens_out"]
    else:
        pkv.block_tables_compact(s["table"], s["lens"], s["table_out"], s["refs"], s["free_list"], s["free_count"], s["pairs"],
                                 s["pair_count"], c["bs"], workspace=s["ws"])
    pkv.kv_block_copy(s["k"], s["v"], s["pairs"], count=s["pair_count"])
    return got


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------- the least work of a pass

def work(case):
    kind = case["kind"]
    e = 2 if case["new"] == "bf16" else 4
    if kind == "rope":
        T, hq, hkv, d = case["T"], case["hq"], case["hkv"], case["d"]
        row = hq * (e + (2 if case["qout"] == "bf16" else 4)) + 2 * hkv * e * (2 if case["to"] == "cache" else 1)
        return {"bytes": int(T * (row * d + 12)), "flops": int(T * (hq + hkv) * case["rot"] * 3)}
    if kind == "sinks":
        B, hq, hkv, d = case["B"], case["hq"], case["hkv"], case["d"]
        rows = (1 + case["rows"]) / 2
        seen = min((case["lo"] + case["hi"]) / 2, case["window"] + case["sinks"])
        return {"bytes": int(B * seen * hkv * 2 * d * e + B * seen / case["bs"] * 4 + B * rows * hq * (8 * d + 4)),
                "flops": int(4 * B * rows * hq * seen * d)}
    if kind == "verify":
        # a row of the target's probabilities, and one of the draft's where a draft was turned down (about two thirds)
        n = case["B"] * case["V"]
        rows = 1 + (2 / 3 if case["drafted"] == "probs" and case["k"] > 0 else 0)
        return {"bytes": int(n * rows * e + case["B"] * (case["k"] + 1) * 12), "flops": int(n * 2 * rows)}
    block = 2 * case["hkv"] * case["bs"] * case["d"] * e
    blocks = case["B"] * (case["lo"] + case["hi"]) / 2 / case["bs"]
    if kind == "fork":
        copies = case["B"] * (1 - 1 / case["beams"]) * (1 - 1 / case["bs"]) * (1 if case["child"] else 0.7)
        return {"bytes": int(blocks * 8 * (0.5 if case["child"] else 1) + 8 * blocks + copies * 2 * block), "flops": 0}
    blocks *= 0.6     # two thirds of a row's blocks are shared with the first of three
    moves = blocks * (1 - case["fill"])
    return {"bytes": int(blocks / 0.6 * 8 + 8 * blocks / case["fill"] + moves * 2 * block), "flops": 0}


# ------------------------------------------------------------------------------------------- values in 64 bits

def _exact_rope(s):
    c = s["case"]
    rot = c["rot"]
    sign = -1.0 if c["inverse"] else 1.0
    pos = s["positions"].cpu().numpy().astype(np.float64)
    phase = sign * pos[:, None] * _frequencies(c)[None]
    z = torch.from_numpy(_mscale(c) * np.exp(1j * phase)).cuda()[:, None]       # a pair is a complex number

    def turned(x):
        x = x.double()
        pairs = x[..., :rot].reshape(*x.shape[:2], rot // 2, 2) if c["inter"] else \
            torch.stack([x[..., :rot // 2], x[..., rot // 2:rot]], -1)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        y = y.flatten(-2) if c["inter"] else torch.cat([y[..., 0], y[..., 1]], -1)
        return torch.cat([y, x[..., rot:]], -1)

    q, k = turned(s["q"]), turned(s["k_new"])
    if c["to"] == "rows":
        return dict(q=q, k=k)
    got = dict(q=q)
    slots = s["slots"].tolist()
    t = torch.tensor([i for i, x in enumerate(slots) if x >= 0], dtype=torch.int64, device="cuda")
    at = torch.tensor([x for x in slots if x >= 0], dtype=torch.int64, device="cuda")
    for name, rows in (("k", k), ("v", s["v_new"].double())):
        cache = s[name].double().transpose(1, 2).flatten(0, 1)                  # [slots][Hkv][d]
        cache[at] = rows[t]
        got[name] = cache.unflatten(0, (-1, c["bs"])).transpose(1, 2)
    return got


def _exact_sinks(s):
    c = s["case"]
    if c["B"] * c["hkv"] * c["rows"] * 2 > 4096:
        return None
    m = c["hq"] // c["hkv"]
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    flat = [s[x].transpose(1, 2).flatten(0, 1) for x in ("k", "v")]             # [slots][Hkv][d]
    for b, L in enumerate(s["lens_host"]):
        r0, nq = s["cu_host"][b], s["cu_host"][b + 1] - s["cu_host"][b]
        for i in range(nq):
            p = L - nq + i
            t = sorted(set(range(min(c["sinks"], p + 1))) | set(range(max(0, p - c["window"] + 1), p + 1)))
            t = torch.tensor(t, device="cuda")
            at = s["table"][b, t // c["bs"]].long() * c["bs"] + t % c["bs"]
            K, V = (f[at].double() for f in flat)
            z = torch.einsum("hmd,thd->hmt", s["q"][r0 + i].double().view(c["hkv"], m, -1), K) * s["scale"]
            l = torch.logsumexp(z, -1)
            lse[r0 + i] = l.flatten()
            out[r0 + i] = torch.einsum("hmt,thd->hmd", torch.exp(z - l[..., None]), V).flatten(0, 1)
    return dict(out=out, lse=lse)


def _exact_verify(s):
    c = s["case"]
    cu, x, u = s["cu"].tolist(), s["draft_tokens"].tolist(), s["uniforms"].double().tolist()
    accepted, tokens, lens = [], [], []
    for b in range(c["B"]):
        k, at = cu[b + 1] - cu[b], cu[b] + b
        P = s["target"][at:at + k + 1].double().cpu().numpy()
        a = 0
        Q = s["draft"][cu[b]:cu[b + 1]].double().cpu().numpy() if s["draft"] is not None else None
        while a < k:
            token = x[cu[b] + a]
            if not u[at + a] * (Q[a, token] if Q is not None else 1.0) < P[a, token]:
                break
            a += 1
        r = P[a]
        if a < k:
            rest = r.copy()
            if Q is not None:
                rest = np.maximum(r - Q[a], 0)
            else:
                rest[x[cu[b] + a]] = 0
            if rest.sum() > 0:
                r = rest
        sums = np.cumsum(r)
        token = int(np.searchsorted(sums, u[at + k] * sums[-1], side="right"))
        accepted.append(a)
        tokens += x[cu[b]:cu[b] + a] + [token] + [-1] * (k - a)
        lens.append(int(s["lens"][b]) - k + a)
    return dict(accepted=np.array(accepted), tokens=np.array(tokens), lens=np.array(lens))


def _exact_blocks(s):
    c, nb = s["case"], s["nb"]
    bs, B = c["bs"], c["B"]
    old, lens = s["table"].tolist(), s["lens"].tolist()
    parents = s["parents"].tolist() if c["kind"] == "fork" else range(B)
    rows = [old[p][:-(-lens[p] // bs)] if p >= 0 else [] for p in parents]
    lens = [lens[p] if p >= 0 else 0 for p in parents]
    refs = [0] * nb
    for t in rows:
        for x in t:
            refs[x] += 1
    free = [x for x in range(nb - 1, -1, -1) if refs[x] == 0]
    pairs = []
    if c["kind"] == "fork":
        partly = [t[-1] if n % bs else -1 for t, n in zip(rows, lens)]
        keeper = {}
        for b, x in enumerate(partly):
            if x >= 0 and x not in keeper:
                keeper[x] = b if refs[x] == partly.count(x) else -1
        for b, x in enumerate(partly):
            if x >= 0 and keeper[x] != b:
                new = free.pop()
                pairs.append((x, new))
                refs[x] -= 1
                refs[new] = 1
                rows[b] = rows[b][:-1] + [new]
    else:
        used = nb - len(free)
        to = dict(zip([x for x in range(used, nb) if refs[x]], [x for x in range(used) if not refs[x]]))
        pairs = sorted(to.items())
        for src, dst in pairs:
            refs[src], refs[dst] = 0, refs[src]
        rows = [[to.get(x, x) for x in t] for t in rows]
        free = [x for x in range(nb - 1, -1, -1) if refs[x] == 0]
    width = s["table"].shape[1]
    got = dict(table=np.array([t + [-1] * (width - len(t)) for t in rows]), refs=np.array(refs),
               free_list=np.array(free + [-1] * (nb - len(free))), free_count=np.array([len(free)]),
               pairs=np.array(pairs + [(-1, -1)] * (s["pairs"].shape[0] - len(pairs))).reshape(-1, 2),
               pair_count=np.array([len(pairs)]))
    for name in ("k", "v"):
        cache = s[name]
        for src, dst in pairs:
            cache[dst] = cache[src]
        got[name] = cache.double()
    if c["kind"] == "fork":
        got["lens"] = np.array(lens)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "sinks": _exact_sinks, "verify": _exact_verify}.get(case["kind"], _exact_blocks)(s)
