"""Plain definitions, in 64 bits and whole numbers, of the operators around the attention of a serving
loop: rotary positions, windows with first tokens that stay visible, drafted tokens, and block tables
whose rows share blocks.  Row by row, entry by entry; nothing of the library is used."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from .oracle import to_f64, to_numpy


# ------------------------------------------------------------- rotary positions

def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: float = 1.0,
                     low: float = 1.0, high: float = 32.0) -> np.ndarray:
    """Radians per position of the rot / 2 dimension pairs."""
    f = []
    for j in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        x = b ** (-2.0 * j / rot)
        if scaling == "linear":
            x /= factor
        if scaling == "parts":
            r = (original * x / (2 * np.pi) - low) / (high - low)
            r = min(1.0, max(0.0, r))
            x = r * x + (1 - r) * x / factor
        f.append(x)
    return np.array(f, np.float64)


def rope_rows(x, positions, freq, interleaved: bool = False, mscale: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x [T][H][d] rotated by positions [T]; dimensions from 2 * len(freq) on stay."""
    x = to_f64(x)
    out = x.copy()
    half = len(freq)
    for t, p in enumerate(np.asarray(positions).tolist()):
        for j in range(half):
            phi = (-1.0 if inverse else 1.0) * p * freq[j]
            c, s = mscale * np.cos(phi), mscale * np.sin(phi)
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return out


# ------------------------------------------------- windows with first tokens

def paged_attention_sinks(q, k_cache, v_cache, block_table, context_lens, cu_q, scale: float, window: int, sinks: int):
    """Row at position p sees t <= p with t < sinks or t > p - window (window 0: every t <= p).
    Returns (out [Tq][Hq][d], lse [Tq][Hq])."""
    qd, kc, vc = to_f64(q), to_f64(k_cache), to_f64(v_cache)
    table, lens, cu = (np.asarray(to_numpy(x)).tolist() for x in (block_table, context_lens, cu_q))
    Tq, Hq, d = qd.shape
    _, Hkv, bs, _ = kc.shape
    out, lse = np.zeros((Tq, Hq, d)), np.full((Tq, Hq), -np.inf)
    for b, L in enumerate(lens):
        nq = cu[b + 1] - cu[b]
        for i in range(nq):
            p = L - nq + i
            seen = [t for t in range(p + 1) if window == 0 or t < sinks or t > p - window]
            blk = np.array([table[b][t // bs] for t in seen])
            off = np.array([t % bs for t in seen])
            for h in range(Hq):
                K, V = kc[blk, h // (Hq // Hkv), off], vc[blk, h // (Hq // Hkv), off]
                s = K @ qd[cu[b] + i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                out[cu[b] + i, h] = w @ V / w.sum()
                lse[cu[b] + i, h] = m + np.log(w.sum())
    return out, lse


# --------------------------------------------------------------- drafted tokens

UNIT = 46   # probabilities are summed as whole multiples of 2^-46


def units(p) -> list:
    """Probabilities as the nearest whole multiples of 2^-46 (ties to even); at most 1, 0 for negative ones and NaN."""
    x = np.asarray(p, np.float64)
    x = np.where(x > 0, np.minimum(x, 1.0), 0.0)
    return [int(v) for v in np.rint(np.ldexp(x, UNIT))]   # scaled by a power of two: exact before the rounding


def verify_drafts(target, draft, draft_tokens, cu_drafts, uniforms):
    """Returns (accepted [B], tokens [D + B]); tokens of -2 are not written (a bad cu_drafts)."""
    P = to_f64(target)
    Q = None if draft is None else to_f64(draft)
    x, cu, u = (np.asarray(to_numpy(v)).tolist() for v in (draft_tokens, cu_drafts, uniforms))
    V = P.shape[1]
    accepted, tokens = [], [-2] * P.shape[0]
    for b in range(len(cu) - 1):
        c0, k = cu[b], cu[b + 1] - cu[b]
        if c0 < 0 or k < 0 or cu[b + 1] > len(x):
            accepted.append(0)
            continue
        at = c0 + b
        a = 0
        while a < k:
            t = x[c0 + a]
            if not 0 <= t < V:
                break
            q = 1.0 if Q is None else Q[c0 + a, t]
            if not (np.isfinite(q) and np.isfinite(P[at + a, t]) and Fraction(u[at + a]) * Fraction(q) < Fraction(P[at + a, t])):
                break
            a += 1
        p = units(P[at + a])
        r = p
        if a < k:
            if Q is not None:
                r = [max(0, y - z) for y, z in zip(p, units(Q[c0 + a]))]
            else:
                r = [0 if v == x[c0 + a] else y for v, y in enumerate(p)]
            if sum(r) == 0:
                r = p
        total, token, run = sum(r), -1, 0
        for v, y in enumerate(r):
            run += y
            if total > 0 and run > Fraction(u[at + k]) * total:
                token = v
                break
        accepted.append(a)
        tokens[at:at + k + 1] = x[c0:c0 + a] + [token] + [-1] * (k - a)
    return accepted, tokens


# ------------------------------------------------------ tables that share blocks

def _free(refs):
    return [i for i in range(len(refs) - 1, -1, -1) if refs[i] == 0]


def block_tables_fork(table, lens, parents, bs: int, nb: int, held=None):
    """Returns a dict: table, lens, refs, free_list, free_count, pairs (a list)."""
    B, width = np.asarray(table).shape
    table, lens = np.asarray(table).tolist(), np.asarray(lens).tolist()
    parents = list(range(B)) if parents is None else np.asarray(parents).tolist()
    refs = [1 if held is not None and h else 0 for h in (held if held is not None else [0] * nb)]
    rows, out_lens = [], []
    for p in parents:
        ok = 0 <= p < B and 0 <= lens[p] <= width * bs
        L = lens[p] if ok else 0
        rows.append([x if 0 <= x < nb else -1 for x in table[p][:-(-L // bs)]] if ok else [])
        out_lens.append(L)
    ends = {}      # a block and the rows that end in it, partly filled
    for b, (t, L) in enumerate(zip(rows, out_lens)):
        for j, x in enumerate(t):
            if x < 0:
                continue
            if L % bs and j == len(t) - 1:
                ends.setdefault(x, []).append(b)
            else:
                refs[x] += 1
    wanting = []
    for x, those in ends.items():
        if refs[x] == 0:
            refs[x] = 1
            those = those[1:]
        wanting += [(b, x) for b in those]
    free = _free(refs)
    pairs = []
    for b, x in sorted(wanting):
        if free:
            new = free.pop()
            refs[new] = 1
            rows[b][-1] = new
            pairs.append((x, new))
        else:
            rows[b], out_lens[b] = [], 0
    return dict(table=[t + [-1] * (width - len(t)) for t in rows], lens=out_lens, refs=refs,
                free_list=free + [-1] * (nb - len(free)), free_count=len(free), pairs=pairs)


def block_tables_compact(table, lens, bs: int, nb: int, held=None):
    """Returns a dict: table, refs, free_list, free_count, pairs (a list)."""
    B, width = np.asarray(table).shape
    table, lens = np.asarray(table).tolist(), np.asarray(lens).tolist()
    held = [0] * nb if held is None else list(held)
    refs = [1 if h else 0 for h in held]
    rows = []
    for t, L in zip(table, lens):
        L = L if 0 <= L <= width * bs else 0
        rows.append([x if 0 <= x < nb else -1 for x in t[:-(-L // bs)]])
        for x in rows[-1]:
            if x >= 0:
                refs[x] += 1
    used = sum(r > 0 for r in refs)
    src = [i for i in range(used, nb) if refs[i] and not held[i]]
    dst = [i for i in range(used) if not refs[i]]
    to = dict(zip(src, dst))
    for s, d in to.items():
        refs[s], refs[d] = 0, refs[s]
    rows = [[to.get(x, x) for x in t] for t in rows]
    free = _free(refs)
    return dict(table=[t + [-1] * (width - len(t)) for t in rows], refs=refs, free_list=free + [-1] * (nb - len(free)),
                free_count=len(free), pairs=list(to.items()))
