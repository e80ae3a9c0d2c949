"""The operators of a serving loop together, as a program uses them: tokens placed by the block tables, rotated
and cached, attended through a window with first tokens, drafts verified, rejected ones given back, rows
forked, the pool compacted -- eagerly and as one CUDA graph a step -- against the definitions on the host."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_165_gb300 as pkv
from oracle import serve
from paged_kv_cache_165_gb300 import DeviceBlocks, _build

from helpers import assert_attn_close

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, BS, NB, VOCAB = 5, 8, 2, 64, 16, 80, 211
WINDOW, SINKS, DRAFTS, STEPS = 40, 5, 3, 9
LAYERS = 2
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    pkv.lib()
    pkv.get_device_error()


class Loop:
    """The device's side: static buffers, so that a step can be captured."""

    def __init__(self, dtype):
        self.rows = B * (DRAFTS + 1)                    # query rows of a step at most
        self.blocks = DeviceBlocks(NB, BS, B, 12, self.rows)
        self.k = [torch.zeros((NB, HKV, BS, D), dtype=dtype, device="cuda") for _ in range(LAYERS)]
        self.v = [torch.zeros((NB, HKV, BS, D), dtype=dtype, device="cuda") for _ in range(LAYERS)]
        self.qkv = torch.zeros((LAYERS, self.rows, HQ + 2 * HKV, D), dtype=dtype, device="cuda")
        self.new = torch.zeros(B, **I32)
        self.turns = pkv.rope_turns(D, scaling="linear", factor=2.0)
        self.q = torch.zeros((self.rows, HQ, D), device="cuda")
        self.out = torch.zeros((LAYERS, self.rows, HQ, D), device="cuda")
        n = pkv.paged_attention_sinks_workspace_bytes(B, self.rows, DRAFTS + 1, HQ, HKV, D, BS, 12, WINDOW, SINKS)
        self.ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
        self.target = torch.zeros((self.rows, VOCAB), device="cuda")
        self.draft = torch.zeros((self.rows - B, VOCAB), device="cuda")
        self.draft_tokens = torch.zeros(self.rows - B, **I32)
        self.u = torch.zeros(self.rows, device="cuda")
        self.cu_drafts = torch.zeros(B + 1, **I32)
        self.accepted = torch.zeros(B, **I32)
        self.tokens = torch.zeros(self.rows, **I32)
        self.row = torch.arange(self.rows, device="cuda")
        self.each = torch.arange(B + 1, **I32)

    def step(self):
        blocks = self.blocks
        before = blocks.context_lens.clone()
        slots = blocks.extend(self.new)
        seq = torch.searchsorted(blocks.cu_new[1:].contiguous(), self.row, right=True).clamp(max=B - 1)
        positions = (before[seq] + self.row - blocks.cu_new[seq]).int()
        for layer in range(LAYERS):
            x = self.qkv[layer]
            pkv.rope_append(self.q, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.k[layer], self.v[layer], positions, slots,
                            self.turns)
            pkv.paged_attention_sinks(self.out[layer], self.q, self.k[layer], self.v[layer], blocks.block_table, blocks.context_lens,
                                      1 / math.sqrt(D), WINDOW, SINKS, cu_q=blocks.cu_new, max_q=DRAFTS + 1, workspace=self.ws)
        torch.sub(blocks.cu_new, self.each, out=self.cu_drafts)
        pkv.verify_drafts(self.accepted, self.tokens, self.target, self.draft_tokens, self.cu_drafts, self.u, draft_probs=self.draft,
                          context_lens=blocks.context_lens, context_lens_out=blocks.context_lens)
        self.settle()

    def settle(self):
        self.blocks.settle()
        self.copy()

    def copy(self):
        for layer in range(LAYERS):
            self.blocks.copy(self.k[layer], self.v[layer])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_serving_loop(dtype, captured):
    rng = np.random.default_rng(3)
    g = torch.Generator().manual_seed(5)
    loop = Loop(dtype)
    graph = None
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            loop.step()                                 # no row asks for a token: nothing but empty sequences
            s.synchronize()
        assert not loop.blocks.context_lens.any() and pkv.get_device_error() in (0, pkv.DEVERR["cu_seqlens"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loop.step()
    freq = serve.rope_frequencies(D, scaling="linear", factor=2.0)
    held = [[[] for _ in range(B)] for _ in range(LAYERS)]   # (rotated k, v) of every token of every row
    for step in range(STEPS):
        ks = rng.integers(0, DRAFTS + 1, B)
        if step == 0:
            ks[:] = DRAFTS
        new = ks + 1
        cu = np.concatenate([[0], np.cumsum(new)])
        T, n = int(cu[-1]), int(ks.sum())
        qkv = torch.randn((LAYERS, T, HQ + 2 * HKV, D), generator=g).to(dtype)
        target = torch.softmax(torch.randn((T, VOCAB), generator=g) * 2, 1)
        seq = np.repeat(np.arange(B), ks)
        draft = torch.softmax(torch.log(target[torch.from_numpy(np.arange(n) + seq)]) + 0.5 * torch.randn((n, VOCAB), generator=g), 1)
        toks = torch.multinomial(draft, 1, generator=g)[:, 0].int()
        u = torch.rand(T, generator=g)
        loop.new.copy_(torch.from_numpy(new.astype(np.int32)))
        loop.qkv[:, :T] = qkv.cuda()
        loop.target[:T], loop.draft[:n], loop.draft_tokens[:n], loop.u[:T] = target.cuda(), draft.cuda(), toks.cuda(), u.cuda()
        loop.out.fill_(float("nan"))
        graph.replay() if captured else loop.step()
        torch.cuda.synchronize()
        assert pkv.get_device_error() == 0
        # the same on the host
        lens = [len(h) for h in held[0]]
        positions = np.concatenate([np.arange(L, L + m) for L, m in zip(lens, new)])
        accepted, tokens = serve.verify_drafts(target, draft, toks, cu - np.arange(B + 1), u)
        assert loop.accepted.tolist() == accepted and loop.tokens[:T].tolist() == tokens
        for layer in range(LAYERS):
            q = serve.rope_rows(qkv[layer, :, :HQ], positions, freq)
            k = torch.from_numpy(serve.rope_rows(qkv[layer, :, HQ:HQ + HKV], positions, freq)).to(dtype).double().numpy()
            v = qkv[layer, :, HQ + HKV:].double().numpy()
            for b in range(B):
                held[layer][b] = held[layer][b] + [(k[t], v[t]) for t in range(cu[b], cu[b + 1])]
            width = max(len(h) for h in held[layer])
            cache = [np.zeros((B * width, HKV, 1, D)) for _ in range(2)]      # a block for every token
            for b, h in enumerate(held[layer]):
                for t, kv in enumerate(h):
                    for c, x in zip(cache, kv):
                        c[b * width + t, :, 0] = x
            table = np.arange(B * width).reshape(B, width)
            want, _ = serve.paged_attention_sinks(q, cache[0], cache[1], table, [len(h) for h in held[layer]], cu, 1 / math.sqrt(D),
                                                  WINDOW, SINKS)
            # K is rounded to its type on both sides from values that differ by fp32's rounding: now and then to the
            # next bf16, 2^-8 of one key's element
            assert_attn_close(loop.out[layer, :T], want, f"step {step}", 2e-3)
        for layer in range(LAYERS):
            held[layer] = [h[:len(h) - (k - a)] for h, k, a in zip(held[layer], ks, accepted)]
        assert loop.blocks.context_lens.tolist() == [len(h) for h in held[0]]
        used = sum(-(-len(h) // BS) for h in held[0])
        if step < 3:
            assert int(loop.blocks.free_count) == NB - used      # everything else has come back
        if step == 3:      # row 0 is continued in row 4 as well, row 2 starts again
            parents = [0, 1, -1, 3, 0]
            loop.blocks.fork(torch.tensor(parents, **I32))
            loop.copy()
            held = [[list(h[p]) if p >= 0 else [] for p in parents] for h in held]
        if step == 6:
            loop.blocks.compact()
            loop.copy()
            assert int(loop.blocks.block_table.max()) < NB - int(loop.blocks.free_count)
        assert pkv.get_device_error() == 0


def test_dependents_read_what_the_kernel_before_them_wrote():
    # The attention lets the next kernel's blocks be scheduled while it runs, and writes its outputs last: they serve as
    # positions, random numbers and a pair count here, each read by a call right behind the attention.
    T, hq, hkv, d, bs, ctx = 64, 32, 8, 64, 16, 2048
    g = torch.Generator().manual_seed(3)
    nb = T * ctx // bs
    kc, vc = (torch.rand((nb, hkv, bs, d), generator=g).bfloat16().cuda() for _ in range(2))
    less = -vc
    table = torch.arange(nb, **I32).view(T, -1)
    lens = torch.full((T,), ctx, **I32)
    q = torch.randn((T, hq, d), generator=g).cuda()
    out = torch.empty((T, hq, d), device="cuda")
    n = pkv.paged_attention_sinks_workspace_bytes(T, T, 1, hq, hkv, d, bs, ctx // bs, 1024, 4)
    ws = torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
    bits = out.view(torch.int32).flatten()
    turns, x = pkv.rope_turns(128), torch.randn((4096, 4, 128), generator=g).cuda()
    probs = torch.softmax(torch.randn((T, 999), generator=g), 1).cuda()
    cu = torch.arange(T + 1, **I32).mul_(0)
    none = torch.zeros(0, **I32)
    moved = torch.stack([torch.arange(100, **I32), torch.arange(100, 200, **I32)], 1)

    def calls():
        rotated, tokens, accepted = torch.empty_like(x), torch.full((T,), -9, **I32), torch.full((T,), -9, **I32)
        k2, v2 = kc[:200].clone(), vc[:200].clone()
        yield rotated, lambda: pkv.rope(rotated, x, None, None, bits[:4096], turns)
        yield tokens, lambda: pkv.verify_drafts(accepted, tokens, probs, none, cu, out.flatten()[:T])
        yield k2, lambda: pkv.kv_block_copy(k2, v2, moved, count=bits[:1])

    def attend(values):
        pkv.paged_attention_sinks(out, q, kc, values, table, lens, 0.125, 1024, 4, workspace=ws)

    for i in range(3):
        got = []
        for waits in (True, False):
            for j, (result, call) in enumerate(calls()):
                if i == j:
                    torch.cuda.synchronize()
                    attend(less)                        # what stands there before: the same with the other sign
                    attend(vc)
                    if waits:
                        torch.cuda.synchronize()
                    call()
                    got.append(result.clone())
        torch.cuda.synchronize()
        assert torch.equal(*got), i
    pkv.get_device_error()                              # a count beyond the list


def test_graphs_in_which_copies_and_fills_come_before_the_calls():
    # memory nodes right before kernels that start as dependents: inputs copied in, outputs filled, every replay
    g = torch.Generator().manual_seed(8)
    x, turns = torch.randn((500, 4, 64), generator=g).cuda(), pkv.rope_turns(64)
    given, positions = torch.zeros(500, **I32), torch.zeros(500, **I32)
    rotated = torch.zeros_like(x)
    u_given, u, cu = torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda"), torch.arange(7, **I32).mul_(0)
    probs = torch.softmax(torch.randn((6, 300), generator=g), 1).cuda()
    accepted, tokens, none = torch.zeros(6, **I32), torch.zeros(6, **I32), torch.zeros(0, **I32)
    table, lens = torch.arange(12, **I32).view(3, 4), torch.zeros(3, **I32)
    lens_given, blocks = torch.zeros(3, **I32), DeviceBlocks(20, 4, 3, 4, 0)
    cache = torch.randn((20, 1, 4, 8), generator=g).cuda()
    k, v = torch.zeros_like(cache), torch.zeros_like(cache)

    def step():
        positions.copy_(given)
        pkv.rope(rotated, x, None, None, positions, turns)
        u.copy_(u_given)
        pkv.verify_drafts(accepted, tokens, probs, none, cu, u)
        blocks.block_table.copy_(table)
        blocks.context_lens.copy_(lens_given)
        blocks.fork(lens)                              # every row takes row 0's sequence
        k.copy_(cache)
        v.zero_()
        blocks.copy(k, v)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(5):
        given.copy_(torch.randint(0, 10 ** 6, (500,), generator=g, dtype=torch.int32))
        u_given.copy_(torch.rand(6, generator=g))
        lens_given.copy_(torch.tensor([n + 5, 3, 1], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(x)
        pkv.rope(want, x, None, None, given, turns)
        assert torch.equal(rotated, want)
        assert tokens.tolist() == serve.verify_drafts(probs, None, [], [0] * 7, u_given)[1]
        forked = serve.block_tables_fork(table.cpu(), [n + 5, 3, 1], [0, 0, 0], 4, 20)
        assert blocks.block_table.tolist() == forked["table"] and blocks.context_lens.tolist() == forked["lens"]
        wanted = cache.clone()
        for a, b in forked["pairs"]:
            wanted[b] = cache[a]
        assert torch.equal(k, wanted) and not v.any()
    assert pkv.get_device_error() == 0
