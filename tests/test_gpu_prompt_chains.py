"""Chains of the prompt side's calls, whose kernels start while the ones before them still run: each overwrites
what the call before it read.  The same bits as with a wait after every call; captured behind and between copies
and fills, and on branches that join; beside the DiT's attention on another stream."""
import pytest
import torch

import rope_block_sparse_b200 as h3a
import prompt_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

KV = 2


def randn(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def dev(x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def starts(lengths):
    return dev([0] + torch.tensor(lengths).cumsum(0).tolist())


class Chain:
    """A layer's calls over buffers of their own: q rotated in place, attention over it, and the norm of what came
    out written over q (and the sum over the residual), round after round."""

    def __init__(self, lq, cached, heads, d):
        self.lq, self.lk = lq, [a + b for a, b in zip(lq, cached)]
        n = sum(lq)
        self.first = randn(n, heads * d, seed=1), randn(n, heads * d, seed=2)
        self.k, self.v = randn(sum(self.lk), KV, d, seed=3), randn(sum(self.lk), KV, d, seed=4)
        self.gamma = torch.ones(heads * d, device="cuda")
        self.positions = torch.arange(n, device="cuda", dtype=torch.int32)
        self.plan = h3a.rope_plan(d)
        self.sq, self.sk = starts(lq), starts(self.lk)
        self.q, self.f = (torch.empty_like(t) for t in self.first)
        self.o = torch.empty(n, heads, d, device="cuda", dtype=torch.bfloat16)
        size = h3a.packed_attention_workspace_size(self.o, self.k, len(lq), max(lq), max(self.lk))
        self.ws = torch.empty(size, device="cuda", dtype=torch.uint8) if size else None

    def reset(self):
        self.q.copy_(self.first[0])
        self.f.copy_(self.first[1])

    def round(self, after=lambda: None):
        q = self.q.view_as(self.o)
        h3a.rope(q, None, self.positions, self.plan, inplace=True)
        after()
        h3a.packed_attention(q, self.k, self.v, self.sq, self.sk, max(self.lq), max(self.lk), workspace=self.ws, out=self.o)
        after()
        h3a.residual_rmsnorm(self.o.view_as(self.f), self.f, self.gamma, out=(self.f, self.q, None))
        after()

    def result(self):
        return self.q.clone(), self.f.clone(), self.o.clone()


CHAINS = {"short_prompts": ([37, 1, 130, 64], [0] * 4, 8), "two_tiles": ([700, 300], [0, 900], 8), "parts": ([70], [9000], 4),
          "single_short": ([1] * 5, [60, 3, 200, 17, 0], 8), "single_long": ([1] * 3, [9000, 5, 4000], 8), "many": ([200] * 40, [0] * 40, 8)}


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("name", CHAINS)
def test_chain_without_waits(name, d):
    lq, cached, heads = CHAINS[name]
    c = Chain(lq, cached, heads, d)
    c.reset()
    for _ in range(12):
        c.round(torch.cuda.synchronize)
    want = c.result()
    # two rounds of it by the 64-bit forms would drift apart by their roundings; one is checked
    c.reset()
    c.round()
    turned = c.first[0].view_as(c.o)
    f = [10000.0 ** (-2 * j / d) for j in range(d // 2)]
    rotated = h3a.rope(turned, None, c.positions, c.plan)[0]
    ref.within(rotated, *ref.rope(turned, c.positions, f, False))
    o, _, bound, _ = ref.attention(rotated, c.k, c.v, c.sq.tolist(), c.sk.tolist())
    ref.within(c.o, o, bound)
    for _ in range(5):
        c.reset()
        for _ in range(12):
            c.round()
        assert same(c.result(), want)


@pytest.mark.parametrize("name", CHAINS)
def test_captured_behind_copies_and_fills(name):
    """A copy, a fill, the calls, and again: nodes of other kinds before, between and behind the kernels."""
    lq, cached, heads = CHAINS[name]
    c = Chain(lq, cached, heads, 128)
    c.reset()
    c.round()
    c.round()
    want = c.result()
    kept = torch.empty_like(c.o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.q.copy_(c.first[0])
        c.f.copy_(c.first[1])
        c.o.zero_()
        c.round()
        kept.copy_(c.o)
        c.o.zero_()
        c.round()
    for t in (c.q, c.f, c.o):
        t.fill_(3.0)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert same(c.result(), want) and not torch.equal(kept, c.o)


def test_captured_branches_that_join():
    """Two chains on streams of their own, forked from one and joined into a norm that reads both."""
    a, b = Chain([37, 1, 130, 64], [0] * 4, 8, 64), Chain([232], [2000], 8, 64)
    gamma = torch.ones(8 * 64, device="cuda")
    for c in (a, b):
        c.reset()
        c.round()
    want = h3a.residual_rmsnorm(a.q, b.q, gamma)[:2]
    out = tuple(torch.zeros_like(t) for t in want)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        a.reset(), b.reset()
        for s, c in zip(sides, (a, b)):
            s.wait_stream(main)
            with torch.cuda.stream(s):
                c.round()
        for s in sides:
            main.wait_stream(s)
        h3a.residual_rmsnorm(a.q, b.q, gamma, out=(*out, None))
    for _ in range(5):
        for t in out:
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert same(out, want)


def test_beside_the_dit_attention():
    """Prompts on one stream, the DiT's attention on another: both use tensor memory."""
    grid = (3, 16, 16)
    q, k, v = (randn(1, 768, 4, 96, seed=s) for s in (5, 6, 7))
    chains = [Chain([300, 20, 77], [0, 0, 50], 8, d) for d in (64, 128)]
    alone = h3a.attention(q, k, v)
    want = []
    for c in chains:
        c.reset()
        for _ in range(10):
            c.round()
        want.append(c.result())
    sides = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for c in chains:
        c.reset()
    torch.cuda.synchronize()
    found = []
    for _ in range(10):
        for s, c in zip(sides, chains):
            with torch.cuda.stream(s):
                c.round()
        with torch.cuda.stream(sides[2]):
            found.append(h3a.attention(q, k, v))
    torch.cuda.synchronize()
    assert grid[0] * grid[1] * grid[2] == q.shape[1] and all(torch.equal(o, alone) for o in found)
    assert all(same(c.result(), w) for c, w in zip(chains, want))
    assert h3a.last_device_error() == 0
