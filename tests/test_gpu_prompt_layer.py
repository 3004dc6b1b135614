"""The prompt side's operators together, as a text model's layer uses them: residual norm to 8 bits, a product,
rotary positions in place on the fused projection, attention over the packed prompts; then single tokens over
the cache that the prompts left.  Also calls that overlap on two streams and from two threads."""
import threading

import pytest
import torch

import rope_block_sparse_b200 as h3a
import prompt_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

HEADS, KV, D, WIDTH = 8, 2, 64, 512
LENGTHS = [37, 1, 130, 64]
ROOM = 160


def starts(lengths):
    return torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def weights():
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn((HEADS + 2 * KV) * D, WIDTH, generator=g, device="cuda").to(torch.bfloat16) * WIDTH ** -0.5
    return w.to(torch.bfloat16), 1 + 0.1 * torch.randn(WIDTH, generator=g, device="cuda")


def project(y8, scale, w):
    """The product after the norm: 8-bit rows with their scales against 16-bit weights."""
    return ((y8.float() * scale[:, None]) @ w.float().T).to(torch.bfloat16).view(-1, HEADS + 2 * KV, D)


def test_prompts_then_single_tokens():
    """Tokens one at a time over the cache give what the whole prompt gives (the last rows of each prompt)."""
    w, gamma = weights()
    g = torch.Generator(device="cuda").manual_seed(2)
    n = sum(LENGTHS)
    x, f = (torch.randn(n, WIDTH, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    plan = h3a.rope_plan(D, 10000.0, scaling="parts", factor=4.0, original_length=64)
    st = starts(LENGTHS)
    positions = torch.cat([torch.arange(i, device="cuda", dtype=torch.int32) for i in LENGTHS])

    h, y8, scale = h3a.residual_rmsnorm(x, f, gamma, scales="row")
    qkv = project(y8, scale, w)
    before = qkv.clone()
    q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
    h3a.rope(q, k, positions, plan, inplace=True)
    o = h3a.packed_attention(q, k, v, st, st, max(LENGTHS), max(LENGTHS))

    # each stage against its 64-bit form, fed with what the stage before it wrote
    want_h, want_y = ref.rmsnorm(x, f, gamma, 1e-6)
    assert torch.equal(h, want_h)
    back = y8.double() * scale.double()[:, None]
    # e4m3: half a step relative, or 2^-10 of the scale among the subnormals; fp32 before it
    ref.within(back, want_y, want_y.abs() * (2.0 ** -4 + 8 * ref.RMSNORM_RELATIVE) + 1.001 * 2.0 ** -10 * scale.double()[:, None])
    freq = [plan.turns[j] / 2.0 ** 64 * 2 * torch.pi for j in range(plan.pairs)]
    for got, was in ((q, before[:, :HEADS]), (k, before[:, HEADS:HEADS + KV])):
        ref.within(got, *ref.rope(was, positions, freq, False))
    assert torch.equal(v, before[:, HEADS + KV:])
    want, _, bound, _ = ref.attention(q, k, v, st.tolist(), st.tolist())
    ref.within(o, want, bound)

    # the cache: keys and values of all but each prompt's last token, then that token alone
    count = len(LENGTHS)
    cache_k = torch.full((count * ROOM, KV, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    cache_v = torch.full_like(cache_k, float("nan"))
    for s, length in enumerate(LENGTHS):
        a = int(st[s])
        cache_k[s * ROOM:s * ROOM + length] = k[a:a + length]
        cache_v[s * ROOM:s * ROOM + length] = v[a:a + length]
    last = (st[1:] - 1).long()
    q1, _ = h3a.rope(before[last, :HEADS], None, positions[last], plan)
    assert torch.equal(q1, q[last])
    ones = torch.arange(count + 1, device="cuda", dtype=torch.int32)
    o1 = h3a.packed_attention(q1, cache_k, cache_v, ones, ones * ROOM, 1, ROOM,
                              lengths_k=torch.tensor(LENGTHS, device="cuda", dtype=torch.int32))
    # another kernel and another order of sums: both within the bound of the exact rows
    ref.within(o1, want[last], bound[last])


def test_two_streams_and_two_threads_at_once():
    """Calls that overlap, each with its own outputs and workspace, give what they give alone."""
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(20000, KV, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    qs = [torch.randn(2, HEADS, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    x = torch.randn(5000, WIDTH, generator=g, device="cuda").to(torch.bfloat16)
    gamma = torch.ones(WIDTH, device="cuda")
    st, sk = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), torch.tensor([0, 15000, 20000], dtype=torch.int32, device="cuda")

    def both(q):
        return h3a.packed_attention(q, k, v, st, sk, 1, 15000), h3a.residual_rmsnorm(x, None, gamma, scales="group")[1]

    alone = [both(q) for q in qs]
    torch.cuda.synchronize()
    found = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                found[i] = both(qs[i])
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for got, want in zip(found, alone):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1].view(torch.uint8), want[1].view(torch.uint8))


def test_two_graphs_with_workspaces_of_their_own():
    """Two captured calls replayed in turn and on two streams at once."""
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(9000, KV, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    st, sk = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([0, 9000], dtype=torch.int32, device="cuda")
    calls = []
    for i in range(2):
        q = torch.randn(1, HEADS, D, generator=g, device="cuda").to(torch.bfloat16)
        ws = torch.empty(h3a.packed_attention_workspace_size(q, k, 1, 1, 9000), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)
        want = h3a.packed_attention(q, k, v, st, sk, 1, 9000)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h3a.packed_attention(q, k, v, st, sk, 1, 9000, workspace=ws, out=out)
        calls.append((graph, out, want, q, ws))  # a graph does not keep what it reads alive
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for (graph, out, *_), s in zip(calls, streams):
            with torch.cuda.stream(s):
                out.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, *_ in calls:
        assert torch.equal(out, want)
