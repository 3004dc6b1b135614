"""packed_attention against the 64-bit form: packed prompts, pieces behind caches, single tokens over padded
caches; grouped heads of every ratio; lengths of zero and one, odd ones and ones around the kernels' tiles;
rows without keys; strides; NaN and infinities in what is not attended; streams and graphs."""
import math
import random

import pytest
import torch

import rope_block_sparse_b200 as h3a
import prompt_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, FP16 = torch.bfloat16, torch.float16


def starts(lengths, first=0):
    got = [first]
    for n in lengths:
        got.append(got[-1] + n)
    return got


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(*shape, dtype=BF16, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def check(q, k, v, sq, sk, lengths=None, causal=True, scale=0.0, label="", **kw):
    """Runs the call into buffers of a known value and compares every row, those outside the sequences too."""
    seqs = len(sq) - 1
    lk = lengths if lengths is not None else [b - a for a, b in zip(sk, sk[1:])]
    out = torch.full(q.shape, 3.0, device="cuda", dtype=q.dtype)
    kw.setdefault("max_q", max(b - a for a, b in zip(sq, sq[1:])))
    kw.setdefault("max_k", max(lk))
    o, lse = h3a.packed_attention(q, k, v, dev(sq), dev(sk), lengths_k=None if lengths is None else dev(lengths),
                                  causal=causal, scale=scale, return_lse=True, out=out, **kw)
    torch.cuda.synchronize()
    assert h3a.last_device_error() == 0
    want, want_lse, bound, lse_bound = ref.attention(q, k, v, sq, sk, lengths, causal, scale or None)
    a, b = sq[0], sq[-1]
    ref.within(o[a:b], want[a:b], bound[a:b], label + " o")
    ref.within(lse[a:b], want_lse[a:b], lse_bound[a:b], label + " lse")
    assert (o[:a] == 3.0).all() and (o[b:] == 3.0).all(), label + ": rows outside the sequences were written"
    return o, lse


def make(lq, lk, heads, kv, d, dtype=BF16, seed=0, extra=0):
    return (randn(sum(lq) + extra, heads, d, dtype=dtype, seed=seed), randn(sum(lk) + extra, kv, d, dtype=dtype, seed=seed + 1),
            randn(sum(lk) + extra, kv, d, dtype=dtype, seed=seed + 2))


# queries of each sequence, keys already cached before them, heads, kv heads
PACKS = {
    "one_token": ([1], [0], 1, 1),
    "tiny": ([1, 2, 3], [0, 0, 0], 4, 2),
    "around_a_tile": ([127, 128, 129, 1, 255, 257], [0] * 6, 4, 1),
    "every_head_its_keys": ([300, 5, 64], [0, 0, 0], 3, 3),
    "seven_a_group": ([100, 37, 1, 0, 213], [0] * 5, 14, 2),
    "empty_ones": ([0, 5, 0, 0, 130, 0], [0, 0, 0, 3, 0, 0], 8, 2),
    "pieces": ([17, 64, 1, 130, 33], [1000, 3, 511, 257, 128], 8, 2),
    "all_heads_share": ([40, 3], [0, 77], 24, 1),
    "wide_group": ([3, 1, 9], [0, 200, 17], 128, 1),
    "odd_group": ([50, 20], [0, 300], 33, 1),
    "long": ([1000, 2100], [0, 0], 2, 1),
    "single_tokens": ([1] * 9, [0, 1, 15, 16, 17, 127, 128, 500, 3000], 8, 2),
    "single_tokens_16_a_group": ([1] * 3, [700, 64, 2], 32, 2),
    "few_tokens": ([4, 2, 3, 1], [900, 0, 63, 5], 4, 1),
    "chunk_of_a_long_one": ([70], [5000], 4, 2),
    "one_tile_behind_a_long_one": ([9, 30, 2, 0, 32], [4000, 9000, 100, 70, 3001], 8, 2),
}


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 96), (BF16, 64), (FP16, 128), (FP16, 64), (FP16, 96)], ids=str)
@pytest.mark.parametrize("pack", PACKS)
def test_packed_causal(pack, dtype, d):
    lq, cached, heads, kv = PACKS[pack]
    lk = [a + b for a, b in zip(lq, cached)]
    q, k, v = make(lq, lk, heads, kv, d, dtype, seed=len(pack))
    check(q, k, v, starts(lq), starts(lk), label=pack)


@pytest.mark.parametrize("pack", ["tiny", "around_a_tile", "seven_a_group", "pieces", "single_tokens", "chunk_of_a_long_one"])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_packed_bidirectional(pack, d):
    lq, cached, heads, kv = PACKS[pack]
    lk = [a + b for a, b in zip(lq, cached)]
    q, k, v = make(lq, lk, heads, kv, d, seed=7)
    check(q, k, v, starts(lq), starts(lk), causal=False, label=pack)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("lq,lk", [([200, 3, 1, 50], [60, 0, 0, 49]), ([9, 4], [5, 1]), ([1, 1], [0, 3])], ids=str)
def test_queries_without_keys(lq, lk, group, d):
    """Fewer keys than queries: the first rows attend nothing and are zeros with a log-sum-exp of -inf."""
    q, k, v = make(lq, lk, 2 * group, 2, d, seed=11, extra=1)
    o, lse = check(q, k, v, starts(lq), starts(lk))
    assert not o[:max(0, lq[0] - lk[0])].any() and (lse[:max(0, lq[0] - lk[0])] == -math.inf).all()


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("lq", [1, 3, 40])
def test_padded_cache(lq, d):
    """lengths_k: a cache of one capacity for all; what lies behind the used rows is NaN."""
    lengths, room = [0, 1, 63, 64, 65, 640, 33, 300], 640
    n = len(lengths)
    q = randn(lq * n, 8, d, seed=1)
    k, v = randn(room * n, 2, d, seed=2), randn(room * n, 2, d, seed=3)
    for s, used in enumerate(lengths):
        k[s * room + used:(s + 1) * room] = math.nan
        v[s * room + used:(s + 1) * room] = math.nan
    check(q, k, v, starts([lq] * n), starts([room] * n), lengths=lengths)
    check(q, k, v, starts([lq] * n), starts([room] * n), lengths=lengths, causal=False)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("lq,used", [([1, 1, 1, 1, 1], [300, 0, 300, 640, 64]), ([1, 4, 2, 3, 1], [9000, 120, 9000, 8999, 1]),
                                     ([40, 1, 150, 7, 33], [300, 20, 300, 640, 0])], ids=str)
def test_cache_slots_in_any_order(lq, used, d):
    """lengths_k: the sequences' slots in any order, one of them read by two sequences."""
    room = max(used)
    k, v = randn(room * 4, 2, d, seed=2), randn(room * 4, 2, d, seed=3)
    slots = [room * i for i in (3, 1, 3, 0, 2)] + [0]
    check(randn(sum(lq), 8, d, seed=1), k, v, starts(lq), slots, lengths=used)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("lq,cached", [([150, 200], [0, 40]), ([5, 2], [60, 3]), ([300], [700])], ids=str)
def test_nonfinite_where_not_attended(lq, cached, group, d):
    """An infinity or NaN in a key or value reaches the queries that attend it and no other."""
    lk = [a + b for a, b in zip(lq, cached)]
    q, k, v = make(lq, lk, 2 * group, 2, d, seed=5)
    sk = starts(lk)
    end = sk[1]
    v[end - 1, 0, 3] = math.inf      # the last key: the last query alone
    v[end - 2, 0, 3] = -math.inf     # so the last query has both: NaN
    v[end - 2, 1, d - 1] = math.nan
    v[max(0, end - 4), 1, 0] = math.inf
    check(q, k, v, starts(lq), sk, label="v")
    k[end - 1] = math.nan
    o, lse = h3a.packed_attention(q, k, v, dev(starts(lq)), dev(sk), max(lq), max(lk), return_lse=True)
    last = lq[0] - 1
    assert lse[last].isnan().all() and lse[:last].isfinite().all()
    assert o[last].isnan().all()


@pytest.mark.parametrize("lq,cached,heads,kv", [([3, 1, 4], [9000, 40, 700], 8, 2), ([130], [9000], 2, 2), ([30, 9], [9000, 500], 8, 2)], ids=str)
@pytest.mark.parametrize("d", [64, 96, 128])
def test_nonfinite_where_not_attended_in_parts(lq, cached, heads, kv, d):
    """The same with keys cut into parts: infinities near the diagonal, NaN in the middle for everyone."""
    lk = [a + b for a, b in zip(lq, cached)]
    q, k, v = make(lq, lk, heads, kv, d, seed=6)
    v[lk[0] - 1, 0, 5] = -math.inf
    v[lk[0] - 2, kv - 1, d - 2] = math.nan
    v[4321, 0, 9] = math.inf
    check(q, k, v, starts(lq), starts(lk))


@pytest.mark.parametrize("lk", [[30, 40], [9000, 500]], ids=str)
@pytest.mark.parametrize("most", [1, 2, 5, 40])
def test_rows_past_max_q_are_left(lk, most):
    """max_q smaller than the sequences: the rows up to it are right, the others as they were."""
    lq = [50, 3] if most == 40 else [7, 3]
    q, k, v = make(lq, lk, 4, 2, 64)
    out = torch.full_like(q, 3.0)
    o, lse = h3a.packed_attention(q, k, v, dev(starts(lq)), dev(starts(lk)), most, max(lk), out=out, return_lse=True)
    want, want_lse, bound, lse_bound = ref.attention(q, k, v, starts(lq), starts(lk))
    for a, n in zip(starts(lq), lq):
        m = min(n, most)
        ref.within(o[a:a + m], want[a:a + m], bound[a:a + m])
        ref.within(lse[a:a + m], want_lse[a:a + m], lse_bound[a:a + m])
        assert (o[a + m:a + n] == 3.0).all()


@pytest.mark.parametrize("lq", [1, 20])
def test_many_sequences(lq):
    """More sequences than are tried or counted at once, most of them short, some empty."""
    rng = random.Random(lq)
    n = 1300
    lk = [rng.choice([0, 1, 5, 17, 30]) + (lq if lq > 1 else 0) for _ in range(n)]
    lk[777] = 6000
    lqs = [rng.choice([0, lq, 1]) for _ in range(n)]
    q, k, v = make(lqs, lk, 4, 2, 64, seed=3)
    check(q, k, v, starts(lqs), starts(lk))
    check(q, k, v, starts(lqs), starts(lk), causal=False)


@pytest.mark.parametrize("kv,heads", [(3, 3), (28, 28), (64, 128), (300, 300), (1, 16)])
def test_streamed_heads(kv, heads):
    """Long caches with numbers of kv heads that do and do not divide the GPU."""
    lk = [3000, 1, 64, 2500]
    q, k, v = make([1] * 4, lk, heads, kv, 64, seed=8)
    check(q, k, v, starts([1] * 4), starts(lk))


def test_neighbours_are_not_touched():
    """Sequences of NaN around one of numbers, and tensors whose rows go on behind the last sequence."""
    lq = [60, 70, 50]
    q, k, v = make(lq, lq, 4, 2, 128, extra=40)
    st = starts(lq, first=20)
    for t in (q, k, v):
        t[:st[1]] = math.nan
        t[st[2]:] = math.nan
    o, lse = h3a.packed_attention(q, k, v, dev(st), dev(st), 70, 70, return_lse=True)
    want, want_lse, bound, lse_bound = ref.attention(q, k, v, st[1:3], st[1:3])
    ref.within(o[st[1]:st[2]], want[st[1]:st[2]], bound[st[1]:st[2]])
    ref.within(lse[st[1]:st[2]], want_lse[st[1]:st[2]], lse_bound[st[1]:st[2]])
    out = torch.full_like(q, 3.0)
    h3a.packed_attention(q, k, v, dev(st), dev(st), 70, 70, out=out)
    assert (out[:20] == 3.0).all() and (out[st[3]:] == 3.0).all()


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("lq", [[1, 1, 1], [90, 7, 200]], ids=str)
def test_strides(lq, d):
    """Views of a fused projection, head-major storage, an output that is a slice of a wider buffer."""
    lk = [a + 100 for a in lq] if lq[0] == 1 else lq
    q, k, v = make(lq, lk, 6, 2, d, seed=9)
    want, lse = check(q, k, v, starts(lq), starts(lk))
    fused = torch.zeros(sum(lk), 10, d + 8, device="cuda", dtype=BF16)
    kf, vf = fused[:, 6:8, :d], fused[:, 8:, :d]
    kf.copy_(k), vf.copy_(v)
    head_major = q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((sum(lq), 8, d + 16), 7.0, device="cuda", dtype=BF16)
    out = wide[:, 1:7, 8:8 + d]
    h3a.packed_attention(head_major, kf, vf, dev(starts(lq)), dev(starts(lk)), max(lq), max(lk), out=out)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert (wide == 7.0).all()


@pytest.mark.parametrize("scale", [0.02, 0.4, 1.0])
@pytest.mark.parametrize("lq,lk", [([1, 1], [4000, 77]), ([300], [300])], ids=str)
def test_scales_and_sharp_rows(scale, lq, lk):
    """Logits of up to a few hundred, growing along the keys so that the running maximum moves again and again."""
    q, k, v = make(lq, lk, 4, 2, 128, seed=13)
    k *= torch.linspace(0.1, 4.0, len(k), device="cuda").to(BF16)[:, None, None]
    check(q, k, v, starts(lq), starts(lk), scale=scale)


def test_large_logits_fp16():
    q, k, v = make([128, 200], [128, 200], 4, 4, 64, FP16, seed=17)
    check(q * 30, k * 30, v, starts([128, 200]), starts([128, 200]))


@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(seed):
    rng = random.Random(seed)
    kv, d = rng.choice([1, 2, 3]), rng.choice([64, 96, 128])
    heads = kv * rng.choice([1, 2, 3, 5, 8, 13])
    n = rng.randint(1, 12)
    lq = [rng.choice([0, 1, 2, rng.randint(1, 400)]) for _ in range(n)] + [1]
    lk = [max(0, a + rng.choice([0, 0, -rng.randint(0, 50), rng.randint(0, 700)])) for a in lq]
    q, k, v = make(lq, lk, heads, kv, d, rng.choice([BF16, FP16]), seed=seed, extra=rng.randint(0, 3))
    check(q, k, v, starts(lq), starts(lk), causal=rng.random() < 0.8, max_k=rng.choice([max(lk), 1, 100000]))


def test_a_row_does_not_depend_on_its_batch():
    """The same prompt alone and inside a batch of the same plan gives the same bits, twice."""
    lq = [200, 90, 200]
    q, k, v = make(lq, lq, 4, 2, 128)
    for t in (q, k, v):
        t[290:] = t[:200]
    st = dev(starts(lq))
    o = h3a.packed_attention(q, k, v, st, st, 200, 200)
    assert torch.equal(o[:200], o[290:])
    assert torch.equal(o, h3a.packed_attention(q, k, v, st, st, 200, 200))


def test_long_cache_past_32_bits():
    """Element offsets past 2^31 (a cache of 4.4 GB of which two short stretches are used)."""
    room = 1 << 21
    k = torch.zeros(room, 8, 128, device="cuda", dtype=BF16)  # 2^31 elements
    v = torch.zeros(room, 8, 128, device="cuda", dtype=BF16)
    used = 500
    for at, seed in ((0, 1), (room - used, 2)):
        k[at:at + used] = randn(used, 8, 128, seed=seed)
        v[at:at + used] = randn(used, 8, 128, seed=seed + 10)
    for lq in (1, 40):
        q = randn(2 * lq, 16, 128, seed=3)
        o = h3a.packed_attention(q, k, v, dev([0, lq, 2 * lq]), dev([0, room - used, room]), lq, used, lengths_k=dev([used, used]))
        ks, vs = (torch.cat((t[:used], t[-used:])) for t in (k, v))
        want, _, bound, _ = ref.attention(q, ks, vs, [0, lq, 2 * lq], [0, used, 2 * used])
        ref.within(o, want, bound, f"lq {lq}")


@pytest.mark.parametrize("lq", [1, 150])
def test_graph_and_other_stream(lq):
    """Captured with its own workspace and replayed on new inputs; the same call on a side stream."""
    n, cached = 3, 2000
    q, k, v = make([lq] * n, [lq + cached] * n, 8, 2, 128, seed=21)
    sq, sk = dev(starts([lq] * n)), dev(starts([lq + cached] * n))
    size = h3a.packed_attention_workspace_size(q, k, n, lq, lq + cached)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = h3a.packed_attention(q, k, v, sq, sk, lq, lq + cached, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            h3a.packed_attention(q, k, v, sq, sk, lq, lq + cached, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    q.copy_(randn(*q.shape, seed=99))
    g.replay()
    torch.cuda.synchronize()
    want = h3a.packed_attention(q, k, v, sq, sk, lq, lq + cached)
    assert torch.equal(out, want)


def test_bad_indices_stay_inside_the_tensors():
    """Index values that do not fit are cut: the call ends, and sequences that do fit are right."""
    q, k, v = make([50, 40], [50, 40], 4, 2, 64)
    out = torch.full_like(q, 3.0)
    h3a.packed_attention(q, k, v, dev([0, 50, 1 << 30]), dev([0, 50, 1 << 30]), 50, 50, out=out)
    want, _, bound, _ = ref.attention(q, k, v, [0, 50, 90], [0, 50, 90])
    ref.within(out, want, bound)
    h3a.packed_attention(q, k, v, dev([0, -5, 90]), dev([-7, 60, 20]), 90, 50, lengths_k=dev([-3, 1 << 30]), out=out)
    torch.cuda.synchronize()
    assert h3a.last_device_error() == 0


def test_empty_batch_and_refusals():
    q, k, v = make([8], [8], 4, 2, 64)
    st = dev([0, 8])
    assert h3a.packed_attention(q[:0], k[:0], v[:0], dev([0, 0]), dev([0, 0]), 0, 0).shape == (0, 4, 64)
    o = h3a.packed_attention(q, k[:0], v[:0], st, dev([0, 0]), 8, 0)
    assert not o.any()
    with pytest.raises(h3a.H3AError, match="UNSUPPORTED"):
        h3a.packed_attention(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous(), st, st, 8, 8)
    with pytest.raises(h3a.H3AError, match="INVALID_ARG"):
        h3a.packed_attention(q[:, :3].contiguous(), k, v, st, st, 8, 8)
    with pytest.raises(h3a.H3AError, match="INVALID_ARG"):
        h3a.packed_attention(q, k, v, st, st, 8, 8, scale=-1.0)
    with pytest.raises(ValueError, match="starts_k"):
        h3a.packed_attention(q, k, v, st, dev([0, 4, 8]), 8, 8)
    with pytest.raises(ValueError, match="element type"):
        h3a.packed_attention(q, k.half(), v, st, st, 8, 8)
    with pytest.raises(h3a.H3AError, match="WORKSPACE"):
        lots = randn(20000, 2, 64)
        h3a.packed_attention(q[:1], lots, lots, dev([0, 1]), dev([0, 20000]), 1, 20000, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
