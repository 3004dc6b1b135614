"""The prompt side's entry points without a GPU: refusals, rotary plans, workspace sizes.  Every call that
takes pointers fails validation before it reaches a kernel."""
import ctypes
import math

import pytest
import torch

from rope_block_sparse_b200 import h3a

NO_GPU = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: CPU-only check")
GOOD, ODD = 0x10000, 0x10008  # never dereferenced


def plan_values(plan):
    return [plan.turns[j] / 2 ** 64 * 2 * math.pi for j in range(plan.pairs)]


@pytest.mark.parametrize("r", [2, 50, 128, 256])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
def test_rope_plan_frequencies(r, scaling):
    theta, s, trained, lo, hi = 500000.0, 8.0, 8192, 1.0, 4.0
    plan = h3a.rope_plan(r, theta, True, scaling, s, trained, lo, hi, amplitude=1.25)
    assert (plan.pairs, plan.interleaved, plan.amplitude) == (r // 2, 1, 1.25)
    for j, got in enumerate(plan_values(plan)):
        base = theta * s ** (r / (r - 2)) if scaling == "base" and r > 2 else theta
        f = base ** (-2 * j / r)
        if scaling == "linear":
            f /= s
        if scaling == "parts":
            w = min(max((trained * f / (2 * math.pi) - lo) / (hi - lo), 0.0), 1.0)
            f = w * f + (1 - w) * f / s
        assert abs(got - f) <= 2.0 ** -48 * f + 2.0 ** -60, (j, got, f)


def test_rope_plan_base_scaling_stretches_only_the_slow_end():
    plain, wide = plan_values(h3a.rope_plan(64)), plan_values(h3a.rope_plan(64, scaling="base", factor=4.0))
    assert wide[0] == plain[0] and abs(wide[-1] * 4 / plain[-1] - 1) < 1e-9


def test_rope_plan_is_made_once_and_refuses():
    assert h3a.rope_plan(64) is h3a.rope_plan(64, 10000.0)
    assert plan_values(h3a.rope_plan(4, frequencies=[2 * math.pi * 5.25, -math.pi / 2])) == pytest.approx([math.pi / 2, 1.5 * math.pi])
    for kw in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=64, theta=0.0), dict(rotary_dim=64, factor=0.0),
               dict(rotary_dim=64, scaling="parts"), dict(rotary_dim=64, amplitude=math.inf), dict(rotary_dim=64, theta=math.nan),
               dict(rotary_dim=64, scaling="parts", original_length=1, low_turns=2.0, high_turns=2.0),
               dict(rotary_dim=2, frequencies=[math.inf])):
        with pytest.raises(h3a.H3AError, match="INVALID_ARG"):
            h3a.rope_plan(**kw)
    with pytest.raises(h3a.H3AError, match="UNSUPPORTED"):
        h3a.rope_plan(258)
    with pytest.raises(ValueError, match="scaling"):
        h3a.rope_plan(64, scaling="other")
    with pytest.raises(ValueError, match="frequencies"):
        h3a.rope_plan(64, frequencies=[1.0])


@NO_GPU
def test_rope_refusals():
    lib = h3a.load()
    plan = h3a.rope_plan(64)

    def call(q=GOOD, qo=GOOD, d=(8, 128, 1024, 128, 1024, 128), k=None, ko=None, dk=None, dtype=0, pos=GOOD, n=4, plan=plan):
        dk = h3a.HeadsDesc(*dk) if dk else None
        return lib.h3a_rope(q, qo, h3a.HeadsDesc(*d) if d else None, k, ko, dk, dtype, pos, n, plan, 0, None)

    assert call(q=None) == 1 and call(qo=None) == 1 and call(pos=None) == 1
    assert call(q=ODD) == 1 and call(qo=ODD) == 1 and call(pos=GOOD + 2) == 1
    assert call(dtype=2) == 1 and call(n=-1) == 1 and call(d=None) == 1 and call(plan=None) == 1
    assert call(plan=h3a.RopePlan()) == 1                         # not made by the plan calls
    assert call(d=(0, 128, 1024, 128, 1024, 128)) == 1
    assert call(d=(8, 32, 1024, 128, 1024, 128)) == 1              # 64 rotated channels in a head of 32
    assert call(d=(8, 132, 2048, 256, 2048, 256)) == 1             # head_dim no multiple of 8
    assert call(d=(8, 128, 1028, 128, 1024, 128)) == 1
    assert call(d=(8, 128, 1024, 64, 1024, 128)) == 1              # heads overlap
    assert call(d=(8, 128, 1024, 128, 2048, 128)) == 1             # in place with other strides
    assert call(d=(8, 520, 8192, 520, 8192, 520)) == 2
    assert call(n=2 ** 31) == 2
    assert call(k=GOOD) == 1                                       # k without its layout
    assert call(k=GOOD, ko=None, dk=(8, 128, 1024, 128, 1024, 128)) == 1
    assert call(k=GOOD, ko=GOOD, dk=(8, 64, 1024, 128, 1024, 128)) == 1   # another head_dim
    assert call(d=(40000, 128, 40000 * 128, 128, 40000 * 128, 128), k=GOOD, ko=GOOD, dk=(40000, 128, 40000 * 128, 128, 40000 * 128, 128)) == 2
    assert call(q=None, qo=None, pos=None, n=0) == 0               # nothing to do


@NO_GPU
def test_rmsnorm_refusals():
    lib = h3a.load()

    def call(x=GOOD, xs=64, f=GOOD, fs=64, g=GOOD, rows=4, c=64, dtype=0, eps=1e-6, scales=1, h=GOOD + 4096, hs=64, y=GOOD + 8192, ys=64, s=GOOD):
        return lib.h3a_residual_rmsnorm(x, xs, f, fs, g, rows, c, dtype, eps, scales, h, hs, y, ys, s, None)

    assert call(x=None) == 1 and call(g=None) == 1 and call(y=None) == 1 and call(h=None) == 1 and call(s=None) == 1
    assert call(x=ODD) == 1 and call(f=ODD) == 1 and call(h=ODD) == 1 and call(y=ODD) == 1 and call(g=ODD) == 1 and call(s=GOOD + 2) == 1
    assert call(c=60, xs=64) == 1 and call(c=0) == 1 and call(rows=-1) == 1 and call(dtype=5) == 1 and call(scales=3) == 1
    assert call(eps=-1.0) == 1 and call(eps=math.nan) == 1
    assert call(xs=56) == 1 and call(fs=68) == 1 and call(hs=60) == 1 and call(ys=63) == 1
    assert call(h=GOOD, hs=128) == 1                                # in place over x with another stride
    assert call(c=16392, xs=16392, fs=16392, hs=16392, ys=16392) == 2
    assert call(rows=2 ** 31) == 2
    assert call(x=None, f=None, g=None, y=None, s=None, rows=0) == 0


def packed(**kw):
    d = dict(dtype=0, seqs=2, heads=8, kv_heads=2, head_dim=128, total_q=64, total_k=512, max_q=32, max_k=256, q_stride_n=1024,
             q_stride_h=128, k_stride_n=256, k_stride_h=128, v_stride_n=256, v_stride_h=128, o_stride_n=1024, o_stride_h=128,
             causal=1, scale=0.0)
    d.update(kw)
    return h3a.PackedDesc(*(d[name] for name, _ in h3a.PackedDesc._fields_))


def test_packed_workspace_size():
    lib = h3a.load()
    n = ctypes.c_size_t(7)

    def size(**kw):
        assert lib.h3a_packed_attention_workspace_size(packed(**kw), n) == 0
        return n.value

    assert size(max_k=100) == 0                                  # one part: nothing to join
    # a single token over a long cache: two parts of 16 rows with their log-sum-exps for each of two CTAs a
    # multiprocessor (148), and a pair of numbers for the sequence
    assert size(seqs=1, total_q=1, max_q=1, total_k=100000, max_k=100000) == 148 * 2 * 2 * 16 * (128 + 1) * 4 + 256
    # a piece of a prompt behind a long cache: whole parts of every row
    parts = size(seqs=1, total_q=64, max_q=64, total_k=100000, max_k=100000)
    assert parts % (64 * 8 * (128 + 1) * 4) == 0 and 2 <= parts // (64 * 8 * (128 + 1) * 4) <= 64
    assert lib.h3a_packed_attention_workspace_size(packed(), None) == 1
    assert lib.h3a_packed_attention_workspace_size(None, n) == 1


@NO_GPU
def test_packed_refusals():
    lib = h3a.load()

    def call(q=GOOD, k=GOOD, v=GOOD, sq=GOOD, sk=GOOD, lk=None, o=GOOD, lse=None, ws=GOOD, wsb=1 << 40, **kw):
        return lib.h3a_packed_attention(q, k, v, packed(**kw), sq, sk, lk, o, lse, ws, wsb, None)

    for name in ("q", "k", "v", "o"):
        assert call(**{name: None}) == 1 and call(**{name: ODD}) == 1, name
    assert call(sq=None) == 1 and call(sk=None) == 1 and call(sq=GOOD + 2) == 1 and call(lk=GOOD + 1) == 1 and call(lse=GOOD + 2) == 1
    assert call(dtype=2) == 1 and call(seqs=0) == 1 and call(heads=7) == 1 and call(kv_heads=0) == 1
    assert call(total_q=-1) == 1 and call(max_q=-1) == 1 and call(max_k=-1) == 1
    assert call(scale=-0.5) == 1 and call(scale=math.inf) == 1 and call(scale=math.nan) == 1
    for name in ("q", "k", "v", "o"):
        assert call(**{name + "_stride_n": 1028}) == 1, name
        assert call(**{name + "_stride_h": 64}) == 1, name
    for d in (32, 80, 256):
        assert call(head_dim=d, q_stride_h=256, k_stride_h=256, v_stride_h=256, o_stride_h=256, q_stride_n=2048, k_stride_n=512,
                    v_stride_n=512, o_stride_n=2048) == 2
    assert call(heads=258, kv_heads=2, q_stride_n=65536, o_stride_n=65536) == 2      # 129 heads to a kv head
    assert call(total_q=2 ** 31) == 2 and call(total_k=2 ** 31) == 2
    long = dict(total_k=1 << 20, max_k=1 << 20, max_q=1, total_q=2)
    assert call(ws=None, **long) == 5 and call(ws=ODD, **long) == 5 and call(wsb=64, **long) == 5
    assert call(total_q=0, q=None, o=None) == 0 and call(max_q=0) == 0               # no query: nothing to do


def test_prompt_side_refuses_cpu_tensors():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        h3a.rope(q, q, torch.zeros(4, dtype=torch.int32), h3a.rope_plan(64))
    with pytest.raises(ValueError, match="CUDA"):
        h3a.residual_rmsnorm(q[:, 0], None, torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        h3a.packed_attention(q, q, q, i, i, 4, 4)
