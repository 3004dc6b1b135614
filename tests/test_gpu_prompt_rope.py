"""rope / rope_plan against the 64-bit form: both layouts, parts of heads, odd numbers of pairs, every
scaling, far and negative positions, strided slices, in place, inverse, single tokens."""
import math

import pytest
import torch

import rope_block_sparse_b200 as h3a
import prompt_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def frequencies(r, theta, scaling="none", s=1.0, trained=1, lo=1.0, hi=32.0):
    got = []
    for j in range(r // 2):
        base = theta * s ** (r / (r - 2)) if scaling == "base" and r > 2 else theta
        f = base ** (-2 * j / r)
        if scaling == "linear":
            f /= s
        if scaling == "parts":
            w = min(max((trained * f / (2 * math.pi) - lo) / (hi - lo), 0.0), 1.0)
            f = f * w + f / s * (1 - w)
        got.append(f)
    return got


def randn(*shape, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def check(x, y, positions, freq, interleaved, amplitude=1.0, inverse=False, label=""):
    want, bound = ref.rope(x, positions, freq, interleaved, amplitude, inverse)
    ref.within(y, want, bound, label)


# tokens, heads, kv heads, head_dim, rotated channels
SHAPES = [(1, 1, 1, 64, 64), (16, 32, 8, 128, 128), (77, 28, 4, 96, 48), (1025, 5, 1, 128, 50), (3, 2, 2, 8, 2),
          (333, 7, 7, 96, 12), (5, 3, 1, 512, 256), (2500, 8, 2, 128, 16), (9, 1, 1, 136, 136), (7, 130, 3, 64, 64),
          (50, 9, 3, 128, 24), (4000, 4, 1, 128, 50), (3000, 5, 2, 96, 24), (5000, 1, 1, 96, 10), (2600, 3, 1, 128, 128), (40000, 1, 1, 8, 6),
          (3001, 2, 1, 512, 254)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope_matches(shape, interleaved, dtype):
    n, h, kv, d, r = shape
    q, k = randn(n, h, d, dtype=dtype, seed=1), randn(n, kv, d, dtype=dtype, seed=2)
    positions = torch.randint(0, 1 << 20, (n,), device="cuda", dtype=torch.int32, generator=torch.Generator(device="cuda").manual_seed(3))
    yq, yk = h3a.rope(q, k, positions, h3a.rope_plan(r, 500000.0, interleaved))
    f = frequencies(r, 500000.0)
    check(q, yq, positions, f, interleaved, label="q")
    check(k, yk, positions, f, interleaved, label="k")
    assert torch.equal(yq[..., r:], q[..., r:])


@pytest.mark.parametrize("scaling,s,amplitude", [("linear", 4.0, 1.0), ("base", 8.0, 1.0), ("parts", 8.0, 1.2079)])
def test_rope_scalings(scaling, s, amplitude):
    q = randn(200, 4, 128)
    positions = torch.arange(200, device="cuda", dtype=torch.int32) * 6553
    plan = h3a.rope_plan(128, 10000.0, scaling=scaling, factor=s, original_length=4096, low_turns=1.0, high_turns=4.0, amplitude=amplitude)
    y, none = h3a.rope(q, None, positions, plan)
    assert none is None
    f = frequencies(128, 10000.0, scaling, s, 4096, 1.0, 4.0)
    check(q, y, positions, f, False, amplitude, label=scaling)
    own = h3a.rope_plan(128, frequencies=f, amplitude=amplitude)
    assert torch.equal(h3a.rope(q, None, positions, own)[0], y)


def test_rope_far_and_negative_positions():
    """Any int32 position: whole turns drop out exactly, so position p and p + 2^20 agree where 2^20 turns are whole."""
    q = randn(8, 2, 64)
    positions = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 123456789, -987654321], device="cuda", dtype=torch.int32)
    f = [2 * math.pi * (2 * j + 1) / 2 ** 24 for j in range(32)]  # turns are multiples of 2^-24: exact in 64 bits
    y, _ = h3a.rope(q, None, positions, h3a.rope_plan(64, frequencies=f))
    whole = positions.long()[:, None] * torch.tensor([2 * j + 1 for j in range(32)], device="cuda") % 2 ** 24
    angle = whole.double() * (2 * math.pi / 2 ** 24)
    a, b = q[..., :32].double(), q[..., 32:].double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    want = torch.cat((a * c - b * s, a * s + b * c), -1)
    # frequencies come through a double's 2^-53 of a turn, times 2^31 positions: 2^-22 of a turn, 2 pi 2^-22 in angle
    reach = (a.abs() + b.abs()).repeat(1, 1, 2) * (2.0 ** -21 + 2 * math.pi * 2.0 ** -22)
    ref.within(y, want, reach + 2.0 ** -8 * (want.abs() + reach))


@pytest.mark.parametrize("r", [96, 50, 64])
def test_rope_strided_in_place_and_out(r):
    """q and k as slices of one fused projection: copies, in place (the rest of the buffer untouched), given outputs."""
    qkv = randn(301, 6 + 2 * 2, 96, seed=5)
    positions = torch.randint(0, 9000, (301,), device="cuda", dtype=torch.int32)
    plan = h3a.rope_plan(r, interleaved=True)
    yq, yk = h3a.rope(qkv[:, :6], qkv[:, 6:8], positions, plan)
    check(qkv[:, :6], yq, positions, frequencies(r, 10000.0), True)
    mine = qkv.clone()
    h3a.rope(mine[:, :6], mine[:, 6:8], positions, plan, inplace=True)
    assert torch.equal(mine[:, :6], yq) and torch.equal(mine[:, 6:8], yk) and torch.equal(mine[:, 8:], qkv[:, 8:])
    wide = torch.full((2, 301, 10, 104), 3.0, device="cuda", dtype=torch.bfloat16)
    out = (wide[0, :, 1:7, 8:], wide[1, :, 4:6, :96])
    h3a.rope(qkv[:, :6], qkv[:, 6:8], positions, plan, out=out)
    assert torch.equal(out[0], yq) and torch.equal(out[1], yk)
    out[0].fill_(3.0), out[1].fill_(3.0)
    assert (wide == 3.0).all()
    # one side in place, the other not
    both = h3a.rope(mine[:, :6], qkv[:, 6:8], positions, plan, out=(mine[:, :6], out[1]))
    assert torch.equal(out[1], yk) and both[0].data_ptr() == mine.data_ptr()


def test_rope_inverse_is_the_transpose():
    """<R x, y> = <x, R^T y>: the inverse call is the gradient's map."""
    x, y = randn(64, 3, 128, seed=1), randn(64, 3, 128, seed=2)
    positions = torch.randint(0, 100000, (64,), device="cuda", dtype=torch.int32)
    plan = h3a.rope_plan(128, scaling="parts", factor=4.0, original_length=2048)
    back, _ = h3a.rope(y, None, positions, plan, inverse=True)
    check(y, back, positions, frequencies(128, 10000.0, "parts", 4.0, 2048), False, inverse=True)
    turned, _ = h3a.rope(x, None, positions, plan)
    again, _ = h3a.rope(turned, None, positions, plan, inverse=True)
    # two roundings of values of the pair's length
    size = (x.double()[..., :64] ** 2 + x.double()[..., 64:] ** 2).sqrt().repeat(1, 1, 2)
    assert ((again.double() - x.double()).abs() <= size * 2 * 2.0 ** -8 * 1.5).all()
    # differences: the map is linear, so f(x + d) - f(x) = R d exactly in 64 bits
    left = (ref.rope(x, positions, frequencies(128, 10000.0, "parts", 4.0, 2048), False)[0] * y.double()).sum()
    right = (x.double() * ref.rope(y, positions, frequencies(128, 10000.0, "parts", 4.0, 2048), False, inverse=True)[0]).sum()
    assert abs(float(left - right)) <= 1e-9 * float((x.double().norm() * y.double().norm()))


def test_rope_passes_what_it_does_not_rotate():
    """NaN and infinities past the rotated channels come through bit for bit and touch nothing else."""
    q = randn(5, 2, 64)
    q[..., 32:40] = math.nan
    q[..., 40:48] = math.inf
    y, _ = h3a.rope(q, None, torch.arange(5, device="cuda", dtype=torch.int32), h3a.rope_plan(32))
    assert torch.equal(y[..., 32:].view(torch.int16), q[..., 32:].view(torch.int16)) and y[..., :32].isfinite().all()


def test_rope_empty_and_refusals():
    plan = h3a.rope_plan(64)
    q = randn(4, 2, 64)
    p = torch.arange(4, device="cuda", dtype=torch.int32)
    y, _ = h3a.rope(q[:0], None, p[:0], plan)
    assert y.shape == (0, 2, 64)
    with pytest.raises(ValueError, match="int32"):
        h3a.rope(q, None, p.long(), plan)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        h3a.rope(q.float(), None, p, plan)
    with pytest.raises(ValueError, match="same tokens"):
        h3a.rope(q, q[:2], p, plan)
    with pytest.raises(h3a.H3AError, match="INVALID_ARG"):
        h3a.rope(q[..., :32].contiguous(), None, p, plan)  # rotates more than the head has
    with pytest.raises(h3a.H3AError, match="INVALID_ARG"):
        h3a.rope(randn(4, 2, 65)[..., 1:], None, p, plan)  # strides and start not on 16 bytes
