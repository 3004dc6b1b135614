"""rope's inverse against the 64-bit form and, by its own outputs, as the transpose: every way the pairs are
loaded (a multiple of 8 or of 4 pairs, other numbers of neighbours and of halves), with an amplitude."""
import math

import pytest
import torch

import rope_block_sparse_b200 as h3a
import prompt_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def randn(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("amplitude", [1.0, 1.2079])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [128, 24, 50, 2])
def test_inverse_is_the_transpose(rotary, interleaved, amplitude, dtype):
    x, y = randn(301, 3, 128, dtype=dtype, seed=1), randn(301, 3, 128, dtype=dtype, seed=2)
    positions = torch.randint(-1000, 100000, (301,), device="cuda", dtype=torch.int32, generator=torch.Generator(device="cuda").manual_seed(3))
    f = [10000.0 ** (-2 * j / rotary) for j in range(rotary // 2)]
    plan = h3a.rope_plan(rotary, interleaved=interleaved, amplitude=amplitude)
    turned, back = h3a.rope(x, y, positions, plan)[0], h3a.rope(x, y, positions, plan, inverse=True)[1]
    want_turned, off_turned = ref.rope(x, positions, f, interleaved, amplitude)
    want_back, off_back = ref.rope(y, positions, f, interleaved, amplitude, inverse=True)
    ref.within(turned, want_turned, off_turned, "R x")
    ref.within(back, want_back, off_back, "R^T y")
    # <R x, y> = <x, R^T y>, off by what the outputs' roundings may add up to, and fp64's own
    left, right = (turned.double() * y.double()).sum(), (x.double() * back.double()).sum()
    room = (off_turned * y.double().abs()).sum() + (x.double().abs() * off_back).sum()
    assert abs(float(left - right)) <= float(room) + 1e-9 * float(x.double().norm() * y.double().norm())
    # the sign matters: the forward map of y is another one
    assert not torch.equal(back, h3a.rope(y, None, positions, plan)[0])
    in_place = y.clone()
    h3a.rope(in_place, None, positions, plan, inverse=True, inplace=True)
    assert torch.equal(in_place, back)


def test_a_quarter_turn_each_way():
    """Position 1 at a quarter of a turn: (a, b) goes to (-b, a), and the inverse to (b, -a), exactly."""
    for interleaved in (False, True):
        x = randn(1, 2, 16, dtype=torch.bfloat16, seed=4)
        plan = h3a.rope_plan(16, interleaved=interleaved, frequencies=[math.pi / 2] * 8)
        a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :8], x[..., 8:])
        one = torch.ones(1, device="cuda", dtype=torch.int32)
        join = (lambda u, v: torch.stack((u, v), -1).flatten(-2)) if interleaved else (lambda u, v: torch.cat((u, v), -1))
        assert torch.equal(h3a.rope(x, None, one, plan)[0], join(-b, a))
        assert torch.equal(h3a.rope(x, None, one, plan, inverse=True)[0], join(b, -a))
