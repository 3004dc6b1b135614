"""rope_plan's arguments, without a GPU: what a plan is made from is the value at the call."""
import numpy as np
import pytest
import torch

from rope_block_sparse_b200 import h3a


def turns(plan):
    return list(plan.turns[:plan.pairs])


@pytest.mark.parametrize("name,first,then,kw", [
    ("theta", 10000.0, 500000.0, {}),
    ("factor", 2.0, 8.0, dict(scaling="linear")),
    ("amplitude", 1.0, 1.25, {}),
    ("original_length", 64, 4096, dict(scaling="parts", factor=4.0)),
    ("low_turns", 1.0, 2.0, dict(scaling="parts", factor=4.0, original_length=4096)),
    ("high_turns", 32.0, 8.0, dict(scaling="parts", factor=4.0, original_length=4096)),
    ("rotary_dim", 64, 32, {}),
    ("interleaved", False, True, {}),
])
def test_a_tensor_written_to_later_gets_its_new_plan(name, first, then, kw):
    """A number in a 0-d tensor: the same tensor with another value in it is another argument."""
    kw = {"rotary_dim": 64, **kw}
    number = torch.tensor(first, dtype=torch.float64 if isinstance(first, float) else None)
    before = h3a.rope_plan(**{**kw, name: number})
    number.fill_(then)
    after = h3a.rope_plan(**{**kw, name: number})
    for got, value in ((before, first), (after, then)):
        want = h3a.rope_plan(**{**kw, name: value})
        assert bytes(got) == bytes(want)
    assert bytes(before) != bytes(after)


def test_numpy_numbers():
    want = h3a.rope_plan(64, 500000.0, scaling="linear", factor=4.0)
    assert turns(h3a.rope_plan(np.int64(64), np.float64(500000.0), scaling="linear", factor=np.float32(4.0))) == turns(want)
    array = np.array(4.0)
    assert turns(h3a.rope_plan(64, 500000.0, scaling="linear", factor=array)) == turns(want)
    array[...] = 2.0
    assert turns(h3a.rope_plan(64, 500000.0, scaling="linear", factor=array)) == turns(h3a.rope_plan(64, 500000.0, scaling="linear", factor=2.0))


def test_plans_of_equal_numbers_are_one():
    """Plain numbers find their plan however they are written, tensors find it by value."""
    want = h3a.rope_plan(96, 10000.0, scaling="linear", factor=2.0)
    assert h3a.rope_plan(96, 10000, False, "linear", 2) is want
    assert h3a.rope_plan(96, 10000, False, "linear", torch.tensor(2.0)) is want


@pytest.mark.parametrize("kw", [dict(rotary_dim=64.7), dict(rotary_dim=torch.tensor(64.5)), dict(rotary_dim=float("nan")), dict(rotary_dim=float("inf")),
                                dict(rotary_dim=2 ** 32 + 64), dict(rotary_dim=64, scaling="parts", original_length=100.5),
                                dict(rotary_dim=64, scaling="parts", original_length=2 ** 64 + 100)], ids=str)
def test_numbers_that_are_not_whole_are_refused(kw):
    """Neither cut to a whole number nor to the C call's type."""
    with pytest.raises(ValueError, match=next(n for n in ("original_length", "rotary_dim") if n in kw)):
        h3a.rope_plan(**kw)


def test_whole_numbers_in_any_form():
    want = h3a.rope_plan(64, scaling="parts", factor=2.0, original_length=4096)
    for r, n in ((64.0, 4096.0), (torch.tensor(64), torch.tensor(4096.0)), (np.int32(64), np.float32(4096))):
        assert bytes(h3a.rope_plan(r, scaling="parts", factor=2.0, original_length=n)) == bytes(want)


@pytest.mark.parametrize("kw", [dict(amplitude=1e39), dict(amplitude=-1e300), dict(scaling="base", theta=1e300, factor=1e300),
                                dict(frequencies=[0.5] * 32, amplitude=1e39)], ids=str)
def test_numbers_that_are_infinite_in_the_plan_are_refused(kw):
    """Finite as given, but the amplitude is kept in 32 bits, and a stretched base may leave 64."""
    with pytest.raises(h3a.H3AError, match="INVALID_ARG"):
        h3a.rope_plan(64, **kw)
