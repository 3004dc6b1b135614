"""Given outputs of the prompt side's calls: all that the call writes and nothing else, or it is refused.  No
GPU: what is given or None is looked at before the tensors are."""
import itertools

import pytest
import torch

from rope_block_sparse_b200 import h3a

X = torch.zeros(4, 64, dtype=torch.bfloat16)
Y8 = torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
S = torch.zeros(4)
GAMMA = torch.ones(64)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("scales", [None, "row"])
@pytest.mark.parametrize("given", list(itertools.product([True, False], repeat=3)), ids=str)
def test_rmsnorm_outputs_are_whole(given, scales, residual):
    out = tuple(t.clone() if g else None for g, t in zip(given, (X, X if scales is None else Y8, S)))
    whole = given == (residual, True, scales is not None)
    # what is whole, or all None (fresh ones), goes on to the tensors, which are not on a GPU here
    match = "CUDA" if whole or not any(given) else "out must hold"
    with pytest.raises(ValueError, match=match):
        h3a.residual_rmsnorm(X, X if residual else None, GAMMA, scales=scales, out=out)


@pytest.mark.parametrize("with_k", [True, False])
@pytest.mark.parametrize("given", list(itertools.product([True, False], repeat=2)), ids=str)
def test_rope_outputs_are_whole(given, with_k):
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    out = tuple(q.clone() if g else None for g in given)
    match = "CUDA" if given == (True, with_k) or not any(given) else "out must hold"
    with pytest.raises(ValueError, match=match):
        h3a.rope(q, q if with_k else None, torch.zeros(4, dtype=torch.int32), h3a.rope_plan(64), out=out)


def test_rope_in_place_has_no_other_output():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="inplace"):
        h3a.rope(q, q, torch.zeros(4, dtype=torch.int32), h3a.rope_plan(64), inplace=True, out=(q.clone(), q.clone()))
