"""Numbers that the prompt side's kernels take in 32 bits, without a GPU: one that is another number there is
refused (before the tensors are looked at)."""
import pytest
import torch

from rope_block_sparse_b200 import h3a
from test_prompt_abi import GOOD, NO_GPU, packed

Q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
I = torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("scale,match", [(1e-60, "scale"), (0.0, "CUDA"), (1e-30, "CUDA"), (0.125, "CUDA")])
def test_a_scale_that_would_select_the_default(scale, match):
    with pytest.raises(ValueError, match=match):
        h3a.packed_attention(Q, Q, Q, I, I, 4, 4, scale=scale)


@pytest.mark.parametrize("eps,match", [(1e-60, "eps"), (0.0, "CUDA"), (1e-30, "CUDA"), (1e-6, "CUDA")])
def test_an_eps_that_would_be_none(eps, match):
    with pytest.raises(ValueError, match=match):
        h3a.residual_rmsnorm(Q[:, 0], None, torch.ones(64), eps)


@NO_GPU
def test_a_scale_that_is_infinite_in_the_kernels_units():
    """Logits are kept times log2 e: 2^127.6 is finite and that is not."""
    def call(scale):
        return h3a.load().h3a_packed_attention(GOOD, GOOD, GOOD, packed(scale=scale, max_q=0), GOOD, GOOD, None, GOOD, None, None, 0, None)

    assert call(2.0 ** 127.6) == 1 and call(2.0 ** 127) == 0  # no query counts: nothing is launched
