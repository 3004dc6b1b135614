"""packed_attention_workspace_size: what the call itself needs, without a GPU."""
import ctypes

import pytest
import torch

from rope_block_sparse_b200 import h3a


def needed(total_q, total_k, heads, kv, d, seqs, max_q, max_k, causal):
    """Bytes by the C call, for contiguous tensors."""
    n = ctypes.c_size_t(0)
    desc = h3a.PackedDesc(0, seqs, heads, kv, d, total_q, total_k, max_q, max_k, heads * d, d, kv * d, d, kv * d, d, heads * d, d, causal, 0.0)
    assert h3a.load().h3a_packed_attention_workspace_size(desc, n) == 0
    return n.value


def meta(rows, heads, d):
    return torch.empty(rows, heads, d, dtype=torch.bfloat16, device="meta")


# total_q, total_k, heads, kv heads, head_dim: one sequence, whose number of parts depends on the mask
SHAPES = [(2583, 12909, 8, 2, 64), (7286, 39934, 2, 2, 128), (6245, 6245, 4, 4, 96)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_the_mask_counts(shape, causal):
    nq, nk, h, kv, d = shape
    size = h3a.packed_attention_workspace_size(meta(nq, h, d), meta(nk, kv, d), 1, nq, nk, causal=causal)
    assert size == needed(nq, nk, h, kv, d, 1, nq, nk, causal)


def test_the_shapes_above_differ_by_the_mask():
    for nq, nk, h, kv, d in SHAPES:
        assert needed(nq, nk, h, kv, d, 1, nq, nk, 1) != needed(nq, nk, h, kv, d, 1, nq, nk, 0)


def test_causal_is_the_default_as_in_the_call():
    nq, nk, h, kv, d = SHAPES[0]
    assert h3a.packed_attention_workspace_size(meta(nq, h, d), meta(nk, kv, d), 1, nq, nk) == needed(*SHAPES[0], 1, nq, nk, 1)
    assert h3a.packed_attention_workspace_size(meta(nq, h, d), meta(nk, kv, d), 1, nq, nk, False) == needed(*SHAPES[0], 1, nq, nk, 0)
