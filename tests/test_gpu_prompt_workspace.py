"""packed_attention with a caller's workspace of exactly the size that packed_attention_workspace_size names."""
import pytest
import torch

import rope_block_sparse_b200 as h3a
import prompt_reference as ref

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


def dev(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,heads,kv,d", [(2583, 12909, 8, 2, 64), (70, 9000, 4, 2, 128), (1, 20000, 8, 2, 96)], ids=str)
def test_size_is_what_the_call_takes(lq, lk, heads, kv, d, causal):
    q, k, v = randn(lq, heads, d, seed=1), randn(lk, kv, d, seed=2), randn(lk, kv, d, seed=3)
    size = h3a.packed_attention_workspace_size(q, k, 1, lq, lk, causal=causal)
    assert size > 0
    room = torch.full((size + 256,), 171, dtype=torch.uint8, device="cuda")
    o = h3a.packed_attention(q, k, v, dev(0, lq), dev(0, lk), lq, lk, causal=causal, workspace=room[:size])
    assert (room[size:] == 171).all()
    rows = torch.arange(0, lq, max(1, lq // 60), device="cuda")
    for r in rows.tolist():  # each against its own keys, the last lk - lq + r + 1 of them causal
        seen = lk - lq + r + 1 if causal else lk
        want, _, bound, _ = ref.attention(q[r:r + 1], k[:seen], v[:seen], [0, 1], [0, seen])
        ref.within(o[r:r + 1], want, bound, f"row {r}")
    with pytest.raises(h3a.H3AError, match="WORKSPACE"):
        h3a.packed_attention(q, k, v, dev(0, lq), dev(0, lk), lq, lk, causal=causal, workspace=room[:size - 256])
