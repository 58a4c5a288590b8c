"""A capacity that the means do not belong to is refused (no GPU)."""
import pytest
import torch

from block_sparse_attention_tok_b200 import sparstar as S


@pytest.mark.parametrize("capacity", [0, 128, 256, 385, 1 << 40, -1])
def test_refuses_a_capacity_of_other_blocks(capacity):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    means, kv_len = torch.zeros(2, 2, 3, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="capacity"):
        S.token_select(q, means, kv_len, 2, capacity=capacity)


@pytest.mark.parametrize("capacity", [None, 257, 300, 384])
def test_takes_one_of_the_same_blocks(capacity):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    means, kv_len = torch.zeros(2, 2, 3, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):  # the next thing that is checked
        S.token_select(q, means, kv_len, 2, capacity=capacity)
