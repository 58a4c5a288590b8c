"""The workspace of token_forward: its shapes and what it refuses (no GPU)."""
import pytest
import torch

from block_sparse_attention_tok_b200 import sparstar as S


def test_holds_the_lists_of_one_shape():
    ws = S.TokenWorkspace(3, 8, 2, 1000, 64, 5, "cpu")
    assert ws.idx.shape == (3, 2, 5) and ws.cnt.shape == (3, 2)
    assert all(t.dtype == torch.int32 and t.is_contiguous() for t in (ws.idx, ws.cnt))
    ws.idx.fill_(1)
    ws.cnt.fill_(2)
    assert (ws.idx == 1).all() and ws.buf.numel() == ws.idx.numel() + ws.cnt.numel()
    ws.check(3, 8, 2, 1000, 64, 5)
    assert S.TokenWorkspace(0, 8, 2, 1000, 64, 5, "cpu").idx.shape == (0, 2, 5)


@pytest.mark.parametrize("shape", [(2, 8, 2, 1000, 64, 5), (3, 4, 2, 1000, 64, 5), (3, 8, 1, 1000, 64, 5),
                                   (3, 8, 2, 999, 64, 5), (3, 8, 2, 1000, 128, 5), (3, 8, 2, 1000, 64, 6)])
def test_refuses_a_call_of_another_shape(shape):
    with pytest.raises(ValueError, match="workspace is for"):
        S.TokenWorkspace(3, 8, 2, 1000, 64, 5, "cpu").check(*shape)


@pytest.mark.parametrize("shape", [(-1, 8, 2, 1000, 64, 5), (3, 0, 2, 1000, 64, 5), (3, 8, 0, 1000, 64, 5),
                                   (3, 8, 2, 0, 64, 5), (3, 8, 2, 1000, 0, 5), (3, 8, 2, 1000, 64, 0)])
def test_refuses_sizes_that_no_call_has(shape):
    with pytest.raises(ValueError, match="no call has"):
        S.TokenWorkspace(*shape, "cpu")
