"""Views whose sequences the gradient of the norm has no use for are refused, as the forward call refuses
them (no GPU)."""
import pytest

from block_sparse_attention_tok_b200 import sparstar as S
from tests.test_norm_rope_checks import bwd

X, Y = S.View(0x1000, 512, 128, 8), S.View(0x2000, 128, 12800, 8)


@pytest.mark.parametrize("over", [dict(dq=Y), dict(dk=Y), dict(dv=Y), dict(q=X), dict(k=X), dict(dqi=X), dict(dki=X),
                                  dict(dvi=X)])
def test_gradient_refuses_a_sequence_stride(over):
    assert bwd(S.load(), **over, ws=None) == S.ERR_ARG  # without a workspace: refused there at the latest
