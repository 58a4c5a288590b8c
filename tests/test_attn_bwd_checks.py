"""Refusals and workspace sizes of the attention gradient (no GPU)."""
import ctypes

import pytest
import torch

from block_sparse_attention_tok_b200 import sparstar as S
from tests import attn_bwd_ref as R


def call(**over):
    a = dict(do=0x1000, q=0x1000, k=0x1000, v=0x1000, o=0x1000, lse=0x1000, heads=2, n_q=300, n_kv=500, d=128,
             block=128, idx=0x1000, cnt=0x1000, kmax=4, scale=0.0, dq=0x1000, dk=0x1000, dv=0x1000, ws=0x1000,
             nbytes=1 << 30)
    a.update(over)
    return S.load().sparstar_attn_bwd(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(heads=0), S.ERR_ARG), (dict(n_q=-1), S.ERR_ARG), (dict(n_kv=0), S.ERR_ARG), (dict(kmax=0), S.ERR_ARG),
    (dict(d=96), S.ERR_UNSUPPORTED), (dict(block=32), S.ERR_UNSUPPORTED), (dict(heads=70000), S.ERR_UNSUPPORTED),
    (dict(n_kv=49152 * 128 + 1), S.ERR_UNSUPPORTED), (dict(n_kv=49152 * 64 + 1, block=64), S.ERR_UNSUPPORTED),
    (dict(n_q=2 ** 31), S.ERR_UNSUPPORTED), (dict(n_q=2 ** 30, kmax=2 ** 20), S.ERR_UNSUPPORTED),
    (dict(scale=float("nan")), S.ERR_ARG), (dict(scale=float("inf")), S.ERR_ARG),
    (dict(do=None), S.ERR_ARG), (dict(q=0x1008), S.ERR_ARG), (dict(k=None), S.ERR_ARG), (dict(v=0x1004), S.ERR_ARG),
    (dict(o=None), S.ERR_ARG), (dict(lse=None), S.ERR_ARG), (dict(lse=0x1002), S.ERR_ARG), (dict(idx=None), S.ERR_ARG),
    (dict(cnt=0x1001), S.ERR_ARG), (dict(dq=None), S.ERR_ARG), (dict(dk=None), S.ERR_ARG), (dict(dv=0x1008), S.ERR_ARG),
    (dict(ws=None), S.ERR_WORKSPACE), (dict(ws=0x1080), S.ERR_WORKSPACE), (dict(nbytes=100), S.ERR_WORKSPACE),
])
def test_refuses(over, code):
    assert call(**over) == code


@pytest.mark.parametrize("heads,n_q,n_kv,block,kmax", [(2, 300, 500, 128, 4), (1, 1, 1, 64, 1), (4, 72192, 144896, 128, 107)])
def test_workspace_size(heads, n_q, n_kv, block, kmax):
    def al(x):
        return (x + 255) // 256 * 256
    nqb, nkb = -(-n_q // block), -(-n_kv // block)
    chunks = -(-nqb // 32)
    share = max(16, -(-heads * nqb * kmax // 148))      # entries of a part of a long list
    parts = 0 if nqb * kmax <= share else min(2 * heads * nqb * kmax // share, 296)
    want = (256 + al(296 * 8 * 4) + al(296 * 20) + parts * 2 * block * 128 * 4 + 2 * al(heads * nqb * block * 4) + 2 * al(heads * chunks * nkb * 4) + al(heads * chunks * 4)
            + al(heads * (nkb + 1) * 4) + al(heads * nqb * kmax * 4))
    assert S.attn_bwd_workspace_size(heads, n_q, n_kv, 128, kmax, block) == want
    with pytest.raises(S.SparstarError):
        S.attn_bwd_workspace_size(heads, n_q, n_kv, 100, kmax, block)
    assert S.load().sparstar_attn_bwd_workspace_size(1, 1, 1, 128, 128, 1, None) == S.ERR_ARG
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def test_reference_gradient_against_autograd():
    """The formula that the kernels are held to is the derivative of the forward pass."""
    g = torch.Generator().manual_seed(1)
    n_q, n_kv, d, block = 20, 45, 8, 8
    q, k, v = (torch.randn(n, d, generator=g, dtype=torch.float64).requires_grad_() for n in (n_q, n_kv, n_kv))
    idx = torch.tensor([[0, 5, 2], [1, 1, 4], [3, 0, 0]], dtype=torch.int32)
    cnt = torch.tensor([3, 2, 1], dtype=torch.int32)
    w = R.multiplicity(idx, cnt, n_q, n_kv, block)
    assert w[0, 40] == 1 and w[8, 8] == 2 and w[16, 0] == 0
    o, lse = R.head_forward(q, k, v, w, 0.3)
    do = torch.randn(o.shape, generator=g, dtype=torch.float64)
    (o * do).sum().backward()
    for x, (val, tol, _) in zip((q, k, v), R.head_backward(do, *(t.detach() for t in (q, k, v, o, lse)), w, 0.3)):
        assert torch.allclose(x.grad, val, rtol=1e-12, atol=1e-12) and (tol > 0).all()
