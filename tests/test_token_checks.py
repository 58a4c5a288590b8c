"""Refusals of the single-token entry points, before any device is touched (no GPU)."""
import pytest
import torch

from block_sparse_attention_tok_b200 import sparstar as S
from tests import token_ref as R

BASE = dict(q=0x1000, k=0x1000, v=0x1000, kv_len=0x1000, means=0x1000, b=2, hq=8, hk=2, cap=1000, d=128, keep=8, sink=1,
            recent=1, scale=0.0, idx=0x1000, cnt=0x1000, o=0x1000, lse=0x1000)


def forward(**over):
    a = dict(BASE, **over)
    return S.load().sparstar_token_forward(*a.values(), None)


def attn(**over):
    a = dict(BASE, **over)
    return S.load().sparstar_token_attn(a["q"], a["k"], a["v"], a["kv_len"], a["b"], a["hq"], a["hk"], a["cap"], a["d"],
                                        a["idx"], a["cnt"], a["keep"], a["scale"], a["o"], a["lse"], None)


def select(**over):
    a = dict(BASE, **over)
    return S.load().sparstar_token_select(a["q"], a["means"], a["kv_len"], a["b"], a["hq"], a["hk"], a["cap"], a["d"],
                                          a["keep"], a["sink"], a["recent"], a["idx"], a["cnt"], None)


def means(**over):
    a = dict(BASE, **over)
    return S.load().sparstar_block_means(a["k"], a["kv_len"], a["b"], a["hk"], a["cap"], a["d"], 0, a["means"], None)


@pytest.mark.parametrize("fn", [forward, attn, select, means])
@pytest.mark.parametrize("over,code", [
    (dict(b=-1), S.ERR_ARG), (dict(hk=0), S.ERR_ARG), (dict(cap=0), S.ERR_ARG), (dict(d=96), S.ERR_UNSUPPORTED),
    (dict(b=65536), S.ERR_UNSUPPORTED), (dict(hk=70000, hq=70000), S.ERR_UNSUPPORTED),
    (dict(cap=16384 * 128 + 1), S.ERR_UNSUPPORTED), (dict(kv_len=None), S.ERR_ARG), (dict(kv_len=0x1002), S.ERR_ARG),
])
def test_sizes_and_lengths(fn, over, code):
    assert fn(**over) == code


@pytest.mark.parametrize("fn,over,code", [
    (f, o, c) for fs, o, c in [
        ((forward, attn, select), dict(hq=9), S.ERR_ARG), ((forward, attn, select), dict(hq=34), S.ERR_UNSUPPORTED),
        ((forward, attn, select), dict(hq=0), S.ERR_ARG), ((forward, attn, select), dict(keep=0), S.ERR_ARG),
        ((forward, attn, select), dict(q=0x1008), S.ERR_ARG), ((forward, attn, select), dict(idx=None), S.ERR_ARG),
        ((forward, attn, select), dict(cnt=0x1001), S.ERR_ARG), ((forward, select), dict(sink=-1), S.ERR_ARG),
        ((forward, select), dict(recent=0), S.ERR_ARG), ((forward, select), dict(sink=8), S.ERR_ARG),
        ((forward, select), dict(recent=9), S.ERR_ARG), ((forward, select), dict(means=0x1004), S.ERR_ARG),
        ((forward, select), dict(sink=2 ** 31 - 1), S.ERR_ARG),
        ((forward, attn), dict(k=None), S.ERR_ARG), ((forward, attn), dict(v=0x1008), S.ERR_ARG),
        ((forward, attn), dict(o=None), S.ERR_ARG), ((forward, attn), dict(lse=0x1002), S.ERR_ARG),
        ((forward, attn), dict(scale=float("nan")), S.ERR_ARG), ((means,), dict(k=0x1008), S.ERR_ARG),
        ((means,), dict(means=None), S.ERR_ARG),
    ] for f in fs])
def test_arguments(fn, over, code):
    assert fn(**over) == code


def test_no_sequences_is_a_no_op():
    assert [f(b=0) for f in (forward, attn, select, means)] == [S.OK] * 4


def test_binding_refuses_wrong_tensors():
    k = torch.zeros(2, 2, 300, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    m = torch.zeros(2, 2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        S.token_forward(q, k, k, n, m, 2)
    with pytest.raises(ValueError, match="means"):
        S.token_forward(q, k, k, n, m[:, :, :2], 2)
    with pytest.raises(ValueError, match="kv_len"):
        S.block_means(k, n.long())
    with pytest.raises(ValueError, match="multiple"):
        S.token_forward(q[:, :3].contiguous(), k, k, n, m, 2)
    with pytest.raises(ValueError, match="cache"):
        S.block_means(k.float(), n)


def test_reference_choice():
    means = torch.tensor([[9.0], [1.0], [3.0], [3.0], [float("nan")], [2.0], [0.0]])
    q = torch.ones(2, 1)
    assert R.choose(q, means, 7 * 128, 4, 1, 1) == [0, 2, 3, 6]
    assert R.choose(q, means, 7 * 128, 3, 1, 1) == [0, 2, 6]
    assert R.choose(q, means, 7 * 128, 6, 0, 1) == [0, 1, 2, 3, 5, 6]
    assert R.choose(q, means, 130, 6, 0, 1) == [0, 1]
    assert R.choose(q, means, 0, 6, 0, 1) == []
