"""Refusals of the norm-with-rotation entry points, before any device is touched (no GPU)."""
import pytest
import torch

from block_sparse_attention_tok_b200 import sparstar as S

V = S.View
OK_X, OK_Y = V(0x1000, 512, 128, 0), V(0x2000, 128, 12800, 0)
NONE = V(None, 0, 0, 0)


def fwd(lib, **over):
    a = dict(q=OK_X, k=OK_X, v=OK_X, dt=S.BF16, n=100, hq=4, hk=4, d=128, wq=0x100, wk=0x100, cos=0x100, sin=0x100,
             eps=1e-6, il=0, qo=OK_Y, ko=OK_Y, vo=OK_Y, rows=None, off=0, cap=100)
    a.update(over)
    return lib.sparstar_qk_norm_rope(a["q"], a["k"], a["v"], a["dt"], a["n"], a["hq"], a["hk"], a["d"], a["wq"],
                                     a["wk"], a["cos"], a["sin"], a["eps"], a["il"], a["qo"], a["ko"], a["vo"],
                                     a["rows"], a["off"], a["cap"], None)


@pytest.mark.parametrize("over,code", [
    (dict(d=96), S.ERR_UNSUPPORTED), (dict(dt=2), S.ERR_ARG), (dict(n=-1), S.ERR_ARG), (dict(hq=0), S.ERR_ARG),
    (dict(hk=-1), S.ERR_ARG), (dict(hq=70000), S.ERR_UNSUPPORTED), (dict(n=2 ** 31), S.ERR_UNSUPPORTED),
    (dict(eps=-1.0), S.ERR_ARG), (dict(eps=float("nan")), S.ERR_ARG), (dict(eps=float("inf")), S.ERR_ARG),
    (dict(cos=None), S.ERR_ARG), (dict(sin=None), S.ERR_ARG), (dict(cos=0x104), S.ERR_ARG), (dict(wq=0x104), S.ERR_ARG),
    (dict(q=V(None, 512, 128, 0)), S.ERR_ARG), (dict(q=V(0x1008, 512, 128, 0)), S.ERR_ARG),
    (dict(q=V(0x1000, 516, 128, 0)), S.ERR_ARG), (dict(q=V(0x1000, 0, 128, 0)), S.ERR_ARG),
    (dict(q=V(0x1000, 512, 128, 8)), S.ERR_ARG), (dict(qo=V(0x2000, 128, 12800, 8)), S.ERR_ARG),
    (dict(ko=V(0x2000, 128, 12800, 8)), S.ERR_ARG), (dict(ko=V(None, 128, 12800, 0)), S.ERR_ARG),
    (dict(v=NONE), S.ERR_ARG), (dict(vo=NONE), S.ERR_ARG), (dict(off=1), S.ERR_ARG), (dict(off=-1), S.ERR_ARG),
    (dict(cap=99), S.ERR_ARG), (dict(rows=0x102), S.ERR_ARG),
])
def test_forward_refuses(over, code):
    assert fwd(S.load(), **over) == code


def bwd(lib, **over):
    a = dict(dq=OK_Y, dk=OK_Y, dv=OK_Y, q=OK_X, k=OK_X, dt=S.FP32, n=100, hq=4, hk=4, d=128, eps=1e-6, off=0, dqi=OK_X,
             dki=OK_X, dvi=OK_X, dwq=0x100, dwk=0x100, ws=0x1000, nbytes=1 << 30)
    a.update(over)
    return lib.sparstar_qk_norm_rope_bwd(a["dq"], a["dk"], a["dv"], a["q"], a["k"], a["dt"], a["n"], a["hq"], a["hk"],
                                         a["d"], None, None, None, None, a["eps"], 0, a["off"], a["dqi"], a["dki"],
                                         a["dvi"], a["dwq"], a["dwk"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("over,code", [
    (dict(d=32), S.ERR_UNSUPPORTED), (dict(off=-1), S.ERR_ARG), (dict(q=V(0x1000, 514, 128, 0)), S.ERR_ARG),
    (dict(k=NONE), S.ERR_ARG), (dict(dvi=NONE), S.ERR_ARG), (dict(dq=V(0x2002, 128, 12800, 0)), S.ERR_ARG),
    (dict(dwq=0x101), S.ERR_ARG), (dict(ws=None), S.ERR_WORKSPACE), (dict(ws=0x1008), S.ERR_WORKSPACE),
    (dict(nbytes=1000), S.ERR_WORKSPACE),
])
def test_gradient_refuses(over, code):
    assert bwd(S.load(), **over) == code


def test_no_tokens_is_a_no_op_and_workspace_is_sized():
    assert fwd(S.load(), n=0) == S.OK
    import ctypes
    out = ctypes.c_size_t()
    assert S.load().sparstar_qk_norm_rope_bwd_workspace_size(128, ctypes.byref(out)) == S.OK
    assert out.value == 1024 * 128 * 4
    assert S.load().sparstar_qk_norm_rope_bwd_workspace_size(96, ctypes.byref(out)) == S.ERR_UNSUPPORTED


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    q, k = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        S.qk_norm_rope(q, k)
    with pytest.raises(ValueError, match="k must be"):
        S.qk_norm_rope(q, k[:3])
    with pytest.raises(ValueError, match="contiguous"):
        S.qk_norm_rope(q.repeat(1, 1, 2)[..., ::2], k)
    with pytest.raises(ValueError, match="q must be"):
        S.qk_norm_rope(q.half(), k)
    with pytest.raises(ValueError, match="come together"):
        S.qk_norm_rope(q, k, cos=torch.zeros(4, 32))
    with pytest.raises(ValueError, match="cos must be"):
        S.qk_norm_rope(q, k, cos=torch.zeros(4, 64), sin=torch.zeros(4, 64))
    with pytest.raises(ValueError, match="v comes with k"):
        S.qk_norm_rope(q, None, k)
