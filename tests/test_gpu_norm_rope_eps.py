"""The norm with rotation and its gradient where eps decides: none at all, one of the size of the mean
square, one beyond it; with tokens and heads that leave places of a tile empty. Bounds of
tests/norm_rope_ref.py: eps adds two roundings below the root (its own to fp32 and the sum), u / 2 each
behind it, which the 16 u of the forward bound and the 64 u of the gradient's have room for."""
import pytest
import torch

from tests import norm_rope_ref as R
from tests.test_gpu_norm_rope import check, make, rope_args

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


def run(S, n, hq, hk, d, dtype, eps, scale, interleaved=False):
    t = make(n, hq, hk, d, dtype, n + hq + d, scale=scale)
    q_out, k_out, v_out = S.qk_norm_rope(t["q"], t["k"], t["v"], eps=eps, interleaved=interleaved, **rope_args(t))
    got = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], dv=t["dv"], eps=eps, interleaved=interleaved,
                             **rope_args(t))
    for name, x, w, y, dy, dx, dw, h in (("q", t["q"], t["wq"], q_out, t["dq"], got[0], got[3], hq),
                                         ("k", t["k"], t["wk"], k_out, t["dk"], got[1], got[4], hk)):
        assert all(torch.isfinite(r).all() for r in (y, dx, dw)), name
        ref, tol = R.forward(x, w, t["cos"], t["sin"], eps, interleaved)
        check(y, ref.transpose(0, 1), tol.transpose(0, 1), name)
        ref, tol, dw_ref, sums = R.backward(x, dy.transpose(0, 1), w, t["cos"], t["sin"], eps, interleaved, dtype)
        check(dx, ref, tol, "d" + name)
        check(dw, dw_ref, R.dw_tol(n, hq + 2 * hk, d, sums), "dw" + name)
    assert torch.equal(v_out, t["v"].bfloat16().transpose(0, 1)) and torch.equal(got[2], t["dv"].to(dtype).transpose(0, 1))
    assert S.device_status() == S.OK


@pytest.mark.parametrize("eps,scale", [(0.0, 1.5), (0.0, 1e-3), (1e-6, 1e-3), (0.5, 1.5), (0.5, 1e-3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (17, 5, 3), (70, 6, 2), (2049, 9, 3)])
def test_eps(S, n, hq, hk, d, dtype, eps, scale):
    run(S, n, hq, hk, d, dtype, eps, scale)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_one_token_of_whole_items_of_heads(S, d, dtype, interleaved):
    run(S, 1, 32, 8, d, dtype, 1e-6, 1.5, interleaved)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_against_differences_where_eps_decides(S, dtype):
    """As tests/test_gpu_norm_rope.py has it, with eps near the mean square (about 2.25)."""
    t = make(24, 3, 2, 64, dtype, 10)
    eps = 1.75
    got = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], eps=eps, **rope_args(t))
    g = torch.Generator(device="cuda").manual_seed(12)
    for x, dy, w, dx, dw in ((t["q"], t["dq"], t["wq"], got[0], got[3]), (t["k"], t["dk"], t["wk"], got[1], got[4])):
        dy = dy.double().transpose(0, 1)

        def loss(xx, ww):
            u = xx / (xx.square().mean(-1, keepdim=True) + eps).sqrt() * ww
            return (R.turn(u, t["cos"], t["sin"], False) * dy).sum().item()

        _, tol, _, sums = R.backward(x, dy, w, t["cos"], t["sin"], eps, False, dtype)
        xd, wd = x.double(), w.double()
        for _ in range(3):
            e = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
            diff = (loss(xd + 1e-5 * e, wd) - loss(xd - 1e-5 * e, wd)) / 2e-5
            assert abs(diff - (dx.double() * e).sum().item()) <= (tol * e.abs()).sum().item() + 1e-6
            f = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
            diff = (loss(xd, wd + 1e-5 * f) - loss(xd, wd - 1e-5 * f)) / 2e-5
            assert abs(diff - (dw.double() * f).sum().item()) <= (R.dw_tol(24, 5, 64, sums) * f.abs()).sum().item() + 1e-6
