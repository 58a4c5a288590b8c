"""The bounds of the norm's tests tell a wrong eps from the right one where eps is near the mean square
(no GPU): a form with twice the eps, with none, or with it added behind the root lies outside them."""
import pytest
import torch

from tests import norm_rope_ref as R

EPS = 1e-6


def inputs():
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(17, 5, 64, generator=g, dtype=torch.float64) for _ in range(2))
    a = torch.rand(17, 32, generator=g, dtype=torch.float64)
    return 1e-3 * x, dy, 1 + 0.3 * torch.randn(64, generator=g), a.cos().float(), a.sin().float()


@pytest.mark.parametrize("wrong", [0.0, 2 * EPS, EPS / 64])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_another_eps_is_outside(wrong, dtype):
    x, dy, w, cos, sin = inputs()
    y, tol = R.forward(x, w, cos, sin, EPS, False)
    assert ((R.forward(x, w, cos, sin, wrong, False)[0] - y).abs() > tol).any()
    dx, tol, dw, sums = R.backward(x, dy, w, cos, sin, EPS, False, dtype)
    dx2, _, dw2, _ = R.backward(x, dy, w, cos, sin, wrong, False, dtype)
    assert ((dx2 - dx).abs() > tol).any() and ((dw2 - dw).abs() > R.dw_tol(17, 11, 64, sums)).any()


def test_eps_behind_the_root_is_outside():
    x, _, w, cos, sin = inputs()
    y, tol = R.forward(x, w, cos, sin, EPS, False)
    u = x / (x.square().mean(-1, keepdim=True).sqrt() + EPS) * w.double()
    assert ((R.turn(u, cos, sin, False) - y).abs() > tol).any()
