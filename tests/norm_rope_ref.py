"""fp64 form of the norm with rotation and its gradient, and the error bounds of its fp32 kernels.

Bounds. The kernels compute in fp32 (half step u = 2^-24) and round each output once.
Forward: the sum of squares of d values takes at most 8 + 4 dependent roundings of positive
terms and a division by d that is exact: relative error below 12 u, halved by the square root;
rsqrt adds at most 2 units = 4 u, and the products by r and w two more roundings: below 12 u on
each coordinate of u = w r x. The turn adds two products and a sum (3 u): below 16 u = 2^-20 of
|a| + |b| in all. A bf16 output adds half a step, 2^-8 of the value.
Gradient: g = w R^T dy has below 4 u of |w| (|a| + |b|); xh = r x below 11 u; the mean of g xh adds
at most 12 roundings and the two errors: below 30 u of its sum of absolute values; the difference
and the product by r add 3 u and r's own 10 u: below 64 u = 2^-18 of
r (|g|_max + |xh| mean(|g|_max |xh|)), |g|_max = |w| (|a| + |b|). A bf16 output adds 2^-8 of the value.
dw: each term has below 16 u of (|a| + |b|) |xh|; the sum's longest chain is (terms of a lane) +
(32 groups at most) + (32 rows of a slice at most) + 32 slices.
"""
import torch

U = 2.0 ** -24


def pairs(d, interleaved, device):
    a = torch.arange(0, d, 2, device=device) if interleaved else torch.arange(d // 2, device=device)
    return a, a + (1 if interleaved else d // 2)


def turn(x, cos, sin, interleaved):
    """x [N, H, d] fp64 turned by cos, sin [N, d/2]."""
    if cos is None:
        return x.clone()
    a, b = pairs(x.shape[-1], interleaved, x.device)
    c, s = cos.double()[:, None], sin.double()[:, None]
    y = torch.empty_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def pair_abs(x, interleaved, rotated):
    """|a| + |b| at both members of each pair (|x| where nothing is turned)."""
    if not rotated:
        return x.abs()
    a, b = pairs(x.shape[-1], interleaved, x.device)
    y = torch.empty_like(x)
    y[..., a] = y[..., b] = x[..., a].abs() + x[..., b].abs()
    return y


def forward(x, w, cos, sin, eps, interleaved):
    """(y [N, H, d] fp64, bound of a bf16 kernel output's error)."""
    x = x.double()
    u = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if w is None else w.double())
    y = turn(u, cos, sin, interleaved)
    tol = 2.0 ** -20 * pair_abs(u, interleaved, cos is not None)
    return y, tol + 2.0 ** -8 * (y.abs() + tol) + 2.0 ** -134


def backward(x, dy, w, cos, sin, eps, interleaved, out_dtype):
    """(dx, bound, dw, sum over the terms of dw of their absolute values) in fp64; dy [N, H, d]."""
    x, dy = x.double(), dy.double()
    wd = torch.ones(x.shape[-1], device=x.device, dtype=torch.float64) if w is None else w.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xh = x * r
    dn = turn(dy, cos, None if sin is None else -sin.double(), interleaved)
    g = dn * wd
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    most = pair_abs(dy, interleaved, cos is not None)
    gm = most * wd.abs()
    tol = 2.0 ** -18 * r * (gm + xh.abs() * (gm * xh.abs()).mean(-1, keepdim=True))
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (dx.abs() + tol)
    return dx, tol + 2.0 ** -134, (dn * xh).sum((0, 1)), (most * xh.abs()).sum((0, 1))


def dw_tol(n, heads, d, sums):
    """Bound of dw's error from its terms' sums of absolute values (see above). A lane adds up to
    four terms of every item of its CTA; with at least 50 of the 444 CTAs (3 an SM) for a kind that
    moves a ninth of the bytes or more, as the cases here do, that is 4 (items / 50 + 1) at most."""
    groups = 256 // (d // 8)
    items = -(-n // groups) * -(-heads // 2)
    chain = 4 * (-(-items // 50) + 1) + 32 + 32 + 32
    return (16 + chain) * U * sums + 1e-30
