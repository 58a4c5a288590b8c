"""fp64 gradient of the block-sparse attention from its formula, and the error bounds of the
kernels.

Bounds, with h = 2^-8 (half a step of bf16, relative) and u = 2^-24:
  P: the logit's fp32 sum of d products is off by at most d u sum_c |q_c k_c|, scaled by s below
    2^-13 of P for the inputs here (sum |q k| s below 16 at d = 128); the scale, lse2 and exp2 add below
    2^-17: P's own error is below 2^-12 P.
  dv = sum P do, P rounded to bf16: (h + 2^-12) sum P |do|, the fp32 sum below 2^-12 of that too.
  dS = P (dP - delta): P's error and the fp32 sums of dP and delta (d u each) are below
    2^-11 P (sum |do v| + sum |do o|); as an operand it is rounded to bf16: h |dS|.
  dq = s sum dS k, dk = s sum dS q: the same through |k| and |q|.
  Each output is rounded once: h of the value.
"""
import math

import torch

H8 = 2.0 ** -8


def multiplicity(idx, cnt, n_q, n_kv, block):
    """How often each (query token, KV token) pair of one head is kept: fp64 [Nq, Nkv]."""
    nkb = -(-n_kv // block)
    w = torch.zeros(idx.shape[0], nkb, dtype=torch.float64, device=idx.device)
    for i, c in enumerate(cnt.tolist()):
        w[i].index_add_(0, idx[i, :c].long(), torch.ones(c, dtype=torch.float64, device=idx.device))
    return w.repeat_interleave(block, 0)[:n_q].repeat_interleave(block, 1)[:, :n_kv]


def head_forward(q, k, v, w, scale):
    """Exact (o, lse) in fp64 of one head with multiplicities w."""
    s = scale * (q @ k.T)
    lse = torch.logsumexp(torch.where(w > 0, s + w.clamp(min=1e-300).log(), -math.inf), dim=1)
    p = torch.exp(s - lse[:, None]) * w
    return p @ v, lse


def head_backward(do, q, k, v, o, lse, w, scale):
    """((dq, bound, floor), (dk, ...), (dv, ...)) of one head, all fp64; `floor` is the part of the
    bound that comes from fp32 sums and does not shrink with dS."""
    p = torch.exp(scale * (q @ k.T) - lse[:, None]) * w
    delta = (do * o).sum(1, keepdim=True)
    ds = p * (do @ v.T - delta)
    size = p * (do.abs() @ v.abs().T + (do * o).abs().sum(1, keepdim=True))
    low = 2.0 ** -11 * size
    e = H8 * ds.abs() + low
    res = []
    for val, err, floor in (
            (scale * (ds @ k), scale * (e @ k.abs()), scale * (low @ k.abs())),
            (scale * (ds.T @ q), scale * (e.T @ q.abs()), scale * (low.T @ q.abs())),
            (p.T @ do, (H8 + 2.0 ** -11) * (p.T @ do.abs()), 2.0 ** -11 * (p.T @ do.abs()))):
        res.append((val, err + H8 * (val.abs() + err) + 1e-30, floor))
    return res
