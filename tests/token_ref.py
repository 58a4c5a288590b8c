"""fp64 selection and attention of one query token over a cache, in plain Python and torch, and the
error bound of the kernel.

Bound: each probability has an error below 2^-12 of it from the fp32 logit (a sum of d products,
as in tests/attn_bwd_ref.py) and exp2, and half a bf16 step, 2^-8, as an operand of the second
product; the denominator is summed in fp32 from unrounded values. So o is off by at most
(2^-8 + 2^-11) sum p |v| before its own rounding (2^-8 of the value), and lse by 2^-12 + 2^-20 |lse|.
"""
import math

import torch


def choose(q, means, n, keep, n_sink, n_recent):
    """Kept blocks of one (sequence, key head): q [G, d], means [nb, d], n tokens."""
    nb = -(-n // 128)
    if nb <= keep:
        return list(range(nb))
    qs = q.double().sum(0)
    score = (means.double() * qs).sum(1).tolist()
    rest = range(n_sink, nb - n_recent)

    def order(j):  # NaN last, then falling score, then rising block
        s = score[j]
        return (1, 0.0, j) if math.isnan(s) else (0, -s, j)

    best = sorted(rest, key=order)[:keep - n_sink - n_recent]
    return sorted(list(range(n_sink)) + best + list(range(nb - n_recent, nb)))


def attend(q, k, v, n, blocks, scale):
    """(o, bound, lse) of q [G, d] over the tokens of `blocks` of k, v [S, d]."""
    at = [t for j in blocks for t in range(j * 128, min((j + 1) * 128, n))]
    if not at:
        z = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        return z, z, torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=q.device)
    at = torch.tensor(at, device=q.device)
    w = scale * q.double() @ k[at].double().T
    lse = torch.logsumexp(w, 1)
    p = torch.exp(w - lse[:, None])
    o = p @ v[at].double()
    err = (2.0 ** -8 + 2.0 ** -11) * (p @ v[at].double().abs())
    return o, err + 2.0 ** -8 * (o.abs() + err), lse
