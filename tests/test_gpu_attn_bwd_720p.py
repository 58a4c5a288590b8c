"""The attention gradient at the size of a final scale, blocks of it against the fp64 form."""
import math

import pytest
import torch

from tests import attn_bwd_ref as R
from tests.test_gpu_attn_bwd import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


def test_blocks_of_the_720p_final_scale(S):
    """One head, 72,187 queries (five short of whole blocks) on 144,891 tokens: dq of some query blocks over
    their lists, dk and dv of some KV blocks over the queries that keep them, one in every list among them.
    Sums over n query blocks are longer than the bounds' 2^-12 of a sum's absolute values counts: 8 n fp32
    additions of 16 products each, 2^-23 of those values each at most, so 8 n 2^-12 of the 2^-11 part more."""
    n_text, n_ctx, n_cur, block, d = 512, 72192, 72187, 128, 128
    n_q, n_kv = n_cur, n_text + n_ctx + n_cur
    q, k, v, do = inputs(1, n_q, n_kv, d, 43)
    o, lse, idx, cnt = S.forward(q, k, v, n_text, n_ctx, n_cur, 2, 0.09375)
    dq, dk, dv = S.attn_bwd(do, q, k, v, o, lse, idx, cnt)
    assert S.device_status() == S.OK
    nqb, nkb = idx.shape[1], -(-n_kv // block)
    kept = torch.zeros(nqb, nkb, dtype=torch.bool, device="cuda").scatter_(1, idx[0].long(), True)

    def tokens(blocks, n):
        t = (blocks[:, None] * block + torch.arange(block, device="cuda")).flatten()
        return t[t < n]

    def compare(name, got, ref, n=0):
        val, tol, floor = ref
        more = 8 * n * 2.0 ** -12 * floor * (1 + R.H8)
        tol, floor = tol + more, floor + more
        err = (got.double() - val).abs()
        assert (err <= tol).all(), f"{name}: {(err / tol).max().item():.3g} of the bound"
        assert torch.linalg.norm(err) <= 2.0 ** -7 * torch.linalg.norm(val) + torch.linalg.norm(floor), name

    def part(rows, cols):
        one = torch.ones(rows.numel(), cols.numel(), dtype=torch.float64, device="cuda")
        t = [x[0, rows].double() for x in (do, q)] + [x[0, cols].double() for x in (k, v)]
        return R.head_backward(*t, o[0, rows].double(), lse[0, rows].double(), one, 1 / math.sqrt(d))

    for i in (0, 1, 300, nqb - 1):
        rows = tokens(torch.tensor([i], device="cuda"), n_q)
        compare(f"dq {i}", dq[0, rows], part(rows, tokens(idx[0, i].long(), n_kv))[0])
    counts = kept.sum(0)
    for j in (0, 3, int(counts[4:].argmax()) + 4, nkb - 1, int((counts - 20).abs().argmin())):
        cols = tokens(torch.tensor([j], device="cuda"), n_kv)
        if counts[j] == 0:
            assert not dk[0, cols].any() and not dv[0, cols].any()
            continue
        _, rk, rv = part(tokens(kept[:, j].nonzero()[:, 0], n_q), cols)
        compare(f"dk {j}", dk[0, cols], rk, int(counts[j]))
        compare(f"dv {j}", dv[0, cols], rv, int(counts[j]))
