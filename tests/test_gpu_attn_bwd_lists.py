"""Lists of the attention gradient that name blocks more than once: right, and not slower by orders of
magnitude."""
import math

import pytest
import torch

from tests.test_gpu_attn_bwd import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


@pytest.mark.parametrize("d", [64, 128])
def test_entries_drawn_with_replacement_in_more_chunks_than_warps(S, d):
    """1,100 rows (35 chunks of 32) of up to 40 entries over 9 blocks: most are listed several times, one
    of them more than 32 times within a chunk; two chunks have distinct entries only."""
    block, nqb = 64, 1100
    n_q, n_kv = nqb * block - 11, 9 * block - 20
    q, k, v, do = inputs(1, n_q, n_kv, d, 41)
    g = torch.Generator().manual_seed(41)
    idx = torch.randint(0, 9, (1, nqb, 40), generator=g, dtype=torch.int32)
    idx[0, 200:230, :39] = 4
    cnt = torch.randint(1, 41, (1, nqb), generator=g, dtype=torch.int32)
    cnt[0, 200:230] = 39
    for i in (*range(32, 64), *range(1088, 1100)):
        c = int(torch.randint(1, 10, (1,), generator=g))
        idx[0, i, :c] = torch.randperm(9, generator=g)[:c].int()
        cnt[0, i] = c
    check(S, do, q, k, v, idx.cuda(), cnt.cuda(), block)


def test_a_block_listed_twice_does_not_slow_the_call_down(S):
    """One head of 1,000 query blocks that keep 200 of 2,000 KV blocks each, as they are and with one entry
    of one row of every 32 repeated. The sums grow by 32 of 200,000 tiles; twice the time leaves room for
    the lists, while a search of every list for every block takes ten times as long."""
    block, nqb, nkb, kmax = 64, 1000, 2000, 200
    q, k, v, do = inputs(1, nqb * block, nkb * block, 64, 42)
    g = torch.Generator(device="cuda").manual_seed(42)
    idx = torch.rand(1, nqb, nkb, generator=g, device="cuda").topk(kmax, dim=2).indices.to(torch.int32)
    cnt = torch.full((1, nqb), kmax, dtype=torch.int32, device="cuda")
    again = idx.clone()
    again[0, ::32, 7] = again[0, ::32, 150]
    times = []
    for lists in (idx, again):
        o, lse = S.attn(q, k, v, lists, cnt, block=block)
        ws = S.AttnBwdWorkspace(1, nqb * block, nkb * block, 64, kmax, "cuda", block)
        best = math.inf
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            S.attn_bwd(do, q, k, v, o, lse, lists, cnt, workspace=ws, block=block)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert S.device_status() == S.OK
    assert times[1] <= 2 * times[0], times
