"""Gradient of the block-sparse attention on the GPU against the fp64 formula, within the bounds
derived in tests/attn_bwd_ref.py."""
import math

import pytest
import torch

from block_sparse_attention_tok_b200 import synth
from tests import attn_bwd_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


def inputs(H, n_q, n_kv, d, seed):
    q, k, v = synth.make_qkv(n_q, n_kv, H, d, [seed + i for i in range(H)], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    return q, k, v, torch.randn(q.shape, generator=g, device="cuda").bfloat16()


def random_lists(H, n_q, n_kv, block, seed, most=None):
    """Lists of 1 to `most` distinct blocks per row, in random order; the rest of the row is junk
    that is never read."""
    nqb, nkb = -(-n_q // block), -(-n_kv // block)
    most = nkb if most is None else min(most, nkb)
    g = torch.Generator().manual_seed(seed)
    idx = torch.full((H, nqb, most), -7, dtype=torch.int32)
    cnt = torch.randint(1, most + 1, (H, nqb), generator=g, dtype=torch.int32)
    for h in range(H):
        for i in range(nqb):
            c = int(cnt[h, i])
            idx[h, i, :c] = torch.randperm(nkb, generator=g)[:c].int()
    return idx.cuda(), cnt.cuda()


def check(S, do, q, k, v, idx, cnt, block, sm_scale=0.0, o=None, lse=None):
    H, n_q, d = q.shape
    n_kv = k.shape[1]
    if o is None:
        o, lse = S.attn(q, k, v, idx, cnt, sm_scale=sm_scale, block=block)
    got = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, sm_scale=sm_scale, block=block)
    assert S.device_status() == S.OK
    scale = sm_scale if sm_scale > 0 else 1 / math.sqrt(d)
    for h in range(H):
        w = R.multiplicity(idx[h], cnt[h], n_q, n_kv, block)
        ref = R.head_backward(*(t[h].double() for t in (do, q, k, v, o, lse)), w, scale)
        for name, x, (val, tol, floor) in zip(("dq", "dk", "dv"), got, ref):
            err = (x[h].double() - val).abs()
            assert (err <= tol).all(), f"{name} head {h}: {(err / tol).max().item():.3g} of the bound"
            # The roundings are independent, so they do not add up like the bound's sums. The fp32
            # part stands beside them: where a row keeps one token, dP = delta and dS is exactly 0
            # (2^-7 of it allows nothing), while the two fp32 sums differ by their own roundings.
            most = 2.0 ** -7 * torch.linalg.norm(val) + torch.linalg.norm(floor)
            assert torch.linalg.norm(err) <= most, f"{name} head {h}: norm"
    return got


@pytest.mark.parametrize("block", [128, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_q,n_kv", [(128, 128), (1, 1), (1, 300), (5, 64), (130, 129), (64, 1000), (257, 511),
                                      (1024, 2048), (1000, 2111)])
def test_random_lists(S, n_q, n_kv, d, block):
    q, k, v, do = inputs(2, n_q, n_kv, d, n_q + 3 * n_kv + d)
    idx, cnt = random_lists(2, n_q, n_kv, block, n_q + d)
    check(S, do, q, k, v, idx, cnt, block)


@pytest.mark.parametrize("block", [128, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_selected_lists_on_more_items_than_sms(S, d, block):
    n_text, n_ctx, n_cur = 200, 3000, 4100
    q, k, v, do = inputs(5, n_cur, n_text + n_ctx + n_cur, d, 50 + d)
    idx, cnt, _ = S.select(q, k, n_text, n_ctx, n_cur, 2, 0.15, block=block)
    check(S, do, q, k, v, idx, cnt, block)


@pytest.mark.parametrize("block", [128, 64])
def test_blocks_that_no_query_keeps_get_zero(S, block):
    q, k, v, do = inputs(3, 500, 1500, 128, 9)
    idx, cnt = random_lists(3, 500, 1500, block, 9, most=2)
    _, dk, dv = check(S, do, q, k, v, idx, cnt, block)
    for h in range(3):
        kept = R.multiplicity(idx[h], cnt[h], 500, 1500, block).sum(0) > 0
        assert not kept.all()
        assert (dk[h][~kept] == 0).all() and (dv[h][~kept] == 0).all()


@pytest.mark.parametrize("block", [128, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_lists_split_into_parts(S, d, block):
    """One head whose ragged last block every query block keeps, another one that they keep twice, and
    blocks that few keep: the long lists are split, and the parts added up the same way every time."""
    n_q, n_kv = 130 * block + 7, 12 * block - 30
    q, k, v, do = inputs(1, n_q, n_kv, d, 22)
    nqb = -(-n_q // block)
    g = torch.Generator().manual_seed(22)
    idx = torch.stack([torch.tensor([11, 3, int(torch.randint(4, 11, (1,), generator=g)), 3]) for _ in range(nqb)])
    idx = idx.to(torch.int32)[None].cuda().contiguous()
    cnt = torch.full((1, nqb), 4, dtype=torch.int32, device="cuda")
    o, lse = S.attn(q, k, v, idx, cnt, block=block)
    want = check(S, do, q, k, v, idx, cnt, block, o=o, lse=lse)
    for _ in range(5):
        got = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, block=block)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_every_block_kept_by_every_query(S):
    q, k, v, do = inputs(2, 700, 900, 128, 10)
    nqb, nkb = 6, 8
    idx = torch.arange(nkb, dtype=torch.int32, device="cuda").expand(2, nqb, nkb).contiguous()
    cnt = torch.full((2, nqb), nkb, dtype=torch.int32, device="cuda")
    check(S, do, q, k, v, idx, cnt, 128, sm_scale=0.05)


@pytest.mark.parametrize("block", [128, 64])
def test_a_block_listed_twice_counts_twice(S, block):
    q, k, v, do = inputs(1, 300, 700, 64, 11)
    nqb = -(-300 // block)
    idx = torch.tensor([3, 1, 3, 3, 0], dtype=torch.int32, device="cuda").expand(1, nqb, 5).contiguous()
    cnt = torch.full((1, nqb), 4, dtype=torch.int32, device="cuda")
    check(S, do, q, k, v, idx, cnt, block)


@pytest.mark.parametrize("block", [128, 64])
def test_blocks_listed_twice_in_some_chunks_of_many_rows(S, block):
    n_q, n_kv = 70 * block + 3, 9 * block + 1
    q, k, v, do = inputs(2, n_q, n_kv, 64, 21)
    idx, cnt = random_lists(2, n_q, n_kv, block, 21)
    for h, i in ((0, 40), (0, 41), (1, 0), (1, 70)):  # chunks of 32 rows: 1, 1, 0, 2
        cnt[h, i] = 5
        idx[h, i, :5] = torch.tensor([4, 9, 4, 0, 9])
    check(S, do, q, k, v, idx, cnt, block)


@pytest.mark.parametrize("block", [128, 64])
def test_long_lists_of_one_block(S, block):
    """Every query block keeps one and the same KV block: one item walks all of them."""
    q, k, v, do = inputs(2, 6000, 600, 128, 12)
    nqb = -(-6000 // block)
    idx = torch.full((2, nqb, 1), 2, dtype=torch.int32, device="cuda")
    cnt = torch.ones(2, nqb, dtype=torch.int32, device="cuda")
    check(S, do, q, k, v, idx, cnt, block)


def test_large_logits_and_outliers(S):
    q, k, v, do = inputs(1, 256, 512, 128, 13)
    q = (q * 6).contiguous()
    q[0, 5] = 0
    v[0, 7] *= 100
    idx, cnt = random_lists(1, 256, 512, 128, 13)
    o, lse = S.attn(q, k, v, idx, cnt)
    got = S.attn_bwd(do, q, k, v, o, lse, idx, cnt)
    # logits reach 6 sum |q k| s below 96: P's error is six times the bound's assumption, so the
    # 2^-11 terms grow to 2^-8
    w = R.multiplicity(idx[0], cnt[0], 256, 512, 128)
    t = [x[0].double() for x in (do, q, k, v, o, lse)]
    scale = 1 / math.sqrt(128)
    p = torch.exp(scale * (t[1] @ t[2].T) - t[5][:, None]) * w
    size = p * (t[0].abs() @ t[3].abs().T + (t[0] * t[4]).abs().sum(1, keepdim=True))
    more = (scale * 2.0 ** -8 * size @ t[2].abs(), scale * 2.0 ** -8 * size.T @ t[1].abs(),
            2.0 ** -8 * p.T @ t[0].abs())
    for x, (val, tol, _), m in zip(got, R.head_backward(*t, w, scale), more):
        assert ((x[0].double() - val).abs() <= tol + m).all()


def test_against_differences_of_the_loss(S):
    """<grad, e> against central differences of L = sum(do * o) with o exact in fp64. Beyond the
    kernels' bounds, delta comes from the bf16 o: off by at most 2^-8 sum |do o| a row."""
    H, n_q, n_kv, block = 1, 200, 400, 128
    q, k, v, do = inputs(H, n_q, n_kv, 64, 14)
    idx, cnt = random_lists(H, n_q, n_kv, block, 14)
    o, lse = S.attn(q, k, v, idx, cnt)
    got = S.attn_bwd(do, q, k, v, o, lse, idx, cnt)
    w = R.multiplicity(idx[0], cnt[0], n_q, n_kv, block)
    scale = 1 / 8
    x = [t[0].double() for t in (q, k, v)]
    dod, od = do[0].double(), o[0].double()
    bounds = [b for _, b, _ in R.head_backward(dod, *x, od, lse[0].double(), w, scale)]
    p = torch.exp(scale * (x[0] @ x[1].T) - lse[0].double()[:, None]) * w
    off = p * (2.0 ** -8 * (dod * od).abs().sum(1, keepdim=True))
    bounds[0] = bounds[0] + scale * off @ x[1].abs()
    bounds[1] = bounds[1] + scale * off.T @ x[0].abs()
    g = torch.Generator(device="cuda").manual_seed(15)

    def loss(*a):
        return (R.head_forward(*a, w, scale)[0] * dod).sum().item()

    for i in range(3):
        for _ in range(3):
            e = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
            up, dn = list(x), list(x)
            up[i], dn[i] = x[i] + 1e-4 * e, x[i] - 1e-4 * e
            diff = (loss(*up) - loss(*dn)) / 2e-4
            assert abs(diff - (got[i][0].double() * e).sum().item()) <= (bounds[i] * e.abs()).sum().item() + 1e-5


def test_reproducible_and_independent_of_buffers(S):
    n_text, n_ctx, n_cur = 256, 2000, 3001
    q, k, v, do = inputs(3, n_cur, n_text + n_ctx + n_cur, 128, 16)
    o, lse, idx, cnt = S.forward(q, k, v, n_text, n_ctx, n_cur, 2, 0.2)
    ws = S.AttnBwdWorkspace(3, n_cur, k.shape[1], 128, idx.shape[-1], "cuda")
    ws.buf.fill_(255)
    first = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, workspace=ws)
    first = [t.clone() for t in first]
    outs = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    for fill in (0, 127):
        ws.buf.fill_(fill)
        again = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
        assert S.device_status() == S.OK
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("block", [128, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_many_runs_of_many_tiles_agree(S, d, block):
    """Warps that run ahead of others must not be counted for the tile that those still work on: with
    few items, long lists and many runs such an early count would show as differing bits."""
    H, n_q, n_kv = 2, 4 * block, 96 * block + 5
    q, k, v, do = inputs(H, n_q, n_kv, d, 19)
    idx, cnt = random_lists(H, n_q, n_kv, block, 19)
    o, lse = S.attn(q, k, v, idx, cnt, block=block)
    want = check(S, do, q, k, v, idx, cnt, block, o=o, lse=lse)
    for _ in range(30):
        got = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, block=block)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_list_order_changes_only_rounding_and_out_of_range_entries_are_reported(S):
    q, k, v, do = inputs(1, 256, 512, 64, 17)
    idx = torch.tensor([[[0, 2, 3, 9], [1, 0, -1, 2]]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[3, 2]], dtype=torch.int32, device="cuda")
    check(S, do, q, k, v, idx, cnt, 128)
    o, lse = S.attn(q, k, v, idx, cnt)
    cnt_bad = torch.tensor([[4, 9]], dtype=torch.int32, device="cuda")
    S.attn_bwd(do, q, k, v, o, lse, idx, cnt_bad)
    assert S.device_status() == S.ERR_DEVICE_BOUNDS and S.device_status() == S.OK


def test_no_queries_give_zero_gradients(S):
    q = torch.empty(2, 0, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(2, 200, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 0, device="cuda")
    idx = torch.empty(2, 0, 1, dtype=torch.int32, device="cuda")
    cnt = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    dq, dk, dv = S.attn_bwd(q, q, k, k, q, lse, idx, cnt, dk=torch.ones_like(k), dv=torch.ones_like(k))
    torch.cuda.synchronize()
    assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()


def test_the_largest_number_of_kv_blocks(S):
    n_q, n_kv, d, block = 100, 49152 * 64 - 3, 64, 64
    g = torch.Generator(device="cuda").manual_seed(40)
    k, v = (torch.randn(1, n_kv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q, do = (torch.randn(1, n_q, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    idx = torch.tensor([[[49151, 0, 30000], [7, 49151, 20000]]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[3, 2]], dtype=torch.int32, device="cuda")
    o, lse = S.attn(q, k, v, idx, cnt, block=block)
    dq, dk, dv = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, block=block)
    assert S.device_status() == S.OK
    used = torch.tensor([0, 7, 30000, 49151], device="cuda")
    rows = (used[:, None] * block + torch.arange(block, device="cuda")).flatten()
    rows = rows[rows < n_kv]
    w = torch.zeros(n_q, rows.numel(), dtype=torch.float64, device="cuda")
    for i, keep in enumerate(([49151, 0, 30000], [7, 49151])):
        for j in keep:
            w[i * block:(i + 1) * block, rows // block == j] = 1
    ref = R.head_backward(*(t[0].double() for t in (do, q)), k[0, rows].double(), v[0, rows].double(), o[0].double(),
                          lse[0].double(), w, 1 / 8)
    for x, (val, tol, _) in zip((dq[0], dk[0, rows], dv[0, rows]), ref):
        assert ((x.double() - val).abs() <= tol).all()
    for x in (dk, dv):
        x[0, rows] = 0
        assert not x.any()


def test_two_calls_at_once(S):
    """Two shapes on two streams, each with its own workspace, many times over."""
    cases = []
    for i, (n_q, n_kv, d, block) in enumerate(((700, 1500, 128, 128), (500, 900, 64, 64))):
        q, k, v, do = inputs(2, n_q, n_kv, d, 30 + i)
        idx, cnt = random_lists(2, n_q, n_kv, block, 30 + i)
        o, lse = S.attn(q, k, v, idx, cnt, block=block)
        args = (do, q, k, v, o, lse, idx, cnt)
        cases.append((args, block, [t.clone() for t in S.attn_bwd(*args, block=block)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for args, block, want, stream in cases:
            got.append((S.attn_bwd(*args, block=block, stream=stream), want))
    torch.cuda.synchronize()
    assert S.device_status() == S.OK
    assert all(torch.equal(a, b) for g, w in got for a, b in zip(g, w))


def test_on_a_side_stream_and_in_a_graph(S):
    q, k, v, do = inputs(2, 500, 900, 128, 18)
    idx, cnt = random_lists(2, 500, 900, 128, 18)
    o, lse = S.attn(q, k, v, idx, cnt)
    want = [t.clone() for t in S.attn_bwd(do, q, k, v, o, lse, idx, cnt)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = S.attn_bwd(do, q, k, v, o, lse, idx, cnt)
    for t in got:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
