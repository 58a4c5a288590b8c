"""One query token per sequence over a cache, on the GPU: block means, selection (exact) and
attention (within the bound of tests/token_ref.py) against the fp64 form."""
import math

import pytest
import torch

from tests import token_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


def make(lens, hq, hk, s, d, seed, junk=True):
    """A cache whose rows behind each sequence's tokens hold infinities and NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = len(lens)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    nb = -(-s // 128)
    k = rnd(b, hk, nb, 128, d) + 0.5 * rnd(b, hk, nb, 1, d)
    k = k.reshape(b, hk, nb * 128, d)[:, :, :s].bfloat16().contiguous()
    v = rnd(b, hk, s, d).bfloat16()
    if junk:
        for i, n in enumerate(lens):
            for x, bad in ((k, float("nan")), (v, float("inf"))):
                x[i, :, n:] = bad
                x[i, :, n + 1::2] = float("nan")
    q = rnd(b, hq, d).bfloat16()
    return q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check_lists(idx, cnt, want):
    b, hk, keep = idx.shape
    got, gc = idx.cpu(), cnt.cpu()
    for i in range(b):
        for h in range(hk):
            w = want[i][h]
            assert int(gc[i, h]) == len(w)
            assert got[i, h].tolist() == w + [-1] * (keep - len(w)), (i, h)


def check_attention(q, k, v, lens, lists, o, lse, scale=None):
    b, hk = k.shape[:2]
    group = q.shape[1] // hk
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    for i in range(b):
        for h in range(hk):
            sl = slice(h * group, (h + 1) * group)
            ref, tol, lr = R.attend(q[i, sl], k[i, h], v[i, h], lens[i], lists[i][h], scale)
            err = (o[i, sl].double() - ref).abs()
            assert (err <= tol).all(), f"{i} {h}: {(err - tol).max().item():.3e} over"
            if lists[i][h] and lens[i]:
                assert ((lse[i, sl].double() - lr).abs() <= 2.0 ** -12 + 2.0 ** -20 * lr.abs()).all()
            else:
                assert (lse[i, sl] == -math.inf).all() and (o[i, sl] == 0).all()


def run_all(S, lens, hq, hk, s, d, keep, sink, recent, seed):
    q, k, v, kv_len = make(lens, hq, hk, s, d, seed)
    means = S.block_means(k, kv_len)
    assert S.device_status() == S.OK
    for i, n in enumerate(lens):
        nb = -(-n // 128)
        for j in range(means.shape[2]):
            if j >= nb:
                assert (means[i, :, j] == 0).all()
                continue
            x = k[i, :, j * 128:min((j + 1) * 128, n)].double()
            # fp32 sum of at most 128 values in a tree of chains, then a division: 2^-24 times the
            # chain of 8 + 4 + 8 + 1 roundings
            assert ((means[i, :, j].double() - x.mean(1)).abs() <= 21 * 2.0 ** -24 * x.abs().mean(1)).all()
    if recent:  # the forced blocks' means are not needed
        for i, n in enumerate(lens):
            nb = -(-n // 128)
            means[i, :, max(nb - recent, 0):] = float("nan")
            means[i, :, :sink] = float("nan")
    group = hq // hk
    want = [[R.choose(q[i, h * group:(h + 1) * group], means[i, h], n, keep, sink, recent) for h in range(hk)]
            for i, n in enumerate(lens)]
    idx, cnt = S.token_select(q, means, kv_len, keep, sink, recent)
    check_lists(idx, cnt, want)
    o, lse = S.token_attn(q, k, v, kv_len, idx, cnt)
    check_attention(q, k, v, lens, want, o, lse)
    o2, lse2, idx2, cnt2 = S.token_forward(q, k, v, kv_len, means, keep, sink, recent)
    assert torch.equal(idx, idx2) and torch.equal(cnt, cnt2)
    check_attention(q, k, v, lens, want, o2, lse2)  # the forced blocks come first there: another order of sums
    assert S.device_status() == S.OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (8, 2), (5, 1), (32, 2)])
@pytest.mark.parametrize("lens,s", [([1], 1), ([0, 1, 127, 128, 129], 130), ([700, 0, 1500, 1409], 1500)])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 1), (4, 1, 1), (3, 1, 2), (9, 0, 3)])
def test_small(S, lens, s, hq, hk, d, keep, sink, recent):
    run_all(S, lens, hq, hk, s, d, keep, sink, recent, 31 * len(lens) + s + hq + keep)


@pytest.mark.parametrize("lens,hq,hk,s,d,keep,sink,recent", [
    ([9000], 4, 1, 9000, 128, 20, 1, 2),              # clusters of eight
    ([6400, 5000, 6399], 8, 8, 6400, 64, 8, 0, 1),    # clusters of four
    ([2000 + 37 * i for i in range(40)], 8, 8, 3500, 128, 6, 1, 1),  # more key heads than SMs: no cluster
    ([20000, 3], 16, 1, 20000, 128, 120, 2, 3),
])
def test_larger(S, lens, hq, hk, s, d, keep, sink, recent):
    run_all(S, lens, hq, hk, s, d, keep, sink, recent, s + keep)


def scores_case(S, values, keep, sink=0, recent=1, hk=1, b=1):
    """Selection over means whose first coordinate is the score (q is the first unit vector)."""
    nb = len(values) + recent
    means = torch.zeros(b, hk, nb, 64, device="cuda")
    means[:, :, :len(values), 0] = torch.tensor(values, device="cuda")
    q = torch.zeros(b, hk, 64, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1
    kv_len = torch.full((b,), nb * 128, dtype=torch.int32, device="cuda")
    idx, cnt = S.token_select(q, means, kv_len, keep, sink, recent)
    assert (cnt == min(keep, nb)).all()
    want = R.choose(q[0], means[0, 0], nb * 128, keep, sink, recent)
    got = idx.cpu()
    assert all(got[i, h].tolist() == want for i in range(b) for h in range(hk))


def test_ties_go_to_the_lower_block(S):
    inf, nan = float("inf"), float("nan")
    scores_case(S, [1.0] * 300, 40)
    scores_case(S, [0.0, -0.0] * 200, 77)
    scores_case(S, [float(i % 3) for i in range(500)], 250)
    scores_case(S, [1.0, 2.0, inf, -inf, 2.0, 0.0, -1.0, inf], 4)


def test_nan_ranks_below_everything(S):
    # a mean of NaN or infinity makes its block's whole dot product NaN with the other coordinates'
    # zeros, so the score itself is drawn through the first coordinate alone where it is finite
    nb = 9
    means = torch.zeros(1, 1, nb + 1, 64, device="cuda")
    means[0, 0, :nb, 0] = torch.tensor([0.5, -3.0, 0.0, 2.0, -1e30, 7.0, 1.0, 1.5, -0.5])
    means[0, 0, 3] = float("nan")
    means[0, 0, 5, 1] = float("inf")   # inf times the query's 0: NaN
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1
    kv_len = torch.tensor([(nb + 1) * 128], dtype=torch.int32, device="cuda")
    for keep in range(1, nb + 1):
        idx, _ = S.token_select(q, means, kv_len, keep, 0, 1)
        assert idx[0, 0].tolist() == R.choose(q[0], means[0, 0], (nb + 1) * 128, keep, 0, 1)


@pytest.mark.parametrize("n", [130, 1000, 4097, 16380])
def test_selection_sizes(S, n):
    g = torch.Generator().manual_seed(n)
    values = torch.randn(n, generator=g).tolist()
    for keep in (1 + 1, n // 7 + 1, n - 1):
        scores_case(S, values, keep, hk=2)
    near = (1.0 + torch.randperm(n, generator=g).double() * 2.0 ** -22).float().tolist()  # ranks in the last bits
    scores_case(S, near, n // 3 + 1, hk=2)


def test_ties_at_the_cut_among_many(S):
    """A few equal or nearly equal scores where the last kept block is chosen, in lists of every path
    (ranked by each CTA, by one CTA with some blocks scored again, by one CTA with all scored again)."""
    g = torch.Generator().manual_seed(3)
    for n in (100, 400, 3000):
        base = torch.rand(n, generator=g) * 4 - 2
        tied = torch.randperm(n, generator=g)[:60]
        base[tied] = 0.5
        above = int((base > 0.5).sum())
        for taken in (1, 17, 59):
            scores_case(S, base.tolist(), above + taken + 1, hk=3)
        near = base.clone()
        near[tied] += torch.arange(60).float() * 2.0 ** -23
        scores_case(S, near.tolist(), above + 30 + 1, hk=3)


@pytest.mark.parametrize("n", [90, 700])
def test_scores_that_are_not_finite_among_others(S, n):
    g = torch.Generator().manual_seed(n)
    means = torch.randn(1, 2, n + 1, 64, generator=g).cuda()
    means[0, :, 5] = float("inf")
    means[0, :, 17, 3] = float("nan")
    means[0, 1, 40] = 3e38   # sums beyond fp32, not beyond fp64
    means[0, 1, 41] = -3e38
    q = torch.randn(1, 4, 64, generator=g).bfloat16().cuda()
    kv_len = torch.tensor([(n + 1) * 128], dtype=torch.int32, device="cuda")
    for keep in (2, n // 3, n - 1):
        idx, _ = S.token_select(q, means, kv_len, keep, 0, 1)
        for h in range(2):
            want = R.choose(q[0, 2 * h:2 * h + 2], means[0, h], (n + 1) * 128, keep, 0, 1)
            assert idx[0, h].tolist() == want


def test_scores_below_the_normal_range_still_rank(S):
    g = torch.Generator().manual_seed(5)
    for n in (100, 500):
        values = (torch.randint(1, 2000, (n,), generator=g).double() * 2.0 ** -149).float()
        means = torch.zeros(1, 1, n + 1, 64, device="cuda")
        means[0, 0, :n, :4] = values[torch.randint(0, n, (n, 4), generator=g)].cuda()
        q = torch.tensor([0.75, -0.5, 1.25, 0.3125] + [0.0] * 60).bfloat16().reshape(1, 1, 64).cuda()
        kv_len = torch.tensor([(n + 1) * 128], dtype=torch.int32, device="cuda")
        idx, _ = S.token_select(q, means, kv_len, n // 3, 0, 1)
        assert idx[0, 0].tolist() == R.choose(q[0], means[0, 0], (n + 1) * 128, n // 3, 0, 1)


def test_near_scores_are_told_apart_beyond_fp32(S):
    """Scores that differ by less than fp32 sums resolve still rank by their fp64 values."""
    means = torch.zeros(1, 1, 4, 64, device="cuda")
    means[0, 0, :3, 0] = 2.0 ** 20
    means[0, 0, 1, 1] = 2.0 ** -20
    means[0, 0, 2, 1] = 2.0 ** -19
    q = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    kv_len = torch.tensor([512], dtype=torch.int32, device="cuda")
    idx, _ = S.token_select(q, means, kv_len, 2, 0, 1)
    assert idx[0, 0].tolist() == [2, 3]


def test_attention_over_any_list(S):
    lens, keep = [1000, 500, 1000], 6
    q, k, v, kv_len = make(lens, 4, 2, 1000, 128, 3)
    idx = torch.tensor([[7, 0, 3, 3, 99, 99], [5, 6, 99, 99, 99, 99]], dtype=torch.int32, device="cuda")
    idx = idx.expand(3, 2, 6).contiguous()
    idx[1] = torch.tensor([3, 3, 0, 99, 99, 99])
    cnt = torch.tensor([[4, 2], [3, 3], [0, 1]], dtype=torch.int32, device="cuda")
    lists = [[idx[i, h, :cnt[i, h]].tolist() for h in range(2)] for i in range(3)]
    o, lse = S.token_attn(q, k, v, kv_len, idx, cnt, sm_scale=0.11)
    assert S.device_status() == S.OK
    check_attention(q, k, v, lens, lists, o, lse, 0.11)
    o2, none = S.token_attn(q, k, v, kv_len, idx, cnt, sm_scale=0.11, want_lse=False)
    assert none is None and torch.equal(o, o2)


def test_entries_without_tokens_are_skipped_and_reported(S):
    lens = [300]
    q, k, v, kv_len = make(lens, 2, 1, 1000, 64, 4)
    idx = torch.tensor([[[0, -5, 3, 2, 2 ** 30]]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[9]], dtype=torch.int32, device="cuda")
    o, lse = S.token_attn(q, k, v, kv_len, idx, cnt)
    assert S.device_status() == S.ERR_DEVICE_BOUNDS and S.device_status() == S.OK
    check_attention(q, k, v, lens, [[[0, 2]]], o, lse)
    for bad, n in ((-3, 0), (5000, 1000)):
        q, k, v, _ = make([n], 2, 1, 1000, 64, 5, junk=False)
        far = torch.tensor([bad], dtype=torch.int32, device="cuda")
        means = S.block_means(k, far)
        o, lse, idx2, cnt2 = S.token_forward(q, k, v, far, means, 8)
        assert S.device_status() == S.ERR_DEVICE_BOUNDS and S.device_status() == S.OK
        check_attention(q, k, v, [n], [[list(range(-(-n // 128)))]], o, lse)


def test_tail_means_alone_change(S):
    lens = [1, 128, 129, 0, 640]
    _, k, _, kv_len = make(lens, 2, 2, 640, 128, 6)
    full = S.block_means(k, kv_len)
    means = torch.full_like(full, 5.0)
    out = S.block_means(k, kv_len, means, tail_only=True)
    assert out is means
    want = torch.full_like(full, 5.0)
    for i, n in enumerate(lens):
        if n:
            want[i, :, (n - 1) // 128] = full[i, :, (n - 1) // 128]
    assert torch.equal(means, want)


def test_cache_beyond_32_bit_offsets(S):
    """The last rows of a cache of 2.4e9 elements."""
    hk, s, d = 9, 16384 * 128, 128
    k = torch.zeros(1, hk, s, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(1, hk, s, d, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    blocks = [0, 9000, 16383]
    for j in blocks:
        for x in (k, v):
            x[:, :, j * 128:(j + 1) * 128] = torch.randn(1, hk, 128, d, generator=g, device="cuda").bfloat16()
    q = torch.randn(1, hk, d, generator=g, device="cuda").bfloat16()
    kv_len = torch.tensor([s - 5], dtype=torch.int32, device="cuda")
    idx = torch.tensor(blocks, dtype=torch.int32, device="cuda").expand(1, hk, 3).contiguous()
    cnt = torch.full((1, hk), 3, dtype=torch.int32, device="cuda")
    o, lse = S.token_attn(q, k, v, kv_len, idx, cnt)
    check_attention(q, k, v, [s - 5], [[blocks] * hk], o, lse)
    means = S.block_means(k, kv_len)
    assert S.device_status() == S.OK
    x = k[0, hk - 1, 16383 * 128:s - 5].double()
    assert ((means[0, hk - 1, 16383].double() - x.mean(0)).abs() <= 21 * 2.0 ** -24 * x.abs().mean(0)).all()
    idx, _ = S.token_select(q, means, kv_len, 4, 1, 1)
    assert all(idx[0, h].tolist() == R.choose(q[0, h:h + 1], means[0, h], s - 5, 4, 1, 1) for h in range(hk))


def test_on_a_side_stream_and_in_a_graph_and_twice(S):
    lens = [900, 1300]
    q, k, v, kv_len = make(lens, 8, 2, 1300, 128, 8)
    means = S.block_means(k, kv_len)
    want = S.token_forward(q, k, v, kv_len, means, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = S.token_forward(q, k, v, kv_len, means, 5, stream=side)
    again = S.token_forward(q, k, v, kv_len, means, 5)  # the two may run at once
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.block_means(k, kv_len, means, tail_only=True)
        got = S.token_forward(q, k, v, kv_len, means, 5)
    kv_len -= 130  # a replay takes the lengths as they are then
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want = S.token_forward(q, k, v, kv_len, S.block_means(k, kv_len), 5)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("d", [128, 64])
def test_a_full_gpu_of_uneven_sequences_gives_the_same_bits_every_time(S, d):
    """Sequences of every length side by side, so that a stage may be refilled the moment it is given
    back: a copy that overtakes a read shows as differing bits, and against the fp64 form."""
    b, hq, hk, s, keep = 48, 32, 8, 16384, 32
    lens = [s - int((s - 500) * ((i * 0.618034) % 1.0)) for i in range(b)]
    q, k, v, kv_len = make(lens, hq, hk, s, d, 9, junk=False)
    means = S.block_means(k, kv_len)
    want = S.token_forward(q, k, v, kv_len, means, keep, 1, 2)
    lists = [[want[2][i, h, :int(want[3][i, h])].tolist() for h in range(hk)] for i in range(b)]
    check_attention(q, k, v, lens, lists, want[0], want[1])
    attn = S.token_attn(q, k, v, kv_len, want[2], want[3])
    check_attention(q, k, v, lens, lists, *attn)
    for _ in range(60):
        got = S.token_forward(q, k, v, kv_len, means, keep, 1, 2)
        again = S.token_attn(q, k, v, kv_len, want[2], want[3])
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert all(torch.equal(x, y) for x, y in zip(attn, again))


def test_no_sequences(S):
    k = torch.empty(0, 2, 300, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv_len = torch.empty(0, dtype=torch.int32, device="cuda")
    means = S.block_means(k, kv_len)
    o, lse, idx, cnt = S.token_forward(q, k, k, kv_len, means, 4)
    assert o.shape == (0, 4, 64) and idx.shape == (0, 2, 4)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk", [1, 160])  # clusters of several CTAs, and CTAs alone
def test_a_nan_query_head_gives_nan_and_leaves_the_others(S, d, hk):
    group, lens = 4, [700, 128, 0, 1, 1000]
    q, k, v, kl = make(lens, group * hk, hk, 1024, d, 21)
    cnt = ((kl + 127) // 128)[:, None].expand(-1, hk).contiguous()
    idx = torch.arange(8, dtype=torch.int32, device="cuda").expand(len(lens), hk, 8).contiguous()
    want, want_lse = S.token_attn(q, k, v, kl, idx, cnt)
    q[:, 2::group] = float("nan")
    q[:, 1::group, 5] = float("inf")
    o, lse = S.token_attn(q, k, v, kl, idx, cnt)
    means = S.block_means(k, kl)
    o2, lse2, _, _ = S.token_forward(q, k, v, kl, means, 8)
    for got, got_lse in ((o, lse), (o2, lse2)):
        for i, n in enumerate(lens):
            for g in range(group):
                x, y = got[i, g::group], got_lse[i, g::group]
                if g == 2 and n:
                    assert x.isnan().all() and y.isnan().all()
                elif g != 1 or n == 0:
                    assert torch.equal(x, want[i, g::group]) and torch.equal(y, want_lse[i, g::group])
    assert S.device_status() == 0
