"""Norm of queries and keys with the position rotation, forward and gradient, on the GPU against
the fp64 form, within the bounds derived in tests/norm_rope_ref.py."""
import pytest
import torch

from tests import norm_rope_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


def make(n, hq, hk, d, dtype, seed, rope=True, weights=True, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = (scale * rnd(n, hq + 2 * hk, d)).to(dtype)
    a = 7.0 * torch.rand(n, d // 2, generator=g, device="cuda", dtype=torch.float64)
    return dict(q=x[:, :hq], k=x[:, hq:hq + hk], v=x[:, hq + hk:], wq=1 + 0.3 * rnd(d) if weights else None,
                wk=1 - 0.3 * rnd(d) if weights else None, cos=a.cos().float() if rope else None,
                sin=a.sin().float() if rope else None,
                dq=rnd(hq, n, d).bfloat16(), dk=rnd(hk, n, d).bfloat16(), dv=rnd(hk, n, d).bfloat16())


def rope_args(t):
    return {key: t[key] for key in ("wq", "wk", "cos", "sin")}


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: {(err - tol).max().item():.3e} over, max err {err.max().item():.3e}"


def check_forward(t, q_out, k_out, v_out, interleaved, eps=1e-6):
    for name, x, w, y in (("q", t["q"], t["wq"], q_out), ("k", t["k"], t["wk"], k_out)):
        ref, tol = R.forward(x, w, t["cos"], t["sin"], eps, interleaved)
        check(y, ref.transpose(0, 1), tol.transpose(0, 1), name)
    assert torch.equal(v_out, t["v"].bfloat16().transpose(0, 1))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 1), (1, 28, 7), (15, 3, 1), (17, 5, 5), (333, 8, 2), (2049, 6, 3)])
def test_forward_and_gradient(S, n, hq, hk, d, dtype, interleaved):
    t = make(n, hq, hk, d, dtype, 11 * n + hq + d)
    out = S.qk_norm_rope(t["q"], t["k"], t["v"], interleaved=interleaved, **rope_args(t))
    check_forward(t, *out, interleaved)
    got = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], dv=t["dv"], interleaved=interleaved, **rope_args(t))
    for name, x, dy, w, dx, dw, h in (("q", t["q"], t["dq"], t["wq"], got[0], got[3], hq),
                                      ("k", t["k"], t["dk"], t["wk"], got[1], got[4], hk)):
        ref, tol, dw_ref, sums = R.backward(x, dy.transpose(0, 1), w, t["cos"], t["sin"], 1e-6, interleaved, dtype)
        check(dx, ref, tol, "d" + name)
        check(dw, dw_ref, R.dw_tol(n, hq + 2 * hk, d, sums), "dw" + name)
    assert torch.equal(got[2], t["dv"].to(dtype).transpose(0, 1))
    assert S.device_status() == S.OK


@pytest.mark.parametrize("rope,weights", [(False, True), (True, False), (False, False)])
def test_without_rotation_or_weights(S, rope, weights):
    t = make(70, 4, 2, 128, torch.bfloat16, 3, rope, weights)
    out = S.qk_norm_rope(t["q"], t["k"], t["v"], **rope_args(t))
    check_forward(t, *out, False)
    got = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], dv=t["dv"], **rope_args(t))
    for x, dy, w, dx, dw in ((t["q"], t["dq"], t["wq"], got[0], got[3]), (t["k"], t["dk"], t["wk"], got[1], got[4])):
        ref, tol, dw_ref, sums = R.backward(x, dy.transpose(0, 1), w, t["cos"], t["sin"], 1e-6, False, x.dtype)
        check(dx, ref, tol, "dx")
        check(dw, dw_ref, R.dw_tol(70, 8, 128, sums), "dw")


def test_queries_alone(S):
    t = make(40, 3, 1, 64, torch.float32, 5)
    q_out, k_out, v_out = S.qk_norm_rope(t["q"], wq=t["wq"], cos=t["cos"], sin=t["sin"])
    assert k_out is None and v_out is None
    ref, tol = R.forward(t["q"], t["wq"], t["cos"], t["sin"], 1e-6, False)
    check(q_out, ref.transpose(0, 1), tol.transpose(0, 1), "q")
    dx, dk, dv, dw, dwk = S.qk_norm_rope_bwd(t["dq"], None, t["q"], wq=t["wq"], cos=t["cos"], sin=t["sin"])
    assert dk is None and dv is None and dwk is None
    ref, tol, dw_ref, sums = R.backward(t["q"], t["dq"].transpose(0, 1), t["wq"], t["cos"], t["sin"], 1e-6, False,
                                        torch.float32)
    check(dx, ref, tol, "dq")
    check(dw, dw_ref, R.dw_tol(40, 3, 64, sums), "dw")


def test_keys_go_behind_the_context_and_other_rows_stay(S):
    t = make(50, 4, 2, 128, torch.bfloat16, 6)
    k_all = torch.full((2, 200, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v_all = torch.full((2, 200, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    plain = S.qk_norm_rope(t["q"], t["k"], t["v"], **rope_args(t))
    out = S.qk_norm_rope(t["q"], t["k"], t["v"], k_out=k_all, v_out=v_all, kv_offset=120, **rope_args(t))
    assert out[1] is k_all and torch.equal(out[0], plain[0])
    for all_, new, fill in ((k_all, plain[1], 7.0), (v_all, plain[2], 9.0)):
        assert torch.equal(all_[:, 120:170], new)
        assert (all_[:, :120] == fill).all() and (all_[:, 170:] == fill).all()
    dk = torch.zeros(2, 200, 128, dtype=torch.bfloat16, device="cuda")
    dk[:, 120:170] = t["dk"]
    a = S.qk_norm_rope_bwd(t["dq"], dk, t["q"], t["k"], kv_offset=120, **rope_args(t))
    b = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], **rope_args(t))
    assert all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


@pytest.mark.parametrize("n", [1, 5, 40])
def test_one_token_of_each_sequence_into_a_cache(S, n):
    t = make(n, 8, 2, 128, torch.bfloat16, 7)
    cap = 33
    caches = [torch.full((n, 2, cap, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rows = (torch.arange(n, device="cuda", dtype=torch.int32) * 7) % cap
    if n > 2:
        rows[2] = -1                                                     # padding: left out
    qbuf = torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda")   # [sequence, head, d]
    plain = S.qk_norm_rope(t["q"], t["k"], t["v"], **rope_args(t))
    S.qk_norm_rope(t["q"], t["k"], t["v"], q_out=qbuf.transpose(0, 1), k_out=caches[0], v_out=caches[1], kv_rows=rows,
                   **rope_args(t))
    assert S.device_status() == S.OK
    assert torch.equal(qbuf.transpose(0, 1), plain[0])
    for cache, new in zip(caches, plain[1:]):
        want = torch.full_like(cache, 3.0)
        for i, r in enumerate(rows.tolist()):
            if r >= 0:
                want[i, :, r] = new[:, i]
        assert torch.equal(cache, want)


def test_a_row_past_the_cache_is_left_out_and_reported(S):
    t = make(3, 2, 1, 64, torch.bfloat16, 8)
    k_out = torch.full((1, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    v_out = k_out.clone()
    rows = torch.tensor([1, 4, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    S.qk_norm_rope(t["q"], t["k"], t["v"], k_out=k_out, v_out=v_out, kv_rows=rows, **rope_args(t))
    assert S.device_status() == S.ERR_DEVICE_BOUNDS and S.device_status() == S.OK
    assert (k_out[0, [0, 2, 3]] == 3.0).all() and not (k_out[0, 1] == 3.0).any()


def test_zero_rows_give_zero_and_special_values_stay_in_their_vectors(S):
    t = make(20, 2, 2, 128, torch.bfloat16, 9)
    x = torch.cat([t["q"], t["k"], t["v"]], dim=1)
    x[3, 0] = 0.0
    x[4, 1, 5] = float("inf")
    x[5, 0, 77] = float("nan")
    q, k, v = x[:, :2], x[:, 2:4], x[:, 4:]
    q_out, k_out, _ = S.qk_norm_rope(q, k, v, **rope_args(t))
    assert (q_out[0, 3] == 0).all()
    assert not torch.isfinite(q_out[1, 4]).all() and torch.isnan(q_out[0, 5]).all()
    ok = torch.ones(2, 20, dtype=torch.bool, device="cuda")
    ok[1, 4] = ok[0, 5] = False
    ref, tol = R.forward(q, t["wq"], t["cos"], t["sin"], 1e-6, False)
    err = (q_out.double() - ref.transpose(0, 1)).abs()
    assert (err <= tol.transpose(0, 1))[ok].all() and torch.isfinite(k_out).all()


def test_gradient_against_differences(S):
    """<dx, e> and <dw, e> against central differences of L = sum(dy * y) in fp64 (step 1e-5: the
    truncation error is of third order, 1e-10 of L's scale, and its cancellation 1e-16 / 1e-5)."""
    t = make(24, 3, 2, 64, torch.float32, 10)
    got = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], interleaved=True, **rope_args(t))
    g = torch.Generator(device="cuda").manual_seed(12)
    for x, dy, w, dx, dw in ((t["q"], t["dq"], t["wq"], got[0], got[3]), (t["k"], t["dk"], t["wk"], got[1], got[4])):
        dy = dy.double().transpose(0, 1)

        def loss(xx, ww):
            u = xx / (xx.square().mean(-1, keepdim=True) + 1e-6).sqrt() * ww
            return (R.turn(u, t["cos"], t["sin"], True) * dy).sum().item()

        xd, wd = x.double(), w.double()
        for _ in range(3):
            e = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
            diff = (loss(xd + 1e-5 * e, wd) - loss(xd - 1e-5 * e, wd)) / 2e-5
            assert abs(diff - (dx.double() * e).sum().item()) <= 2.0 ** -18 * (dx.double() * e).abs().sum().item() + 1e-6
            f = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
            diff = (loss(xd, wd + 1e-5 * f) - loss(xd, wd - 1e-5 * f)) / 2e-5
            _, _, _, sums = R.backward(x, dy, w, t["cos"], t["sin"], 1e-6, True, torch.float32)
            assert abs(diff - (dw.double() * f).sum().item()) <= (R.dw_tol(24, 5, 64, sums) * f.abs()).sum().item() + 1e-6


def test_reproducible_and_into_strided_outputs(S):
    t = make(700, 6, 2, 128, torch.bfloat16, 13)
    first = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], dv=t["dv"], **rope_args(t))
    fused = torch.full((700, 12, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    again = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], dv=t["dv"], dq_in=fused[:, :6], dk_in=fused[:, 6:8],
                               dv_in=fused[:, 8:10], **rope_args(t))
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert (fused[:, 10:] == 5.0).all()


def test_no_tokens(S):
    t = make(0, 2, 1, 64, torch.bfloat16, 14)
    q_out, k_out, v_out = S.qk_norm_rope(t["q"], t["k"], t["v"], **rope_args(t))
    assert q_out.shape == (2, 0, 64) and k_out.shape == (1, 0, 64)
    got = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], dv=t["dv"], **rope_args(t))
    assert (got[3] == 0).all() and (got[4] == 0).all()


def test_on_a_side_stream_and_in_a_graph(S):
    t = make(64, 4, 2, 128, torch.bfloat16, 15)
    want = S.qk_norm_rope(t["q"], t["k"], t["v"], **rope_args(t))
    want_b = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], **rope_args(t))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = S.qk_norm_rope(t["q"], t["k"], t["v"], stream=side, **rope_args(t))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = S.qk_norm_rope(t["q"], t["k"], t["v"], **rope_args(t))
        got = S.qk_norm_rope_bwd(t["dq"], t["dk"], t["q"], t["k"], **rope_args(t))
    for x in (*out, *got):
        if x is not None:
            x.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.equal(a, b) for a, b in zip(got, want_b) if a is not None)
