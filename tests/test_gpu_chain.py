"""The operators together, as a layer uses them.

Training: fused projection -> qk_norm_rope (the new keys behind the context's) -> selection and
attention -> a loss -> attn_bwd -> qk_norm_rope_bwd, against fp64 autograd over the same kept lists.
Serving: a prompt's cache through qk_norm_rope and block_means, then single tokens through qk_norm_rope
into the cache, block_means of the newest block and token_forward, against fp64 over the same inputs."""
import math

import pytest
import torch

from tests import attn_bwd_ref as RB
from tests import norm_rope_ref as RN
from tests import token_ref as RT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


def angles(n, d, start=0):
    a = (start + torch.arange(n, dtype=torch.float64))[:, None] * 10000.0 ** (-torch.arange(0, d, 2).double() / d)
    return a.cos().float().cuda(), a.sin().float().cuda()


def norm_rope64(x, w, cos, sin, interleaved):
    u = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
    c, s = cos.double()[:, None], sin.double()[:, None]
    if interleaved:
        a, b = u[..., 0::2], u[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = u.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


@pytest.mark.parametrize("block,interleaved,dtype", [(128, False, torch.bfloat16), (64, True, torch.float32)])
def test_training_step(S, block, interleaved, dtype):
    H, d, n_text, n_ctx, n_cur = 2, 64, 200, 700, 900
    g = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    n_kv = n_text + n_ctx + n_cur
    x = rnd(n_cur, 3 * H, d).to(dtype)
    wq, wk = 1 + 0.2 * rnd(d), 1 + 0.2 * rnd(d)
    cos, sin = angles(n_cur, d)
    k, v = (rnd(H, n_kv, d).bfloat16() for _ in range(2))
    do = rnd(H, n_cur, d).bfloat16()
    rope = dict(wq=wq, wk=wk, cos=cos, sin=sin, interleaved=interleaved)
    at = n_text + n_ctx
    q, _, _ = S.qk_norm_rope(x[:, :H], x[:, H:2 * H], x[:, 2 * H:], k_out=k, v_out=v, kv_offset=at, **rope)
    o, lse, idx, cnt = S.forward(q, k, v, n_text, n_ctx, n_cur, 2, 0.3, block=block)
    dq, dk, dv = S.attn_bwd(do, q, k, v, o, lse, idx, cnt, block=block)
    dx = torch.empty_like(x)
    _, _, _, dwq, dwk = S.qk_norm_rope_bwd(dq, dk, x[:, :H], x[:, H:2 * H], dv=dv, kv_offset=at, dq_in=dx[:, :H],
                                           dk_in=dx[:, H:2 * H], dv_in=dx[:, 2 * H:], **rope)
    assert S.device_status() == S.OK

    xr = x.double().requires_grad_()
    wqr, wkr = wq.double().requires_grad_(), wk.double().requires_grad_()
    qr = norm_rope64(xr[:, :H], wqr, cos, sin, interleaved).transpose(0, 1)
    kr = torch.cat((k[:, :at].double(), norm_rope64(xr[:, H:2 * H], wkr, cos, sin, interleaved).transpose(0, 1)), 1)
    vr = torch.cat((v[:, :at].double(), xr[:, 2 * H:].transpose(0, 1)), 1)
    loss = 0.0
    for h in range(H):
        w = RB.multiplicity(idx[h], cnt[h], n_cur, n_kv, block)
        loss = loss + (RB.head_forward(qr[h], kr[h], vr[h], w, 1 / math.sqrt(d))[0] * do[h].double()).sum()
    loss.backward()
    # Six bf16 roundings lie on the way (q, k, v, o, P, dS, and dq, dk, dv), each 2^-8 at most and
    # independent over many terms: 2^-5 of the norm leaves them twice their worst sum.
    for name, got, ref in (("dx", dx, xr.grad), ("dwq", dwq, wqr.grad), ("dwk", dwk, wkr.grad)):
        err = torch.linalg.norm(got.double() - ref) / torch.linalg.norm(ref)
        assert err <= 2.0 ** -5, f"{name}: {err.item():.3e}"


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (3, 3, 64)])
def test_prompt_and_steps(S, hq, hk, d):
    b, cap, keep, sink, recent = 3, 1500, 5, 1, 1
    lens = [1021, 640, 127]
    g = torch.Generator(device="cuda").manual_seed(6)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    wq, wk = 1 + 0.2 * rnd(d), 1 + 0.2 * rnd(d)
    kc = torch.full((b, hk, cap, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    for i, n in enumerate(lens):  # prompts go into each sequence's cache
        x = rnd(n, hq + 2 * hk, d).bfloat16()
        cos, sin = angles(n, d)
        S.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], wq=wq, wk=wk, cos=cos, sin=sin, k_out=kc[i],
                       v_out=vc[i])
        ref, tol = RN.forward(x[:, hq:hq + hk], wk, cos, sin, 1e-6, False)
        assert ((kc[i, :, :n].double() - ref.transpose(0, 1)).abs() <= tol.transpose(0, 1)).all()
        assert torch.equal(vc[i, :, :n], x[:, hq + hk:].transpose(0, 1)) and torch.isnan(kc[i, :, n:]).all()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    means = S.block_means(kc, kv_len)
    qbuf = torch.empty(b, hq, d, dtype=torch.bfloat16, device="cuda")
    for step in range(5):  # crosses a block's end in two sequences
        x = rnd(b, hq + 2 * hk, d).bfloat16()
        pos = kv_len.cpu().double()
        a = pos[:, None] * 10000.0 ** (-torch.arange(0, d, 2).double() / d)
        cos, sin = a.cos().float().cuda(), a.sin().float().cuda()
        S.qk_norm_rope(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], wq=wq, wk=wk, cos=cos, sin=sin,
                       q_out=qbuf.transpose(0, 1), k_out=kc, v_out=vc, kv_rows=kv_len)
        kv_len += 1
        S.block_means(kc, kv_len, means, tail_only=True)
        o, lse, idx, cnt = S.token_forward(qbuf, kc, vc, kv_len, means, keep, sink, recent)
        assert S.device_status() == S.OK
        now = [n + step + 1 for n in lens]
        fresh = S.block_means(kc, kv_len)
        for i, n in enumerate(now):
            nb = -(-n // 128)
            assert torch.equal(means[i, :, :nb], fresh[i, :, :nb])
            for h in range(hk):
                sl = slice(h * hq // hk, (h + 1) * hq // hk)
                want = RT.choose(qbuf[i, sl], means[i, h], n, keep, sink, recent)
                assert idx[i, h, :int(cnt[i, h])].tolist() == want
                ref, tol, lr = RT.attend(qbuf[i, sl], kc[i, h], vc[i, h], n, want, 1 / math.sqrt(d))
                assert ((o[i, sl].double() - ref).abs() <= tol).all()
                assert ((lse[i, sl].double() - lr).abs() <= 2.0 ** -12 + 2.0 ** -20 * lr.abs()).all()
