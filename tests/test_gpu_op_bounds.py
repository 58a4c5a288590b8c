"""Writes of the norm with rotation, the attention gradient and the single-token entry points stay
inside their outputs and workspace: each lies in a larger buffer whose bands around it must not
change, at sizes with ragged ends."""
import pytest
import torch

from block_sparse_attention_tok_b200 import synth

pytestmark = pytest.mark.gpu
BAND = 4096  # bytes on either side


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


class Bands:
    def __init__(self):
        self.all = []

    def like(self, shape, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        n = int(torch.Size(shape).numel()) * size
        pad = -n % 256
        raw = torch.full((2 * BAND + n + pad,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, n))
        return raw[BAND:BAND + n].view(dtype).reshape(shape)

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.all:
            assert (raw[:BAND] == 0xA5).all() and (raw[BAND + n:] == 0xA5).all()


@pytest.mark.parametrize("block", [128, 64])
@pytest.mark.parametrize("H,n_q,n_kv,d", [(1, 1, 1, 64), (2, 130, 70, 128), (3, 333, 1001, 64), (2, 1100, 2500, 128)])
def test_attention_gradient(S, H, n_q, n_kv, d, block):
    q, k, v = synth.make_qkv(n_q, n_kv, H, d, list(range(H)), device="cuda")
    nqb, nkb = -(-n_q // block), -(-n_kv // block)
    keep = max(1, nkb // 2)
    b = Bands()
    idx, cnt = b.like((H, nqb, keep), torch.int32), b.like((H, nqb), torch.int32)
    g = torch.Generator().manual_seed(n_q)
    idx.copy_(torch.stack([torch.randperm(nkb, generator=g)[:keep] for _ in range(H * nqb)]).reshape(H, nqb, keep))
    cnt.fill_(keep)
    o, lse = S.attn(q, k, v, idx, cnt, block=block)
    ws = S.AttnBwdWorkspace(H, n_q, n_kv, d, keep, "cuda", block)
    ws.buf = b.like((ws.nbytes,), torch.uint8)
    assert ws.buf.data_ptr() % 256 == 0
    outs = [b.like(t.shape, torch.bfloat16) for t in (q, k, v)]
    S.attn_bwd(torch.ones_like(q), q, k, v, o, lse, idx, cnt, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws,
               block=block)
    assert S.device_status() == S.OK
    b.check()
    assert all(torch.isfinite(t).all() for t in outs)


@pytest.mark.parametrize("n,hq,hk,d", [(1, 1, 1, 64), (33, 5, 2, 128), (1001, 3, 3, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope(S, n, hq, hk, d, dtype):
    b = Bands()
    x = torch.randn(n, hq + 2 * hk, d, device="cuda").to(dtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    out = [b.like((h, n, d), torch.bfloat16) for h in (hq, hk, hk)]
    S.qk_norm_rope(q, k, v, q_out=out[0], k_out=out[1], v_out=out[2])
    grads = [b.like((n, h, d), dtype) for h in (hq, hk, hk)]
    S.qk_norm_rope_bwd(out[0], out[1], q, k, dv=out[2], dq_in=grads[0], dk_in=grads[1], dv_in=grads[2])
    b.check()
    assert all(torch.isfinite(t).all() for t in out + grads)


@pytest.mark.parametrize("lens,hq,hk,s,d,keep", [([1], 1, 1, 1, 64, 1), ([0, 129, 700], 6, 2, 701, 128, 3),
                                                ([30000, 17], 16, 1, 30001, 64, 40)])
def test_tokens(S, lens, hq, hk, s, d, keep):
    b, B = Bands(), len(lens)
    k, v = (torch.randn(B, hk, s, d, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, hq, d, device="cuda").bfloat16()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    means = b.like((B, hk, -(-s // 128), d), torch.float32)
    means.zero_()
    S.block_means(k, kv_len, means)
    S.block_means(k, kv_len, means, tail_only=True)
    idx, cnt = b.like((B, hk, keep), torch.int32), b.like((B, hk), torch.int32)
    o, lse = b.like((B, hq, d), torch.bfloat16), b.like((B, hq), torch.float32)
    S.token_select(q, means, kv_len, keep, 0, 1, idx=idx, cnt=cnt)
    S.token_attn(q, k, v, kv_len, idx, cnt, o=o, lse=lse)
    S.token_forward(q, k, v, kv_len, means, keep, 0, 1, idx=idx, cnt=cnt, o=o, lse=lse)
    assert S.device_status() == S.OK
    b.check()
    assert torch.isfinite(o).all() and torch.isfinite(means).all()
