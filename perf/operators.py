"""Cases, plain forms and 64-bit forms of the operators around the block-sparse attention.

Three groups, as a program uses them together:
  norm_rope       RMS norm of the queries and keys of each head and the position rotation, in one
                  pass that also lays q, k and v out head-major (or into a K/V cache), and its
                  gradient (norm_rope_bwd);
  attn_bwd        gradient of the attention over the kept blocks: dq, dk, dv;
  token           one query token per sequence over a K/V cache: the blocks are scored by the
                  query against the kept block means, the best are attended (token_forward);
                  block_means keeps those means.

With `own` false `run` computes an operator by elementary torch operations in 32 bits (block
scores in 64, where neighbouring ranks decide); with `own` true it calls the library.
"""
import math

import torch

own = False

BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "fp32": FP32}
POOL = 128  # tokens of a pooled cache block


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step of 4 sequences: each sequence's new q is normed and rotated, its new k
        # and v go behind the tokens its cache already holds.
        dict(name="norm_rope_step", op="norm_rope", n=4, hq=32, hk=8, d=128, dtype="bf16", interleaved=False,
             cache=1024),
        # A ragged prompt from fp32 projections, adjacent-pair rotation, narrow heads.
        dict(name="norm_rope_ragged_fp32", op="norm_rope", n=1000, hq=6, hk=6, d=64, dtype="fp32", interleaved=True,
             cache=0),
        # All heads of the 720p final scale.
        dict(name="norm_rope_final720p", op="norm_rope", n=72192, hq=32, hk=32, d=128, dtype="bf16",
             interleaved=False, cache=0),
        # Gradient of the ragged prompt, and of a refined scale in training.
        dict(name="norm_rope_bwd_ragged_fp32", op="norm_rope_bwd", n=1000, hq=6, hk=6, d=64, dtype="fp32",
             interleaved=True),
        dict(name="norm_rope_bwd_18k", op="norm_rope_bwd", n=18432, hq=32, hk=32, d=128, dtype="bf16",
             interleaved=False),
        # The tiny scale: two narrow heads, where launches count.
        dict(name="attn_bwd_tiny", op="attn_bwd", h=2, d=64, n_q=1024, n_text=256, n_ctx=768, n_cur=1024, clip=2,
             density=0.25, block=128),
        # Ragged query and key tails, 64-token blocks.
        dict(name="attn_bwd_ragged_b64", op="attn_bwd", h=4, d=128, n_q=4133, n_text=200, n_ctx=1000, n_cur=4133,
             clip=2, density=0.1875, block=64),
        # One GPU's share (4 heads of 32 split over 8) of the 720p final scale of a later clip.
        dict(name="attn_bwd_final720p_4heads", op="attn_bwd", h=4, d=128, n_q=72192, n_text=512, n_ctx=72192,
             n_cur=72192, clip=2, density=0.09375, block=128),
        # One sequence, every head with its own keys, a short cache: the latency of a step.
        dict(name="token_one_sequence", op="token_forward", b=1, hq=32, hk=32, d=128, s=4000, lo=4000, keep=16,
             sink=1, recent=1),
        # A served batch: 48 sequences of 2,000 to 32,768 tokens, four query heads to a key head.
        dict(name="token_batch_32k", op="token_forward", b=48, hq=32, hk=8, d=128, s=32768, lo=2000, keep=32,
             sink=1, recent=2),
        # Means of a whole prompt's cache, and of the newest block after a step.
        dict(name="means_prompt", op="block_means", b=4, hk=8, d=128, s=32768, lo=9000, tail=False),
        dict(name="means_step", op="block_means", b=48, hk=8, d=128, s=4096, lo=1, tail=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope", "norm_rope_bwd", "attn_bwd", "attn_bwd", "token_forward",
                     "token_forward", "block_means"])
    d = rng.choice([64, 128])
    if op in ("norm_rope", "norm_rope_bwd"):
        group = rng.choice([1, 1, 2, 4])
        hk = rng.choice([1, 2, 3, 5, 8])
        c = dict(op=op, n=_log_int(rng, 1, 72192 if op == "norm_rope" else 18432), hq=hk * group, hk=hk, d=d,
                 dtype=rng.choice(["bf16", "bf16", "fp32"]), interleaved=rng.random() < 0.5)
        if op == "norm_rope":
            c["cache"] = rng.randint(1, 3000) if c["n"] <= 64 else 0
        return c
    if op == "attn_bwd":
        block = rng.choice([128, 128, 64])
        n_cur = _log_int(rng, 1, 9000)
        return dict(op=op, h=rng.randint(1, 6), d=d, n_q=n_cur, n_text=rng.randint(0, 600),
                    n_ctx=_log_int(rng, 1, 9000), n_cur=n_cur, clip=rng.choice([1, 2]),
                    density=rng.choice([0.625, 0.1875, 0.09375, rng.uniform(0.02, 1.0)]), block=block)
    s = _log_int(rng, 1, 32768)
    hk = rng.choice([1, 2, 4, 8])
    b = max(1, min(_log_int(rng, 1, 48), (1 << 21) // (s * hk) + 1))
    if op == "block_means":
        return dict(op=op, b=b, hk=hk, d=d, s=s, lo=rng.randint(1, s), tail=rng.random() < 0.5)
    sink, recent = rng.randint(0, 2), rng.randint(1, 3)
    return dict(op=op, b=b, hq=hk * rng.choice([1, 2, 4, 5, 8, 16]), hk=hk, d=d, s=s, lo=rng.randint(1, s),
                keep=sink + recent + rng.randint(0, 40), sink=sink, recent=recent)


def _lengths(case):
    """Tokens held by each sequence: spread over [lo, s] in a fixed pattern, the first one full."""
    b, s, lo = case["b"], case["s"], case["lo"]
    return [s - int((s - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(b)]


def _budget(case):
    """Forced prefix and kept blocks of a query-block row."""
    block = case["block"]
    nkb = -(-(case["n_text"] + case["n_ctx"] + case["n_cur"]) // block)
    forced = -(-(case["n_text"] + (case["n_ctx"] if case["clip"] == 1 else 0)) // block)
    return nkb, forced, min(max(math.ceil(case["density"] * nkb - 1e-9), forced, 1), nkb)


# ------------------------------------------------------------------------------- inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=FP32)


def _angles(gen, n, d):
    """cos and sin of each token's rotation, from positions that a long video reaches."""
    pos = torch.randint(0, 1 << 17, (1,), generator=gen, device="cuda").double() + torch.arange(n, device="cuda")
    inv = 10000.0 ** (-torch.arange(0, d, 2, device="cuda").double() / d)
    a = pos[:, None] * inv
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        n, hq, hk, d = case["n"], case["hq"], case["hk"], case["d"]
        x = (1.5 * _randn(gen, n, hq + 2 * hk, d)).to(DTYPES[case["dtype"]])  # one fused projection
        st.update(x=x, q=x[:, :hq], k=x[:, hq:hq + hk], v=x[:, hq + hk:], wq=1 + 0.2 * _randn(gen, d),
                  wk=1 + 0.2 * _randn(gen, d))
        st["cos"], st["sin"] = _angles(gen, n, d)
        if op == "norm_rope_bwd":
            st.update(dq=_randn(gen, hq, n, d).to(BF16), dk=_randn(gen, hk, n, d).to(BF16),
                      dv=_randn(gen, hk, n, d).to(BF16))
        elif case["cache"]:
            s = case["cache"]
            st.update(k_cache=torch.zeros(n, hk, s, d, device="cuda", dtype=BF16),
                      v_cache=torch.zeros(n, hk, s, d, device="cuda", dtype=BF16),
                      rows=torch.randint(0, s, (n,), generator=gen, device="cuda", dtype=torch.int32))
        return st
    if op == "attn_bwd":
        h, d, n_q, block = case["h"], case["d"], case["n_q"], case["block"]
        n_kv = case["n_text"] + case["n_ctx"] + case["n_cur"]
        nkb, forced, keep = _budget(case)
        q, v, do = _randn(gen, h, n_q, d), _randn(gen, h, n_kv, d), _randn(gen, h, n_q, d)
        k = _randn(gen, h, n_kv, d)
        off = 0.5 * _randn(gen, h, nkb, d)  # blocks differ, as the selection needs
        k += off.repeat_interleave(block, dim=1)[:, :n_kv]
        st.update(q=q.to(BF16), k=k.to(BF16), v=v.to(BF16), do=do.to(BF16))
        qm, km = _block_mean(st["q"].float(), block), _block_mean(st["k"].float(), block)
        sc = qm @ km.transpose(1, 2)
        sc[:, :, :forced] = math.inf
        st["idx"] = torch.topk(sc, keep, dim=2).indices.sort(dim=2).values.to(torch.int32).contiguous()
        st["cnt"] = torch.full(sc.shape[:2], keep, device="cuda", dtype=torch.int32)
        o, lse = torch.empty(h, n_q, d, device="cuda"), torch.empty(h, n_q, device="cuda")
        for hh, i0, i1, kg, vg, s in _rows_of_blocks(st):
            m = s.amax(dim=2, keepdim=True)
            p = torch.exp(s - m)
            den = p.sum(dim=2, keepdim=True)
            t0, t1 = i0 * block, min(i1 * block, n_q)
            o[hh, t0:t1] = ((p @ vg) / den).reshape(-1, d)[:t1 - t0]
            lse[hh, t0:t1] = (m + torch.log(den)).reshape(-1)[:t1 - t0]
        st.update(o=o.to(BF16), lse=lse)
        if own:
            from block_sparse_attention_tok_b200 import sparstar
            st["ws"] = sparstar.AttnBwdWorkspace(h, n_q, n_kv, d, keep, "cuda", block)
        return st
    lens = _lengths(case)
    b, hk, d, s = case["b"], case["hk"], case["d"], case["s"]
    nb = -(-s // POOL)
    st["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    off = 0.5 * _randn(gen, b, hk, nb, 1, d)
    k = torch.empty(b, hk, nb, POOL, d, device="cuda", dtype=BF16)
    for i in range(b):
        k[i] = (_randn(gen, hk, nb, POOL, d) + off[i]).to(BF16)
    st["k"] = k.reshape(b, hk, nb * POOL, d)[:, :, :s].contiguous()
    st["means"] = torch.zeros(b, hk, nb, d, device="cuda")
    if op == "token_forward":
        v = torch.empty(b, hk, s, d, device="cuda", dtype=BF16)
        for i in range(b):
            v[i] = _randn(gen, hk, s, d).to(BF16)
        st["v"] = v
        st["q"] = _randn(gen, b, case["hq"], d).to(BF16)
        st["means"] = _masked_means(st)
        if own:
            from block_sparse_attention_tok_b200 import sparstar
            st["ws"] = sparstar.TokenWorkspace(b, case["hq"], hk, s, d, case["keep"], "cuda")
    return st


# ------------------------------------------------------------------------------- plain forms

def _norm(x, w, eps):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps) * w


def _pairs(x, interleaved):
    return (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, dim=-1)


def _join(a, b, interleaved):
    return torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)


def _rotate(x, cos, sin, interleaved):
    """x [N, H, d] turned by each token's angles."""
    a, b = _pairs(x, interleaved)
    c, s = cos[:, None], sin[:, None]
    return _join(a * c - b * s, b * c + a * s, interleaved)


EPS = 1e-6


def _plain_norm_rope(st):
    il = st["case"]["interleaved"]
    yq = _rotate(_norm(st["q"].float(), st["wq"], EPS), st["cos"], st["sin"], il).to(BF16)
    yk = _rotate(_norm(st["k"].float(), st["wk"], EPS), st["cos"], st["sin"], il).to(BF16)
    v = st["v"].to(BF16)
    if "k_cache" in st:
        at = torch.arange(yk.shape[0], device="cuda")
        st["k_cache"][at, :, st["rows"].long()] = yk
        st["v_cache"][at, :, st["rows"].long()] = v
        return yq.transpose(0, 1).contiguous(), st["k_cache"], st["v_cache"]
    return tuple(t.transpose(0, 1).contiguous() for t in (yq, yk, v))


def _plain_norm_rope_bwd(st):
    il = st["case"]["interleaved"]
    grads, dws = [], []
    for x, dy, w in ((st["q"], st["dq"], st["wq"]), (st["k"], st["dk"], st["wk"])):
        x = x.float()
        dn = _rotate(dy.float().transpose(0, 1), st["cos"], -st["sin"], il)
        r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
        xh = x * r
        g = dn * w
        dws.append((dn * xh).sum(dim=(0, 1)))
        grads.append((r * (g - xh * (g * xh).mean(dim=-1, keepdim=True))).to(st["q"].dtype))
    dv = st["dv"].transpose(0, 1).to(st["q"].dtype).contiguous()
    return grads[0], grads[1], dv, dws[0], dws[1]


def _block_mean(x, block):
    """Mean of each block of tokens of x [H, N, d], a ragged last one over its own tokens."""
    n = x.shape[1]
    nb = -(-n // block)
    pad = torch.nn.functional.pad(x, (0, 0, 0, nb * block - n)).reshape(x.shape[0], nb, block, -1)
    num = torch.full((nb,), float(block), device=x.device)
    num[-1] = n - (nb - 1) * block
    return pad.sum(dim=2) / num[:, None]


def _rows_of_blocks(st):
    """Runs of query blocks of a head with their gathered keys, values and scaled logits."""
    case = st["case"]
    block, d, n_q = case["block"], case["d"], case["n_q"]
    h, nqb, keep = st["idx"].shape
    n_kv = st["k"].shape[1]
    nkb = -(-n_kv // block)
    scale = 1 / math.sqrt(d)
    run = max(1, (1 << 26) // (block * block * keep))

    def blocks(x, n):
        return torch.nn.functional.pad(x.float(), (0, 0, 0, n * block - x.shape[0])).reshape(n, block, d)

    for hh in range(h):
        kb, vb, qb = blocks(st["k"][hh], nkb), blocks(st["v"][hh], nkb), blocks(st["q"][hh], nqb)
        for i0 in range(0, nqb, run):
            i1 = min(i0 + run, nqb)
            sel = st["idx"][hh, i0:i1].long()
            kg, vg = kb[sel].reshape(i1 - i0, -1, d), vb[sel].reshape(i1 - i0, -1, d)
            s = (qb[i0:i1] @ kg.transpose(1, 2)) * scale
            gone = (sel[:, :, None] * block + torch.arange(block, device="cuda")).reshape(i1 - i0, 1, -1) >= n_kv
            yield hh, i0, i1, kg, vg, s.masked_fill_(gone, -math.inf)


def _plain_attn_bwd(st):
    case = st["case"]
    block, d, n_q = case["block"], case["d"], case["n_q"]
    h, nqb, _ = st["idx"].shape
    n_kv = st["k"].shape[1]
    nkb = -(-n_kv // block)
    scale = 1 / math.sqrt(d)
    dq = torch.empty(h, n_q, d, device="cuda", dtype=BF16)
    dk, dv = (torch.zeros(h, nkb, block, d, device="cuda") for _ in range(2))
    for hh, i0, i1, kg, vg, s in _rows_of_blocks(st):
        t0, t1 = i0 * block, min(i1 * block, n_q)
        pad = (i1 - i0) * block - (t1 - t0)

        def rows(x):
            return torch.nn.functional.pad(x[hh, t0:t1].float(), (0, 0, 0, pad)).reshape(i1 - i0, block, d)

        q, o, do = rows(st["q"]), rows(st["o"]), rows(st["do"])
        lse = torch.nn.functional.pad(st["lse"][hh, t0:t1], (0, pad), value=math.inf).reshape(i1 - i0, block, 1)
        p = torch.exp(s - lse)
        ds = p * (do @ vg.transpose(1, 2) - (do * o).sum(dim=2, keepdim=True))
        sel = st["idx"][hh, i0:i1].long().reshape(-1)
        dq[hh, t0:t1] = ((ds @ kg) * scale).reshape(-1, d)[:t1 - t0].to(BF16)
        dk[hh].index_add_(0, sel, ((ds.transpose(1, 2) @ q) * scale).reshape(-1, block, d))
        dv[hh].index_add_(0, sel, (p.transpose(1, 2) @ do).reshape(-1, block, d))
    return dq, *(x.reshape(h, -1, d)[:, :n_kv].to(BF16).contiguous() for x in (dk, dv))


def _masked_means(st):
    """The state's means with those of every block that holds tokens put in."""
    case, k, lens = st["case"], st["k"], st["lens"].long()
    b, hk, s, d = k.shape
    nb = -(-s // POOL)
    pad = torch.nn.functional.pad(k, (0, 0, 0, nb * POOL - s)).reshape(b, hk, nb, POOL, d)
    at = torch.arange(nb * POOL, device="cuda").reshape(nb, POOL)
    live = at[None] < lens[:, None, None]
    num = live.sum(dim=2)
    sums = torch.stack([(pad[i].float() * live[i][None, :, :, None]).sum(dim=2) for i in range(b)])
    put = num > 0
    if case.get("tail"):
        put = put & (torch.arange(nb, device="cuda")[None] == (lens[:, None] - 1) // POOL)
    means = sums / num.clamp(min=1)[:, None, :, None]
    return torch.where(put[:, None, :, None], means, st["means"])


def _plain_token_forward(st):
    case, lens = st["case"], st["lens"].long()
    b, hk, s, d = st["k"].shape
    hq, keep, sink, recent = case["hq"], case["keep"], case["sink"], case["recent"]
    group, nb = hq // hk, -(-s // POOL)
    nblk = (lens + POOL - 1) // POOL
    j = torch.arange(nb, device="cuda")
    qs = st["q"].double().reshape(b, hk, group, d).sum(dim=2)
    score = (st["means"].double() @ qs[..., None])[..., 0]
    forced = (j < sink) | (j >= nblk[:, None] - recent)
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((j < nblk[:, None])[:, None], score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices
    width = min(keep, nb)
    cnt = nblk.clamp(max=keep)
    sel = torch.where(torch.arange(width, device="cuda") < cnt[:, None, None], order[:, :, :width], nb)
    sel = sel.sort(dim=2).values
    kb = torch.nn.functional.pad(st["k"], (0, 0, 0, nb * POOL - s)).reshape(b, hk, nb, POOL, d)
    vb = torch.nn.functional.pad(st["v"], (0, 0, 0, nb * POOL - s)).reshape(b, hk, nb, POOL, d)
    o = torch.empty(b, hq, d, device="cuda", dtype=BF16)
    lse = torch.empty(b, hq, device="cuda")
    heads = torch.arange(hk, device="cuda")[:, None]
    for i in range(b):
        rows = sel[i].clamp(max=nb - 1)
        kg, vg = (x[i][heads, rows].reshape(hk, -1, d).float() for x in (kb, vb))
        q = st["q"][i].float().reshape(hk, group, d)
        w = (q @ kg.transpose(1, 2)) / math.sqrt(d)
        at = (sel[i][:, :, None] * POOL + torch.arange(POOL, device="cuda")).reshape(hk, 1, -1)
        w = w.masked_fill(at >= lens[i], -math.inf)
        m = w.amax(dim=2, keepdim=True)
        p = torch.exp(w - m)
        den = p.sum(dim=2, keepdim=True)
        o[i] = ((p @ vg) / den).reshape(hq, d).to(BF16)
        lse[i] = (m + torch.log(den)).reshape(hq)
    idx = torch.full((b, hk, keep), -1, device="cuda", dtype=torch.int32)
    idx[:, :, :width] = torch.where(sel < nb, sel, -1).to(torch.int32)
    return o, lse, idx, cnt[:, None].expand(b, hk).to(torch.int32).contiguous()


# ------------------------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        if op == "norm_rope":
            return _plain_norm_rope(st)
        if op == "norm_rope_bwd":
            return _plain_norm_rope_bwd(st)
        if op == "attn_bwd":
            return _plain_attn_bwd(st)
        if op == "token_forward":
            return _plain_token_forward(st)
        st["means"] = _masked_means(st)
        return st["means"]
    from block_sparse_attention_tok_b200 import sparstar
    if op == "norm_rope":
        rope = dict(wq=st["wq"], wk=st["wk"], cos=st["cos"], sin=st["sin"], eps=EPS, interleaved=case["interleaved"])
        if "k_cache" in st:
            return sparstar.qk_norm_rope(st["q"], st["k"], st["v"], k_out=st["k_cache"], v_out=st["v_cache"],
                                         kv_rows=st["rows"], **rope)
        return sparstar.qk_norm_rope(st["q"], st["k"], st["v"], **rope)
    if op == "norm_rope_bwd":
        return sparstar.qk_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], dv=st["dv"], wq=st["wq"], wk=st["wk"],
                                         cos=st["cos"], sin=st["sin"], eps=EPS, interleaved=case["interleaved"])
    if op == "attn_bwd":
        return sparstar.attn_bwd(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], st["idx"], st["cnt"],
                                 block=case["block"], workspace=st["ws"])
    if op == "token_forward":
        return sparstar.token_forward(st["q"], st["k"], st["v"], st["lens"], st["means"], case["keep"],
                                      n_sink=case["sink"], n_recent=case["recent"], workspace=st["ws"])
    return sparstar.block_means(st["k"], st["lens"], st["means"], tail_only=case["tail"])


def work(case):
    op, d = case["op"], case["d"]
    if op in ("norm_rope", "norm_rope_bwd"):
        n, hq, hk = case["n"], case["hq"], case["hk"]
        e = 2 if case["dtype"] == "bf16" else 4
        if op == "norm_rope":
            return dict(bytes=n * (hq + 2 * hk) * d * (e + 2) + n * d * 4, flops=n * (hq + hk) * d * 8)
        return dict(bytes=n * (hq + hk) * d * (2 + 2 * e) + n * hk * d * (2 + e) + n * d * 4,
                    flops=n * (hq + hk) * d * 16)
    if op == "attn_bwd":
        h, n_q, block = case["h"], case["n_q"], case["block"]
        n_kv = case["n_text"] + case["n_ctx"] + case["n_cur"]
        nkb, _, keep = _budget(case)
        nqb = -(-n_q // block)
        return dict(bytes=h * (4 * (n_q + n_kv) * d * 2 + n_q * 4 + nqb * keep * 4),
                    flops=10 * d * h * n_q * min(keep * block, n_kv))
    lens = _lengths(case)
    hk = case["hk"]
    if op == "block_means":
        tok = sum((n - 1) % POOL + 1 for n in lens) if case["tail"] else sum(lens)
        blocks = len(lens) if case["tail"] else sum(-(-n // POOL) for n in lens)
        return dict(bytes=hk * d * (tok * 2 + blocks * 4), flops=hk * d * tok)
    hq, keep, forced = case["hq"], case["keep"], case["sink"] + case["recent"]
    nbytes = flops = 0
    for n in lens:
        nb = -(-n // POOL)
        scored = nb - forced if nb > keep else 0
        tok = n if nb <= keep else (keep - 1) * POOL + (n - 1) % POOL + 1
        nbytes += hk * d * (scored * 4 + tok * 4) + hq * d * 4 + hk * keep * 4
        flops += hk * scored * d * 2 + 4 * hq * tok * d
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------------------------------------- 64-bit forms

def _exact_turn(x, c, s, interleaved):
    """Each pair of coordinates as a complex number times exp(i angle)."""
    d = x.shape[-1]
    first = torch.arange(0, d, 2, device=x.device) if interleaved else torch.arange(d // 2, device=x.device)
    second = first + (1 if interleaved else d // 2)
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(c, s)
    y = torch.empty_like(x)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm_rope(st):
    il = st["case"]["interleaved"]
    n = st["x"].shape[0]
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        y = torch.empty(x.shape[1], n, x.shape[2], device="cuda", dtype=torch.float64)
        for h in range(x.shape[1]):
            xh = x[:, h].double()
            ms = (xh * xh).sum(dim=-1, keepdim=True) / x.shape[2]
            y[h] = _exact_turn(w.double() * xh / (ms + EPS).sqrt(), st["cos"].double(), st["sin"].double(), il)
        out.append(y)
    v = st["v"].transpose(0, 1).double()
    if "k_cache" in st:
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        for i, r in enumerate(st["rows"].tolist()):
            kc[i, :, r], vc[i, :, r] = out[1][:, i], v[:, i]
        return out[0], kc, vc
    return out[0], out[1], v.contiguous()


def _exact_norm_rope_bwd(st):
    il = st["case"]["interleaved"]
    res = []
    for x, dy, w in ((st["q"], st["dq"], st["wq"]), (st["k"], st["dk"], st["wk"])):
        n, heads, d = x.shape
        dx = torch.empty(n, heads, d, device="cuda", dtype=torch.float64)
        dw = torch.zeros(d, device="cuda", dtype=torch.float64)
        for h in range(heads):
            xh = x[:, h].double()
            norm = ((xh * xh).sum(dim=-1, keepdim=True) / d + EPS).sqrt()
            dn = _exact_turn(dy[h].double(), st["cos"].double(), -st["sin"].double(), il)
            dw += (dn * xh / norm).sum(dim=0)
            dn = dn * w.double()
            dx[:, h] = dn / norm - xh * (dn * xh).sum(dim=-1, keepdim=True) / (d * norm ** 3)
        res.append((dx, dw))
    return res[0][0], res[1][0], st["dv"].transpose(0, 1).double().contiguous(), res[0][1], res[1][1]


def _exact_attn_bwd(st):
    """Over dense rows of logits, with the pairs that are not kept taken out."""
    case = st["case"]
    block, d, h, n_q = case["block"], case["d"], case["h"], case["n_q"]
    n_kv = st["k"].shape[1]
    nkb = -(-n_kv // block)
    scale = 1 / math.sqrt(d)
    dq, dk, dv = (torch.zeros(h, n, d, device="cuda", dtype=torch.float64) for n in (n_q, n_kv, n_kv))
    per = max(1, (1 << 25) // (n_kv * block))
    for hh in range(h):
        k, v = st["k"][hh].double(), st["v"][hh].double()
        for i0 in range(0, st["idx"].shape[1], per):
            sel = st["idx"][hh, i0:i0 + per].long()
            kept = torch.zeros(sel.shape[0], nkb, device="cuda", dtype=torch.bool).scatter_(1, sel, True)
            t0, t1 = i0 * block, min((i0 + sel.shape[0]) * block, n_q)
            kept = kept.repeat_interleave(block, 0)[:t1 - t0].repeat_interleave(block, 1)[:, :n_kv]
            q, o, do = (st[x][hh, t0:t1].double() for x in ("q", "o", "do"))
            p = torch.exp(scale * (q @ k.T) - st["lse"][hh, t0:t1].double()[:, None]) * kept
            dv[hh] += p.T @ do
            ds = scale * p * (do @ v.T - (o * do).sum(dim=1)[:, None])
            dq[hh, t0:t1] = ds @ k
            dk[hh] += ds.T @ q
    return dq, dk, dv


def _exact_token_forward(st):
    case = st["case"]
    hk, group, d = case["hk"], case["hq"] // case["hk"], case["d"]
    o, lse = [], []
    for i, n in enumerate(st["lens"].tolist()):
        nb = -(-n // POOL)
        for g in range(hk):
            q = st["q"][i, g * group:(g + 1) * group].double()
            if nb <= case["keep"]:
                blocks = list(range(nb))
            else:
                forced = list(range(case["sink"])) + list(range(nb - case["recent"], nb))
                rest = range(case["sink"], nb - case["recent"])
                sc = (st["means"][i, g, :nb].double() * q.sum(dim=0)).sum(dim=1).tolist()
                best = sorted(rest, key=lambda j: (-sc[j], j))[:case["keep"] - len(forced)]
                blocks = sorted(forced + best)
            at = torch.cat([torch.arange(j * POOL, min((j + 1) * POOL, n), device="cuda") for j in blocks])
            w = q @ st["k"][i, g, at].double().T / math.sqrt(d)
            lse.append(torch.logsumexp(w, dim=1))
            o.append(torch.exp(w - lse[-1][:, None]) @ st["v"][i, g, at].double())
    b = case["b"]
    return torch.stack(o).reshape(b, -1, d), torch.stack(lse).reshape(b, -1), None, None


def _exact_block_means(st):
    out = st["means"].double()
    for i, n in enumerate(st["lens"].tolist()):
        nb = -(-n // POOL)
        for j in range(nb - 1 if st["case"]["tail"] else 0, nb):
            out[i, :, j] = st["k"][i, :, j * POOL:min((j + 1) * POOL, n)].double().mean(dim=1)
    return out


def exact(case, seed):
    if case["op"] == "attn_bwd" and 10 * case["d"] * case["h"] * case["n_q"] * (
            case["n_text"] + case["n_ctx"] + case["n_cur"]) > 2e13:
        return None
    st = prepare(case, seed)
    form = dict(norm_rope=_exact_norm_rope, norm_rope_bwd=_exact_norm_rope_bwd, attn_bwd=_exact_attn_bwd,
                token_forward=_exact_token_forward, block_means=_exact_block_means)
    return form[case["op"]](st)
