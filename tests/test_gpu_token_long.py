"""Single tokens over caches so long that the scores take the place of the K/V ring in shared memory
(above 1,100 blocks), by clusters and by CTAs alone, beside short and empty sequences; and each entry
point captured into a graph by a process that has not called it before."""
import math
import subprocess
import sys

import pytest
import torch

from tests import token_ref as R
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


@pytest.mark.parametrize("lens,hq,hk,s,d,keep,sink,recent", [
    ([1300 * 128 - 5], 4, 1, 1300 * 128, 128, 40, 1, 2),             # clusters of eight
    ([200_000, 17, 0, 160 * 128, 199_873], 2, 2, 200_001, 64, 3, 0, 1),  # CTAs alone, lists of every kind
    ([16384 * 128 - 1, 150_000], 16, 1, 16384 * 128, 64, 17, 2, 1),  # the longest
])
def test_long_caches(S, lens, hq, hk, s, d, keep, sink, recent):
    b, group = len(lens), hq // hk
    g = torch.Generator(device="cuda").manual_seed(s + keep)
    k, v = (torch.empty(b, hk, s, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x in (k, v):
        for i in range(b):
            x[i] = torch.randn(hk, s, d, generator=g, device="cuda").bfloat16()
            x[i, :, lens[i]:] = math.nan
    q = torch.randn(b, hq, d, generator=g, device="cuda").bfloat16()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    means = S.block_means(k, kv_len)
    want = [[R.choose(q[i, h * group:(h + 1) * group], means[i, h], n, keep, sink, recent) for h in range(hk)]
            for i, n in enumerate(lens)]
    ws = S.TokenWorkspace(b, hq, hk, s, d, keep, "cuda")
    for _ in range(5):
        o, lse, idx, cnt = S.token_forward(q, k, v, kv_len, means, keep, sink, recent, workspace=ws)
        alone, cnt2 = S.token_select(q, means, kv_len, keep, sink, recent, capacity=s)
        assert S.device_status() == S.OK and torch.equal(idx, alone) and torch.equal(cnt, cnt2)
    for i, n in enumerate(lens):
        for h in range(hk):
            w = want[i][h]
            assert idx[i, h].tolist() == w + [-1] * (keep - len(w)) and int(cnt[i, h]) == len(w)
            sl = slice(h * group, (h + 1) * group)
            ref, tol, lr = R.attend(q[i, sl], k[i, h], v[i, h], n, w, 1 / math.sqrt(d))
            assert ((o[i, sl].double() - ref).abs() <= tol).all()
            if n:
                assert ((lse[i, sl].double() - lr).abs() <= 2.0 ** -12 + 2.0 ** -20 * lr.abs()).all()
            else:
                assert (lse[i, sl] == -math.inf).all()


FIRST = """
import torch
from block_sparse_attention_tok_b200 import sparstar as S
g = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *n: torch.randn(*n, generator=g, device="cuda").bfloat16()
if {which!r} == "norm":
    x = rnd(40, 12, 64)
    call = lambda: S.qk_norm_rope_bwd(*S.qk_norm_rope(x[:, :8], x[:, 8:10])[:2], x[:, :8], x[:, 8:10])
elif {which!r} == "gradient":
    q, k, lse = rnd(2, 300, 64), rnd(2, 500, 64), torch.full((2, 300), 5.0, device="cuda")
    idx = torch.arange(3, dtype=torch.int32, device="cuda").expand(2, 3, 3).contiguous()
    cnt = torch.full((2, 3), 3, dtype=torch.int32, device="cuda")
    call = lambda: S.attn_bwd(q, q, k, k, q, lse, idx, cnt)
else:
    q, k, n = rnd(3, 8, 64), rnd(3, 2, 900, 64), torch.tensor([900, 0, 300], dtype=torch.int32, device="cuda")
    m = torch.zeros(3, 2, 8, 64, device="cuda")
    call = lambda: S.token_forward(q, k, k, n, S.block_means(k, n, m), 3)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
want = call()
assert S.device_status() == S.OK
assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)
"""


@pytest.mark.parametrize("which", ["norm", "gradient", "token"])
def test_the_first_call_of_a_process_may_be_captured(S, which):
    run = subprocess.run([sys.executable, "-c", FIRST.format(which=which)], capture_output=True, text=True, timeout=300,
                         cwd=ROOT)
    assert run.returncode == 0, run.stderr[-2000:]
