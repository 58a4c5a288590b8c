"""token_forward with a workspace: the same results as without one, several steps over, in a graph
and beside another call."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


def make(S, lens, hq, hk, s, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(len(lens), hk, s, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda").bfloat16()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return q, k, v, kv_len, S.block_means(k, kv_len)


# every block kept, few candidates, many candidates over a cluster's CTAs, and an empty sequence
@pytest.mark.parametrize("lens,hq,hk,s,d,keep,sink,recent", [
    ([1], 1, 1, 1, 64, 1, 0, 1), ([700, 0, 129], 6, 2, 701, 128, 9, 1, 2), ([3000, 2999, 640], 8, 2, 3000, 64, 5, 1, 1),
    ([30000, 17], 16, 1, 30001, 128, 40, 2, 3),
])
def test_same_results_with_and_without(S, lens, hq, hk, s, d, keep, sink, recent):
    ws = S.TokenWorkspace(len(lens), hq, hk, s, d, keep, "cuda")
    for seed in (1, 2):  # the second call overwrites the lists of the first
        args = (*make(S, lens, hq, hk, s, d, seed), keep, sink, recent)
        want = S.token_forward(*args)
        ws.buf.fill_(2 ** 30)
        got = S.token_forward(*args, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert got[2] is ws.idx and got[3] is ws.cnt
        mine = torch.empty_like(ws.idx)
        ws.idx.fill_(7)
        got = S.token_forward(*args, idx=mine, workspace=ws)  # given lists come first
        assert got[2] is mine and torch.equal(mine, want[2]) and (ws.idx == 7).all()
    assert S.device_status() == S.OK


def test_two_calls_at_once_and_in_a_graph(S):
    shape = ([900, 1300], 8, 2, 1300, 128)
    cases = [(*make(S, *shape, seed), 5) for seed in (3, 4)]
    want = [S.token_forward(*c) for c in cases]
    ws = [S.TokenWorkspace(2, 8, 2, 1300, 128, 5, "cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [S.token_forward(*c, workspace=w, stream=st) for c, w, st in zip(cases, ws, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = S.token_forward(*cases[0], workspace=ws[0])
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want[0], got))


def test_refuses_a_workspace_of_another_shape(S):
    args = (*make(S, [300, 200], 4, 2, 300, 64, 5), 2)
    with pytest.raises(ValueError, match="workspace is for"):
        S.token_forward(*args, workspace=S.TokenWorkspace(2, 4, 2, 300, 64, 3, "cuda"))
    with pytest.raises(ValueError, match="tensors are on"):
        S.token_forward(*args, workspace=S.TokenWorkspace(2, 4, 2, 300, 64, 2, "cpu"))
