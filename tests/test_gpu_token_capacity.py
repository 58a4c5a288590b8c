"""token_select held to the cache's own capacity, where that ends within a block."""
import pytest
import torch

from tests import token_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S(cuda_lib):
    from block_sparse_attention_tok_b200 import sparstar
    return sparstar


@pytest.mark.parametrize("capacity", [1281, 1300, 1407, 1408])
def test_lengths_past_the_capacity_are_reported(S, capacity):
    g = torch.Generator(device="cuda").manual_seed(capacity)
    q = torch.randn(3, 4, 64, generator=g, device="cuda").bfloat16()
    means = torch.randn(3, 2, 11, 64, generator=g, device="cuda")
    for last, code in ((capacity, S.OK), (1408, S.OK if capacity == 1408 else S.ERR_DEVICE_BOUNDS),
                       (1409, S.ERR_DEVICE_BOUNDS)):
        kv_len = torch.tensor([capacity, 700, last], dtype=torch.int32, device="cuda")
        idx, cnt = S.token_select(q, means, kv_len, 4, 1, 1, capacity=capacity)
        assert S.device_status() == code
        for i, n in enumerate((capacity, 700, capacity)):
            for h in range(2):
                want = R.choose(q[i, 2 * h:2 * h + 2], means[i, h], n, 4, 1, 1)
                assert idx[i, h, :int(cnt[i, h])].tolist() == want
    idx2, _ = S.token_select(q, means, kv_len.clamp(max=1408), 4, 1, 1)  # whole blocks where none is given
    assert S.device_status() == S.OK and torch.equal(idx, idx2)
