"""Draft verification where a request is short of work or a decision hangs on little: against the same 64-bit restatement."""
import pytest
import torch

from tests.test_gpu_verify import call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b", [1, 38, 39, 76, 77, 152, 153])
@pytest.mark.parametrize("v", [1, 2, 5, 8, 31])
def test_clusters_with_next_to_nothing_to_scan(b, v):
    """Requests of a few tokens: a cluster's CTAs send their shares to each other as soon as they can, some of them before others do
    anything.  Batches on both sides of every size of cluster, and the calls behind each other."""
    a = make(b, 2, v, torch.bfloat16, greedy=0.2, lens=True, seed=100 * b + v)
    tokens, counts = (x.clone() for x in call(a))
    check(a)
    for _ in range(20):
        a["tokens"].fill_(-9), a["counts"].fill_(-9)
        call(a)
        assert torch.equal(a["tokens"], tokens) and torch.equal(a["counts"], counts)
