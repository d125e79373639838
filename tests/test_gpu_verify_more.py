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


@pytest.mark.parametrize("dtype,body", [(torch.float32, 6.0), (torch.float32, 7.0), (torch.float32, 11.0), (torch.bfloat16, 7.0)])
@pytest.mark.parametrize("tau", [0.7213449, 0.55, 1.0])
def test_a_rows_sum_is_right_to_a_step_in_a_million(dtype, body, tau):
    """Drafts that are certain and have the largest logit stand while u z < 1: requests with u on both sides of 1 / z say what z is.

    The sum's exponents have a rounding of 2^-23.7 at most in their scale, taken times at most 7.5 (the weights' mean distance from a chunk's
    maximum, of a sum of which they are 0.9): 4.6e-7; an exponential's own 2^-22.5 = 1.7e-7; the sums' roundings, which average out, under
    2^-23 = 1.2e-7: 7.5e-7 in all.  0.7213449 is a temperature whose scale is rounded by that 2^-23.7.
    """
    v, b = 131072, 65
    g = torch.Generator(device="cuda").manual_seed(int(body))
    row = -(body + torch.rand((v,), generator=g, device="cuda") - 0.5) * tau
    row[::4096 if dtype == torch.float32 else 8192] = 0.0
    row = row.to(dtype)
    t = torch.tensor(tau, dtype=torch.float32)
    z = float((row.double() / float(t)).exp().sum())
    uniform = torch.tensor([1 / z], dtype=torch.float32)
    steps = torch.arange(-32, 33, dtype=torch.int32)
    uniform = (uniform.view(torch.int32) + steps).view(torch.float32).cuda()[:, None]
    a = dict(logits=row.expand(b, 2, v).contiguous(), draft_tokens=torch.zeros((b, 1), dtype=torch.int32, device="cuda"), uniform=uniform,
             noise=torch.ones((b, v), device="cuda"), tokens=torch.empty((b, 2), dtype=torch.int32, device="cuda"),
             counts=torch.empty((b,), dtype=torch.int32, device="cuda"), temperature=torch.full((b,), tau, device="cuda"))
    _, counts = call(a)
    off = (uniform[:, 0].double() * z - 1).cpu()
    sure = off.abs() > 7.5e-7
    assert bool(sure[0]) and bool(sure[-1])
    assert torch.equal((counts.cpu() == 2)[sure], (off < 0)[sure])
