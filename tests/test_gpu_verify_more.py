"""Draft verification where a request is short of work or a decision hangs on little: against the same 64-bit restatement."""
import math

import pytest
import torch

import gated_delta_rule_23_gb300 as kda
from gated_delta_rule_23_gb300._native import KDA_ERR_INVALID_ARGUMENT, KDAError
from tests.test_gpu_verify import call, check, expected, make

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


# -------------------------------------------------------------------------------------------- greedy requests whose logits tie
def tied(b, k, v, dtype, seed):
    """Rows with several largest logits, some of them in other chunks and some NaN before them; drafts that are the first, a later one, or none."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = make(b, k, v, dtype, probs=False, seed=seed)
    a["temperature"] = torch.zeros((b,), device="cuda")
    first = torch.randint(0, v, (b, k + 1), generator=g, device="cuda")
    for _ in range(3):
        at = torch.randint(0, v, (b, k + 1), generator=g, device="cuda")
        a["logits"].scatter_(2, at[..., None], 40.0)
        first = torch.minimum(first, at)
    a["logits"].scatter_(2, first[..., None], 40.0)
    a["logits"][:, :, 0][first > 0] = math.nan
    which = torch.rand((b, k), generator=g, device="cuda")
    a["draft_tokens"].copy_(torch.where(which < 0.75, first[:, :k], torch.where(which < 0.9, at[:, :k], a["draft_tokens"].long())))
    return a, first


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,k,v", [(1, 4, 1), (7, 4, 3), (40, 3, 1000), (9, 5, 8191), (200, 3, 5001), (3, 31, 40003), (2, 4, 1 << 20)])
def test_greedy_tokens_are_those_of_single_steps(dtype, b, k, v):
    """With first_largest every token is the row's first largest, whatever the drafts; also beside requests that sample."""
    a, first = tied(b, k, v, dtype, seed=b + v)
    tokens, counts = call(a, first_largest=True)
    taken = (a["draft_tokens"] == first[:, :k]).long().cumprod(1).sum(1)
    assert torch.equal(counts.long(), taken + 1)
    at = torch.arange(k + 1, device="cuda")
    assert torch.equal(tokens.long(), torch.where(at <= taken[:, None], first, -1))
    # one token at a time: the same call with no drafts, on the rows in turn
    alone = torch.empty((b, 1), dtype=torch.int32, device="cuda")
    one = torch.empty((b,), dtype=torch.int32, device="cuda")
    kda.kda_verify_drafts(a["logits"][:, 0].contiguous()[:, None], torch.empty((b, 0), dtype=torch.int32, device="cuda"),
                          torch.empty((b, 0), device="cuda"), a["noise"], alone, one, temperature=a["temperature"], first_largest=True)
    assert torch.equal(alone[:, 0], tokens[:, 0])
    # requests that sample do not change by it
    a["temperature"][::2] = 0.8
    tokens, counts = (x.clone() for x in call(a, first_largest=True))
    call(a)
    assert torch.equal(tokens[::2], a["tokens"][::2]) and torch.equal(counts[::2], a["counts"][::2])
    check(a)                                                          # any of the largest stands where that is not asked for


def test_a_row_without_a_maximum_under_the_first_of_the_largest():
    a, _ = tied(4, 2, 300, torch.float32, seed=3)
    a["logits"][0] = -math.inf
    a["logits"][1] = math.nan
    a["logits"][2, 0, 7] = math.inf
    a["draft_tokens"][2, 0] = 7
    tokens, counts = call(a, first_largest=True)
    assert counts[:3].tolist() == [1, 1, 1] and tokens[:3].tolist() == [[-1, -1, -1]] * 3


def test_the_first_of_the_largest_with_a_workspace():
    a, first = tied(6, 4, 20000, torch.bfloat16, seed=4)
    ws = torch.empty((kda.verify_drafts_workspace_size(6, 4, 20000),), dtype=torch.uint8, device="cuda")
    tokens, counts = (x.clone() for x in call(a, first_largest=True))
    a["tokens"].fill_(-9)
    call(a, first_largest=True, workspace=ws)
    assert torch.equal(a["tokens"], tokens) and torch.equal(a["counts"], counts)
    for small in (ws[:-8], ws[:0]):
        with pytest.raises(KDAError) as e:
            call(a, workspace=small)
        assert e.value.status == KDA_ERR_INVALID_ARGUMENT


# -------------------------------------------------------------------------------------------- temperatures and rows without a maximum
@pytest.mark.parametrize("tau", [1.0, 30.0, 1e4, 1e30, 3e38])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_high_temperatures_over_many_chunks(tau, dtype):
    """Against the restatement: weights of all tokens come near 1, and each counts."""
    a = make(4, 2, 70001, dtype, seed=21)
    a["temperature"].fill_(tau)
    a["logits"][:, :, 60000] = 40.0
    a["draft_tokens"][:2, 0] = 60000
    call(a)
    check(a)


def test_a_row_of_nan_after_an_accepted_draft():
    """The first draft stands (its test is 0 < p), the row behind it has no maximum: one token, and then none."""
    a = make(3, 2, 700, seed=22)
    a["uniform"].zero_()
    a["logits"][1, 1:] = math.nan
    a["logits"][2, 1:] = -math.inf
    tokens, counts = call(a)
    # (0 < 0 at a row without a maximum is no matter of rounding, so the restatement's tokens count as they are)
    want, many, _ = expected(a)
    assert counts.tolist() == many.tolist() == [3, 2, 2] and tokens.tolist() == want.tolist()
    for b in (1, 2):
        assert tokens[b].tolist() == [int(a["draft_tokens"][b, 0]), -1, -1]
