"""Draft verification against its 64-bit restatement.

The outputs are whole numbers, equal unless a decision is a matter of rounding: a probability is a quotient of fp32 exponentials, each off by a
few 2^-23 (the exponent's own rounding among it: logits under 64 in magnitude, 2^-18 at most), so requests whose test or whose
race is decided by less than 2^-16 of the value are left out of the comparison; there are few of them.
"""
import math

import pytest
import torch

import gated_delta_rule_23_gb300 as kda
from gated_delta_rule_23_gb300._native import KDA_ERR_INVALID_ARGUMENT, KDAError
from tests import linear_ref

pytestmark = pytest.mark.gpu


def make(b, k, v, dtype=torch.float32, probs=True, greedy=0.0, lens=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    logits = 3 * torch.randn((b, k + 1, v), generator=g, device="cuda")
    guess = torch.softmax(logits[:, :k] + torch.randn((b, k, v), generator=g, device="cuda"), -1)
    drafts = (guess / (-torch.log(rand(b, k, v).clamp(min=1e-9))).clamp(min=1e-9)).argmax(-1) if k else torch.zeros((b, 0), device="cuda")
    temperature = 0.5 + rand(b)
    temperature[rand(b) < greedy] = 0.0
    return dict(logits=logits.to(dtype), draft_tokens=drafts.to(torch.int32), uniform=rand(b, k),
                noise=(-torch.log(rand(b, v).clamp(min=1e-9))).clamp(min=1e-9),
                tokens=torch.full((b, k + 1), -9, dtype=torch.int32, device="cuda"),
                counts=torch.full((b,), -9, dtype=torch.int32, device="cuda"), draft_probs=guess if probs else None,
                temperature=temperature,
                draft_lens=torch.randint(0, k + 1, (b,), generator=g, device="cuda", dtype=torch.int32) if lens else None)


def call(a, **kw):
    kda.kda_verify_drafts(**{**a, **kw})
    kda.device_status()
    return a["tokens"], a["counts"]


def expected(a):
    b, rows = a["logits"].shape[:2]
    lens = a["draft_lens"].tolist() if a["draft_lens"] is not None else [rows - 1] * b
    tau = a["temperature"].tolist() if a["temperature"] is not None else [1.0] * b
    return linear_ref.verify(a["logits"], a["draft_tokens"].cpu(), a["draft_probs"], a["uniform"].cpu(), a["noise"], tau, lens)


def check(a):
    tokens, counts, near = expected(a)
    sure = near > 2.0 ** -16
    assert int((~sure).sum()) <= max(1, len(sure) // 50)
    assert torch.equal(a["counts"].cpu().long()[sure], counts[sure])
    assert torch.equal(a["tokens"].cpu().long()[sure], tokens[sure])
    return tokens, counts


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("b,k,v", [(1, 1, 1), (3, 2, 7), (5, 4, 33), (2, 31, 100), (40, 3, 1000), (3, 4, 8191), (2, 3, 16385),
                                   (3, 1, 40003), (2, 5, 131072)])
def test_sizes(dtype, probs, b, k, v):
    a = make(b, k, v, dtype, probs, greedy=0.2, lens=b > 2, seed=v)
    call(a)
    check(a)


def test_no_drafts():
    for lens in (None, "some"):
        a = make(6, 0 if lens is None else 3, 500, seed=1)
        if lens:
            a["draft_lens"] = torch.tensor([0, 3, 0, 1, 2, 0], dtype=torch.int32, device="cuda")
        call(a)
        check(a)


def test_certain_acceptance_and_certain_rejection():
    a = make(8, 4, 300, seed=2)
    a["uniform"].zero_()                              # 0 < p: all accepted
    call(a)
    assert bool((a["counts"] == 5).all()) and torch.equal(a["tokens"][:, :4], a["draft_tokens"])
    check(a)
    a["uniform"].fill_(1.0)
    a["draft_probs"].fill_(2.0)                       # never below p: all rejected; nothing is left over, so the race is on p
    call(a)
    assert bool((a["counts"] == 1).all()) and bool((a["tokens"][:, 1:] == -1).all())
    check(a)


def test_greedy_ties_and_drafts():
    a = make(4, 3, 5000, torch.bfloat16, probs=False, seed=3)
    a["temperature"] = torch.zeros((4,), device="cuda")
    a["logits"][:, :, 17] = a["logits"][:, :, 4000] = 50.0      # tied at the top
    a["draft_tokens"][:] = torch.tensor([[17, 4000, 17], [4000, 4000, 5], [3, 17, 17], [17, 17, 4999]], device="cuda")
    tokens, counts = call(a)
    assert counts.tolist() == [4, 3, 1, 3]
    assert tokens.tolist() == [[17, 4000, 17, 17], [4000, 4000, 17, -1], [17, -1, -1, -1], [17, 17, 17, -1]]


def test_equal_racers_go_to_the_lower_index():
    a = make(3, 1, 9000, seed=4)
    a["draft_lens"] = torch.zeros((3,), dtype=torch.int32, device="cuda")
    a["logits"].zero_()
    a["noise"].fill_(1.0)
    a["noise"][1, :4500] = 2.0
    tokens, counts = call(a)
    assert tokens[:, 0].tolist() == [0, 4500, 0] and counts.tolist() == [1, 1, 1]


def test_masked_logits_nan_and_rows_without_a_maximum():
    a = make(6, 2, 700, seed=5)
    a["logits"][:, :, ::2] = -math.inf                # a grammar's mask
    a["logits"][:, :, 1] = math.nan
    a["logits"][2] = -math.inf                        # nothing allowed
    a["logits"][3, 1:] = math.nan
    a["logits"][4, 0, 9] = math.inf
    tokens, counts = call(a)
    check(a)
    assert tokens[2].tolist() == [-1, -1, -1] and int(counts[2]) == 1
    assert int(tokens[3, int(counts[3]) - 1]) == (-1 if int(counts[3]) == 2 else int(tokens[3, 0]))
    assert int(tokens[4, 0]) == -1 and int(counts[4]) == 1
    for b in (0, 1, 5):
        got = [x for x in tokens[b].tolist() if x >= 0]
        assert all(x % 2 == 1 and x != 1 for x in got)


def test_the_types_lowest_value_as_a_mask():
    for dtype in (torch.float32, torch.bfloat16):
        a = make(4, 2, 700, dtype, seed=6)
        a["logits"][:, :, :650] = torch.finfo(dtype).min
        tokens, _ = call(a)
        check(a)
        assert all(x >= 650 or x == -1 or x in a["draft_tokens"].tolist()[i] for i, t in enumerate(tokens.tolist()) for x in t)


def test_small_and_large_temperatures():
    a = make(6, 2, 900, seed=7)
    a["temperature"] = torch.tensor([1e-45, 1e-20, 1e-3, 100.0, 1e30, 3e38], device="cuda")
    call(a)
    tokens, _ = check(a)
    best = a["logits"].argmax(-1).tolist()
    for i in range(2):
        assert all(x in (-1, best[i][j]) for j, x in enumerate(tokens[i].tolist()))


@pytest.mark.parametrize("bad", [-1.0, math.nan, math.inf])
def test_a_bad_temperature_is_reported_and_taken_as_0(bad):
    a = make(3, 2, 900, seed=8)
    a["temperature"][1] = bad
    with pytest.raises(KDAError) as e:
        call(a)
    assert e.value.status == KDA_ERR_INVALID_ARGUMENT
    kda.device_status()
    a["temperature"][1] = 0.0
    check(a)


def test_bad_drafts_and_counts_are_reported():
    a = make(4, 3, 900, seed=9)
    a["uniform"].zero_()
    a["draft_tokens"][1, 1] = 900
    a["draft_tokens"][2, 0] = -1
    with pytest.raises(KDAError):
        call(a)
    assert a["counts"].tolist() == [4, 2, 1, 4]
    check(a)
    a = make(4, 3, 900, seed=9)
    a["draft_lens"] = torch.tensor([-2, 9, 1, 0], dtype=torch.int32, device="cuda")
    with pytest.raises(KDAError):
        call(a)
    a["draft_lens"] = torch.tensor([0, 3, 1, 0], dtype=torch.int32, device="cuda")
    check(a)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rows_apart_and_off_16_bytes(dtype, shift):
    b, k, v = 3, 3, 5001
    a = make(b, k, v, dtype, seed=10 + shift)
    store = torch.full((b * (k + 1) * (v + 6) + shift,), 99.0, dtype=dtype, device="cuda")
    view = store[shift:].view(b, k + 1, v + 6)[..., :v]
    view.copy_(a["logits"])
    a["logits"] = view
    call(a)
    check(a)


def test_noise_that_is_not_positive():
    a = make(3, 1, 600, seed=12)
    a["draft_lens"] = torch.zeros((3,), dtype=torch.int32, device="cuda")
    a["noise"][0, 100:] = math.nan
    a["noise"][1, 100:] = -1.0
    a["noise"][2, 77] = 0.0
    tokens, _ = call(a)
    check(a)
    assert 0 <= int(tokens[0, 0]) < 100 and 0 <= int(tokens[1, 0]) < 100 and int(tokens[2, 0]) == 77
    a["noise"].fill_(-1e-9)                           # nothing can be drawn
    tokens, counts = call(a)
    check(a)
    assert bool((tokens == -1).all()) and bool((counts == 1).all())


def test_the_tokens_follow_the_targets_distribution():
    """Drafts from another distribution, 200,000 requests: the first token's frequencies are the target's.  A frequency of n requests is off
    by more than 5 standard deviations sqrt(p (1 - p) / n) once in two million."""
    n, v = 200000, 6
    g = torch.Generator(device="cuda").manual_seed(13)
    target = torch.tensor([1.0, 0.2, -1.0, 0.7, -2.0, 0.0], device="cuda")
    draft = torch.softmax(torch.tensor([-1.0, 1.0, 0.0, 0.5, 0.0, -3.0], device="cuda"), 0)
    drafts = torch.multinomial(draft.expand(n, v), 1, generator=g).to(torch.int32)
    tokens, counts = torch.empty((n, 2), dtype=torch.int32, device="cuda"), torch.empty((n,), dtype=torch.int32, device="cuda")
    noise = torch.empty((n, v), device="cuda").exponential_(generator=g).clamp(min=1e-20)
    kda.kda_verify_drafts(target.expand(n, 2, v).contiguous(), drafts, torch.rand((n, 1), generator=g, device="cuda"), noise, tokens,
                          counts, draft_probs=draft.expand(n, 1, v).contiguous())
    p = torch.softmax(target.double(), 0)
    got = torch.bincount(tokens[:, 0].long(), minlength=v).double() / n
    assert bool(((got - p).abs() <= 5 * (p * (1 - p) / n).sqrt()).all())
    taken = torch.minimum(p, draft.double()).sum()
    assert abs(float((counts == 2).double().mean() - taken)) <= 5 * float(taken * (1 - taken) / n) ** 0.5


def test_on_a_side_stream_and_in_a_graph():
    a = make(5, 4, 20000, torch.bfloat16, seed=14)
    tokens, counts = (x.clone() for x in call(a))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a["tokens"].fill_(-9)
    kda.kda_verify_drafts(**a, stream=side)
    side.synchronize()
    assert torch.equal(a["tokens"], tokens)
    ws = torch.empty((kda.verify_drafts_workspace_size(5, 4, 20000),), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_verify_drafts(**a, workspace=ws)
    uniform = a["uniform"].clone()
    for u in (uniform, 1 - uniform, uniform * 0):
        a["uniform"].copy_(u)
        graph.replay()
        check(a)
    a["uniform"].copy_(uniform)
    graph.replay()
    assert torch.equal(a["tokens"], tokens) and torch.equal(a["counts"], counts)


def test_what_the_binding_refuses():
    a = make(3, 2, 50, seed=15)
    wrong = [dict(logits=a["logits"].half()), dict(logits=a["logits"][0]), dict(draft_tokens=a["draft_tokens"].long()),
             dict(draft_tokens=a["draft_tokens"][:, :1]), dict(uniform=a["uniform"].double()), dict(noise=a["noise"][:, :49]),
             dict(noise=a["noise"].t().contiguous().t()), dict(tokens=a["tokens"][:, :2]), dict(counts=a["counts"].long()),
             dict(draft_probs=a["draft_probs"].bfloat16()), dict(draft_probs=a["draft_probs"][:, :1]),
             dict(temperature=a["temperature"].double()), dict(draft_lens=torch.zeros((2,), dtype=torch.int32, device="cuda")),
             dict(logits=a["logits"][..., ::2]), dict(noise=a["noise"].cpu()), dict(workspace=torch.zeros((4,), device="cuda"))]
    for kw in wrong:
        with pytest.raises((TypeError, ValueError)):
            kda.kda_verify_drafts(**{**a, **kw})


def test_guards_around_the_outputs():
    a = make(7, 3, 999, seed=16)
    tokens, counts = torch.full((9, 4), -7, dtype=torch.int32, device="cuda"), torch.full((16,), -7, dtype=torch.int32, device="cuda")
    a["tokens"], a["counts"] = tokens[1:8], counts[4:11]
    call(a)
    check(a)
    assert bool((tokens[0] == -7).all()) and bool((tokens[8] == -7).all())
    assert bool((counts[:4] == -7).all()) and bool((counts[11:] == -7).all())


@pytest.mark.parametrize("b", [39, 77, 153, 400])
def test_batches_of_every_size_of_cluster(b):
    a = make(b, 2, 2000, torch.bfloat16, greedy=0.1, lens=True, seed=b)
    call(a)
    check(a)


@pytest.mark.parametrize("tau", [1e-45, 1e-38, 1e-30, 1e-3, 1e30])
def test_extreme_temperatures_over_many_chunks(tau):
    """Exponents past fp32's range between the chunks of a row: what is far from the maximum has no weight, and no NaN comes of it."""
    a = make(4, 2, 70001, torch.bfloat16, seed=17)
    a["temperature"].fill_(tau)
    a["logits"][:, :, 60000] = 40.0
    a["draft_tokens"][:, 0] = 60000
    tokens, counts = call(a)
    if tau < 1.0:
        a["draft_probs"][:] = 0.0
        a["draft_probs"][:, :, 60000] = 1.0
        tokens, counts = call(a)
        assert bool((tokens[:, 0] == 60000).all())
    assert bool((tokens.gather(1, counts.long()[:, None] - 1) >= 0).all())
