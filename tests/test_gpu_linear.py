"""Linear attention with a decay for each head against its 64-bit restatement.

Tolerances.  A value rounded to bf16 is off by at most 2^-8 of itself (half a step).  With M what an output would be if
nothing cancelled (the recurrence on magnitudes): the output is rounded once, 2^-8 |o|; on the tensor cores a score or a state's
element that makes part of it is rounded once, 2^-8 M; what
fp32 adds (sums of up to 128 products, exponentials, one factor a chunk) stays under 2^-13 M.  States: 2^-17 M for the two bf16
terms of a key, 2^-8 |s| for a bf16 state's own rounding, and 2^-16 M for fp32 sums over a sequence.
The norms' bars are for inputs whose roundings are independent: each has a standard deviation of at most 2^-8 / sqrt(3) of
its value, of which two add up as the root of their squares: 3.2e-3.
"""
import math

import pytest
import torch

import gated_delta_rule_23_gb300 as kda
from gated_delta_rule_23_gb300._native import (KDA_DEFAULT_WAIT_POLLS, KDA_ERR_INVALID_ARGUMENT, KDA_ERR_TIMEOUT,
                                               KDAError)
from tests import linear_ref

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(lengths, h, hkv, d, layout, seed=0, decay="both", state=torch.float32, initial=True, total=None):
    """Inputs of a call; layout: "batch" (equal lengths), "lens" (padded on the right) or "cu" (side by side)."""
    g = gen(seed)
    n = len(lengths)
    b, t = (1, sum(lengths)) if layout == "cu" else (n, total or max(lengths))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x = normal(b, t, (h + 2 * hkv) * d).to(torch.bfloat16)
    a = dict(q=x[..., :h * d].unflatten(-1, (h, d)), k=x[..., h * d:(h + hkv) * d].unflatten(-1, (hkv, d)),
             v=x[..., (h + hkv) * d:].unflatten(-1, (hkv, d)), log_decay=None, gate=None, lens=None, cu_seqlens=None)
    if decay in ("head", "both"):
        a["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, h + 1, device="cuda") / h)
    if decay in ("token", "both"):
        a["gate"] = -torch.nn.functional.softplus(2 * normal(b, t, h) - 3)
    if layout == "cu":
        a["cu_seqlens"] = torch.tensor([sum(lengths[:i]) for i in range(n + 1)], dtype=torch.int64, device="cuda")
    if layout == "lens":
        a["lens"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    a["initial_state"] = (3 * normal(n, h, d, d)).to(state) if initial else None
    a["final_state"] = torch.full((n, h, d, d), 7.0, device="cuda", dtype=state)
    a["out"] = torch.full((b, t, h, d), 5.0, device="cuda", dtype=torch.bfloat16)
    return a


def ranges_of(a):
    b, t = a["q"].shape[:2]
    if a["cu_seqlens"] is not None:
        cu = a["cu_seqlens"].tolist()
        return [(x, y - x) for x, y in zip(cu, cu[1:])]
    lens = a["lens"].tolist() if a["lens"] is not None else [t] * b
    return [(i * t, x) for i, x in enumerate(lens)]


def call(a, **kw):
    kda.kda_linear_attn(**{**a, **kw})
    kda.device_status()
    return a["out"], a["final_state"]


def logs(a):
    b, t, h = a["q"].shape[:3]
    x = torch.zeros((b * t, h), dtype=torch.float64, device="cuda")
    if a["log_decay"] is not None:
        x = x + a["log_decay"].double()
    if a["gate"] is not None:
        x = x + a["gate"].double().flatten(0, 1)
    return x


def check(a, out, fin, scale=None, norms=True, start=None):
    d = a["q"].shape[-1]
    scale = d ** -0.5 if scale is None else scale
    init = a["initial_state"] if start is None else start
    o, s, mag, size = linear_ref.linear(a["q"].flatten(0, 1), a["k"].flatten(0, 1), a["v"].flatten(0, 1), logs(a), scale,
                                        init, ranges_of(a))
    got = out.flatten(0, 1).double()
    live = ~o.isnan().all(-1).all(-1)
    half = fin is not None and fin.dtype == torch.bfloat16
    bound = BF16 * o.abs() + (BF16 + 2.0 ** -13) * mag
    off = (got - o).abs()
    assert bool((off <= bound)[live].all()), float((off / bound.clamp(min=1e-30))[live].max())
    assert bool((got[~live] == 5.0).all()), "rows behind the sequences were written"
    if norms and live.any() and float(o[live].norm()) > 0:
        assert float((got - o)[live].norm() / o[live].norm()) <= 3.2e-3 + 2.0 ** -13
    if fin is not None:
        bound = (BF16 if half else 0.0) * s.abs() + (2.0 ** -17 + 2.0 ** -16) * size
        off = (fin.double() - s).abs()
        assert bool((off <= bound).all()), float((off / bound.clamp(min=1e-30)).max())


EDGES = [1, 2, 5, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 200, 333]


@pytest.mark.parametrize("t", EDGES)
@pytest.mark.parametrize("h,hkv,d,state", [(4, 4, 128, torch.float32), (6, 2, 64, torch.bfloat16), (3, 1, 128, torch.bfloat16),
                                           (2, 2, 64, torch.float32)])
def test_lengths(t, h, hkv, d, state):
    a = make([t, t], h, hkv, d, "batch", seed=t, state=state)
    check(a, *call(a))


@pytest.mark.parametrize("layout", ["lens", "cu"])
@pytest.mark.parametrize("lengths", [[0, 1, 5, 3], [70, 0, 1, 64, 129], [1], [16, 0, 0], [300, 7, 65, 63, 64, 200]])
@pytest.mark.parametrize("d,state", [(128, torch.float32), (64, torch.bfloat16)])
def test_ragged(layout, lengths, d, state):
    a = make(lengths, 4, 2, d, layout, seed=len(lengths), state=state, total=max(lengths) + 3)
    check(a, *call(a))


@pytest.mark.parametrize("decay", ["", "head", "token", "both"])
@pytest.mark.parametrize("t", [3, 150])
def test_decays(decay, t):
    a = make([t, t], 4, 4, 128, "batch", seed=3, decay=decay)
    check(a, *call(a))


@pytest.mark.parametrize("t", [4, 100])
@pytest.mark.parametrize("initial,final", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_states_present_or_not(t, initial, final, state):
    a = make([t, t - 1], 3, 3, 128, "lens", seed=5, initial=initial, state=state)
    if not final:
        a["final_state"] = None
    check(a, *call(a))


@pytest.mark.parametrize("t", [1, 7, 130])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_state_in_place(t, state):
    a = make([t, t], 4, 4, 128, "batch", seed=6, state=state)
    start = a["initial_state"].clone()
    a["final_state"] = a["initial_state"]
    out, fin = call(a)
    check(a, out, fin, start=start)
    b = make([t, t], 4, 4, 128, "batch", seed=6, state=state)
    out2, fin2 = call(b)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)


@pytest.mark.parametrize("t", [5, 200])
def test_resumed_in_pieces(t):
    """Two calls in a row, the first one's final state into the second, are one call."""
    whole = make([2 * t], 4, 2, 128, "batch", seed=8)
    check(whole, *call(whole))
    first = {**whole, **{x: whole[x][:, :t] for x in ("q", "k", "v")}, "gate": whole["gate"][:, :t].contiguous(),
             "out": torch.empty_like(whole["out"][:, :t].contiguous()), "final_state": torch.empty_like(whole["final_state"])}
    kda.kda_linear_attn(**first)
    second = {**whole, **{x: whole[x][:, t:] for x in ("q", "k", "v")}, "gate": whole["gate"][:, t:].contiguous(),
              "out": torch.full_like(first["out"], 5.0), "initial_state": first["final_state"],
              "final_state": torch.empty_like(whole["final_state"])}
    out, fin = call(second)
    check(second, out, fin)
    assert float((fin - whole["final_state"]).norm() / fin.norm()) <= 2.0 ** -15


@pytest.mark.parametrize("t", [3, 100, 700])
def test_a_gate_of_minus_infinity_clears_the_state(t):
    a = make([t], 4, 4, 128, "batch", seed=9)
    at = sorted({0, t // 2, t - 1, min(70, t - 1)})
    a["gate"][:, at] = -math.inf
    out, fin = call(a)
    check(a, out, fin)
    # nothing of what came before is left
    b = {x: (y.clone() if isinstance(y, torch.Tensor) else y) for x, y in a.items()}
    b["v"] = a["v"].clone()
    b["v"][:, :t // 2] = 100.0
    out2, fin2 = call(b)
    assert torch.equal(out[:, t // 2:], out2[:, t // 2:]) and torch.equal(fin, fin2)


@pytest.mark.parametrize("strong", [-3.0, -20.0, -90.0])
def test_strong_decays_beside_weak_ones(strong):
    a = make([190], 2, 2, 128, "batch", seed=10, decay="token")
    a["gate"][:] = -1e-4
    a["gate"][:, ::3] = strong
    check(a, *call(a), norms=False)


@pytest.mark.parametrize("t", [2, 90])
def test_a_positive_decay_is_reported_and_taken_as_0(t):
    a = make([t], 2, 2, 128, "batch", seed=11, decay="token")
    a["gate"][0, t // 2, 1] = 0.5
    with pytest.raises(KDAError) as e:
        call(a)
    assert e.value.status == KDA_ERR_INVALID_ARGUMENT
    kda.device_status()
    a["gate"][0, t // 2, 1] = 0.0
    check(a, a["out"], a["final_state"])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 3, 64, 70, 127, 149])
@pytest.mark.parametrize("d", [64, 128])
def test_a_value_that_is_not_finite_reaches_no_earlier_token(bad, at, d):
    a = make([150, 150], 2, 2, d, "batch", seed=12)
    clean = make([150, 150], 2, 2, d, "batch", seed=12)
    call(clean)
    a["v"][0, at, 1, 5] = bad
    out, fin = call(a)
    column = torch.zeros_like(out, dtype=torch.bool)
    column[0, :, 1, 5] = True
    assert torch.equal(out[~column], clean["out"][~column])
    assert not bool(out[0, at:, 1, 5].isfinite().any())
    # what of the column comes before it may be summed in another order: a bf16 step
    before, was = out[0, :at, 1, 5].double(), clean["out"][0, :at, 1, 5].double()
    assert bool(((before - was).abs() <= 2 * BF16 * was.abs() + 2.0 ** -13).all())
    row = torch.zeros_like(fin, dtype=torch.bool)
    row[0, 1, 5] = True
    assert torch.equal(fin[~row], clean["final_state"][~row]) and not bool(fin[row].isfinite().any())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("at", [0, 5, 63, 66])
def test_a_key_or_query_that_is_not_finite_reaches_no_earlier_token(bad, at):
    a = make([100], 2, 2, 128, "batch", seed=13)
    clean = make([100], 2, 2, 128, "batch", seed=13)
    call(clean)
    a["k"][0, at, 0, 7] = bad
    out, fin = call(a)
    assert torch.equal(out[:, :at], clean["out"][:, :at]) and torch.equal(out[:, :, 1], clean["out"][:, :, 1])
    assert not bool(out[:, at:, 0].isfinite().any())
    assert torch.equal(fin[:, 1], clean["final_state"][:, 1]) and not bool(fin[:, 0, :, 7].isfinite().any())
    b = make([100], 2, 2, 128, "batch", seed=13)
    b["q"][0, at, 0, 7] = bad
    out, fin = call(b)
    other = torch.ones_like(out, dtype=torch.bool)
    other[0, at, 0] = False
    assert torch.equal(out[other], clean["out"][other]) and torch.equal(fin, clean["final_state"])
    assert not bool(out[0, at, 0].isfinite().any())


def test_what_lies_behind_a_sequence_does_not_reach_it():
    """Padding and the next sequence's tokens may hold anything."""
    for layout in ("lens", "cu"):
        a = make([70, 5, 130], 2, 1, 128, layout, seed=14, total=140)
        out, fin = (x.clone() for x in call(a))
        first, count = ranges_of(a)[0]
        for x in ("k", "v", "q"):
            flat = a[x].flatten(0, 1)
            flat[first + count:first + count + 5] = math.nan
            assert bool(a[x].isnan().any())
        a["gate"].flatten(0, 1)[first + count:first + count + 5] = math.nan
        a["out"].fill_(5.0)
        out2, fin2 = call(a)
        keep = slice(first, first + count)
        assert torch.equal(out.flatten(0, 1)[keep], out2.flatten(0, 1)[keep]) and torch.equal(fin[0], fin2[0])


def test_lens_out_of_range_are_reported_and_clamped():
    a = make([4, 4, 4], 2, 2, 64, "lens", seed=15)
    a["lens"].copy_(torch.tensor([-3, 9, 2], dtype=torch.int32))
    with pytest.raises(KDAError) as e:
        call(a)
    assert e.value.status == KDA_ERR_INVALID_ARGUMENT
    a["lens"].copy_(torch.tensor([0, 4, 2], dtype=torch.int32))
    check(a, a["out"], a["final_state"])


@pytest.mark.parametrize("cu", [[0, 400, 300], [0, -5, 300], [7, 9, 300], [0, 100, 1 << 40], [300, 200, 100]])
def test_malformed_cu_seqlens_stay_inside_the_buffers(cu):
    a = make([150, 150], 2, 2, 128, "cu", seed=16)
    guard = torch.full((3, 300, 2, 128), 3.0, device="cuda", dtype=torch.bfloat16)
    a["cu_seqlens"].copy_(torch.tensor(cu))
    a["out"] = guard[1:2]
    with pytest.raises(KDAError) as e:
        call(a)
    assert e.value.status == KDA_ERR_INVALID_ARGUMENT
    assert bool((guard[0] == 3).all()) and bool((guard[2] == 3).all())


@pytest.mark.parametrize("t", [3, 300])
def test_on_a_side_stream_and_in_a_graph(t):
    a = make([t, t], 4, 2, 128, "batch", seed=17)
    out, fin = (x.clone() for x in call(a))
    side = torch.cuda.Stream()
    a["out"].fill_(5.0), a["final_state"].fill_(7.0)
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_linear_attn(**a, stream=side)
    side.synchronize()
    assert torch.equal(a["out"], out) and torch.equal(a["final_state"], fin)
    size = kda.linear_attn_workspace_size(2, t, 4, 128)
    ws = torch.empty((max(size, 1),), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_linear_attn(**a, workspace=ws)
    v = a["v"].clone()
    for factor in (1.0, -2.0):
        a["v"].copy_(v * factor)
        a["out"].fill_(5.0)
        graph.replay()
        check(a, a["out"], a["final_state"])


def test_tokens_far_apart():
    """Offsets past 2^31 elements."""
    t, far = 20, 1 << 27
    store = torch.empty(((t - 1) * far + 3 * 128,), dtype=torch.bfloat16, device="cuda")
    a = make([t], 1, 1, 128, "batch", seed=18)
    for i, x in enumerate("qkv"):
        view = store[i * 128:].as_strided((1, t, 1, 128), (t * far, far, 128, 1))
        view.copy_(a[x])
        a[x] = view
    check(a, *call(a))
    b = {**a, "lens": torch.tensor([t - 1], dtype=torch.int32, device="cuda"), "out": torch.full_like(a["out"], 5.0)}
    check(b, *call(b))


def test_no_tokens_at_all():
    a = make([0, 0], 2, 2, 128, "cu", seed=19)
    _, fin = call(a)
    assert torch.equal(fin, a["initial_state"])
    a["initial_state"] = None
    _, fin = call(a)
    assert bool((fin == 0).all())


@pytest.mark.parametrize("scale", [0.0, -1.5, 0.3])
@pytest.mark.parametrize("t", [2, 70])
def test_scale(scale, t):
    a = make([t], 2, 2, 64, "batch", seed=20)
    check(a, *call(a, scale=scale), scale=scale)


@pytest.mark.parametrize("n,t,h,layout", [(1, 2100, 2, "batch"), (1, 4099, 1, "batch"), (3, 1000, 2, "cu"), (2, 900, 3, "lens"),
                                          (40, 65, 6, "batch")])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_long_sequences_on_few_heads(n, t, h, layout, state):
    r = [t] * n if layout == "batch" else [t - 37 * i for i in range(n)]
    a = make(r, h, 1, 128, layout, seed=21, state=state)
    if a["log_decay"] is not None:
        a["log_decay"] *= 0.01                      # long memories
        a["gate"] *= 0.02
    check(a, *call(a))


def test_the_same_bits_every_time():
    a = make([700, 300, 5], 4, 2, 128, "cu", seed=22)
    out, fin = (x.clone() for x in call(a))
    for _ in range(5):
        out2, fin2 = call(a)
        assert torch.equal(out, out2) and torch.equal(fin, fin2)


@pytest.mark.parametrize("n,each", [(33, 40), (129, 21), (200, 70)])
def test_many_sequences(n, each):
    """More than are sorted by length, and more than a warp looks at in one step."""
    r = [(i * 37) % each for i in range(n)]
    a = make(r, 2, 1, 64, "cu", seed=23)
    check(a, *call(a))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["cu", "lens"])
def test_groups_of_ragged_sequences(d, layout):
    """Few heads, long sequences among short and empty ones: groups of chunks side by side, of one sequence and of several."""
    a = make([3000, 0, 40, 1], 2, 1, d, layout, seed=24)
    a["log_decay"] *= 0.01
    a["gate"] *= 0.02
    a["gate"].flatten(0, 1)[1500] = -math.inf
    assert kda.linear_attn_workspace_size(4, a["q"].shape[1], 2, d, varlen=layout == "cu") > 0
    check(a, *call(a))


@pytest.mark.parametrize("t", [4, 100, 2500])
def test_states_off_32_bytes(t):
    a = make([t], 2, 2, 128, "batch", seed=25)
    size = a["initial_state"].numel()
    for x in ("initial_state", "final_state"):
        store = torch.full((size + 8,), 9.0, device="cuda")
        view = store[4:4 + size].view_as(a[x])
        view.copy_(a[x])
        a[x] = view
        a["guard_" + x] = store
    guards = [a.pop("guard_initial_state"), a.pop("guard_final_state")]
    check(a, *call(a))
    for g in guards:
        assert bool((g[:4] == 9).all()) and bool((g[-4:] == 9).all())


@pytest.mark.parametrize("t", [70, 3000])
def test_a_wait_that_gives_up_is_reported(t):
    a = make([t, t], 3, 3, 128, "batch", seed=26)
    lib = kda.load()
    lib.kda_set_wait_limit(0)
    try:
        with pytest.raises(KDAError) as e:
            call(a)
        assert e.value.status == KDA_ERR_TIMEOUT
    finally:
        lib.kda_set_wait_limit(KDA_DEFAULT_WAIT_POLLS)
    a["out"].fill_(5.0)
    check(a, *call(a))


@pytest.mark.parametrize("t", [70, 3000])
def test_waits_that_give_up_in_some_warps_alone(t):
    """Whatever comes of such a call, it ends, and the next one is right."""
    a = make([t, t], 3, 3, 128, "batch", seed=27)
    lib = kda.load()
    try:
        for polls in (1, 2, 5):
            lib.kda_set_wait_limit(polls)
            try:
                call(a)
            except KDAError as e:
                assert e.status == KDA_ERR_TIMEOUT
    finally:
        lib.kda_set_wait_limit(KDA_DEFAULT_WAIT_POLLS)
    a["out"].fill_(5.0)
    check(a, *call(a))


def test_two_graphs_with_workspaces_of_their_own():
    """Captured calls in groups, replayed on two streams at once."""
    calls, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        a = make([2500], 2, 2, 128, "batch", seed=27 + i)
        call(a)
        ws = torch.empty((kda.linear_attn_workspace_size(1, 2500, 2, 128),), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.kda_linear_attn(**a, workspace=ws)
        calls.append((a, ws)), graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, _ in calls:
        check(a, a["out"], a["final_state"])


def test_what_the_binding_refuses():
    a = make([20, 20], 4, 2, 64, "batch", seed=29)
    f32 = torch.float32
    wrong = [dict(q=a["q"].float()), dict(k=a["k"][:, :, :1]), dict(v=a["v"][:1]), dict(out=a["out"].float()),
             dict(out=a["out"].transpose(0, 1).contiguous().transpose(0, 1)), dict(log_decay=a["log_decay"].bfloat16()),
             dict(log_decay=a["log_decay"][:3]), dict(gate=a["gate"][:, :10]), dict(gate=a["gate"].bfloat16()),
             dict(initial_state=a["initial_state"].half()), dict(initial_state=a["initial_state"].bfloat16()),
             dict(final_state=a["final_state"][:1]), dict(lens=torch.zeros((2,), dtype=torch.int64, device="cuda")),
             dict(lens=torch.zeros((3,), dtype=torch.int32, device="cuda")),
             dict(cu_seqlens=torch.zeros((3,), dtype=torch.int64, device="cuda")), dict(q=a["q"][..., ::2]),
             dict(workspace=torch.zeros((4,), dtype=f32, device="cuda")), dict(v=a["v"].cpu())]
    for kw in wrong:
        with pytest.raises((TypeError, ValueError)):
            kda.kda_linear_attn(**{**a, **kw})
    with pytest.raises(KDAError):
        kda.kda_linear_attn(**{**a, "out": a["q"].contiguous(), "q": a["q"].contiguous()}, scale=math.nan)
    with pytest.raises(KDAError):
        same = a["q"].contiguous()
        kda.kda_linear_attn(**{**a, "out": same, "q": same})


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout,lengths", [("batch", [2500]), ("cu", [2000, 70, 0]), ("cu", [1985]), ("lens", [2113, 1])])
def test_state_in_place_with_groups(state, layout, lengths):
    """Groups of a sequence run side by side; the last one may end before the first one begins."""
    a = make(lengths, 2, 2, 128, layout, seed=30, state=state)
    b = make(lengths, 2, 2, 128, layout, seed=30, state=state)
    for x in (a, b):
        x["log_decay"] *= 0.001
        x["gate"] *= 0.002
    start = a["initial_state"].clone()
    a["final_state"] = a["initial_state"]
    out, fin = call(a)
    check(a, out, fin, start=start)
    out2, fin2 = call(b)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)


def test_a_thousand_sequences():
    r = [(i * 29) % 41 for i in range(1000)]
    a = make(r, 1, 1, 64, "cu", seed=31)
    check(a, *call(a))
