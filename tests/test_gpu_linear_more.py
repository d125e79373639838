"""Linear attention at the corners of its two kernels: against the same 64-bit restatement, within the bounds of tests/test_gpu_linear.py."""
import math

import pytest
import torch

import gated_delta_rule_23_gb300 as kda
from gated_delta_rule_23_gb300._native import KDA_ERR_INVALID_ARGUMENT, KDAError
from tests import linear_ref
from tests.test_gpu_linear import BF16, call, logs, make, ranges_of

pytestmark = pytest.mark.gpu


def same_kind(got, want):
    """Infinities of either sign and NaN where the other has them."""
    return (torch.equal(got.isnan(), want.isnan()) and torch.equal(got == math.inf, want == math.inf) and
            torch.equal(got == -math.inf, want == -math.inf))


# -------------------------------------------------------------------------------------------- states that are not finite
@pytest.mark.parametrize("decay", [0.0, -1e-3, -0.3, -3.0])
@pytest.mark.parametrize("d,state", [(128, torch.float32), (64, torch.bfloat16)])
@pytest.mark.parametrize("layout,lengths", [("lens", [0, 3, 5]), ("lens", [0, 70, 129]), ("cu", [0, 64, 200, 0, 1]), ("lens", [2500, 0]),
                                            ("cu", [1500, 0, 900])])
def test_an_infinite_state_stays_infinite(layout, lengths, d, state, decay):
    """e^a x infinity is infinity for every a, in both kernels, and a sequence of no tokens hands its state on as it is."""
    a = make(lengths, 2, 1, d, layout, seed=50, decay="head", state=state, total=max(lengths) + 1)
    a["log_decay"].fill_(decay / 64)                              # (of a chunk: decay)
    for n in range(len(lengths)):
        for i, x in enumerate((math.inf, -math.inf, math.nan)):
            a["initial_state"][n, i % 2, 5 + 29 * i, 7 * i + n] = x
    out, fin = call(a)
    o, s, mag, size = linear_ref.linear(a["q"].flatten(0, 1), a["k"].flatten(0, 1), a["v"].flatten(0, 1), logs(a), d ** -0.5,
                                        a["initial_state"], ranges_of(a))
    assert same_kind(fin, s)
    for n, count in enumerate(lengths):
        if count == 0:
            assert torch.equal(fin[n].nan_to_num(), a["initial_state"][n].nan_to_num())
    fine = s.isfinite()
    half = BF16 if state == torch.bfloat16 else 0.0
    assert bool(((fin.double() - s).abs() <= half * s.abs() + (2.0 ** -17 + 2.0 ** -16) * size)[fine].all())
    # (rows that no sequence has are NaN in the restatement)
    live = torch.zeros_like(o, dtype=torch.bool)
    for first, count in ranges_of(a):
        live[first:first + count] = True
    got = out.flatten(0, 1).double()
    assert same_kind(got[live], o[live])
    fine = live & o.isfinite()
    assert bool(((got - o).abs() <= BF16 * o.abs() + (BF16 + 2.0 ** -13) * mag)[fine].all())
    assert bool((got[~live] == 5.0).all())


# -------------------------------------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(4))
def test_many_values_that_are_not_finite(d, seed):
    """Columns of one warp that take their outputs again from different tokens on, or not at all: each token's outputs before its column's
    first bad value are what the finite values make of them, and those of other columns do not change by a bit."""
    a = make([150, 90], 2, 1, d, "lens", seed=60 + seed, total=160)
    clean = {x: (y.clone() if isinstance(y, torch.Tensor) else y) for x, y in a.items()}
    call(clean)
    g = torch.Generator().manual_seed(seed)
    first = torch.full((2, d), 1 << 20)                           # first bad token of a sequence's column
    for n, count in ((0, 150), (1, 90)):
        for _ in range(d // 3):
            t, c = int(torch.randint(count, (1,), generator=g)), int(torch.randint(d, (1,), generator=g))
            a["v"][n, t, 0, c] = (math.nan, math.inf, -math.inf)[t % 3]
            first[n, c] = min(int(first[n, c]), t)
    out, fin = call(a)
    o, s, mag, size = linear_ref.linear(a["q"].flatten(0, 1), a["k"].flatten(0, 1), a["v"].flatten(0, 1), logs(a), d ** -0.5,
                                        a["initial_state"], ranges_of(a))
    o, mag = o.view(out.shape), mag.view(out.shape)
    t = torch.arange(160)[None, :, None]
    live = (t < torch.tensor([150, 90])[:, None, None]).expand(2, 160, d)
    before = (live & (t < first[:, None])).cuda()[:, :, None].expand(out.shape)
    behind = (live & (t >= first[:, None])).cuda()[:, :, None].expand(out.shape)
    assert bool(((out.double() - o).abs() <= BF16 * o.abs() + (BF16 + 2.0 ** -13) * mag)[before].all())
    assert not bool(out[behind].isfinite().any())
    untouched = (first == 1 << 20).cuda()
    for n in range(2):
        assert torch.equal(out[n][..., untouched[n]], clean["out"][n][..., untouched[n]])
        assert torch.equal(fin[n][:, untouched[n]], clean["final_state"][n][:, untouched[n]])
        assert not bool(fin[n][:, ~untouched[n]].isfinite().any())


# -------------------------------------------------------------------------------------------- bars of each kernel's own
def restated(a):
    o, s, mag, size = linear_ref.linear(a["q"].flatten(0, 1), a["k"].flatten(0, 1), a["v"].flatten(0, 1), logs(a),
                                        a["q"].shape[-1] ** -0.5, a["initial_state"], ranges_of(a))
    return o, s, mag, size, ~o.isnan().all(-1).all(-1)


def takes_tokens(a):
    """Whether a call goes token by token (sizes alone say so)."""
    t, h, d = a["q"].shape[1:]
    return t <= (16 if d == 64 else 14 if len(ranges_of(a)) * h <= 1024 else 8)


@pytest.mark.parametrize("layout,lengths", [("batch", [1] * 5), ("batch", [2, 2]), ("batch", [8] * 200), ("batch", [14] * 3), ("lens", [0, 13, 1, 7]),
                                            ("lens", [0, 5, 3, 8] * 80), ("cu", [1, 0, 9, 4]), ("cu", [1] * 14)])
@pytest.mark.parametrize("h,hkv,d,state", [(6, 2, 128, torch.float32), (6, 2, 128, torch.bfloat16), (8, 8, 64, torch.float32),
                                           (8, 1, 64, torch.bfloat16)])
def test_token_by_token_is_fp32(layout, lengths, h, hkv, d, state):
    """Token by token all but the outputs' (and a bf16 state's) own rounding is fp32's.

    Per token a state takes expf's two units, 2^-22, the rounding of its argument, |a| e^a 2^-24 under 2^-25, and one fma, 2^-24 (products of
    bf16 numbers are exact): under 1.4 x 2^-22 of the magnitudes.  An output's sum adds at most 13 roundings of 2^-24 and its scale's, 4 x 2^-22.
    A bf16 rounding is off by 2^-8 of the value at most, and by 2^-8 / sqrt(3) in the norm; fp32's, independent but for a head's common
    decay, by 2^-23 a token, as the root of the number of tokens.
    """
    a = make(lengths, h, hkv, d, layout, seed=70, state=state)
    assert takes_tokens(a)
    out, fin = call(a)
    o, s, mag, size, live = restated(a)
    tokens = max(lengths)
    got = out.flatten(0, 1).double()
    assert bool(((got - o).abs() <= BF16 * o.abs() + (1.4 * tokens + 4) * 2.0 ** -22 * mag)[live].all())
    assert float((got - o)[live].norm() / o[live].norm()) <= BF16 / 3 ** 0.5
    half = BF16 if state == torch.bfloat16 else 0.0
    assert bool(((fin.double() - s).abs() <= half * s.abs() + 1.4 * tokens * 2.0 ** -22 * size).all())
    if state == torch.float32:
        assert float((fin.double() - s).norm() / s.norm()) <= (2 + tokens ** 0.5) * 2.0 ** -23


@pytest.mark.parametrize("layout,lengths", [("batch", [64]), ("batch", [100, 100]), ("batch", [1000, 1000]), ("lens", [15, 300, 64, 0]), ("cu", [700, 2, 65, 900]),
                                            ("batch", [2500])])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slow", [1.0, 0.01])
def test_fp32_states_of_chunks_in_the_norm(layout, lengths, d, slow):
    """A decayed value is two bf16 terms of a factor that is two terms itself: each pair leaves off 2^-17 of it at most, independently from token to
    token, so the norm is off by sqrt(2) 2^-17 / sqrt(3), and fp32's sums add far less: under 2^-17."""
    a = make(lengths, 4, 2, d, layout, seed=71, state=torch.float32)
    a["log_decay"] *= slow
    a["gate"] *= slow
    assert not takes_tokens(a)
    _, fin = call(a)
    _, s, _, _, _ = restated(a)
    assert float((fin.double() - s).norm() / s.norm()) <= 2.0 ** -17


# -------------------------------------------------------------------------------------------- malformed arrays, every kernel
def guarded(shape, dtype, value):
    """A tensor between two stretches that nothing may touch, and these."""
    size = math.prod(shape)
    store = torch.full((size + 2048,), value, dtype=dtype, device="cuda")
    return store[1024:1024 + size].view(shape), (store[:1024], store[1024 + size:])


def run_guarded(a, total):
    n, h, d = len(ranges_of(a)), a["q"].shape[2], a["q"].shape[3]
    varlen = a["cu_seqlens"] is not None
    need = kda.linear_attn_workspace_size(n, total, h, d, varlen=varlen)
    ws, edges = guarded((need,), torch.uint8, 7)
    a["out"], out_edges = guarded(a["out"].shape, torch.bfloat16, 5.0)
    a["final_state"], fin_edges = guarded(a["final_state"].shape, a["final_state"].dtype, 9.0)
    with pytest.raises(KDAError) as e:
        call(a, workspace=ws if need else None)
    assert e.value.status == KDA_ERR_INVALID_ARGUMENT
    kda.device_status()
    for e, value in ((edges, 7), (out_edges, 5.0), (fin_edges, 9.0)):
        assert all(bool((x == value).all()) for x in e)
    return need


@pytest.mark.parametrize("total,lengths", [(10, [5, 5]), (300, [150, 150]), (3000, [1500, 1500])])
@pytest.mark.parametrize("cu", [[0, 4 / 3, 1], [0, -0.1, 1], [0.1, 0.15, 1], [0, 1 / 3, 1e9], [1, 2 / 3, 1 / 3], [-1e9, 1e9, -1e9], [0, 1, 1 / 2]])
@pytest.mark.parametrize("d", [64, 128])
def test_a_malformed_cu_seqlens_in_every_kernel(total, lengths, cu, d):
    """Token by token, in chunks, and in groups: reported, and nothing outside the outputs and the workspace is written."""
    a = make(lengths, 2, 2, d, "cu", seed=80)
    a["cu_seqlens"].copy_(torch.tensor([int(x * total) for x in cu]))
    need = run_guarded(a, total)
    assert (need > 0) == (total == 3000)


@pytest.mark.parametrize("t", [4, 150, 2500])
@pytest.mark.parametrize("d", [64, 128])
def test_lens_out_of_range_in_every_kernel(t, d):
    a = make([t, t, t], 2, 1, d, "lens", seed=81)
    a["lens"].copy_(torch.tensor([-3, t + 9, t // 2], dtype=torch.int32))
    need = run_guarded(a, t)
    assert (need > 0) == (t == 2500)
    # clamped: what the call makes of them in range
    a["lens"].copy_(torch.tensor([0, t, t // 2], dtype=torch.int32))
    o, s, mag, size, live = restated(a)
    got = a["out"].flatten(0, 1).double()
    assert bool(((got - o).abs() <= BF16 * o.abs() + (BF16 + 2.0 ** -13) * mag)[live].all()) and bool((got[~live] == 5.0).all())
    assert bool(((a["final_state"].double() - s).abs() <= (2.0 ** -17 + 2.0 ** -16) * size).all())
