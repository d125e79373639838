"""Linear attention at the corners of its two kernels: against the same 64-bit restatement, within the bounds of tests/test_gpu_linear.py."""
import math

import pytest
import torch

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
