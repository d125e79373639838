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
