"""CPU check that the bars of the token-by-token kernel's tests tell fp32 from a bf16 rounding in the wrong place: planted in the restatement."""
import torch

from tests import linear_ref


def run(read=lambda s: s, scores=lambda x: x):
    """The recurrence in 64 bits on bf16 inputs, with what an output reads of the state, or the products it sums, changed."""
    g = torch.Generator().manual_seed(0)
    t, h, d = 8, 64, 64
    q, k, v = (torch.randn((t, h, d), generator=g).bfloat16() for _ in range(3))
    a = -torch.rand((t, h), generator=g)
    init = torch.randn((1, h, d, d), generator=g)
    o = linear_ref.linear(q, k, v, a, d ** -0.5, init, [(0, t)])[0]
    s, out = init[0].double(), torch.empty((t, h, d), dtype=torch.float64)
    for i in range(t):
        s = a[i].double().exp()[:, None, None] * s + v[i].double()[:, :, None] * k[i].double()[:, None, :]
        out[i] = d ** -0.5 * scores(read(s) * q[i].double()[:, None]).sum(-1)
    return float((out.bfloat16().double() - o).norm() / o.norm())


def test_the_bar_holds_for_one_rounding_and_not_for_two():
    bar = 2.0 ** -8 / 3 ** 0.5
    assert run() <= bar
    assert run(read=lambda s: s.bfloat16().double()) > bar
    assert run(scores=lambda x: x.bfloat16().double()) > bar
