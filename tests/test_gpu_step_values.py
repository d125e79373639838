"""GPU tests of windowed attention on values at the ends of bf16's range: large finite ones, infinities and NaN, in sight and
out of it.  The reference and the tolerances are those of tests/test_gpu_step_batches.py."""
import math

import pytest
import torch

from tests import step_ref
from tests.test_gpu_step import _check_attn, _gen, kda  # noqa: F401
from tests.test_gpu_step_batches import _reference

pytestmark = pytest.mark.gpu


def _call(kda, q, k, v, table, lens, window, sinks=0):  # noqa: F811
    out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:3], math.nan, device="cuda")
    kda.kda_window_attn(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, window, sinks=sinks, lse=lse)
    kda.device_status()
    return out, lse


# new tokens, query heads over 1, window: the decode kernel alone, as a cluster, with splits through memory; the tile kernel
# as a cluster and through memory
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new, hq, length, window", [(1, 4, 90, 60), (3, 4, 1300, 1200), (1, 2, 9000, 8800), (150, 3, 400, 90),
                                                     (40, 8, 9000, 8800)])
def test_attn_large_values(kda, new, hq, length, window, dim):  # noqa: F811
    """Finite values whose sums pass fp32's range while the output, a mean of them, does not."""
    gen = _gen(new + dim)
    k, v, table = step_ref.make_cache([length], 1, dim, 16, gen, "cuda")
    v.copy_(torch.where(v.isnan(), v, (3e38 - 1e37 * v.abs().clamp(max=4)).to(torch.bfloat16)))
    v[..., 1::2] *= -1
    q = torch.randn((1, new, hq, dim), generator=gen, device="cuda").mul(0.3).to(torch.bfloat16)
    out, lse = _call(kda, q, k, v, table, [length], window, 2)
    rows = slice(0, new, max(1, new // 8))               # a few rows: the reference holds every key
    ref = _reference(q[0], k, v, table, length, 0, window, 2, dim ** -0.5)
    assert bool(torch.isfinite(out).all())
    _check_attn([out[0][rows]], [lse[0][rows]], [tuple(x[rows] for x in ref)], dim)


def _same_kind(got, want, mag):
    """NaN for NaN, an infinity for the same infinity, and the finite ones within the tolerance."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.isposinf(got), torch.isposinf(want)) and torch.equal(torch.isneginf(got), torch.isneginf(want))
    fine = torch.isfinite(want)
    u = 2.0 ** -8
    assert bool(((got - want).abs()[fine] <= (u * want.abs() + (u + 2.0 ** -13) * mag)[fine]).all())


@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new, hq, length, window, sinks", [(3, 4, 300, 60, 3), (30, 8, 700, 90, 0), (150, 3, 400, 90, 5),
                                                            (60, 8, 2600, 2400, 0), (20, 8, 9000, 8800, 40)])
def test_attn_infinity_in_sight_beside_a_value_out_of_sight(kda, new, hq, length, window, sinks, value, own):  # noqa: F811
    """A row that sees an infinity in a column where a row it does not see holds another value that is not finite: the
    output is the infinity.  And the other way round: a row that sees neither is not touched."""
    gen = _gen(new)
    k, v, table = step_ref.make_cache([length], 1, 128, 16, gen, "cuda")

    def put(j, column, x):
        v[int(table[0, j // 16]), 0, j % 16, column] = x
    first = length - new                              # position of the first row
    put(length - 1, 5, value)                         # seen by the last row alone,
    put(length - 2, 5, math.inf)                      # beside what the one before sees at its own position
    put(first - window + 1, 70, value)                # the first row's oldest key, which the others do not see
    put(first + 1, 70, math.inf)                      # the second row's own
    if not own:
        put(first, 9, -math.inf)                      # every row sees this, at a position that is not its own but for the first,
        put(length - 1, 9, value)                     # and only the last one this
    if not own and sinks:
        put(sinks, 100, value)                        # behind the sinks: nobody sees it
        put(0, 101, math.inf)                         # a sink: all do
    q = torch.randn((1, new, hq, 128), generator=gen, device="cuda").mul(0.3).to(torch.bfloat16)
    out, lse = _call(kda, q, k, v, table, [length], window, sinks)
    rows = sorted({0, 1, 2, new // 2, max(new - 3, 0), new - 2, new - 1})
    for i in rows:                                    # a row at a time: the reference takes in what the row sees and no more
        o, l, mag, _ = step_ref.attention([q[0, i:i + 1]], k, v, table, [first + i + 1], [1], window, sinks, 128 ** -0.5)[0]
        _same_kind(out[0, i:i + 1], o, mag)
        assert bool(((lse[0, i:i + 1].double() - l).abs() <= 1e-4 * (1 + l.abs())).all())


def _best_time(f, repeats=5):
    best = math.inf
    for _ in range(repeats):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("batch, new, length, window, at", [(1, 2048, 2048, 2048, 3), (64, 1, 3000, 2000, 2990)])
def test_attn_value_in_sight_holds_nobody_up(kda, batch, new, length, window, at, value):  # noqa: F811
    """Rows that rightly see a value that is not finite are not worked out key by key: that would be a thousand times the call's time
    for the prompt, over sixty times for the decode step."""
    gen = _gen(3)
    k, v, table = step_ref.make_cache([length] * batch, 4, 128, 64, gen, "cuda")
    q = torch.randn((batch, new, 32, 128), generator=gen, device="cuda").to(torch.bfloat16)
    out, lens = torch.empty_like(q), torch.full((batch,), length, dtype=torch.int32, device="cuda")

    def call():
        kda.kda_window_attn(q, k, v, table, lens, out, window)
    call()
    clean = _best_time(call)
    v[int(table[0, at // 64]), :, at % 64, 17] = value
    assert _best_time(call) <= 10 * clean


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new, hq, length, window", [(1, 4, 90, 60), (3, 4, 1300, 1200), (150, 3, 400, 90), (40, 8, 9000, 8800)])
def test_attn_value_in_sight_among_large_ones(kda, new, hq, length, window, value):  # noqa: F811
    """Finite values whose sums pass fp32's range beside one that is not finite: the output is of its kind."""
    gen = _gen(new)
    k, v, table = step_ref.make_cache([length], 1, 128, 16, gen, "cuda")
    wide = v[..., 30:40]                              # the other columns stay finite in any form
    wide.copy_(torch.where(wide.isnan(), wide, (3e38 - 1e37 * wide.abs().clamp(max=4)).to(torch.bfloat16)))
    at = length - 1 - new // 2                        # rows before its position do not see it
    v[int(table[0, at // 16]), 0, at % 16, 30:40] = value
    q = torch.randn((1, new, hq, 128), generator=gen, device="cuda").mul(0.3).to(torch.bfloat16)
    out, _ = _call(kda, q, k, v, table, [length], window)
    for i in sorted({0, max(new // 2 - 1, 0), new // 2, new - 1}):
        o, _, mag, _ = step_ref.attention([q[0, i:i + 1]], k, v, table, [length - new + i + 1], [1], window, 0, 128 ** -0.5)[0]
        _same_kind(out[0, i:i + 1], o, mag)


@pytest.mark.parametrize("new, hq", [(1, 4), (3, 4), (150, 3)])
def test_attn_value_of_a_key_without_weight(kda, new, hq):  # noqa: F811
    """A key whose score is -infinity has weight 0, and 0 x NaN is NaN, also in rows that are taken again (here for large values)
    and where it is the first key that the row sees."""
    gen = _gen(new)
    length = 200
    k, v, table = step_ref.make_cache([length], 1, 128, 16, gen, "cuda")
    v.copy_(torch.where(v.isnan(), v, (3e38 - 1e37 * v.abs().clamp(max=4)).to(torch.bfloat16)))
    page = int(table[0, 0])
    k[page, 0, 0] = -math.inf
    v[page, 0, 0, 9] = math.nan
    q = torch.randn((1, new, hq, 128), generator=gen, device="cuda").abs().mul(0.3).to(torch.bfloat16)
    out, lse = _call(kda, q, k, v, table, [length], 200)
    for i in sorted({0, new // 2, new - 1}):
        o, l, mag, _ = step_ref.attention([q[0, i:i + 1]], k, v, table, [length - new + i + 1], [1], 200, 0, 128 ** -0.5)[0]
        _same_kind(out[0, i:i + 1], o, mag)
        assert bool(torch.isnan(out[0, i, :, 9]).all()) and bool(((lse[0, i].double() - l[0]).abs() <= 1e-4 * (1 + l[0].abs())).all())
