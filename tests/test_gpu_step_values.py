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
