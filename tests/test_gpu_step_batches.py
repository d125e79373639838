"""GPU tests of windowed attention over batches of more query tiles than the GPU has SMs, with empty slots among them.

The tile kernel's CTAs then walk several (query tile, key head) items each, and some of them hold no visible key: sequences
without any token in the cache, and rows before the first one (padding on the left).  Tolerances are those of
tests/test_gpu_step.py; the 64-bit reference is the same definition, a sequence at a time.
"""
import math

import pytest
import torch

from tests import step_ref
from tests.test_gpu_step import _check_attn, _gen, _ragged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_23_gb300 as m
    return m


def _reference(q, k_cache, v_cache, table, length, n, window, sinks, scale):
    """out, lse, sum p |v| and scale max sum |q k| of one sequence's queries [Q, Hq, D], in 64 bits."""
    new, hq, dim = q.shape
    hkv = k_cache.shape[1]
    out = torch.zeros((new, hq, dim), dtype=torch.float64, device=q.device)
    lse = torch.full((new, hq), -math.inf, dtype=torch.float64, device=q.device)
    if length == 0:
        return out, lse, torch.zeros_like(out), torch.zeros_like(lse)
    k = step_ref.gather(k_cache, table, n, list(range(length))).repeat_interleave(hq // hkv, 1)
    v = step_ref.gather(v_cache, table, n, list(range(length))).repeat_interleave(hq // hkv, 1)
    p = torch.arange(length - new, length, device=q.device)[:, None]
    j = torch.arange(length, device=q.device)[None]
    seen = (j <= p) & ((j > p - window) | (j < sinks))
    x = q.double()
    s = (scale * torch.einsum("qhd,jhd->hqj", x, k)).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None])
    big = (scale * torch.einsum("qhd,jhd->hqj", x.abs(), k.abs())).masked_fill(~seen, 0.0).amax(-1)
    return (torch.einsum("hqj,jhd->qhd", w, v), lse.T, torch.einsum("hqj,jhd->qhd", w, v.abs()), big.T)


def _batch(lens, new, hq, hkv, dim, page, ragged, seed):
    gen = _gen(seed)
    k, v, table = step_ref.make_cache(lens, hkv, dim, page, gen, "cuda")
    qs = [torch.randn((n, hq, dim), generator=gen, device="cuda").to(torch.bfloat16) for n in new]
    q = torch.cat(qs)[None] if ragged else torch.stack(qs)
    return qs, q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


# lens (repeated over the batch), sequences, new tokens of each, hq, hkv, dim, window, sinks.  With 152 SMs: 1024, 1536, 320 and
# 1280 items of up to 256 rows.
BATCHES = [
    ([0, 40, 700], 64, 300, 8, 8, 128, 500, 3),
    ([0, 40, 700], 64, 300, 8, 8, 64, 500, 3),
    ([700, 0, 0, 0, 0, 0, 0, 40], 64, 760, 8, 8, 128, 1000, 0),
    ([330, 0, 5, 300, 0, 0, 40, 257], 40, 64, 64, 8, 64, 100, 0),
    ([20, 0, 300, 8], 160, 33, 64, 8, 128, 200, 4),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", BATCHES, ids=[str(i) for i in range(len(BATCHES))])
def test_attn_batches_with_empty_slots(kda, case, ragged):
    lens, count, new, hq, hkv, dim, window, sinks = case
    lens = (lens * count)[:count]
    new = [max(1, new - 7 * (i % 5)) if ragged else new for i in range(count)]
    qs, q, k, v, table, lens_t = _batch(lens, new, hq, hkv, dim, 16, ragged, count)
    got = []
    for _ in range(2):
        out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:3], math.nan, device="cuda")
        kda.kda_window_attn(q, k, v, table, lens_t, out, window, sinks=sinks, lse=lse,
                            cu_seqlens=_ragged(new) if ragged else None)
        kda.device_status()
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    ref = [_reference(x, k, v, table, lens[n], n, window, sinks, dim ** -0.5) for n, x in enumerate(qs)]
    outs = list(out[0].split(new)) if ragged else list(out)
    lses = list(lse[0].split(new)) if ragged else list(lse)
    _check_attn(outs, lses, ref, dim)


def test_reference_is_the_definition():
    """The vectorised reference against tests/step_ref.py's, row by row."""
    lens, new = [37, 0, 5], [9, 4, 8]
    qs, _, k, v, table, _ = _batch(lens, new, 4, 2, 64, 16, True, 1)
    rows = step_ref.attention(qs, k, v, table, lens, new, 12, 2, 0.125)
    for n, x in enumerate(qs):
        for a, b in zip(_reference(x, k, v, table, lens[n], n, 12, 2, 0.125), rows[n]):
            assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("polls", [0, 1])
def test_attn_waits_that_give_up_in_a_walk_over_items(kda, dim, polls):
    """CTAs with several items whose waits get no poll, or one: the call ends and says so where a wait gave up, and the next
    call works."""
    from gated_delta_rule_23_gb300 import _native
    lib = _native.load()
    lens, new = [300, 0, 40, 260] * 16, [300] * 64
    qs, q, k, v, table, lens_t = _batch(lens, new, 8, 8, dim, 16, False, 5)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    try:
        lib.kda_set_wait_limit(polls)
        kda.kda_window_attn(q, k, v, table, lens_t, out, 200, lse=lse)
        try:
            kda.device_status()
            assert polls > 0
        except kda.KDAError as e:
            assert e.status == _native.KDA_ERR_TIMEOUT
    finally:
        lib.kda_set_wait_limit(_native.KDA_DEFAULT_WAIT_POLLS)
    kda.kda_window_attn(q, k, v, table, lens_t, out, 200, lse=lse)
    kda.device_status()
    ref = [_reference(x, k, v, table, lens[n], n, 200, 0, dim ** -0.5) for n, x in enumerate(qs[:8])]
    _check_attn(list(out[:8]), list(lse[:8]), ref, dim)
