"""GPU tests of the decoder-step operators against 64-bit restatements.

Tolerances.  u = 2^-8 is bf16's unit roundoff.
* Append: one rounding of an fp32 result: |d| <= u |ref| + 2^-20 (|x| + |y|).
* Attention: the probabilities are rounded to bf16 (u each, so u sum p |v|) and the output once more (u |ref|); the fp32
  scores, exponentials and sums add less than 2^-13 sum p |v| at these sizes.  lse: the fp32 dot products are off by at
  most D 2^-24 scale sum |q k|, the rest by 2^-18 (1 + |lse|).
* Beam scores: fp32 sums and logarithm: 2^-20 (1 + |score|); a chosen candidate's 64-bit score is that near the true
  k-th best; exact ties are checked exactly.
* Reorder: bytes.
"""
import math

import pytest
import torch

from tests import step_ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def kda():
    import gated_delta_rule_23_gb300 as m
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ragged(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int64, device="cuda")


def _check_attn(out, lse, ref, dim):
    for (o, l, mag, big), got, got_lse in zip(ref, out, lse):
        tol = U * o.abs() + (U + 2.0 ** -13) * mag
        err = (got.double() - o).abs()
        assert bool((err <= tol).all()), float((err - tol).max())
        none = torch.isinf(l)
        assert torch.equal(none, torch.isinf(got_lse)) and bool((got_lse[none] < 0).all())
        e = (got_lse.double() - l)[~none].abs()
        assert bool((e <= dim * 2.0 ** -24 * big[~none] + 2.0 ** -18 * (1 + l[~none].abs())).all()), e.max()


def _attn(kda, lens, new, hq, hkv, dim, page, window, sinks, ragged, seed=0, scale=None, keep=None, big_q=1.0,
          edit=None, stream=None, workspace=False):
    gen = _gen(seed)
    k, v, table = step_ref.make_cache(lens, hkv, dim, page, gen, "cuda", keep=keep)
    if edit:
        edit(k, v, table)
    qs = [torch.randn((n, hq, dim), generator=gen, device="cuda").mul(big_q).to(torch.bfloat16) for n in new]
    q = torch.cat(qs)[None] if ragged else torch.stack(qs)
    out = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:3], math.nan, device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = {}
    if workspace:
        size = kda.window_attn_workspace_size(window, sinks, len(lens), q.shape[1], hq, hkv, dim, page,
                                              table.shape[1], varlen=ragged)
        kw["workspace"] = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    kda.kda_window_attn(q, k, v, table, lens_t, out, window, sinks=sinks, scale=scale, lse=lse,
                        cu_seqlens=_ragged(new) if ragged else None, stream=stream, **kw)
    kda.device_status(stream)
    ref = step_ref.attention(qs, k, v, table.cpu().cuda(), lens, new, window, sinks, scale or dim ** -0.5)
    outs = list(out[0].split(new)) if ragged else list(out)
    lses = list(lse[0].split(new)) if ragged else list(lse)
    _check_attn(outs, lses, ref, dim)
    return out, lse


# lens, new, hq, hkv, dim, page, window, sinks, ragged
ATTN = [
    ([1], [1], 1, 1, 128, 16, 1, 0, False),
    ([5], [1], 4, 1, 64, 16, 3, 1, False),
    ([700], [1], 8, 1, 128, 16, 600, 4, False),
    ([129, 128, 127, 1], [1, 1, 1, 1], 8, 2, 128, 16, 4096, 0, False),
    ([300, 17, 64, 65], [1, 1, 1, 1], 12, 1, 128, 32, 100, 33, False),
    ([2000, 90], [1, 1], 6, 3, 64, 64, 1500, 5, False),
    ([513, 40], [1, 1], 40, 1, 128, 16, 300, 2, False),
    ([70, 300], [2, 2], 8, 1, 128, 16, 65, 3, False),
    ([70, 300], [5, 5], 24, 2, 64, 32, 40, 0, False),
    ([64], [64], 2, 1, 128, 16, 64, 0, False),
    ([130, 257], [130, 130], 4, 2, 128, 128, 33, 1, False),
    ([300], [300], 3, 3, 64, 256, 1000, 0, False),
    ([400, 333], [111, 111], 14, 2, 64, 16, 129, 37, False),
    ([150, 1, 77, 300, 33], [150, 1, 70, 2, 33], 8, 2, 128, 32, 48, 4, True),
    ([10, 0, 200, 40], [10, 0, 129, 1], 5, 1, 128, 64, 50, 20, True),
    ([600, 90], [1, 40], 64, 1, 128, 16, 200, 130, True),
    ([300], [260], 2, 2, 128, 16, 2 ** 31 - 1, 0, False),
]


@pytest.mark.parametrize("case", ATTN, ids=[str(i) for i in range(len(ATTN))])
def test_attn(kda, case):
    _attn(kda, *case)


@pytest.mark.parametrize("case", [ATTN[i] for i in (2, 5, 9, 13)], ids=["2", "5", "9", "13"])
def test_attn_workspace(kda, case):
    """The caller's workspace (filled with NaN patterns) gives the same bits as the pool's."""
    a = _attn(kda, *case)
    b = _attn(kda, *case, workspace=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("lens, new", [([0, 3, 200], [1, 1, 1]), ([0, 2, 300], [4, 4, 4]), ([0, 60, 300], [200, 200, 200])])
def test_attn_rows_that_see_nothing(kda, lens, new, ragged):
    """Queries before the cache's first token, and sequences without any, give 0 and -inf."""
    _attn(kda, lens, new, 8, 2, 128, 16, 40, 2, ragged)


@pytest.mark.parametrize("new", [1, 3, 150])
def test_attn_given_back_pages(kda, new):
    """Pages between the sinks and the window may be unmapped."""
    lens, page, window, sinks = [700, 400], 16, 100, 5
    _attn(kda, lens, [new] * 2, 8, 2, 128, page, window, sinks, False,
          keep=lambda n, p: p < 1 or (p + 1) * page > lens[n] - new - window + 1)


# Query rows in several tiles of 16: tokens that two tiles share, a last tile of one row, 256 rows and one more, sequences
# shorter than their tokens, windows of one key and of fewer keys than a tile has tokens; few and many key heads.
ROW_TILES = [
    ([900], [6], 6, 2, 128, 16, 200, 3), ([33], [33], 5, 5, 64, 32, 9, 0), ([700, 20], [17, 17], 10, 2, 128, 16, 1, 1),
    ([400, 0, 7], [11, 11, 11], 24, 2, 64, 128, 150, 4), ([2000], [32], 8, 1, 128, 64, 1024, 4),
    ([2000], [257], 1, 1, 128, 16, 600, 0), ([1500], [3], 64, 1, 128, 16, 1000, 0), ([260, 255], [256, 256], 1, 1, 64, 16, 40, 2),
    ([600] * 12, [20] * 12, 4, 2, 128, 32, 100, 2), ([3000], [9], 16, 8, 64, 16, 2500, 1), ([1200], [2], 13, 1, 128, 16, 1100, 0),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", ROW_TILES, ids=[str(i) for i in range(len(ROW_TILES))])
def test_attn_row_tiles(kda, case, ragged):
    _attn(kda, *case, ragged)


# Query tiles of 256 rows with their keys in splits: 2, 4, 8 and many of them, splits that hold no key of a half's rows, rows that
# see nothing.
SPLIT_TILES = [
    ([700], [300], 2, 1, 128, 16, 500, 0), ([1500], [300], 2, 1, 64, 32, 1300, 3), ([2600], [258], 1, 1, 128, 64, 2500, 5),
    ([9000], [40], 8, 1, 128, 16, 8800, 1), ([3000, 90, 30], [100, 90, 40], 14, 2, 64, 16, 2100, 37),
    ([3000], [257], 1, 1, 64, 128, 30, 2500), ([2000], [600], 8, 8, 128, 32, 40, 0), ([20, 2000], [300, 300], 3, 1, 128, 16, 1000, 0),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("case", SPLIT_TILES, ids=[str(i) for i in range(len(SPLIT_TILES))])
def test_attn_split_tiles(kda, case, ragged):
    if len(set(case[1])) > 1 and not ragged:
        case = (case[0], [case[1][0]] * len(case[1])) + case[2:]
    a, b = (_attn(kda, *case, ragged) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("lens, window", [(700, 301), (2600, 2031)])
def test_attn_split_tiles_values_out_of_sight(kda, lens, window, value):
    """Keys and values just before every row's window, in the tiles that the splits do bring in."""
    def edit(k, v, table):
        for j in range(lens - 258 - window - 15, lens - 258 - window + 1):
            at = int(table[0, j // 16])
            k[at, :, j % 16], v[at, :, j % 16] = value, value
    _attn(kda, [lens], [258], 1, 1, 128, 16, window, 0, False, edit=edit)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("new, hq", [(1, 8), (2, 4), (140, 4)])
def test_attn_values_out_of_sight(kda, value, new, hq):
    """Infinities and NaN in keys and values outside a query's window do not reach it, also where the pages are shared
    with visible ones and where other queries of the call do see them."""
    lens, page, window, sinks = [300], 32, 60, 3
    hit = [sinks, 100, 239 - new, 299 if new > 1 else 2]     # the last is seen by the last query only

    def edit(k, v, table):
        for j in hit[:3]:
            at = int(table[0, j // page])
            k[at, :, j % page], v[at, :, j % page] = value, value
        if new > 1:
            at = int(table[0, hit[3] // page])
            v[at, :, hit[3] % page] = value
    gen = _gen(3)
    k, v, table = step_ref.make_cache(lens, 2, 128, page, gen, "cuda")
    edit(k, v, table)
    q = torch.randn((1, new, hq, 128), generator=gen, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((1, new, hq), device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kda.kda_window_attn(q, k, v, table, lens_t, out, window, sinks=sinks, lse=lse)
    kda.device_status()
    keep = list(range(new if new == 1 else new - 1))
    # rows that see one of the bad positions are not held to anything
    clean = [i for i in keep if not any(j <= 300 - new + i and (j > 300 - new + i - window or j < sinks) for j in hit[:3])]
    assert len(clean) >= len(keep) // 3
    ref = step_ref.attention([q[0]], k, v, table, lens, [new], window, sinks, 128 ** -0.5)[0]
    _check_attn([out[0][clean]], [lse[0][clean]], [tuple(x[clean] for x in ref)], 128)


@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("new", [1, 3, 600])
def test_attn_values_in_sight(kda, where, new):
    """NaN that a row does see is in its output, in the columns it belongs to; the other rows and columns are not touched."""
    gen = _gen(31)
    lens, window = [900], 200
    k, v, table = step_ref.make_cache(lens, 1, 128, 16, gen, "cuda")
    q = torch.randn((1, new, 4, 128), generator=gen, device="cuda").to(torch.bfloat16)
    bad = 900 - 1 - new // 2                          # a position that some rows see, from its own row on
    page, row = int(table[0, bad // 16]), bad % 16
    if where == "q":
        q[0, bad - (900 - new), 2, 7] = math.nan
    elif where == "k":
        k[page, 0, row, 3] = math.nan
    else:
        v[page, 0, row, 5] = math.inf
        v[page, 0, row, 64] = math.nan
    out, lse = torch.empty_like(q), torch.empty((1, new, 4), device="cuda")
    kda.kda_window_attn(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, window, lse=lse)
    kda.device_status()
    o, ref_lse, mag, big = step_ref.attention([q[0]], k, v, table, lens, [new], window, 0, 128 ** -0.5)[0]
    assert torch.equal(torch.isfinite(out[0].double()), torch.isfinite(o))
    fine = torch.isfinite(o)
    tol = U * o.abs() + (U + 2.0 ** -13) * mag
    assert bool(((out[0].double() - o).abs()[fine] <= tol[fine]).all())
    assert torch.equal(torch.isnan(lse[0]), torch.isnan(ref_lse))


def test_attn_large_scores(kda):
    """Scores in the hundreds: the running maximum moves by large steps."""
    for new, lens in ((1, [500]), (200, [500])):
        _attn(kda, lens, [new], 4, 2, 128, 16, 300, 4, False, big_q=40.0)


@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0])
def test_attn_scale(kda, scale):
    gen = _gen(1)
    k, v, table = step_ref.make_cache([90], 1, 64, 16, gen, "cuda")
    for new in (1, 50):
        q = torch.randn((1, new, 2, 64), generator=gen, device="cuda").to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty((1, new, 2), device="cuda")
        kda.kda_window_attn(q, k, v, table, torch.tensor([90], dtype=torch.int32, device="cuda"), out, 30, scale=scale,
                            lse=lse)
        _check_attn(out, lse, step_ref.attention([q[0]], k, v, table, [90], [new], 30, 0, scale), 64)


def test_attn_strided_queries_and_stream(kda):
    gen = _gen(2)
    k, v, table = step_ref.make_cache([200, 180], 2, 128, 16, gen, "cuda")
    lens = torch.tensor([200, 180], dtype=torch.int32, device="cuda")
    for new in (1, 2, 90):
        rows = torch.randn((2, new, 1000 + 8), generator=gen, device="cuda").to(torch.bfloat16)
        q = rows[..., 8:8 + 4 * 128].unflatten(-1, (4, 128))
        dense = q.contiguous()
        a, b = torch.empty_like(dense), torch.empty_like(dense)
        kda.kda_window_attn(q, k, v, table, lens, a, 77, sinks=1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())     # the inputs were made on the current stream
        kda.kda_window_attn(dense, k, v, table, lens, b, 77, sinks=1, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_attn_repeats_bit_for_bit(kda):
    for case in (ATTN[2], ATTN[12], ATTN[13]):
        a, b = _attn(kda, *case), _attn(kda, *case)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attn_long_cache(kda):
    """Cache rows past 2^31 elements."""
    hkv, page, dim = 8, 128, 128
    pages = 2 ** 31 // (hkv * page * dim) + 9
    k = torch.zeros((pages, hkv, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    gen = _gen(4)
    ids = [pages - 1, pages - 5, pages - 2]
    for i in ids:
        k[i].normal_(generator=gen)
        v[i].normal_(generator=gen)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    for new in (1, 100):
        q = torch.randn((1, new, 16, dim), generator=gen, device="cuda").to(torch.bfloat16)
        out, lse = torch.empty_like(q), torch.empty((1, new, 16), device="cuda")
        kda.kda_window_attn(q, k, v, table, torch.tensor([380], dtype=torch.int32, device="cuda"), out, 250, sinks=2,
                            lse=lse)
        small = k[ids], v[ids], torch.arange(3, dtype=torch.int32, device="cuda")[None]
        _check_attn(out, lse, step_ref.attention([q[0]], *small, [380], [new], 250, 2, dim ** -0.5), dim)
    # and the append that fills them
    x = torch.randn((1, 3, hkv, dim), generator=gen, device="cuda").to(torch.bfloat16)
    kda.kda_kv_append(x, x, k, v, table, torch.tensor([130], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(k[ids[0], :, 127], x[0, 0]) and torch.equal(v[ids[1], :, 1], x[0, 2])


def test_attn_malformed_arrays_are_reported(kda):
    gen = _gen(5)
    k, v, table = step_ref.make_cache([100], 1, 128, 16, gen, "cuda")
    for new in (1, 40):
        q = torch.zeros((1, new, 8, 128), dtype=torch.bfloat16, device="cuda")
        out = torch.empty_like(q)
        for lens, tab in ((100, torch.full_like(table, 10 ** 6)), (100, torch.full_like(table, -7)),
                          (10 ** 6, table), (-3, table)):
            kda.kda_window_attn(q, k, v, tab, torch.tensor([lens], dtype=torch.int32, device="cuda"), out, 50)
            with pytest.raises(kda.KDAError):
                kda.device_status()
            kda.device_status()
        cu = torch.tensor([0, 5 * new], dtype=torch.int64, device="cuda")
        kda.kda_window_attn(q, k, v, table, torch.tensor([100], dtype=torch.int32, device="cuda"), out, 50, cu_seqlens=cu)
        with pytest.raises(kda.KDAError):
            kda.device_status()


@pytest.mark.parametrize("new", [1, 60, 400])
def test_attn_waits_that_give_up_are_reported(kda, new):
    """With no polls allowed every wait gives up at once: the kernels end by themselves and say so, and the next call works."""
    from gated_delta_rule_23_gb300 import _native
    lib = _native.load()
    gen = _gen(9)
    k, v, table = step_ref.make_cache([500], 2, 128, 16, gen, "cuda")
    lens = torch.tensor([500], dtype=torch.int32, device="cuda")
    q = torch.randn((1, new, 8, 128), generator=gen, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    try:
        lib.kda_set_wait_limit(0)
        kda.kda_window_attn(q, k, v, table, lens, out, 300)
        with pytest.raises(kda.KDAError) as e:
            kda.device_status()
        assert e.value.status == _native.KDA_ERR_TIMEOUT
    finally:
        lib.kda_set_wait_limit(_native.KDA_DEFAULT_WAIT_POLLS)
    lse = torch.empty((1, new, 8), device="cuda")
    kda.kda_window_attn(q, k, v, table, lens, out, 300, lse=lse)
    kda.device_status()
    _check_attn(out, lse, step_ref.attention([q[0]], k, v, table, [500], [new], 300, 0, 128 ** -0.5), 128)


# ---------------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens, new, hq, hkv, dim, page, rotary, ragged", [
    ([1], [1], 4, 1, 128, 16, 128, False),
    ([40, 17, 64], [1, 1, 1], 6, 2, 64, 16, 32, False),
    ([300, 260], [250, 250], 3, 3, 128, 64, 64, False),
    ([33, 0, 5, 90], [33, 0, 2, 47], 12, 1, 128, 32, 128, True),
    ([70], [9], 0, 5, 64, 128, 64, False),
    ([3, 50], [8, 8], 2, 2, 128, 16, 16, False),
])
def test_append(kda, lens, new, hq, hkv, dim, page, rotary, ragged, interleaved):
    gen = _gen(7)
    k_cache, v_cache, table = step_ref.make_cache(lens, hkv, dim, page, gen, "cuda")
    before = k_cache.clone(), v_cache.clone()
    b, t = (1, sum(new)) if ragged else (len(new), new[0])
    rows = torch.randn((b, t, (hq + 2 * hkv) * dim + 8), generator=gen, device="cuda").to(torch.bfloat16)
    q = rows[..., :hq * dim].unflatten(-1, (hq, dim)) if hq else None
    k = rows[..., hq * dim:(hq + hkv) * dim].unflatten(-1, (hkv, dim))
    v = rows[..., (hq + hkv) * dim:(hq + 2 * hkv) * dim].unflatten(-1, (hkv, dim))
    angle = torch.rand((max(lens), rotary // 2), generator=gen, device="cuda") * 6.28
    cos, sin = angle.cos(), angle.sin()
    q_out = torch.empty((b, t, hq, dim), dtype=torch.bfloat16, device="cuda") if hq else None
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = _ragged(new) if ragged else None
    kda.kda_kv_append(k, v, k_cache, v_cache, table, lens_t, cos=cos, sin=sin, interleaved=interleaved, q=q, q_out=q_out,
                      cu_seqlens=cu)
    kda.device_status()

    def near(got, x, ref):
        size = x.double().abs().amax(-1, keepdim=True)
        assert bool(((got.double() - ref).abs() <= U * ref.abs() + 2.0 ** -19 * size).all())
    at = 0
    expect_k, expect_v = before
    for n, count in enumerate(new):
        for i in range(count):
            p = lens[n] - count + i
            bi, ti = (0, at + i) if ragged else (n, i)
            if p < 0:
                if hq:
                    assert torch.equal(q_out[bi, ti], q[bi, ti])
                continue
            c, s = cos[p].double(), sin[p].double()
            if hq:
                near(q_out[bi, ti], q[bi, ti], step_ref.rotate(q[bi, ti].double(), c, s, interleaved))
            page_id = int(table[n, p // page])
            near(k_cache[page_id, :, p % page], k[bi, ti], step_ref.rotate(k[bi, ti].double(), c, s, interleaved))
            expect_k[page_id, :, p % page] = k_cache[page_id, :, p % page]
            expect_v[page_id, :, p % page] = v[bi, ti]
        at += count
    # nothing else was written
    assert torch.equal(expect_k.view(torch.int16), k_cache.view(torch.int16))
    assert torch.equal(expect_v.view(torch.int16), v_cache.view(torch.int16))
    if hq:   # in place, without rotation: a copy
        x = q.contiguous()
        kda.kda_kv_append(k, v, k_cache, v_cache, table, lens_t, q=x, q_out=x, cu_seqlens=cu)
        assert torch.equal(x, q)
        y = torch.empty_like(x)
        kda.kda_kv_append(k, v, k_cache, v_cache, table, lens_t, cos=cos, sin=sin, interleaved=interleaved, q=x, q_out=x,
                          cu_seqlens=cu)
        y.copy_(x)
        assert torch.equal(y, q_out)


def test_append_malformed_arrays_are_reported(kda):
    gen = _gen(8)
    k_cache, v_cache, table = step_ref.make_cache([40], 1, 64, 16, gen, "cuda")
    x = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    before = k_cache.clone()
    ang = torch.zeros((40, 32), device="cuda")
    for lens, tab, rows in ((40, torch.full_like(table, 99), 40), (40, -table - 1, 40), (10 ** 6, table, 40), (40, table, 39)):
        kda.kda_kv_append(x, x, k_cache, v_cache, tab, torch.tensor([lens], dtype=torch.int32, device="cuda"),
                          cos=ang[:rows], sin=ang[:rows])
        with pytest.raises(kda.KDAError):
            kda.device_status()
        kda.device_status()
    assert torch.equal(before[:1].view(torch.int16), k_cache[:1].view(torch.int16)) or int(table[0, 2]) == 0


# ---------------------------------------------------------------------------------------------- beams
def _select(kda, logits, scores, k, finished=None, eos=0):
    b = logits.shape[0]
    out = (torch.full((b, k), math.nan, device="cuda"), torch.full((b, k), -1, dtype=torch.int32, device="cuda"),
           torch.full((b, k), -1, dtype=torch.int32, device="cuda"))
    kda.kda_beam_select(logits, scores, *out, finished=finished, eos=eos)
    kda.device_status()
    return out


def _check_select(logits, scores, finished, eos, got):
    best, tokens, parents = got
    b, w, v = logits.shape
    k = best.shape[1]
    ref = step_ref.beam_scores(logits, scores, finished, eos).flatten(1)
    want = torch.sort(ref, dim=1, descending=True).values[:, :k]
    local = parents.long() - w * torch.arange(b, device="cuda")[:, None]
    assert bool(((local >= 0) & (local < w) & (tokens >= 0) & (tokens < v)).all())
    flat = local * v + tokens
    assert all(len(set(r)) == k for r in flat.tolist())
    chosen = torch.gather(ref, 1, flat)
    for x in (best.double(), chosen):
        assert torch.equal(torch.isinf(x), torch.isinf(want))
        fin = ~torch.isinf(want)
        assert bool(((x - want)[fin].abs() <= 2.0 ** -20 * (1 + want[fin].abs())).all()), (x - want)[fin].abs().max()
    # order: scores fall, equal scores by index
    rising = (best[:, 1:] < best[:, :-1]) | ((best[:, 1:] == best[:, :-1]) & (flat[:, 1:] > flat[:, :-1]))
    assert bool(rising.all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b, w, v, k", [(1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 32001, 8), (3, 8, 4099, 16),
                                        (2, 32, 1000, 64), (1, 2, 200003, 64), (40, 4, 257, 4), (1, 1, 8192, 1),
                                        (2, 5, 8193, 10)])
def test_beam_select(kda, b, w, v, k, dtype):
    gen = _gen(b * 7 + w)
    logits = torch.randn((b, w, v), generator=gen, device="cuda").mul(3).to(dtype)
    scores = -10 * torch.rand((b, w), generator=gen, device="cuda")
    _check_select(logits, scores, None, 0, _select(kda, logits, scores, k))
    done = (torch.rand((b, w), generator=gen, device="cuda") < 0.5).to(torch.uint8)
    _check_select(logits, scores, done, v - 1, _select(kda, logits, scores, k, done, v - 1))


@pytest.mark.parametrize("v", [50, 9000, 40000])
def test_beam_masked_logits(kda, v):
    """Banned tokens (-inf, the type's lowest value, NaN), rows with nothing left, beams that are out."""
    gen = _gen(v)
    for dtype in (torch.bfloat16, torch.float32):
        logits = torch.randn((3, 4, v), generator=gen, device="cuda").to(dtype)
        logits[0] = logits[0].masked_fill(torch.rand((4, v), generator=gen, device="cuda") < 0.9, -math.inf)
        logits[0, 1, 3:] = torch.finfo(dtype).min
        logits[0, 2, ::3] = math.nan
        logits[1, 0] = -math.inf
        logits[1, 1] = math.nan
        logits[1, 2, 2:] = -math.inf            # two tokens left
        scores = torch.tensor([[-1., -2., -3., -4.], [0., 0., -1., -math.inf], [0., -math.inf, -math.inf, math.nan]],
                              device="cuda")
        _check_select(logits, scores, None, 0, _select(kda, logits, scores, 16))
        only = torch.full((1, 4, v), -math.inf, device="cuda", dtype=dtype)
        best, tokens, parents = _select(kda, only, scores[:1], 8)
        assert bool(torch.isinf(best).all()) and tokens[0].tolist() == list(range(8)) and parents[0].tolist() == [0] * 8


def test_beam_ties_take_the_lowest_index(kda):
    for v in (100, 5000, 70000):
        same = torch.zeros((2, 3, v), device="cuda")
        zero = torch.zeros((2, 3), device="cuda")
        best, tokens, parents = _select(kda, same, zero, 20)
        assert tokens.tolist() == [list(range(20))] * 2 and parents.tolist() == [[0] * 20, [3] * 20]
        # the same few values over and over, in bf16
        gen = _gen(v)
        x = torch.randint(0, 3, (2, 3, v), generator=gen, device="cuda").to(torch.bfloat16)
        x[:, 1] = x[:, 0]
        x[:, 2] = x[:, 0]
        best, tokens, parents = _select(kda, x, zero, 12)
        want = torch.sort(x.float().flatten(1), dim=1, descending=True, stable=True).indices[:, :12]
        assert torch.equal(tokens.long(), want % v)
        assert torch.equal(parents.long(), want // v + torch.tensor([[0], [3]], device="cuda"))


@pytest.mark.parametrize("v", [300, 20000, 90000])
def test_beam_distinct_logits_of_one_score(kda, v):
    """Logits so near each other that their fp32 scores are equal: the tie goes by index, not by logit."""
    x = torch.full((1, 2, v), -30.0, device="cuda")
    at = torch.tensor([v - 1, v // 2, 250, 40, 7], device="cuda")
    x[0, :, at] = (torch.arange(5, device="cuda") * 1e-8 + 1e-7).flip(0)[None]
    scores = torch.tensor([[-300.0, -300.0]], device="cuda")
    for k in (1, 2, 4, 5, 7, 10):
        best, tokens, parents = _select(kda, x, scores, k)
        m = x.amax(-1, keepdim=True)
        c = (scores[..., None] - m) - (x - m).exp().sum(-1, keepdim=True).log()
        want = torch.sort((c + x).flatten(1), dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(tokens.long(), want % v) and torch.equal(parents.long(), want // v)


def test_beam_strided_logits(kda):
    gen = _gen(11)
    rows = torch.randn((2, 3, 1003), generator=gen, device="cuda")
    scores = torch.zeros((2, 3), device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        x = rows.to(dtype)[..., 1:1001]
        a, b = _select(kda, x, scores, 6), _select(kda, x.contiguous(), scores, 6)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("v", [101, 4097, 33003])
def test_beam_equal_beams_of_odd_rows_tie(kda, v):
    """Equal beams whose rows are aligned differently have equal scores: their candidates tie by beam."""
    gen = _gen(v)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn((1, 1, v), generator=gen, device="cuda").to(dtype).expand(2, 8, v).contiguous()
        best, tokens, parents = _select(kda, x, torch.full((2, 8), -3.0, device="cuda"), 8)
        top = int(x[0, 0].float().argmax())
        assert tokens.tolist() == [[top] * 8] * 2 and parents.tolist() == [list(range(8)), list(range(8, 16))]
        assert bool((best == best[0, 0]).all())


def test_beam_workspace_and_stream(kda):
    gen = _gen(12)
    x = torch.randn((2, 4, 50001), generator=gen, device="cuda")
    scores = torch.zeros((2, 4), device="cuda")
    a = _select(kda, x, scores, 8)
    ws = torch.full((kda.beam_select_workspace_size(2, 4, 50001, 8),), 255, dtype=torch.uint8, device="cuda")
    b = tuple(torch.empty_like(y) for y in a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_beam_select(x, scores, *b, stream=side, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


# ---------------------------------------------------------------------------------------------- reorder
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("groups, beams", [(1, 1), (3, 2), (2, 4), (5, 5), (2, 9), (1, 32)])
def test_reorder(kda, groups, beams, dtype):
    gen = _gen(groups * 40 + beams)
    n = groups * beams
    src = [torch.randint(0, 200, (n, *shape), generator=gen, device="cuda").to(dtype) for shape in ((2, 128, 128), (16,), (7, 48))]
    parents = (torch.randint(0, beams, (groups, beams), generator=gen, device="cuda")
               + beams * torch.arange(groups, device="cuda")[:, None]).flatten().to(torch.int32)
    want = [s[parents.long()] for s in src]
    dst = [torch.empty_like(s) for s in src]
    kda.kda_state_reorder(src, parents, beams, dst=dst)
    assert all(torch.equal(a, b) for a, b in zip(dst, want))
    kda.kda_state_reorder(src, parents, beams)
    kda.device_status()
    assert all(torch.equal(a, b) for a, b in zip(src, want))


def test_reorder_many_tensors(kda):
    gen = _gen(13)
    src = [torch.randn((4, 16 * (1 + i % 5)), generator=gen, device="cuda") for i in range(150)]
    parents = torch.tensor([2, 2, 0, 3], dtype=torch.int32, device="cuda")
    dst = [torch.empty_like(s) for s in src]
    kda.kda_state_reorder(src, parents, 4, dst=dst)
    assert all(torch.equal(d, s[parents.long()]) for s, d in zip(src, dst))


def test_reorder_long_rows(kda):
    """A row of over 2^32 bytes."""
    src = torch.zeros((2, 2 ** 32 + 64), dtype=torch.uint8, device="cuda")
    src[1, -32:] = 7
    src[0, 5] = 9
    kda.kda_state_reorder(src, torch.tensor([1, 0], dtype=torch.int32, device="cuda"), 2)
    assert int(src[0, -32:].sum()) == 224 and int(src[1, 5]) == 9 and int(src[0, 5]) == 0 and int(src[1, -32:].sum()) == 0


def test_reorder_malformed_parents_are_reported(kda):
    x = torch.arange(64, device="cuda", dtype=torch.int32).reshape(4, 16)
    y = torch.empty_like(x)
    for bad in ([0, 4, 2, 3], [-1, 0, 1, 2], [2, 1, 2, 3]):
        kda.kda_state_reorder(x, torch.tensor(bad, dtype=torch.int32, device="cuda"), 2, dst=y)
        with pytest.raises(kda.KDAError):
            kda.device_status()
    kda.device_status()


# ---------------------------------------------------------------------------------------------- the two ways in
def test_calls_the_compiled_binding_declines(kda, monkeypatch):
    """The checked way through ctypes makes the same calls as the compiled binding."""
    from gated_delta_rule_23_gb300 import _native

    class Declines:
        def __getattr__(self, name):
            return lambda *a: None

    def everything():
        gen = _gen(30)
        k_cache, v_cache, table = step_ref.make_cache([90, 40], 2, 64, 16, gen, "cuda")
        lens = torch.tensor([90, 40], dtype=torch.int32, device="cuda")
        x = torch.randn((2, 3, 8, 64), generator=gen, device="cuda").to(torch.bfloat16)
        angle = torch.rand((100, 16), generator=gen, device="cuda")
        q_out, out = torch.empty_like(x), torch.empty_like(x)
        kda.kda_kv_append(x[:, :, :2], x[:, :, 2:4], k_cache, v_cache, table, lens, angle.cos(), angle.sin(), True, x, q_out)
        lse = torch.empty((2, 3, 8), device="cuda")
        kda.kda_window_attn(q_out, k_cache, v_cache, table, lens, out, 2 ** 40, sinks=1, lse=lse)
        logits = torch.randn((2, 2, 77), generator=gen, device="cuda")
        best, tokens, parents = _select(kda, logits, torch.zeros((2, 2), device="cuda"), 2,
                                        torch.tensor([[True, False]] * 2, device="cuda"), 5)
        kda.kda_state_reorder(x.flatten(0, 1)[:4], parents.view(-1), 2)
        torch.cuda.synchronize()
        return [k_cache, v_cache, q_out, out, lse, best, tokens, parents, x]
    a = everything()
    monkeypatch.setattr(_native, "_binding", Declines())
    b = everything()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


# ---------------------------------------------------------------------------------------------- graphs
@pytest.mark.parametrize("new", [1, 70])
def test_calls_in_a_row_read_what_the_ones_before_wrote(kda, new):
    """Steps whose every call takes the output of the call before, with and without a wait after each call."""
    gen = _gen(40)
    hq, hkv, dim, page, steps, beams = 8, 2, 128, 16, 12, 4
    full = 40 + steps * new
    _, _, table = step_ref.make_cache([full] * beams, hkv, dim, page, gen, "cuda")
    k_cache = torch.zeros((int(table.max()) + 1, hkv, page, dim), dtype=torch.bfloat16, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    x = torch.randn((beams, new, hq, dim), generator=gen, device="cuda").to(torch.bfloat16)
    angle = torch.rand((full, dim // 2), generator=gen, device="cuda") * 6.28
    cos, sin = angle.cos(), angle.sin()
    lens = [torch.full((beams,), 40 + (i + 1) * new, dtype=torch.int32, device="cuda") for i in range(steps)]

    def run(wait):
        k_cache.zero_(), v_cache.zero_()
        q, q_rot, out, scores = x.clone(), torch.empty_like(x), torch.empty_like(x), torch.zeros((1, beams), device="cuda")
        sel = (scores, torch.empty((1, beams), dtype=torch.int32, device="cuda"),
               torch.empty((1, beams), dtype=torch.int32, device="cuda"))
        before = torch.zeros((1, beams), device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            kda.kda_kv_append(q[:, :, :hkv], q[:, :, hkv:2 * hkv], k_cache, v_cache, table, lens[i], cos=cos, sin=sin, q=q,
                              q_out=q_rot)
            if wait:
                torch.cuda.synchronize()
            kda.kda_window_attn(q_rot, k_cache, v_cache, table, lens[i], out, 100, sinks=3)
            if wait:
                torch.cuda.synchronize()
            kda.kda_beam_select(out[:, -1].reshape(1, beams, hq * dim), before, *sel)
            if wait:
                torch.cuda.synchronize()
            kda.kda_state_reorder(out, sel[2].view(-1), beams, dst=q)
            if wait:
                torch.cuda.synchronize()
        kda.device_status()
        return [y.clone() for y in (q, out, *sel, k_cache, v_cache)]
    waited = run(True)
    for _ in range(5):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(waited, run(False)))


def test_step_operators_in_a_graph(kda):
    """A captured step replays with the bits of direct calls on the data then in the buffers."""
    gen = _gen(14)
    lens = [130, 99]
    k_cache, v_cache, table = step_ref.make_cache(lens, 2, 128, 16, gen, "cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((2, 1, 8, 128), generator=gen, device="cuda").to(torch.bfloat16)
    k = torch.randn((2, 1, 2, 128), generator=gen, device="cuda").to(torch.bfloat16)
    logits = torch.randn((1, 2, 30000), generator=gen, device="cuda")
    scores = torch.zeros((1, 2), device="cuda")
    state = torch.randn((2, 4, 128, 128), generator=gen, device="cuda")
    out, moved = torch.empty_like(q), torch.empty_like(state)
    sel = (torch.empty((1, 2), device="cuda"), torch.empty((1, 2), dtype=torch.int32, device="cuda"),
           torch.empty((1, 2), dtype=torch.int32, device="cuda"))
    ws = torch.empty(kda.window_attn_workspace_size(64, 3, 2, 1, 8, 2, 128, 16, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    ws2 = torch.empty(kda.beam_select_workspace_size(1, 2, 30000, 2), dtype=torch.uint8, device="cuda")

    def step():
        kda.kda_kv_append(k, k, k_cache, v_cache, table, lens_t)
        kda.kda_window_attn(q, k_cache, v_cache, table, lens_t, out, 64, sinks=3, workspace=ws)
        kda.kda_beam_select(logits, scores, *sel, workspace=ws2)
        kda.kda_state_reorder(state, sel[2].view(-1), 2, dst=moved)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (20, 21):
        fresh = _gen(seed)
        for x in (q, k, logits, state):
            x.normal_(generator=fresh)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, moved, *sel, k_cache, v_cache)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, (out, moved, *sel, k_cache, v_cache)))


@pytest.mark.parametrize("v", [300, 40000])
def test_beam_scores_in_place(kda, v):
    """scores may be beam_scores where K = W, also where the entry is picked over all candidates."""
    x = torch.full((2, 3, v), -30.0, device="cuda")
    at = torch.tensor([v - 1, v // 2, 250, 40, 7], device="cuda")
    x[:, :, at] = (torch.arange(5, device="cuda") * 1e-8 + 1e-7).flip(0)     # distinct logits of one score
    scores = torch.tensor([[-300.0, -300.0, -300.5], [-300.0, -299.0, -300.0]], device="cuda")
    done = torch.tensor([[0, 0, 1], [0, 1, 0]], dtype=torch.uint8, device="cuda")
    want = _select(kda, x, scores, 3, done, 9)
    _check_select(x, scores, done, 9, want)
    place = scores.clone()
    tokens, parents = torch.empty_like(want[1]), torch.empty_like(want[2])
    kda.kda_beam_select(x, place, place, tokens, parents, finished=done, eos=9)
    kda.device_status()
    assert torch.equal(place, want[0]) and torch.equal(tokens, want[1]) and torch.equal(parents, want[2])
    with pytest.raises(kda.KDAError):
        kda.kda_beam_select(x, place, place.view(-1)[:4].view(2, 2), tokens[:, :2].contiguous(), parents[:, :2].contiguous())


def test_reorder_buffers_of_several_tensors(kda):
    """One source for several tensors, neighbours in one allocation, in place beside out of place; tensors swapped by one call
    are refused."""
    gen = _gen(15)
    pool = torch.randn((6, 4, 64), generator=gen, device="cuda")
    before = pool.clone()
    parents = torch.tensor([1, 0, 3, 3], dtype=torch.int32, device="cuda")
    p = parents.long()
    kda.kda_state_reorder([pool[0], pool[0], pool[3], pool[5]], parents, 4, dst=[pool[1], pool[2], pool[3], pool[4]])
    kda.device_status()
    for i, want in ((0, before[0]), (1, before[0][p]), (2, before[0][p]), (3, before[3][p]), (4, before[5][p]), (5, before[5])):
        assert torch.equal(pool[i], want), i
    for src, dst in (([0, 1], [1, 0]), ([0, 1], [2, 2]), ([0, 0], [0, 0]), ([0, 1], [0, 0])):
        with pytest.raises(kda.KDAError):
            kda.kda_state_reorder([pool[i] for i in src], parents, 4, dst=[pool[i] for i in dst])


@pytest.mark.parametrize("place", [0, 50000, 99000])
@pytest.mark.parametrize("k", [1, 4, 8])
def test_beam_bf16_ties_at_the_last_place(kda, k, place):
    """bf16 logits that tie at the K-th place, in rows whose scores are so low that fp32 logits beside them would tie too:
    picked from the short lists, not over all candidates (five times the time for K = 1, and it grows with K)."""
    gen = _gen(k)
    b, w, v = 64, 2, 100000
    logits = torch.randn((b, w, v), generator=gen, device="cuda").to(torch.bfloat16)
    scores = torch.tensor([-20.0, -60.0], device="cuda").repeat(b, 1)
    at = place + 40 * torch.arange(k + 3, device="cuda")
    tied = logits.clone()
    tied[:, 0, at] = 9.0
    distinct = logits.clone()
    distinct[:, 0, at] = (9.0 + 0.0625 * torch.arange(k + 3, device="cuda").flip(0)).to(torch.bfloat16)
    outs = []
    for x in (distinct, tied):
        out = _select(kda, x, scores, k)
        _check_select(x, scores, None, 0, out)
        assert out[1].tolist() == [at[:k].tolist()] * b and out[2].tolist() == [[i * w] * k for i in range(b)]
        outs.append(out)
    times = []
    for x, out in zip((distinct, tied), outs):
        best = math.inf
        for _ in range(7):
            a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            kda.kda_beam_select(x, scores, *out)
            z.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(z))
        times.append(best)
    assert times[1] <= 3 * times[0], times
