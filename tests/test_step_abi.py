"""CPU checks of the decoder-step entry points: what they refuse before any CUDA call, and what the binding refuses."""
import ctypes

import pytest
import torch

from gated_delta_rule_23_gb300 import _native, step
from gated_delta_rule_23_gb300._native import KDA_ERR_INVALID_ARGUMENT, KDA_ERR_UNSUPPORTED

A = 1 << 20   # a fake, aligned device address: a refused call never touches it


@pytest.fixture(scope="module")
def lib():
    return _native.load()


CACHE = dict(cu=None, N=2, T=3, Hq=8, Hkv=2, D=128, pages=10, page=16, max_pages=4)


def _cache(a):
    return [a[x] for x in ("cu", "N", "T", "Hq", "Hkv", "D", "pages", "page", "max_pages")]


def append(lib, **kw):
    a = dict(CACHE, k=A, ks=256, v=A, vs=256, kc=A, vc=A, table=A, lens=A, cos=A, sin=A, rotary=64, positions=9, inter=0,
             q=A, qs=1024, qo=A + (1 << 19))
    a.update(kw)
    return lib.kda_kv_append(a["k"], a["ks"], a["v"], a["vs"], a["kc"], a["vc"], a["table"], a["lens"], a["cos"], a["sin"],
                             a["rotary"], a["positions"], a["inter"], a["q"], a["qs"], a["qo"], *_cache(a), None)


def attn(lib, **kw):
    a = dict(CACHE, q=A, qs=1024, kc=A, vc=A, table=A, lens=A, out=A, lse=None, scale=0.1, window=8, sinks=0)
    a.update(kw)
    return lib.kda_window_attn(a["q"], a["qs"], a["kc"], a["vc"], a["table"], a["lens"], a["out"], a["lse"], a["scale"],
                               a["window"], a["sinks"], *_cache(a), None)


SHARED = [dict(kc=None), dict(vc=None), dict(table=None), dict(lens=None), dict(N=0), dict(T=-1), dict(Hkv=0),
          dict(pages=0), dict(max_pages=0), dict(page=15), dict(page=8), dict(page=24), dict(page=8192), dict(kc=A + 8),
          dict(vc=A + 2), dict(table=A + 2), dict(lens=A + 1), dict(cu=A + 4), dict(q=A + 8)]
LARGE = [dict(D=96), dict(D=256), dict(pages=1 << 30), dict(max_pages=1 << 28), dict(T=1 << 31), dict(N=1 << 20, T=1 << 20)]


@pytest.mark.parametrize("kw", SHARED + [
    dict(k=None), dict(v=None), dict(k=A + 8), dict(ks=255), dict(ks=260), dict(vs=128), dict(qs=1000), dict(q=None),
    dict(qo=None), dict(Hq=-1), dict(cos=None), dict(sin=None), dict(cos=A + 4), dict(rotary=8), dict(rotary=72),
    dict(rotary=144), dict(positions=0), dict(qo=A, qs=2048), dict(qo=A + 8)])
def test_append_refuses(lib, kw):
    assert append(lib, **kw) == KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", SHARED + [
    dict(q=None), dict(out=None), dict(out=A + 2), dict(lse=A + 2), dict(Hq=0), dict(Hq=7), dict(window=0), dict(sinks=-1),
    dict(qs=1000), dict(qs=1028)])
def test_attn_refuses(lib, kw):
    assert attn(lib, **kw) == KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("call", [append, attn])
@pytest.mark.parametrize("kw", LARGE)
def test_sizes_unsupported(lib, call, kw):
    assert call(lib, **kw) == KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -0.1])
def test_attn_scale_unsupported(lib, scale):
    assert attn(lib, scale=scale) == KDA_ERR_UNSUPPORTED


def beam(lib, **kw):
    a = dict(logits=A, dtype=2, stride=100, bs=A, fin=A, eos=3, scores=A, tokens=A, parents=A, B=2, W=3, V=100, K=6)
    a.update(kw)
    return lib.kda_beam_select(a["logits"], a["dtype"], a["stride"], a["bs"], a["fin"], a["eos"], a["scores"], a["tokens"],
                               a["parents"], a["B"], a["W"], a["V"], a["K"], None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(bs=None), dict(scores=None), dict(tokens=None), dict(parents=None), dict(dtype=0), dict(dtype=7),
    dict(stride=99), dict(eos=-1), dict(eos=100), dict(B=0), dict(W=0), dict(W=33), dict(V=0), dict(K=0), dict(K=65),
    dict(V=2, K=7, stride=2, eos=0), dict(logits=A + 2), dict(dtype=1, logits=A + 1), dict(bs=A + 2), dict(tokens=A + 1)])
def test_beam_refuses(lib, kw):
    assert beam(lib, **kw) == KDA_ERR_INVALID_ARGUMENT


def test_beam_unsupported(lib):
    assert beam(lib, V=(1 << 24) + 1, stride=1 << 25) == KDA_ERR_UNSUPPORTED
    assert beam(lib, B=1 << 30, W=4) == KDA_ERR_UNSUPPORTED


def reorder(lib, src=(A,), dst=(A + (1 << 16),), rows=(256,), parents=A, N=4, beams=2):
    n = len(src)
    return lib.kda_state_reorder((ctypes.c_void_p * n)(*src), (ctypes.c_void_p * n)(*dst), (ctypes.c_int64 * n)(*rows), n,
                                 parents, N, beams, None)


@pytest.mark.parametrize("kw", [
    dict(src=(None,)), dict(dst=(None,)), dict(rows=(-16,)), dict(rows=(24,)), dict(src=(A + 8,)), dict(dst=(A + 4,)),
    dict(parents=None), dict(parents=A + 2), dict(N=0), dict(N=5), dict(beams=0), dict(N=66, beams=33),
    dict(dst=(A + 16,)), dict(dst=(A - 512,))])
def test_reorder_refuses(lib, kw):
    assert reorder(lib, **kw) == KDA_ERR_INVALID_ARGUMENT


def test_workspace_sizes_of_invalid_calls(lib):
    assert lib.kda_window_attn_workspace_size(0, 0, 0, 1, 1, 8, 2, 128, 16, 4) == 0
    assert lib.kda_window_attn_workspace_size(8, 0, 0, 1, 1, 8, 3, 128, 16, 4) == 0
    assert lib.kda_beam_select_workspace_size(0, 1, 1, 1) == 0
    assert lib.kda_beam_select_workspace_size(1, 1, 10, 65) == 0


def test_binding_refuses():
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        step.kda_kv_append(x, x, cache, cache, table, lens)
    with pytest.raises(ValueError):
        step.kda_window_attn(x, cache, cache, table, lens, x.clone(), 4)
    with pytest.raises(ValueError):
        step.kda_beam_select(torch.zeros(1, 2, 5), torch.zeros(1, 2), torch.zeros(1, 2), table, table)
    with pytest.raises(ValueError):
        step.kda_state_reorder(torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32), 2)


@pytest.mark.parametrize("make, error", [
    (lambda t: t.float(), TypeError),
    (lambda t: t[:, :3], ValueError),
    (lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), ValueError),
    (lambda t: torch.zeros(2, 4, 2, 129, dtype=t.dtype)[..., :128], ValueError),
    (lambda t: torch.zeros(2, 4, 2 * 128 + 4, dtype=t.dtype)[..., :256].unflatten(-1, (2, 128)), ValueError),
    (lambda t: torch.zeros(2, 5, 2, 128, dtype=t.dtype)[:, :4], ValueError),
    (lambda t: t[:1].expand(2, 4, 2, 128), ValueError),
])
def test_token_strides(make, error):
    t = torch.zeros(2, 4, 2, 128, dtype=torch.bfloat16)
    dev = t.device
    assert step._rows(t, "x", 2, 128, (2, 4), dev) == 256
    wide = torch.zeros(2, 4, 1024, dtype=torch.bfloat16)[..., 8:264].unflatten(-1, (2, 128))
    assert step._rows(wide, "x", 2, 128, (2, 4), dev) == 1024
    with pytest.raises(error):
        step._rows(make(t), "x", 2, 128, (2, 4), dev)
