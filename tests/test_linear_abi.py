"""CPU checks of linear attention and draft verification: what they refuse before any CUDA call, and what the binding refuses."""
import pytest
import torch

from gated_delta_rule_23_gb300 import _native, step
from gated_delta_rule_23_gb300._native import (KDA_DTYPE_BF16, KDA_DTYPE_FP32, KDA_DTYPE_NONE, KDA_ERR_INVALID_ARGUMENT,
                                               KDA_ERR_UNSUPPORTED)

A, STEP = 1 << 30, 1 << 24   # fake, aligned device addresses: a refused call never touches them


@pytest.fixture(scope="module")
def lib():
    return _native.load()


def at(i):
    return A + i * STEP


def linear(lib, **kw):
    a = dict(q=at(0), qs=512, k=at(1), ks=256, v=at(2), vs=256, ld=at(3), gate=at(4), scale=0.1, out=at(5), init=at(6), fin=at(7),
             dtype=KDA_DTYPE_FP32, lens=None, cu=None, N=2, T=3, H=4, Hkv=2, D=128)
    a.update(kw)
    return lib.kda_linear_attn(*(a[x] for x in ("q", "qs", "k", "ks", "v", "vs", "ld", "gate", "scale", "out", "init", "fin", "dtype",
                                                "lens", "cu", "N", "T", "H", "Hkv", "D")), None)


@pytest.mark.parametrize("kw", [
    dict(N=0), dict(T=-1), dict(H=0), dict(Hkv=0), dict(H=5), dict(q=None), dict(k=None), dict(v=None), dict(out=None),
    dict(q=at(0) + 8), dict(k=at(1) + 2), dict(v=at(2) + 4), dict(out=at(5) + 8), dict(ld=at(3) + 2), dict(gate=at(4) + 1),
    dict(init=at(6) + 8), dict(fin=at(7) + 4), dict(lens=at(8) + 2), dict(cu=at(8) + 4), dict(lens=at(8), cu=at(9)),
    dict(qs=508), dict(qs=504), dict(ks=255), dict(vs=128), dict(dtype=KDA_DTYPE_NONE), dict(dtype=7),
    # buffers that one head's work writes and another's reads, or two outputs
    dict(out=at(0)), dict(out=at(1)), dict(out=at(2) - 16), dict(out=at(4)), dict(out=at(6)), dict(out=at(7)), dict(out=at(3)),
    dict(fin=at(0)), dict(fin=at(1)), dict(fin=at(2)), dict(fin=at(4)), dict(fin=at(3)), dict(fin=at(6) + 16),
    dict(lens=at(7)), dict(cu=at(7)), dict(lens=at(5)), dict(cu=at(5))])
def test_linear_refuses(lib, kw):
    assert linear(lib, **kw) == KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [dict(D=96), dict(D=256), dict(scale=float("nan")), dict(scale=float("inf")), dict(T=1 << 31),
                                dict(N=1 << 20, T=1 << 20), dict(N=1 << 20, H=1 << 10, qs=1 << 17)])
def test_linear_unsupported(lib, kw):
    assert linear(lib, **kw) == KDA_ERR_UNSUPPORTED


def test_linear_workspace(lib):
    for bad in ((0, 0, 10, 4, 128), (0, 1, -1, 4, 128), (0, 1, 10, 0, 128), (0, 1, 10, 4, 96), (0, 1, 1 << 31, 4, 128)):
        assert lib.kda_linear_attn_workspace_size(*bad) == 0
    assert step.linear_attn_workspace_size(256, 1, 96, 128) == 0
    with pytest.raises(ValueError):
        step.linear_attn_workspace_size(1 << 40, 1, 96, 128)


def verify(lib, **kw):
    a = dict(logits=at(0), dtype=KDA_DTYPE_FP32, stride=1000, drafts=at(1), probs=at(2), uniform=at(3), noise=at(4), tau=at(5),
             lens=at(6), tokens=at(7), counts=at(8), B=3, K=4, V=1000)
    a.update(kw)
    return lib.kda_verify_drafts(*(a[x] for x in ("logits", "dtype", "stride", "drafts", "probs", "uniform", "noise", "tau", "lens",
                                                  "tokens", "counts", "B", "K", "V")), None)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(K=-1), dict(V=0), dict(dtype=KDA_DTYPE_NONE), dict(dtype=9), dict(stride=999), dict(logits=None),
    dict(drafts=None), dict(uniform=None), dict(noise=None), dict(tokens=None), dict(counts=None), dict(logits=at(0) + 2),
    dict(logits=at(0) + 1, dtype=KDA_DTYPE_BF16), dict(drafts=at(1) + 2), dict(probs=at(2) + 2), dict(uniform=at(3) + 1),
    dict(noise=at(4) + 2), dict(tau=at(5) + 2), dict(lens=at(6) + 2), dict(tokens=at(7) + 2), dict(counts=at(8) + 2),
    dict(counts=at(7)), dict(counts=at(7) + 56)] + [dict(tokens=at(i)) for i in range(7)] + [dict(counts=at(i)) for i in range(7)])
def test_verify_refuses(lib, kw):
    assert verify(lib, **kw) == KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [dict(K=32), dict(V=(1 << 24) + 1, stride=1 << 25), dict(B=1 << 29), dict(B=1 << 28, K=7)])
def test_verify_unsupported(lib, kw):
    assert verify(lib, **kw) == KDA_ERR_UNSUPPORTED


def test_verify_workspace(lib):
    for bad in ((KDA_DTYPE_FP32, 0, 4, 1000), (KDA_DTYPE_FP32, 1, 32, 1000), (KDA_DTYPE_FP32, 1, 4, 0), (5, 1, 4, 1000),
                (KDA_DTYPE_BF16, 1 << 30, 4, 1000)):
        assert lib.kda_verify_drafts_workspace_size(*bad) == 0
    assert step.verify_drafts_workspace_size(3, 4, 1000) >= 15 * 8
    with pytest.raises(TypeError):
        step.verify_drafts_workspace_size(3, 4, 1000, torch.float16)


def test_workspaces_are_checked(lib):
    args = [at(0), KDA_DTYPE_FP32, 1000, at(1), at(2), at(3), at(4), None, None, at(7), at(8), 3, 4, 1000]
    need = lib.kda_verify_drafts_workspace_size(KDA_DTYPE_FP32, 3, 4, 1000)
    for ws, size in ((None, need), (at(9) + 16, need), (at(9), need - 1)):
        assert lib.kda_verify_drafts_ws(*args, ws, size, None) == KDA_ERR_INVALID_ARGUMENT


def test_the_binding_wants_cuda_tensors():
    q = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        step.kda_linear_attn(q, q, q, torch.empty_like(q))
    with pytest.raises(ValueError):
        step.kda_verify_drafts(torch.zeros((1, 2, 5)), torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 1)), torch.zeros((1, 5)),
                               torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32))
