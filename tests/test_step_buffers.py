"""CPU checks of buffers that a decoder-step call would read and write at once: refused before any CUDA call."""
import pytest

from gated_delta_rule_23_gb300._native import KDA_ERR_INVALID_ARGUMENT
from tests.test_step_abi import append, attn, beam, lib, reorder  # noqa: F401

M = 1 << 20
FAR = dict(logits=M, bs=2 * M, fin=3 * M, scores=4 * M, tokens=5 * M, parents=6 * M)      # 2 x 3 beams of 100 fp32 logits, 6 kept


@pytest.mark.parametrize("kw", [
    dict(scores=5 * M), dict(tokens=6 * M + 44), dict(parents=4 * M - 44), dict(tokens=2 * M), dict(parents=2 * M + 20),
    dict(scores=M + 2396), dict(tokens=M - 44), dict(parents=3 * M + 4), dict(scores=2 * M), dict(scores=2 * M, bs=2 * M + 4),
    dict(scores=2 * M + 4, K=3), dict(tokens=2 * M, K=3), dict(scores=2 * M + 16, W=4, K=4)])
def test_selection_refuses_shared_buffers(lib, kw):  # noqa: F811
    """scores in the place of beam_scores is allowed where K = W alone."""
    assert beam(lib, **dict(FAR, **kw)) == KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("src, dst", [
    ((M, 2 * M), (2 * M, M)), ((M, 2 * M), (3 * M, 3 * M)), ((M, 2 * M), (3 * M, 3 * M + 1008)), ((M, M), (M, M)),
    ((M, M + 512), (M, 3 * M)), ((M, M + 512), (M, M + 512)), ((M, 2 * M, 3 * M), (4 * M, 5 * M, 2 * M + 1008)),
    ((M, 4 * M), (M + 1008, 4 * M)), (tuple(M * i for i in range(1, 201)), tuple(M * (201 - i) for i in range(1, 201)))])
def test_reorder_refuses_shared_buffers(lib, src, dst):  # noqa: F811
    """What one tensor of a call is read from or written to is nobody else's destination (4 rows of 256 bytes each)."""
    assert reorder(lib, src=src, dst=dst, rows=(256,) * len(src), parents=M // 2) == KDA_ERR_INVALID_ARGUMENT


def test_reorder_refuses_to_write_its_parents(lib):  # noqa: F811
    assert reorder(lib, src=(M,), dst=(2 * M,), parents=2 * M + 1020) == KDA_ERR_INVALID_ARGUMENT


# q, out and lse of 2 x 3 tokens with 8 heads of 128: q and out 12288 bytes, lse 192
@pytest.mark.parametrize("kw", [
    dict(out=M), dict(out=M + 12272), dict(out=M - 12272), dict(qs=2048, out=M + 5 * 4096 + 2032), dict(lse=M + 12284),
    dict(lse=M - 188), dict(lse=3 * M + 12284), dict(lse=3 * M - 188), dict(out=M, T=1)])
def test_attention_refuses_shared_buffers(lib, kw):  # noqa: F811
    assert attn(lib, **dict(dict(q=M, out=3 * M, lse=5 * M), **kw)) == KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(qo=M + 12272), dict(qo=M - 12272), dict(qs=2048, qo=M + 5 * 4096 + 2032), dict(qo=2 * M), dict(qo=2 * M + 3056),
    dict(qo=3 * M - 12272), dict(q=2 * M, qo=2 * M), dict(vs=512, qo=3 * M + 5 * 1024 + 496)])
def test_append_refuses_shared_buffers(lib, kw):  # noqa: F811
    """q_out may be q, but no other part of it, and nothing of k or v (6 tokens of 2 heads of 128: 3072 bytes)."""
    assert append(lib, **dict(dict(q=M, k=2 * M, v=3 * M, qo=5 * M), **kw)) == KDA_ERR_INVALID_ARGUMENT


# What tests/test_step_abi.py has refused with one address for every buffer, with buffers apart: each for its own reason.
@pytest.mark.parametrize("kw", [
    dict(kc=None), dict(table=None), dict(lens=None), dict(N=0), dict(T=-1), dict(Hkv=0), dict(pages=0), dict(max_pages=0),
    dict(page=15), dict(page=8192), dict(kc=7 * M + 8), dict(table=9 * M + 2), dict(lens=10 * M + 1), dict(cu=11 * M + 4),
    dict(q=None), dict(q=M + 8), dict(out=None), dict(out=3 * M + 2), dict(lse=5 * M + 2), dict(Hq=0), dict(Hq=7),
    dict(window=0), dict(sinks=-1), dict(qs=1000), dict(qs=1028)])
def test_attention_refuses_each_for_itself(lib, kw):  # noqa: F811
    far = dict(q=M, out=3 * M, lse=5 * M, kc=7 * M, vc=8 * M, table=9 * M, lens=10 * M)
    assert attn(lib, **dict(far, **kw)) == KDA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(bs=None), dict(scores=None), dict(tokens=None), dict(parents=None), dict(dtype=0), dict(dtype=7),
    dict(stride=99), dict(eos=-1), dict(eos=100), dict(B=0), dict(W=0), dict(W=33), dict(V=0), dict(K=0), dict(K=65),
    dict(V=2, K=7, stride=2, eos=0), dict(logits=M + 2), dict(dtype=1, logits=M + 1), dict(bs=2 * M + 2), dict(scores=4 * M + 2),
    dict(tokens=5 * M + 1), dict(parents=6 * M + 2)])
def test_selection_refuses_each_for_itself(lib, kw):  # noqa: F811
    assert beam(lib, **dict(FAR, **kw)) == KDA_ERR_INVALID_ARGUMENT
