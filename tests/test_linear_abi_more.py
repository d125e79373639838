"""CPU checks of what linear attention and draft verification refuse of their workspaces and options."""
import random

import pytest

from gated_delta_rule_23_gb300 import _native, step
from gated_delta_rule_23_gb300._native import KDA_DTYPE_FP32, KDA_ERR_INVALID_ARGUMENT, KDA_VERIFY_FIRST_LARGEST
from tests.test_linear_abi import at


@pytest.fixture(scope="module")
def lib():
    return _native.load()


@pytest.mark.parametrize("options,ws,size", [(2, None, 0), (1 << 31, None, 0), (3, None, 0), (KDA_VERIFY_FIRST_LARGEST, None, 1),
                                             (0, at(9) + 16, 1 << 20), (0, at(9), 0), (KDA_VERIFY_FIRST_LARGEST, at(9), 8)])
def test_verify_options_are_checked(lib, options, ws, size):
    args = [at(0), KDA_DTYPE_FP32, 1000, at(1), at(2), at(3), at(4), None, None, at(7), at(8), 3, 4, 1000]
    assert lib.kda_verify_drafts_opt(*args, options, ws, size, None) == KDA_ERR_INVALID_ARGUMENT


# -------------------------------------------------------------------------------------------- linear attention's workspace
def linear_ws(lib, ws, size, **kw):
    a = dict(q=at(0), qs=256, k=at(1), ks=128, v=at(2), vs=128, ld=at(3), gate=at(4), scale=0.1, out=at(5), init=at(6), fin=at(7),
             dtype=KDA_DTYPE_FP32, lens=None, cu=None, N=1, T=8192, H=2, Hkv=1, D=128)
    a.update(kw)
    return lib.kda_linear_attn_ws(*(a[x] for x in ("q", "qs", "k", "ks", "v", "vs", "ld", "gate", "scale", "out", "init", "fin", "dtype",
                                                   "lens", "cu", "N", "T", "H", "Hkv", "D")), ws, size, None)


@pytest.mark.parametrize("varlen", [False, True])
def test_a_call_in_groups_needs_a_workspace_and_gets_no_less(lib, varlen):
    kw = dict(cu=at(8)) if varlen else {}
    need = lib.kda_linear_attn_workspace_size(int(varlen), 1, 8192, 2, 128)
    assert need >= 2 * 2 * (128 * 128 + 2) * 4                    # two groups' states at least
    for ws, size in ((None, 0), (None, need), (at(20) + 16, need), (at(20) + 128, need), (at(20), need - 1), (at(20), 0)):
        assert linear_ws(lib, ws, size, **kw) == KDA_ERR_INVALID_ARGUMENT
    assert step.linear_attn_workspace_size(1, 8192, 2, 128, varlen=varlen) == need


def seq_range(cu, n, total):
    lo = min(max(cu[n], 0), total)
    return lo, max(lo, min(max(cu[n + 1], lo), total)) - lo


def test_groups_of_a_malformed_cu_seqlens_stay_inside_the_workspace(lib):
    """The slots of groups' states, worked out as the kernels do, for any cu_seqlens at all: below what the workspace holds.  (bos / X + n + g for
    group g of sequence n, X tokens a group, and one slot more for the first group's start: the last group's.)"""
    rng = random.Random(0)
    for _ in range(400):
        total, n, h, d = rng.randint(65, 40000), rng.randint(1, 9), rng.randint(1, 8), rng.choice([64, 128])
        size = lib.kda_linear_attn_workspace_size(1, n, total, h, d)
        slots, rest = divmod(size, h * (d * d + 2) * 4)
        assert rest == 0
        cu = [rng.choice([rng.randint(-100, total + 100), 0, total, 1 << 40, -(1 << 40)]) for _ in range(n + 1)]
        if slots == 0:
            continue
        # groups of X tokens, a multiple of 64 that gives this many slots (T // X + N + 1): every such X
        for x in range(64, total + 64, 64):
            if total // x + n + 1 != slots:
                continue
            for i in range(n):
                bos, count = seq_range(cu, i, total)
                assert 0 <= bos and bos + count <= total
                groups = -(-count // x)
                assert bos // x + i + max(groups - 1, 0) < slots
