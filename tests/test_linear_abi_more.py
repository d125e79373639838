"""CPU checks of what linear attention and draft verification refuse of their workspaces and options."""
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
