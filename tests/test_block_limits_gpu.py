"""The block operators at the largest row counts that their argument checks admit, with the tolerances derived in
test_block_gpu."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_block_gpu import (check_linear_backward, check_linear_forward, check_norm_backward,  # noqa: E402
                                  check_norm_forward)

MOST = 1 << 24


@pytest.mark.parametrize("rows,H", [(70001, 5), (MOST, 2), (MOST, 7)])
def test_norm_of_short_rows(rows, H):
    """Rows of fewer than 8 elements, more of them than workgroups."""
    check_norm_forward(rows, H, "f16")
    check_norm_backward(rows, H, "bf16")


@pytest.mark.parametrize("H", [8, 12])
def test_norm_of_most_rows(H):
    check_norm_forward(MOST, H, "bf16")
    check_norm_backward(MOST, H, "f16")


@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
def test_linear_layer_of_most_rows(act):
    check_linear_forward(MOST, 8, 16, act, "f16")
    check_linear_backward(MOST, 16, 8, act, "f16")
