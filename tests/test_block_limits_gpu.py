"""The block operators at the largest row counts that their argument checks admit, with the tolerances derived in
test_block_gpu."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_block_gpu import check_norm_backward, check_norm_forward  # noqa: E402

MOST = 1 << 24


@pytest.mark.parametrize("rows,H", [(70001, 5), (MOST, 2), (MOST, 7)])
def test_norm_of_short_rows(rows, H):
    """Rows of fewer than 8 elements, more of them than workgroups."""
    check_norm_forward(rows, H, "f16")
    check_norm_backward(rows, H, "bf16")
