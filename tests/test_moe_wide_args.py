"""The widths that a gradient of a fused gate and up needs: twice those of its experts (host checks only)."""
import pytest

import moe_decode_ffn_gb300 as m

WIDE, I = 1 << 21, 1 << 20


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.library()


@pytest.mark.parametrize("k,want", [(WIDE, m.SI_OK), (I + 8, m.SI_OK), (WIDE + 8, m.SI_ERR_INVALID_ARG), (WIDE - 4, m.SI_ERR_INVALID_ARG)])
def test_summed_width(lib, k, want):
    """No rows: checked, nothing launched."""
    for cols in (0, 1):
        assert lib.si_moe_matmul(16, m.SI_BF16, 0, k, 16, 1, 8, k, 8 if cols else k, 8 * k, cols, 16, 16, m.SI_BF16, 8, None, 0, None) == want


@pytest.mark.parametrize("n,want", [(WIDE, m.SI_ERR_WORKSPACE), (WIDE + 8, m.SI_ERR_INVALID_ARG)])
def test_rows_of_the_gradient(lib, n, want):
    """A workspace too small is found behind the widths, before any launch."""
    assert lib.si_moe_matmul_grad_w(16, n, 16, 8, m.SI_BF16, 4, 1, n, 8, 16, 16, m.SI_BF16, 256, 255, None) == want
