"""A batch without rows goes through the quantiser and the product."""
import pytest
import torch

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_product_without_rows(dtype):
    some = m.si_quantize_mxfp4(torch.randn(40, 96, device="cuda"))
    none = m.si_quantize_mxfp4(torch.empty(0, 96, device="cuda"))
    for a, w, shape in ((none, some, (0, 40)), (some, none, (40, 0)), (none, none, (0, 0))):
        y = m.si_mxfp4_matmul(*a, *w, dtype=dtype)
        assert y.shape == shape and y.dtype == dtype and y.is_cuda
        out = torch.empty(shape, dtype=dtype, device="cuda")
        assert m.si_mxfp4_matmul(*a, *w, out=out) is out
        assert m.si_mxfp4_matmul(*a, *w, dtype=dtype, stream=torch.cuda.Stream()).shape == shape


def test_product_without_rows_keeps_its_checks():
    some = m.si_quantize_mxfp4(torch.randn(40, 96, device="cuda"))
    none = m.si_quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    with pytest.raises(ValueError):                  # 64 columns against 96
        m.si_mxfp4_matmul(*none, *some)
    none = m.si_quantize_mxfp4(torch.empty(0, 96, device="cuda"))
    with pytest.raises(ValueError):
        m.si_mxfp4_matmul(*none, *some, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.si_mxfp4_matmul(*none, *some, out=torch.empty(1, 40, device="cuda"))
