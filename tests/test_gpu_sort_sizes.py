"""Sizes that the C ABI cannot take (int) are refused, not cut to 32 bits."""
import pytest
import torch

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu

MANY = 2 ** 32 + 1            # 1 in the low 32 bits


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def refused(f):
    with pytest.raises((ValueError, m.SiError)):
        f()


def test_number_of_experts():
    ids = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    for n in (2 ** 32 + 4, 2 ** 31, 1025, 0, -1, -2 ** 32 + 4):
        refused(lambda: m.si_moe_sort(ids, n))
    assert m.si_moe_sort(ids, 4)[2].tolist() == [0, 6, 6, 6, 6]


def test_number_of_tokens():
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB")
    position = torch.empty(MANY, 1, dtype=torch.int32, device="cuda")      # never read
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty(MANY, 1, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(MANY, 1, device="cuda")
    refused(lambda: m.si_moe_sort(position, 2))
    refused(lambda: m.si_moe_gather(x, position, offsets))
    refused(lambda: m.si_moe_gather_backward(x, position))
    refused(lambda: m.si_moe_combine(x, position, w))
    refused(lambda: m.si_moe_combine_backward(x, x, position, offsets, w))
    del x, w, position
    torch.cuda.empty_cache()


def test_workspace_of_too_many_tokens():
    q = lambda r, c: m.si_quantize_mxfp4(torch.randn(2, r, c, device="cuda"))  # noqa: E731
    experts = m.Mxfp4Experts(q(64, 32), q(64, 32), q(32, 64))
    assert m.ffn_mxfp4_workspace_bytes(experts, 1, 1) > 0
    for t, k in ((MANY, 1), (1, MANY), (2 ** 24 + 1, 1), (0, 1), (1, 9)):
        assert m.ffn_mxfp4_workspace_bytes(experts, t, k) == 0
