"""Arguments of the MXFP4 and token-sorting calls are checked on the host (no
device work; every call here is refused or has nothing to do)."""
import ctypes

import pytest
import torch

import moe_decode_ffn_gb300 as m

BAD, UNS, WS = m.SI_ERR_INVALID_ARG, m.SI_ERR_UNSUPPORTED, m.SI_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.library()


def test_scale_bytes(lib):
    assert lib.si_mxfp4_scale_bytes(1, 32) == 512
    assert lib.si_mxfp4_scale_bytes(128, 128) == 512
    assert lib.si_mxfp4_scale_bytes(129, 160) == 4 * 512
    assert lib.si_mxfp4_scale_bytes(0, 32) == 0
    assert lib.si_mxfp4_scale_bytes(4, 48) == 0 and lib.si_mxfp4_scale_bytes(-1, 32) == 0


@pytest.mark.parametrize("args,want", [
    ((16, m.SI_BF16, 1, 4, 48, 48, 0, 16, 16), BAD),       # columns not a multiple of 32
    ((16, m.SI_BF16, 1, 4, 64, 32, 0, 16, 16), BAD),       # rows overlap
    ((16, m.SI_BF16, 2, 4, 64, 64, 128, 16, 16), BAD),     # matrices overlap
    ((16, m.SI_BF16, 2, 4, 64, 100, 64, 16, 16), BAD),     # rows in turn that overlap
    ((16, m.SI_BF16, 2, 4, 64, 128, 32, 16, 16), BAD),
    ((16, m.SI_BF16, 1, 4, 64, -64, 0, 16, 16), BAD),
    ((16, m.SI_BF16, 1, -1, 64, 64, 0, 16, 16), BAD),
    ((16, m.SI_BF16, -1, 4, 64, 64, 0, 16, 16), BAD),
    ((16, m.SI_BF16, 1, 4, 64, 64, 0, 8, 16), BAD),        # misaligned codes
    ((16, m.SI_BF16, 1, 4, 64, 64, 0, 16, 24), BAD),       # misaligned scales
    ((17, m.SI_BF16, 1, 4, 64, 64, 0, 16, 16), BAD),       # misaligned values
    ((None, m.SI_BF16, 1, 4, 64, 64, 0, 16, 16), BAD),
    ((16, m.SI_Q4_K, 1, 4, 64, 64, 0, 16, 16), UNS),
    ((16, m.SI_BF16, 1, 0, 64, 64, 0, 16, 16), m.SI_OK),   # nothing to do
    ((None, m.SI_BF16, 0, 4, 64, 64, 0, None, None), m.SI_OK),
])
def test_quantize_refusals(lib, args, want):
    x, ty, n, rows, cols, rs, ms, c, s = args
    assert lib.si_quantize_mxfp4(x, ty, n, rows, cols, rs, ms, c, s, None) == want
    assert lib.si_dequantize_mxfp4(c, s, n, rows, cols, x, ty, rs, ms, None) == want


def test_matmul_refusals(lib):
    def call(ac=16, asc=16, mm=4, wc=16, wsc=16, n=8, k=64, out=16, ty=m.SI_BF16, ld=8, ws=256, nb=256):
        return lib.si_mxfp4_matmul(ac, asc, mm, wc, wsc, n, k, out, ty, ld, ws, nb, None)
    for kw in ({"ac": None}, {"wsc": None}, {"out": None}, {"mm": 0}, {"n": 0}, {"k": 0}, {"k": 48}, {"ld": 7},
               {"ac": 8}, {"wc": 24}, {"out": 17}, {"k": (1 << 20) + 32}, {"mm": -1}, {"mm": (1 << 30) + 1}):
        assert call(**kw) == BAD, kw
    assert call(ty=m.SI_Q8_0) == UNS
    assert call(mm=1 << 30, n=1 << 30, ld=1 << 30) == UNS      # more tiles than a launch counts
    for kw in ({"ws": 16}, {"nb": 255}):
        assert call(**kw) == WS, kw


def test_sort_and_row_refusals(lib):
    ok = [16, 4, 2, 8, 16, 16, 16, None, 0, None]
    for i, v in ((0, None), (0, 18), (1, 0), (1, -1), (2, 0), (2, 9), (3, 0), (3, 1025), (4, None), (5, None), (6, 17),
                 (1, 1 << 30)):
        a = list(ok)
        a[i] = v
        if i == 1 and v == 1 << 30:
            a[2] = 8                                          # 2^33 pairs
        assert lib.si_moe_sort(*a) == BAD, (i, v)
    size = lib.si_moe_sort_workspace_bytes
    assert size(4, 2, 8) == 0 and size(0, 2, 8) == 0 and size(1000, 9, 8) == 0
    need = size(1000, 8, 8)
    assert need > 0 and need % 256 == 0
    for ws, n in ((None, need), (128, need), (256, need - 1)):
        assert lib.si_moe_sort(16, 1000, 8, 8, 16, 16, 16, ws, n, None) == WS
    g = [16, m.SI_BF16, 4, 2, 64, 16, 16, 16, None]
    for i, v in ((0, None), (0, 17), (2, 0), (3, 0), (3, 9), (4, 0), (4, (1 << 24) + 1), (5, None), (6, None), (7, None)):
        a = list(g)
        a[i] = v
        assert lib.si_moe_gather(*a) == BAD, (i, v)
    assert lib.si_moe_gather(16, m.SI_Q8_0, 4, 2, 64, 16, 16, 16, None) == UNS
    assert lib.si_moe_combine(16, m.SI_F32, 4, 2, 64, 16, None, 16, None) == BAD
    assert lib.si_moe_combine(18, m.SI_F32, 4, 2, 64, 16, 16, 16, None) == BAD
    assert lib.si_moe_gather_backward(16, m.SI_F16, 4, 2, 0, 16, 16, None) == BAD
    assert lib.si_moe_combine_backward(16, 16, m.SI_F16, 4, 2, 8, 16, 16, 16, 16, None, None) == BAD
    assert lib.si_moe_combine_backward(16, 16, m.SI_F16, 4, 2, 8, 16, None, 16, 16, 16, None) == BAD


def test_ffn_refusals(lib):
    def experts(**kw):
        c = m.SiMxfp4Experts(256, 128, 8, 16, 16, 16, 16, 16, 16)
        for k, v in kw.items():
            setattr(c, k, v)
        return ctypes.byref(c)
    size = lib.si_moe_ffn_mxfp4_workspace_bytes
    need = size(experts(), 3, 2)
    assert need > 0 and need % 256 == 0
    assert size(experts(), 300, 2) > need
    for c, t, k in ((experts(hidden=40), 3, 2), (experts(inter=0), 3, 2), (experts(n_experts=0), 3, 2),
                    (experts(n_experts=1025), 3, 2), (experts(), 0, 2), (experts(), 3, 9), (experts(), 3, 0),
                    (experts(), 1 << 24, 2), (None, 3, 2)):
        assert size(c, t, k) == 0
        assert lib.si_moe_ffn_mxfp4(c, t, k, 16, 16, 16, 16, 256, 1 << 40, None) == BAD
    call = lambda c=experts(), x=16, ids=16, w=16, out=16, ws=256, nb=need: lib.si_moe_ffn_mxfp4(  # noqa: E731
        c, 3, 2, x, ids, w, out, ws, nb, None)
    for kw in ({"x": None}, {"ids": None}, {"w": 18}, {"out": 8}, {"c": experts(up_scales=None)},
               {"c": experts(down_codes=8)}):
        assert call(**kw) == BAD, kw
    for kw in ({"ws": None}, {"ws": 128}, {"nb": need - 1}):
        assert call(**kw) == WS, kw


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        m.si_quantize_mxfp4(x)
    with pytest.raises(ValueError):
        m.si_quantize_mxfp4(torch.zeros(4, 40))
    with pytest.raises(ValueError):
        m.si_quantize_mxfp4(torch.zeros(64))
    with pytest.raises(ValueError):
        m.si_quantize_mxfp4(torch.zeros(64, 4).t())
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.si_mxfp4_matmul(u8, torch.zeros(512, dtype=torch.uint8), u8, torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError):
        m.si_moe_sort(torch.zeros(2, 2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        m.Mxfp4Experts((u8, u8), (u8, u8), (u8, u8))
