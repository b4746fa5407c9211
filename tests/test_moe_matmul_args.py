"""Arguments of the products of sorted rows, of the 8-bit activations and of SwiGLU
are checked on the host (no device work; every call here is refused or has nothing
to do)."""
import ctypes

import pytest
import torch

import moe_decode_ffn_gb300 as m

BAD, UNS, WS, OK = m.SI_ERR_INVALID_ARG, m.SI_ERR_UNSUPPORTED, m.SI_ERR_WORKSPACE, m.SI_OK


@pytest.fixture(scope="module")
def lib():
    m.build()
    return m.library()


def refused(call, ok, cases, want):
    for kw in cases:
        assert set(kw) <= set(ok)
        assert call(*{**ok, **kw}.values(), None) == want, kw


def test_product_refusals(lib):
    assert lib.si_moe_matmul_workspace_bytes() == 256
    ok = dict(x=16, type=m.SI_BF16, rows=40, ldx=64, w=16, e=4, n=24, k=64, ldw=64, mat=24 * 64, cols=0, off=16, out=16,
              to=m.SI_BF16, ldo=24, ws=256, nb=256)
    refused(lib.si_moe_matmul, ok, [
        {"x": None}, {"x": 8}, {"w": None}, {"w": 24}, {"off": None}, {"off": 18}, {"out": None}, {"out": 8},
        {"rows": -1}, {"rows": 1 << 31}, {"ldx": 56}, {"ldx": 68}, {"ldx": -64}, {"e": 0}, {"e": 1025}, {"n": 0}, {"n": 12},
        {"n": (1 << 20) + 8}, {"k": 0}, {"k": 60}, {"ldw": 56}, {"ldw": 66}, {"mat": 24 * 64 - 8}, {"mat": 24 * 64 + 4},
        {"cols": 1, "ldw": 16}, {"cols": 1, "ldw": 24, "mat": 24 * 63}, {"ldo": 16}, {"ldo": 28}], BAD)
    refused(lib.si_moe_matmul, ok, [{"type": m.SI_F32}, {"type": m.SI_Q8_0}, {"to": m.SI_F16}, {"to": m.SI_Q8_0},
                                    {"rows": 1 << 30, "n": 1 << 20, "ldo": 1 << 20, "mat": 1 << 26}], UNS)
    refused(lib.si_moe_matmul, ok, [{"ws": 16}, {"nb": 255}], WS)
    refused(lib.si_moe_matmul, ok, [{"rows": 0}, {"rows": 0, "x": None, "out": None}], OK)


def test_gradient_refusals(lib):
    ok = dict(gy=16, ldg=24, x=16, ldx=64, type=m.SI_F16, rows=40, e=4, n=24, k=64, off=16, gw=16, to=m.SI_F32, ws=256,
              nb=256)
    refused(lib.si_moe_matmul_grad_w, ok, [
        {"gy": None}, {"gy": 8}, {"ldg": 16}, {"ldg": 28}, {"x": None}, {"x": 8}, {"ldx": 56}, {"rows": -1},
        {"rows": 1 << 31}, {"e": 0}, {"e": 1025}, {"n": 20}, {"k": 4}, {"off": None}, {"off": 17}, {"gw": None},
        {"gw": 8}], BAD)
    refused(lib.si_moe_matmul_grad_w, ok, [{"type": m.SI_F32}, {"to": m.SI_BF16}, {"e": 1024, "n": 1 << 20, "ldg": 1 << 20, "k": 1 << 20, "ldx": 1 << 20}], UNS)
    refused(lib.si_moe_matmul_grad_w, ok, [{"ws": 16}, {"nb": 255}], WS)


def test_gateup_refusals(lib):
    ok = dict(x=16, type=m.SI_BF16, rows=40, ldx=64, w=16, e=4, inter=24, hidden=64, off=16, h=16, codes=16, scales=16,
              ws=256, nb=256)
    refused(lib.si_moe_gateup, ok, [
        {"x": None}, {"w": 8}, {"off": None}, {"h": None}, {"h": 8}, {"codes": None}, {"codes": 8}, {"scales": None},
        {"ldx": 56}, {"inter": 4}, {"hidden": 68}, {"e": 0}, {"rows": -1}], BAD)
    refused(lib.si_moe_gateup, ok, [{"type": m.SI_F32}], UNS)
    refused(lib.si_moe_gateup, ok, [{"ws": 128}, {"nb": 0}], WS)
    refused(lib.si_moe_gateup, ok, [{"rows": 0, "x": None}], OK)


def test_down_backward_refusals(lib):
    need = lib.si_moe_down_backward_workspace_bytes(40, 4, 24)   # a header of 256 bytes and 40 rows of 4 sums, to the next 256
    assert need == 1024 and lib.si_moe_down_backward_workspace_bytes(-1, 4, 24) == 0
    assert lib.si_moe_down_backward_workspace_bytes(40, 0, 24) == 0 and lib.si_moe_down_backward_workspace_bytes(40, 4, 20) == 0
    ok = dict(gy=16, type=m.SI_BF16, rows=40, ldg=64, down=16, e=4, hidden=64, inter=24, off=16, codes=16, scales=16, w=16,
              order=16, ggu=16, wh=16, gw=16, ws=256, nb=need)
    refused(lib.si_moe_down_backward, ok, [
        {"gy": None}, {"gy": 8}, {"ldg": 56}, {"down": None}, {"down": 8}, {"off": None}, {"codes": None}, {"scales": None},
        {"w": 18}, {"order": 18}, {"ggu": None}, {"ggu": 17}, {"wh": 17}, {"codes": 8}, {"ggu": 8}, {"wh": 24}, {"gw": 18}, {"hidden": 60}, {"inter": 20},
        {"e": 1025}, {"rows": -1}], BAD)
    refused(lib.si_moe_down_backward, ok, [{"type": m.SI_F32}], UNS)
    refused(lib.si_moe_down_backward, ok, [{"ws": None}, {"ws": 128}, {"nb": need - 1}, {"gw": None, "nb": 255}], WS)
    refused(lib.si_moe_down_backward, ok, [{"rows": 0, "gy": None}], OK)


def test_experts_refusals(lib):
    def experts(**kw):
        c = m.SiExperts(m.SI_BF16, 64, 24, 4, 16, 16)
        for name, v in kw.items():
            setattr(c, name, v)
        return ctypes.byref(c)
    size, kept = lib.si_moe_experts_workspace_bytes, lib.si_moe_experts_kept_bytes
    need = size(experts(), 10, 2)
    assert need > 0 and need % 256 == 0 and size(experts(), 1000, 2) > need
    # order and position of 20 pairs, 5 offsets, 48 codes and 2 scales a pair, each to the next 256
    assert kept(experts(), 10, 2) == 3 * 256 + 1024 + 256
    for c, t, k in ((experts(hidden=60), 10, 2), (experts(inter=0), 10, 2), (experts(n_experts=0), 10, 2),
                    (experts(n_experts=1025), 10, 2), (experts(), 0, 2), (experts(), 10, 0), (experts(), 10, 9),
                    (experts(), 1 << 28, 8), (None, 10, 2)):
        assert size(c, t, k) == 0 and kept(c, t, k) == 0
        assert lib.si_moe_experts(c, t, k, 16, 16, 16, 16, None, 256, 1 << 40, None) == BAD
        assert lib.si_moe_experts_backward(c, t, k, 16, 16, 16, 256, 16, 16, 16, 16, 256, 1 << 40, None) == BAD
    ok = dict(L=experts(), t=10, k=2, x=16, ids=16, w=16, y=16, kept=256, ws=256, nb=need)
    refused(lib.si_moe_experts, ok, [{"x": None}, {"x": 8}, {"ids": None}, {"w": None}, {"y": None}, {"y": 8}, {"kept": 128},
                                     {"L": experts(gate_up=None)}, {"L": experts(down=8)}], BAD)
    refused(lib.si_moe_experts, ok, [{"L": experts(type=m.SI_F32)}], UNS)
    refused(lib.si_moe_experts, ok, [{"ws": None}, {"ws": 128}, {"nb": need - 1}], WS)
    ok = dict(L=experts(), t=10, k=2, gy=16, x=16, w=16, kept=256, gx=16, gw=16, ggate_up=16, gdown=16, ws=256, nb=need)
    refused(lib.si_moe_experts_backward, ok, [
        {"gy": None}, {"gy": 8}, {"x": None}, {"x": 24}, {"w": None}, {"kept": None}, {"kept": 128}, {"gx": 8}, {"gw": 18},
        {"ggate_up": 8}, {"gdown": 24}], BAD)
    refused(lib.si_moe_experts_backward, ok, [{"ws": None}, {"nb": need - 1}], WS)


def test_combine_of_fp32_rows_refusals(lib):
    ok = dict(ys=16, t=4, k=2, hidden=64, position=16, w=16, y=16, type=m.SI_BF16)
    refused(lib.si_moe_combine_f32, ok, [{"ys": None}, {"ys": 18}, {"t": 0}, {"k": 9}, {"hidden": 0}, {"position": None},
                                         {"w": 18}, {"y": None}, {"y": 17}], BAD)
    refused(lib.si_moe_combine_f32, ok, [{"type": m.SI_Q8_0}], UNS)


def test_mxint8_refusals(lib):
    ok = dict(x=16, type=m.SI_F32, rows=4, cols=40, ld=40, codes=16, scales=16)
    refused(lib.si_quantize_mxint8, ok, [
        {"x": None}, {"x": 18}, {"rows": -1}, {"cols": 0}, {"cols": -8}, {"ld": 39}, {"codes": None}, {"scales": None},
        {"rows": 1 << 30, "cols": 1 << 30, "ld": 1 << 30}], BAD)
    refused(lib.si_quantize_mxint8, ok, [{"type": m.SI_Q8_0}], UNS)
    refused(lib.si_quantize_mxint8, ok, [{"rows": 0, "x": None}], OK)
    ok = dict(codes=16, scales=16, rows=4, cols=40, y=16, type=m.SI_BF16, ld=40)
    refused(lib.si_dequantize_mxint8, ok, [{"y": None}, {"y": 17}, {"ld": 32}, {"codes": None}, {"scales": None}], BAD)
    refused(lib.si_dequantize_mxint8, ok, [{"type": m.SI_Q4_K}], UNS)


def test_swiglu_refusals(lib):
    ok = dict(gu=16, type=m.SI_BF16, rows=4, inter=40, ld=80, h=16, codes=16, scales=16)
    refused(lib.si_swiglu, ok, [{"gu": None}, {"gu": 17}, {"h": None}, {"inter": 0}, {"ld": 79}, {"rows": -1},
                                {"codes": None}, {"scales": None}], BAD)
    refused(lib.si_swiglu, ok, [{"type": m.SI_Q8_1}], UNS)
    ok = dict(gh=16, type=m.SI_F32, rows=4, inter=40, codes=16, scales=16, w=16, order=16, ggu=16, wh=16, gw=16)
    refused(lib.si_swiglu_backward, ok, [
        {"gh": None}, {"gh": 18}, {"codes": None}, {"scales": None}, {"w": 18}, {"order": 17}, {"ggu": None}, {"wh": 18},
        {"gw": 18}, {"inter": 0}, {"rows": 1 << 31}], BAD)
    refused(lib.si_swiglu_backward, ok, [{"type": m.SI_Q8_1}], UNS)
    refused(lib.si_swiglu_backward, ok, [{"rows": 0}], OK)


def test_binding_refuses_host_tensors(lib):
    x, w, off = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    ids, c = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: m.si_moe_matmul(x, w, off), lambda: m.si_moe_matmul_grad_w(x, x, off),
                 lambda: m.si_moe_matmul_backward(x, x, w, off), lambda: m.si_moe_gateup(x, w, off),
                 lambda: m.si_moe_experts(x, ids, c, w, w), lambda: m.si_quantize_mxint8(x),
                 lambda: m.si_dequantize_mxint8(x, x), lambda: m.si_swiglu(x),
                 lambda: m.si_swiglu_backward(x, (x, x))):
        with pytest.raises(ValueError):
            call()
