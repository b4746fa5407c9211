"""Forward-mode differentiation: dual tensors are refused, not read as plain ones."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu
T, k, E, H, I = 4, 2, 3, 16, 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def calls():
    """name -> (call, its tensors that a gradient reaches)"""
    half = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ids = torch.tensor([[0, 1], [1, 2], [0, 2], [2, 1]], dtype=torch.int32, device="cuda")
    _, position, offsets = m.si_moe_sort(ids, E)
    w = torch.ones(T, k, device="cuda")
    return {
        "gather": (lambda x: m.si_moe_gather(x, position, offsets), [half(T, H)]),
        "combine": (lambda ys, w: m.si_moe_combine(ys, position, w), [half(T * k, H), w]),
        "matmul": (lambda x, w: m.si_moe_matmul(x, w, offsets), [half(T * k, H), half(E, I, H)]),
        "swiglu": (m.si_swiglu, [half(T * k, 2 * I)]),
        "gateup": (lambda x, w: m.si_moe_gateup(x, w, offsets), [half(T * k, H), half(E, 2 * I, H)]),
        "experts": (lambda x, w, a, b: m.si_moe_experts(x, ids, w, a, b), [half(T, H), w, half(E, 2 * I, H), half(E, H, I)]),
    }


@pytest.mark.parametrize("name", ["gather", "combine", "matmul", "swiglu", "gateup", "experts"])
def test_duals_are_refused(name):
    call, tensors = calls()[name]
    want = call(*tensors)
    with fwd.dual_level():
        assert torch.equal(call(*tensors), want)             # plain tensors are welcome
        for i, t in enumerate(tensors):
            for like in (t, t.clone().requires_grad_()):
                dual = fwd.make_dual(like, torch.ones_like(t))
                with pytest.raises(ValueError, match="tangent"):
                    call(*tensors[:i], dual, *tensors[i + 1:])
    assert torch.equal(call(*tensors), want)
