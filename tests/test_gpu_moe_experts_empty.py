"""si_moe_experts of a batch without tokens."""
import pytest
import torch

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu
E, H, I, k = 3, 64, 24, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def inputs(dtype, T=0):
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    return draw(T, H), ids, torch.ones(T, k, device="cuda"), draw(E, 2 * I, H), draw(E, H, I)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ws", [False, True])
def test_empty_results_and_zero_gradients(dtype, ws):
    x, ids, w, gate_up, down = inputs(dtype)
    ws = m.workspace(m.moe_experts_workspace_bytes(4, k, gate_up)) if ws else None
    y = m.si_moe_experts(x, ids, w, gate_up, down, ws=ws)
    assert y.shape == (0, H) and y.dtype is dtype and not y.requires_grad
    leaves = [t.requires_grad_() for t in (x, w, gate_up, down)]
    y = m.si_moe_experts(x, ids, w, gate_up, down, ws=ws)
    assert y.shape == (0, H) and y.requires_grad
    for g, t in zip(torch.autograd.grad(y, leaves, torch.empty_like(y)), leaves):
        assert g.shape == t.shape and g.dtype is t.dtype and not bool(g.any())
    y = m.si_moe_experts(x.detach(), ids, w.detach(), gate_up.detach(), down, ws=ws)   # one leaf alone, into .grad
    down.grad = None
    y.sum().backward()
    assert not bool(down.grad.any()) and gate_up.grad is None


def test_the_same_sizes_are_refused_as_with_tokens():
    for T in (0, 1):
        x, ids, w, gate_up, down = inputs(torch.bfloat16, T)
        many = ids.repeat(1, 5)
        bad = [(x, many, many.float(), gate_up, down), (x, ids[:, :0], w[:, :0], gate_up, down), (x, ids.long(), w, gate_up, down),
               (x, ids, w.half(), gate_up, down), (x.half(), ids, w, gate_up, down), (x[:, :40], ids, w, gate_up, down),
               (x, ids, w, gate_up[:0], down[:0])]
        for args in bad:
            with pytest.raises((ValueError, RuntimeError)):
                m.si_moe_experts(*args)
