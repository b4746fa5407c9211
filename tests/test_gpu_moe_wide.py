"""Experts wider than 2^19, whose gradients meet matrices of more than 2^20 rows."""
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxint8 as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products_at_the_widest(out):
    """Whole numbers of -1 to 1: sums of 2^21 of them are exact in fp32."""
    W, R = 1 << 21, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    whole = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, w, gy, rows = whole(R, W), whole(1, W, 8), whole(R, W), whole(R, 8)
    offsets = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    assert torch.equal(m.si_moe_matmul(x, w.transpose(1, 2), offsets, dtype=out), (x.double() @ w[0].double()).to(out))
    assert torch.equal(m.si_moe_matmul_grad_w(gy, rows, offsets, dtype=out), (gy.double().T @ rows.double()).to(out)[None])


def test_gradients_of_wide_experts():
    """down is zero but for 16 features at either end, so gh and the sums over features have that many
    terms that are not zero; the others' gradients are zeros."""
    T, H, I = 3, 8, (1 << 19) + 8
    g = torch.Generator(device="cuda").manual_seed(2)
    at = torch.cat([torch.arange(16), torch.arange(I - 16, I)]).cuda()
    x = torch.randint(-2, 3, (T, H), generator=g, device="cuda").bfloat16()
    gate_up = (torch.randint(-2, 3, (1, 2 * I, H), generator=g, device="cuda") / 4).bfloat16()   # g and u exact
    down = torch.zeros(1, H, I, dtype=torch.bfloat16, device="cuda")
    down[:, :, at] = torch.randint(-2, 3, (1, H, 32), generator=g, device="cuda").bfloat16()
    gy = torch.randint(-2, 3, (T, H), generator=g, device="cuda").bfloat16()                     # gh exact
    ids, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    leaves = [t.requires_grad_() for t in (x, w, gate_up, down)]
    gx, gw, ggate_up, gdown = torch.autograd.grad(m.si_moe_experts(x, ids, w, gate_up, down), leaves, gy)
    x, gate_up, down, gy = (t.detach().double() for t in (x, gate_up, down, gy))
    gu = x @ gate_up[0].T
    kept = [torch.from_numpy(Q.dequantize(*Q.quantize(v.cpu().numpy()))).cuda() for v in (gu[:, :I], gu[:, I:])]
    gh = (gy @ down[0])[:, at]
    q0, q1 = (v[:, at] for v in kept)
    s = torch.sigmoid(q0)
    gg, gu_ = gh * q1 * s * (1 + q0 * (1 - s)), gh * q0 * s

    # a rounding to bf16 as an operand and one as a result, 2^-8 each; the logistic function within 16 (1 + |g|) + 4 units
    # of 2^-24, |g| at most 8; a sum of n terms n 2^-23 of their magnitudes
    def near(got, want, size, terms, half=2.0 ** -8):
        return bool(((got.double() - want).abs() <= (2 * half + half * half + (terms + 96) * 2.0 ** -23) * size).all())

    both, size = torch.cat([gg, gu_], 1), torch.cat([gh.abs() * q1.abs() * s * (1 + q0.abs() * (1 - s)), gh.abs() * q0.abs() * s], 1)
    rows = torch.cat([at, I + at])
    assert near(gx, both @ gate_up[0, rows], size @ gate_up[0, rows].abs(), 64)
    assert near(ggate_up[0, rows], both.T @ x, size.T @ x.abs(), T)
    rest = torch.ones(2 * I, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert not bool(ggate_up[0, rest].any())
    h = torch.nn.functional.silu(kept[0]) * kept[1]
    assert near(gdown[0], gy.T @ h, gy.abs().T @ h.abs(), T)
    assert near(gw[:, 0], (gh * h[:, at]).sum(1), (gh * h[:, at]).abs().sum(1), 32, 0.0)


def test_a_product_whose_gradient_would_be_too_wide():
    """Refused before the forward pass, not half way through the backward pass."""
    k = (1 << 20) + 8
    x, w = torch.ones(2, k, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 8, k, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    assert bool((m.si_moe_matmul(x, w, offsets, dtype=torch.float32) == k).all())
    for a, b in ((x.clone().requires_grad_(), w), (x, w.clone().requires_grad_())):
        with pytest.raises(ValueError, match="wide"):
            m.si_moe_matmul(a, b, offsets)
        with torch.no_grad():
            assert bool((m.si_moe_matmul(a, b, offsets, dtype=torch.float32) == k).all())
