"""si_moe_gateup through torch's autograd: the gradients that si_moe_matmul and si_swiglu would hand on."""
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxint8 as Q

pytestmark = pytest.mark.gpu
# rows of every expert, rows before the first and behind the last, H, I: in one SM and in pairs
CASES = [([1], 0, 0, 8, 8), ([3, 0, 5], 1, 2, 72, 40), ([40, 0, 17, 129], 2, 7, 136, 136), ([0, 300], 0, 3, 64, 264)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def inputs(counts, head, tail, H, I, dtype):
    g = torch.Generator(device="cuda").manual_seed(H + I)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(dtype)  # noqa: E731
    R, at = head + sum(counts) + tail, [head]
    for c in counts:
        at.append(at[-1] + c)
    offsets = torch.tensor(at, dtype=torch.int32, device="cuda")
    gh = torch.randn(R, I, generator=g, device="cuda").to(dtype)
    return whole(R, H), whole(len(counts), 2 * I, H) / 16, offsets, gh     # g and u exact in fp32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("counts,head,tail,H,I", CASES)
def test_gradients(counts, head, tail, H, I, dtype):
    x, gate_up, offsets, gh = inputs(counts, head, tail, H, I, dtype)
    R = x.shape[0]
    gh[:head], gh[R - tail:] = float("nan"), float("inf")                  # rows of no expert add nothing
    a, b = x.clone().requires_grad_(), gate_up.clone().requires_grad_()
    h, kept = m.si_moe_gateup(a, b, offsets, keep=True)
    want, want_kept = m.si_moe_gateup(x, gate_up, offsets, keep=True)
    assert torch.equal(h, want) and all(torch.equal(p, q) and not p.requires_grad for p, q in zip(kept, want_kept))
    gx, gw = torch.autograd.grad(h, (a, b), gh)
    # equal to the steps
    ggu = m.si_swiglu_backward(gh, kept)[0]
    for got, step in zip((gx, gw), m.si_moe_matmul_backward(ggu, x, gate_up, offsets)):
        assert torch.equal(got, step)
    # and to the formulas from the kept values: ggu is rounded to the type as an operand, the result once more; the
    # logistic function within 16 (1 + |g|) + 4 units of 2^-24; a sum of n terms n 2^-23 of their magnitudes
    half, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    want_x = torch.zeros(R, H, dtype=torch.float64, device="cuda")
    off_x, at = torch.zeros_like(want_x), head
    for e, c in enumerate(counts):
        rows, w = slice(at, at + c), gate_up[e].double()
        at += c
        X, G = x[rows].double(), gh[rows].double()
        gu = X @ w.T
        q0, q1 = (torch.from_numpy(Q.dequantize(*Q.quantize(v.cpu().numpy()))).cuda() for v in (gu[:, :I], gu[:, I:]))
        s = torch.sigmoid(q0)
        d = torch.cat([G * q1 * s * (1 + q0 * (1 - s)), G * q0 * s], 1)
        size = torch.cat([(G * q1).abs() * s * (1 + q0.abs() * (1 - s)), (G * q0).abs() * s], 1)
        off = half * d.abs() + (1 + half) * (16 * (1 + torch.cat([q0, q0], 1).abs()) + 4) * 2.0 ** -24 * size + tiny
        want_x[rows], off_x[rows] = d @ w, off @ w.abs() + 2 * I * 2.0 ** -23 * ((d.abs() + off) @ w.abs())
        want_w, off_w = d.T @ X, off.T @ X.abs() + c * 2.0 ** -23 * ((d.abs() + off).T @ X.abs())
        assert bool(((gw[e].double() - want_w).abs() <= off_w * (1 + half) + half * want_w.abs() + tiny).all())
    assert bool(((gx.double() - want_x).abs() <= off_x * (1 + half) + half * want_x.abs() + tiny).all())


def test_one_gradient_alone_and_none():
    x, gate_up, offsets, gh = inputs([40, 0, 17, 129], 2, 7, 136, 136, torch.bfloat16)
    a, b = x.clone().requires_grad_(), gate_up.clone().requires_grad_()
    gx, gw = torch.autograd.grad(m.si_moe_gateup(a, b, offsets), (a, b), gh)
    assert torch.equal(torch.autograd.grad(m.si_moe_gateup(a, gate_up, offsets), a, gh)[0], gx)
    assert torch.equal(torch.autograd.grad(m.si_moe_gateup(x, b, offsets), b, gh)[0], gw)
    with torch.no_grad():
        assert not m.si_moe_gateup(a, b, offsets).requires_grad
    assert not m.si_moe_gateup(x, gate_up, offsets).requires_grad


def test_on_another_stream():
    x, gate_up, offsets, gh = inputs([40, 0, 17, 129], 2, 7, 136, 136, torch.bfloat16)
    a, b = x.clone().requires_grad_(), gate_up.clone().requires_grad_()
    want = torch.autograd.grad(m.si_moe_gateup(a, b, offsets), (a, b), gh)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h = m.si_moe_gateup(a, b, offsets, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    got = torch.autograd.grad(h, (a, b), gh)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_up_to_the_experts():
    """Sort, gather, gateup, product and combine by hand: every leaf's gradient arrives."""
    T, k, E, H, I = 70, 3, 4, 64, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda c, *s: (torch.randn(*s, generator=g, device="cuda") * c).bfloat16().requires_grad_()  # noqa: E731
    x, gate_up, down = draw(1, T, H), draw(0.1, E, 2 * I, H), draw(0.1, E, H, I)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand(T, k, generator=g, device="cuda").requires_grad_()
    _, position, offsets = m.si_moe_sort(ids, E)
    h = m.si_moe_gateup(m.si_moe_gather(x, position, offsets), gate_up, offsets)
    y = m.si_moe_combine(m.si_moe_matmul(h, down, offsets), position, w)
    grads = torch.autograd.grad(y, (x, w, gate_up, down), torch.ones_like(y))
    once = m.si_moe_experts(x, ids, w, gate_up, down)
    for a, b in zip(grads, torch.autograd.grad(once, (x, w, gate_up, down), torch.ones_like(y))):
        # 16-bit rows between the steps: some roundings of 2^-8 more
        assert float((a.double() - b.double()).norm()) <= 0.02 * float(b.double().norm())


def test_captured_and_replayed():
    args = [40, 0, 17, 129], 2, 7, 136, 136, torch.bfloat16
    x, gate_up, offsets, gh = inputs(*args)
    ws, graph = m.workspace(m.moe_matmul_workspace_bytes()), torch.cuda.CUDAGraph()
    a, b = x.clone().requires_grad_(), gate_up.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                # autograd's own first pass outside the capture
        torch.autograd.grad(m.si_moe_gateup(a, b, offsets, ws=ws), (a, b), gh)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        h = m.si_moe_gateup(a, b, offsets, ws=ws)
        out = h, *torch.autograd.grad(h, (a, b), gh)
    for cut in (1, 2):
        with torch.no_grad():
            a.copy_(x.flip(0)), b.copy_(gate_up.flip(1))
        offsets.copy_(torch.tensor([cut, 100, 100, 130, 150 + cut], device="cuda"))
        gh.copy_(torch.randn(gh.shape, device="cuda"))
        graph.replay()
        c, d = a.detach().clone().requires_grad_(), b.detach().clone().requires_grad_()
        fresh = m.si_moe_gateup(c, d, offsets)
        assert all(torch.equal(p, q) for p, q in zip(out, (fresh, *torch.autograd.grad(fresh, (c, d), gh))))
    assert m.si_workspace_status(ws) == m.SI_OK
