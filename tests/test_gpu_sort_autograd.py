"""Gradients through si_moe_gather and si_moe_combine reach tensors that require
them: equal to the explicit calls, to the formulas in 64 bits (a product or a sum
of n fp32 terms is off by at most n 2^-24 of the terms' magnitudes, and by half a
unit in the last place of its type on top) and to nothing where nothing was kept."""
import pytest
import torch

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# tokens, ranks, experts, hidden, share of dropped pairs
CASES = [(1, 1, 1, 8, 0), (5, 2, 3, 1, 0), (33, 4, 7, 72, 0.4), (64, 8, 128, 512, 0.1), (9, 3, 4, 40, 1.0), (700, 7, 20, 65, 0.2)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def inputs(T, k, E, H, drop, kind):
    g = torch.Generator(device="cuda").manual_seed(T * 31 + H)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < drop, torch.full_like(ids, E + 1), ids)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(TYPES[kind])  # noqa: E731
    w = torch.randn(T, k, generator=g, device="cuda")
    return ids, draw(T, H), draw(T * k, H), w, draw(T, H), draw(T * k, H)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,k,E,H,drop", CASES)
def test_gradients_equal_the_explicit_calls(T, k, E, H, drop, kind):
    ids, x, ys, w, gy, gxs = inputs(T, k, E, H, drop, kind)
    _, position, offsets = m.si_moe_sort(ids, E)
    xs, y = m.si_moe_gather(x, position, offsets), m.si_moe_combine(ys, position, w)
    want = [m.si_moe_gather_backward(gxs, position), *m.si_moe_combine_backward(gy, ys, position, offsets, w)]
    a, b, c = (t.clone().requires_grad_() for t in (x, ys, w))
    out = m.si_moe_gather(a, position, offsets), m.si_moe_combine(b, position, c)
    assert torch.equal(out[0], xs) and torch.equal(out[1], y)
    assert all(o.requires_grad for o in out)
    torch.autograd.backward(out, (gxs, gy))
    for t, g in zip((a, b, c), want):
        assert t.grad.dtype == t.dtype and torch.equal(t.grad, g)
    # one of the two alone
    b, c = ys.clone().requires_grad_(), w.clone().requires_grad_()
    assert torch.equal(torch.autograd.grad(m.si_moe_combine(b, position, w), b, gy)[0], want[1])
    assert torch.equal(torch.autograd.grad(m.si_moe_combine(ys, position, c), c, gy)[0], want[2])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,k,E,H,drop", CASES)
def test_gradients_against_64_bits(T, k, E, H, drop, kind):
    """sum(c * combine(f(gather(x)), w)) with f(v) = v * s, fp64 by autograd of
    plain indexing. The chain rounds xs * s, gys and gxs to the type before gx."""
    ids, x, s, w, gy, _ = inputs(T, k, E, H, drop, kind)
    _, position, offsets = m.si_moe_sort(ids, E)
    a, c = x.clone().requires_grad_(), w.clone().requires_grad_()
    m.si_moe_combine(m.si_moe_gather(a, position, offsets) * s, position, c).backward(gy)
    kept = (position >= 0).double()[..., None]
    at = position.clamp(min=0).long()
    xd, sd, wd, gd = x.double(), s.double()[at] * kept, w.double(), gy.double()
    gx, agx = (wd[..., None] * sd * gd[:, None]).sum(1), (wd[..., None] * sd * gd[:, None]).abs().sum(1)
    gw, agw = (gd * xd)[:, None].mul(sd).sum(2), (gd * xd)[:, None].mul(sd).abs().sum(2)
    half = torch.finfo(TYPES[kind]).eps / 2
    tiny = 2.0 ** -24 * T * k if kind == "f16" else 0        # subnormal results: half a step of 2^-24 each
    near = lambda got, want, tol: bool(((got.double() - want).abs() <= tol).all())  # noqa: E731
    # two roundings of the type below the sum, one of its result (1.01: their products)
    assert near(a.grad, gx, 1.01 * (2 * half + (k + 2) * 2.0 ** -24) * agx + half * (gx.abs() + agx * 3 * half) + tiny * (1 + s.abs().max().double()))
    # one rounding of the type (xs * s) below the sum of H terms
    assert near(c.grad, gw, 1.01 * (half + (H + 2) * 2.0 ** -24) * agw + tiny * gy.abs().max().double() * H)


def test_rows_that_no_pair_has_get_zero():
    """Places of one's own choice, with gaps among them."""
    T, k, H = 6, 2, 24
    position = torch.tensor([[9, 0], [-1, 4], [11, 2], [-1, -1], [5, 100], [7, 10]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    ys, w, gy = (torch.randn(*s, generator=g, device="cuda") for s in ((T * k, H), (T, k), (T, H)))
    junk = [torch.full((T * k, H), float("nan"), device="cuda") for _ in range(4)]      # what freed memory may hold
    del junk
    ys.requires_grad_()
    grad, = torch.autograd.grad(m.si_moe_combine(ys, position, w), ys, gy)
    want = torch.zeros(T * k, H, device="cuda")
    for t in range(T):
        for r in range(k):
            if 0 <= int(position[t, r]) < T * k:
                want[int(position[t, r])] = w[t, r] * gy[t]
    assert torch.equal(grad, want)


def test_without_grad_nothing_is_recorded():
    ids, x, ys, w, gy, _ = inputs(20, 2, 4, 64, 0.1, "bf16")
    _, position, offsets = m.si_moe_sort(ids, 4)
    x.requires_grad_()
    with torch.no_grad():
        assert not m.si_moe_gather(x, position, offsets).requires_grad
    with torch.inference_mode():
        assert not m.si_moe_gather(x, position, offsets).requires_grad
    assert not m.si_moe_combine(ys, position, w).requires_grad


def test_second_derivatives_are_refused():
    ids, x, ys, w, gy, _ = inputs(20, 2, 4, 64, 0.1, "f32")
    _, position, offsets = m.si_moe_sort(ids, 4)
    ys.requires_grad_()
    gy.requires_grad_()
    g, = torch.autograd.grad(m.si_moe_combine(ys, position, w), ys, gy, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_gradients_of_broadcast_and_strided_ones():
    """y.sum().backward() hands an expanded gradient back."""
    ids, x, ys, w, _, _ = inputs(33, 3, 5, 48, 0.2, "f32")
    _, position, offsets = m.si_moe_sort(ids, 5)
    a, b, c = (t.clone().requires_grad_() for t in (x, ys, w))
    m.si_moe_combine(b, position, c).sum().backward()
    gys, gw = m.si_moe_combine_backward(torch.ones_like(x), ys, position, offsets, w)
    assert torch.equal(b.grad, gys) and torch.equal(c.grad, gw)
    m.si_moe_gather(a, position, offsets).t().sum(0).sum().backward()
    assert torch.equal(a.grad, m.si_moe_gather_backward(torch.ones_like(ys), position))


def test_gradients_on_a_given_stream_and_captured():
    ids, x, ys, w, gy, _ = inputs(48, 4, 12, 256, 0.1, "bf16")

    def step(stream=None):
        a, c = x.detach().requires_grad_(), w.detach().requires_grad_()
        _, position, offsets = m.si_moe_sort(ids, 12, stream=stream)
        xs = m.si_moe_gather(a, position, offsets, stream=stream)
        y = m.si_moe_combine(xs, position, c, stream=stream)
        return y.detach(), *torch.autograd.grad(y, (a, c), gy)

    want = step()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = step(other)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in (1, 2):
        ids.copy_(torch.randint(0, 13, ids.shape, generator=torch.Generator().manual_seed(seed)))
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))
