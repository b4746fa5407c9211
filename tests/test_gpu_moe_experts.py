"""The differentiable routed experts, and the gate and up product with SwiGLU.

x and gate_up hold whole numbers from -2 to 2 (gate_up in sixteenths), so that g and
u are exact in fp32 in any order of their sums and so are their 8-bit codes. From there
every step's error is carried along beside its value in 64 bits (class V): a rounding
adds half a unit in the last place, a sum of n terms n 2^-23 of the terms' magnitudes (an
addition on the tensor cores may truncate), and what comes in off by some bound goes
on multiplied by the magnitudes that it meets."""
import numpy as np
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxint8 as Q

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# tokens, ranks, experts, hidden, inter, share of dropped pairs
CASES = [(1, 1, 1, 8, 8, 0), (1, 8, 16, 72, 40, 0), (5, 2, 3, 64, 32, 0.3), (64, 8, 16, 128, 96, 0.1), (70, 3, 2, 200, 136, 0),
         (9, 3, 4, 40, 264, 1.0)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


class V:
    """Values in 64 bits and how far the device's may be from them."""

    def __init__(self, v, off=None):
        self.v, self.off = v, torch.zeros_like(v) if off is None else off

    def matmul(self, o):
        n = self.v.shape[1]
        size = (self.v.abs() + self.off) @ (o.v.abs() + o.off)
        return V(self.v @ o.v, self.off @ (o.v.abs() + o.off) + self.v.abs() @ o.off + n * 2.0 ** -23 * size)

    @property
    def T(self):
        return V(self.v.T, self.off.T)

    def round(self, dtype):
        i = torch.finfo(dtype)
        return V(self.v, self.off + i.eps / 2 * (self.v.abs() + self.off) + i.smallest_normal * i.eps)


def inputs(T, k, E, H, I, drop, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(T * 31 + H + seed)
    dtype = TYPES[kind]
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(dtype)  # noqa: E731
    ids = torch.rand(T, E + 8, generator=g, device="cuda")[:, :E].argsort(1)[:, :k] if E >= k else torch.randint(0, E, (T, k), generator=g, device="cuda")
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < drop, torch.full_like(ids, -1), ids).to(torch.int32)
    x, gate_up = whole(T, H), whole(E, 2 * I, H) / 16
    down = (torch.randn(E, H, I, generator=g, device="cuda") * 0.1).to(dtype)
    w, gy = torch.rand(T, k, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda").to(dtype)
    return x, ids, w, gate_up, down, gy


def silu_off(g, h):
    """Of silu(g) u in fp32: 16 (1 + |g|) + 4 units of 2^-24."""
    return (16 * (1 + g.abs()) + 4) * 2.0 ** -24 * h.abs()


def expected(x, ids, w, gate_up, down, gy):
    """y and the gradients of x, w, gate_up, down as V, pair by pair of an expert."""
    dtype, (T, k), (E, I2, H) = x.dtype, ids.shape, gate_up.shape
    I, z = I2 // 2, lambda *s: V(torch.zeros(*s, dtype=torch.float64, device="cuda"))  # noqa: E731
    y, gx, gw, ggate_up, gdown = z(T, H), z(T, H), z(T, k), z(E, I2, H), z(E, H, I)
    size_y, size_x = z(T, H).v, z(T, H).v
    for e in range(E):
        t, r = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        up, dn, c = V(gate_up[e].double()), V(down[e].double()), w[t, r].double()[:, None]
        X, GY = V(x[t].double()), V(gy[t].double())
        gu = X.v @ up.v.T                        # exact on the device
        g, u = gu[:, :I], gu[:, I:]
        h = torch.nn.functional.silu(g) * u
        h = V(h, silu_off(g, h)).round(dtype)
        ys = h.matmul(dn.T)
        y.v.index_add_(0, t, c * ys.v), y.off.index_add_(0, t, c * ys.off), size_y.index_add_(0, t, c * (ys.v.abs() + ys.off))
        q = [torch.from_numpy(Q.dequantize(*Q.quantize(v.cpu().numpy()))).cuda() for v in (g, u)]
        gh = GY.matmul(dn)
        s = torch.sigmoid(q[0])
        qh = q[0] * s * q[1]
        slope = q[1] * s * (1 + q[0] * (1 - s))
        most = q[1].abs() * s * (1 + q[0].abs() * (1 - s))       # its terms one by one
        f = (16 * (1 + q[0].abs()) + 4) * 2.0 ** -24
        gh_size = gh.v.abs() + gh.off
        gg = V(c * gh.v * slope, c * (gh.off * slope.abs() + f * gh_size * most))
        gu_ = V(c * gh.v * q[0] * s, c * (q[0].abs() * s * (gh.off + f * gh_size)))
        ggu = V(torch.cat([gg.v, gu_.v], 1), torch.cat([gg.off, gu_.off], 1)).round(dtype)
        ch = V(c * qh, c * f * qh.abs()).round(dtype)
        terms = gh_size * qh.abs()
        gw.v[t, r] = (gh.v * qh).sum(1)
        gw.off[t, r] = (gh.off * qh.abs() + (f + I * 2.0 ** -24) * terms).sum(1)
        for out, got in ((gdown, GY.T.matmul(ch)), (ggate_up, ggu.T.matmul(X))):
            got = got.round(dtype)
            out.v[e], out.off[e] = got.v, got.off
        gxs = ggu.matmul(up)
        gx.v.index_add_(0, t, gxs.v), gx.off.index_add_(0, t, gxs.off), size_x.index_add_(0, t, gxs.v.abs() + gxs.off)
    y.off += 2 * k * 2.0 ** -24 * size_y
    gx.off += k * 2.0 ** -24 * size_x
    return y.round(dtype), gx.round(dtype), gw, ggate_up, gdown


def near(got, want, name):
    bad = ~((got.double() - want.v).abs() <= want.off)
    assert not bool(bad.any()), (name, bad.nonzero()[:3], got[bad][:3], want.v[bad][:3], want.off[bad][:3])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("case", CASES)
def test_against_64_bits(case, kind):
    x, ids, w, gate_up, down, gy = inputs(*case, kind)
    leaves = [t.clone().requires_grad_() for t in (x, w, gate_up, down)]
    y = m.si_moe_experts(leaves[0], ids, *leaves[1:])
    assert torch.equal(y, m.si_moe_experts(x, ids, w, gate_up, down))
    got = y.detach(), *torch.autograd.grad(y, leaves, gy)
    for a, b, name in zip(got, expected(x, ids, w, gate_up, down, gy), ("y", "gx", "gw", "ggate_up", "gdown")):
        near(a, b, name)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("case", CASES)
def test_equals_the_calls_that_it_is_made_of(case, kind):
    x, ids, w, gate_up, down, gy = inputs(*case, kind, seed=1)
    E = gate_up.shape[0]
    order, position, offsets = m.si_moe_sort(ids, E)
    xs = m.si_moe_gather(x, position, offsets)
    h, kept = m.si_moe_gateup(xs, gate_up, offsets, keep=True)
    y = m.si_moe_combine(m.si_moe_matmul(h, down, offsets, dtype=torch.float32), position, w, dtype=x.dtype)
    gys = m.si_moe_gather(gy, position, offsets)
    ggu, wh, gw = m.si_moe_down_backward(gys, down, kept, offsets, w, order)
    gxs = m.si_moe_matmul(ggu, gate_up.transpose(1, 2), offsets, dtype=torch.float32)
    ggate_up, gdown = m.si_moe_matmul_grad_w(ggu, xs, offsets), m.si_moe_matmul_grad_w(gys, wh, offsets)
    want = y, m.si_moe_gather_backward(gxs, position, dtype=x.dtype), gw, ggate_up, gdown
    leaves = [t.clone().requires_grad_() for t in (x, w, gate_up, down)]
    out = m.si_moe_experts(leaves[0], ids, *leaves[1:])
    got = out, *torch.autograd.grad(out, leaves, gy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for i in range(4):                           # one leaf alone
        some = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, w, gate_up, down))]
        out = m.si_moe_experts(some[0], ids, *some[1:])
        assert torch.equal(torch.autograd.grad(out, some[i], gy)[0], want[1 + i])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts,H,I", [([1], 8, 8), ([3, 0, 5], 72, 40), ([16, 17, 2], 64, 136), ([200, 0, 130], 136, 264),
                                        ([100, 3], 72, 40), ([65], 64, 512)])
def test_gate_and_up_product(counts, H, I, kind):
    """Codes and scales equal to the exact sums', h within its bound; rows of no expert zero."""
    dtype, head, tail = TYPES[kind], 1, 3
    R, g = head + sum(counts) + tail, torch.Generator(device="cuda").manual_seed(I)
    xs = torch.randint(-2, 3, (R, H), generator=g, device="cuda").to(dtype)
    gate_up = torch.randint(-2, 3, (len(counts), 2 * I, H), generator=g, device="cuda").to(dtype) / 16
    offsets = torch.tensor([head + sum(counts[:e]) for e in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    gu = m.si_moe_matmul(xs, gate_up, offsets, dtype=torch.float32)
    h, (codes, scales) = m.si_moe_gateup(xs, gate_up, offsets, keep=True)
    assert torch.equal(h, m.si_moe_gateup(xs, gate_up, offsets))
    parts = [Q.quantize(v.double().cpu().numpy()) for v in (gu[:, :I], gu[:, I:])]
    assert np.array_equal(codes.cpu().numpy(), np.concatenate([p[0] for p in parts], 1))
    assert np.array_equal(scales.cpu().numpy(), np.concatenate([p[1] for p in parts], 1))
    gd, ud = gu[:, :I].double(), gu[:, I:].double()
    want = torch.nn.functional.silu(gd) * ud
    near(h, V(want, silu_off(gd, want)).round(dtype), "h")
    assert not bool(h[:head].any()) and not bool(h[R - tail:].any()) and not bool(codes[R - tail:].any())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts,H,I", [([1], 8, 8), ([3, 0, 5], 72, 40), ([16, 17, 2], 64, 136), ([200, 0, 130], 136, 264),
                                        ([100, 3], 72, 40), ([290], 64, 512)])
def test_gradient_behind_the_down_product(counts, H, I, kind):
    """Equal to the steps: gh = gy down in fp32 is exact here (whole numbers), so
    si_swiglu_backward of fp32 rows differs by its logistic function alone: an error of
    2 (16 (1 + |g|) + 4) 2^-24 of every term, and each result rounded to its type once."""
    dtype, head, tail = TYPES[kind], 2, 3
    R, E, g_ = head + sum(counts) + tail, len(counts), torch.Generator(device="cuda").manual_seed(I)
    gy = torch.randint(-2, 3, (R, H), generator=g_, device="cuda").to(dtype)
    down = torch.randint(-2, 3, (E, H, I), generator=g_, device="cuda").to(dtype)
    gu = torch.randn(R, 2 * I, generator=g_, device="cuda") * 3
    offsets = torch.tensor([head + sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32, device="cuda")
    _, kept = m.si_swiglu(gu, keep=True)
    order = torch.randperm(R, generator=g_, device="cuda").to(torch.int32)
    order[head + 1] = -1                         # a row without a pair
    w = torch.randn(R, generator=g_, device="cuda")
    gh = m.si_moe_matmul(gy, down.transpose(1, 2), offsets, dtype=torch.float32)
    q = m.si_dequantize_mxint8(*(t.reshape(R * 2, -1) for t in kept), torch.float32).double()
    qg, qu = q[0::2], q[1::2]
    f = 2 * (16 * (1 + qg.abs()) + 4) * 2.0 ** -24
    for args in ((None, None), (w, None), (w, order)):
        want = list(m.si_swiglu_backward(gh, kept, *args))
        for t in want[:2]:                       # rows of no expert: zeros
            t[:head], t[R - tail:] = 0, 0
        got = m.si_moe_down_backward(gy, down, kept, offsets, *args)
        c = torch.ones_like(w) if args[0] is None else w if args[1] is None else torch.where(order >= 0, w[order.long().clamp(min=0)], 0 * w)
        a, s = (c[:, None] * gh).abs().double(), torch.sigmoid(qg)
        sizes = torch.cat([a * qu.abs() * s * (1 + qg.abs() * (1 - s)), a * qg.abs() * s], 1), (c[:, None] * qg * s * qu).abs()
        for x, y, size, ff in zip(got, want, sizes, (torch.cat([f, f], 1), f)):
            near(x, V(y.double(), ff * size).round(dtype), "ggu or wh")
        if args[0] is None:
            assert got[2] is None
        else:
            terms = (gh.double() * qg * s * qu).abs()
            off = (((f + 2 * I * 2.0 ** -24) * terms).sum(1))
            if args[1] is not None:
                off = torch.zeros_like(off).index_copy_(0, order[order >= 0].long(), off[order >= 0])
            near(got[2], V(want[2].double(), off), "gw")


def test_gradients_against_differences():
    """The loss <gy, y> in 64 bits with g and u replaced by their kept values plus what
    a change of x adds: its central differences along random directions."""
    case = (6, 2, 3, 64, 32, 0.0)
    x, ids, w, gate_up, down, gy = inputs(*case, "bf16", seed=3)
    leaves = [t.clone().requires_grad_() for t in (x, w, gate_up, down)]
    grads = torch.autograd.grad(m.si_moe_experts(leaves[0], ids, *leaves[1:]), leaves, gy)
    (T, k), I = ids.shape, gate_up.shape[1] // 2
    e, base = ids.long(), [t.double() for t in (x, w, gate_up, down)]
    gu0 = torch.einsum("th,tkih->tki", base[0], base[2][e])
    kept = [torch.from_numpy(Q.dequantize(*Q.quantize(v.reshape(T * k, I).cpu().numpy()))).cuda().reshape(T, k, I)
            for v in (gu0[..., :I], gu0[..., I:])]
    shift = torch.cat(kept, 2) - gu0

    def loss(x, w, gate_up, down):
        gu = torch.einsum("th,tkih->tki", x, gate_up[e]) + shift
        h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
        return (gy.double() * torch.einsum("tk,tkhi,tki->th", w, down[e], h)).sum()

    r = torch.Generator(device="cuda").manual_seed(11)
    bounds = expected(x, ids, w, gate_up, down, gy)[1:]
    for i, grad in enumerate(grads):
        d = torch.randn(base[i].shape, generator=r, device="cuda", dtype=torch.float64)
        eps = 2.0 ** -12
        up, lo = ([t + s * eps * d if j == i else t for j, t in enumerate(base)] for s in (1, -1))
        diff = (loss(*up) - loss(*lo)) / (2 * eps)
        got = (grad.double() * d).sum()
        # the gradient's own bound along d, and eps^2 times a third derivative of at most the size seen here
        assert abs(diff - got) <= (bounds[i].off * d.abs()).sum() + eps ** 2 * (grad.double().abs() * d.abs()).sum() * 100


def test_captured_and_replayed_beside_a_second_graph():
    case = (20, 2, 4, 64, 32, 0.1)
    x, ids, w, gate_up, down, gy = inputs(*case, "bf16", seed=4)
    ws = m.workspace(m.moe_experts_workspace_bytes(20, 2, gate_up))
    graphs = []
    for _ in range(2):
        leaves = [t.clone().requires_grad_() for t in (x, w, gate_up, down)]
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):            # autograd's own first pass outside the capture
            torch.autograd.grad(m.si_moe_experts(leaves[0], ids, *leaves[1:], ws=ws), leaves, gy)
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            y = m.si_moe_experts(leaves[0], ids, *leaves[1:], ws=ws)
            out = y, *torch.autograd.grad(y, leaves, gy)
        graphs.append((graph, leaves, out))
    other = inputs(*case, "bf16", seed=5)
    ids.copy_(other[1])
    gy.copy_(other[5])
    for i, (graph, leaves, out) in enumerate(graphs):
        with torch.no_grad():
            for t, v in zip(leaves, (other[0], other[2] + i, other[3], other[4])):
                t.copy_(v)
    for graph, _, _ in graphs:
        graph.replay()
    for i, (_, leaves, out) in enumerate(graphs):
        fresh = [t.detach().clone().requires_grad_() for t in leaves]
        y = m.si_moe_experts(fresh[0], ids, *fresh[1:])
        assert all(torch.equal(a, b) for a, b in zip(out, (y, *torch.autograd.grad(y, fresh, gy))))
    assert m.si_workspace_status(ws) == m.SI_OK


def test_on_another_stream():
    x, ids, w, gate_up, down, gy = inputs(30, 2, 4, 64, 32, 0.1, "f16", seed=6)
    want = m.si_moe_experts(x, ids, w, gate_up, down)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    leaves = [t.clone().requires_grad_() for t in (x, w, gate_up, down)]
    side.wait_stream(torch.cuda.current_stream())
    y = m.si_moe_experts(leaves[0], ids, *leaves[1:], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)
    a = torch.autograd.grad(y, leaves, gy)
    fresh = [t.detach().clone().requires_grad_() for t in leaves]
    b = torch.autograd.grad(m.si_moe_experts(fresh[0], ids, *fresh[1:]), fresh, gy)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    x, ids, w, gate_up, down, _ = inputs(4, 2, 3, 64, 32, 0, "bf16")
    bad = [(x[0], ids, w, gate_up, down), (x, ids[:3], w, gate_up, down), (x, ids, w[:, :1], gate_up, down),
           (x, ids, w, gate_up.half(), down), (x, ids, w, gate_up[:, :63], down), (x, ids, w, gate_up, down[:2]),
           (x, ids, w.half(), gate_up, down), (x, ids.long(), w, gate_up, down), (x.float(), ids, w, gate_up.float(), down.float()),
           (x, ids, w, gate_up.transpose(1, 2).contiguous().transpose(1, 2), down)]
    for args in bad:
        with pytest.raises(ValueError):
            m.si_moe_experts(*args)
    off = torch.tensor([0, 2, 5, 8], dtype=torch.int32, device="cuda")
    xs = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: m.si_moe_matmul(xs, gate_up, off[:3]), lambda: m.si_moe_matmul(xs, gate_up, off.long()),
                 lambda: m.si_moe_matmul(xs[:, :56], gate_up, off), lambda: m.si_moe_matmul(xs[:, 4:60], gate_up[:, :, :56], off),
                 lambda: m.si_moe_matmul(xs, gate_up, off, dtype=torch.float16), lambda: m.si_moe_matmul(xs.t(), gate_up, off),
                 lambda: m.si_moe_matmul(xs, gate_up[:, :, ::2], off), lambda: m.si_moe_matmul(xs, gate_up, off, out=xs),
                 lambda: m.si_moe_matmul(xs, gate_up[:, :60], off), lambda: m.si_moe_matmul_grad_w(xs[:7], xs, off),
                 lambda: m.si_moe_matmul_backward(xs, xs, gate_up[:, :32], off), lambda: m.si_moe_matmul(xs[:1].expand(8, 64), gate_up, off),
                 lambda: m.si_swiglu(xs[:, :63]), lambda: m.si_swiglu_backward(xs, (xs, xs)),
                 lambda: m.si_quantize_mxint8(xs.int()), lambda: m.si_dequantize_mxint8(*m.si_quantize_mxint8(xs), dtype=torch.int32)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("hidden", [1, 6, 8, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_fp32_rows_combined_into_another_type(hidden, dtype):
    """The same sums as in fp32, rounded once; gradients as through fp32."""
    g = torch.Generator(device="cuda").manual_seed(hidden)
    ids = torch.randint(0, 6, (33, 3), generator=g, device="cuda", dtype=torch.int32)
    _, position, _ = m.si_moe_sort(ids, 5)
    ys, w = torch.randn(99, hidden, generator=g, device="cuda"), torch.randn(33, 3, generator=g, device="cuda")
    assert torch.equal(m.si_moe_combine(ys, position, w, dtype=dtype), m.si_moe_combine(ys, position, w).to(dtype))
    assert torch.equal(m.si_moe_gather_backward(ys, position, dtype=dtype), m.si_moe_gather_backward(ys, position).to(dtype))
    a, b = (t.clone().requires_grad_() for t in (ys, w))
    gy = torch.randn(33, hidden, generator=g, device="cuda").to(dtype)
    got = torch.autograd.grad(m.si_moe_combine(a, position, b, dtype=dtype), (a, b), gy)
    want = torch.autograd.grad(m.si_moe_combine(a, position, b), (a, b), gy.float())
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    with pytest.raises(ValueError):
        m.si_moe_combine(ys.to(dtype), position, w, dtype=torch.float32)
