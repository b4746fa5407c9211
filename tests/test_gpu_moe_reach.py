"""Calls of the products of sorted rows, of the 8-bit activations and of the experts
that the documentation allows and no other test makes: offsets beyond 32 bits, many
experts, calls on two streams at once, a process whose first calls are captured,
gradients that autograd hands on unaligned or expanded."""
import os
import subprocess
import sys

import pytest
import torch

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()
    yield
    torch.cuda.empty_cache()


def room(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < nbytes:
        pytest.skip(f"needs {nbytes >> 30} GB")


def whole(g, *shape):
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(torch.bfloat16)


def int32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- offsets beyond 2^31 values --------------------------------------------------

def test_product_and_gradients_beyond_32_bits():
    """2.2e9 values of x and of y: the last rows, one expert's own, equal the same rows alone;
    whole numbers, so every sum is exact."""
    R, n, k, tail = 1080000, 2056, 2056, 300
    room(40 << 30)
    assert R * k > 2 ** 31 and (R - tail) * n > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = torch.zeros(R, k, dtype=torch.bfloat16, device="cuda"), whole(g, 3, n, k)
    x[-tail:] = whole(g, tail, k)
    offsets, last = int32(0, 5, R - tail, R), x[-tail:].clone()
    y = m.si_moe_matmul(x, w, offsets)
    assert torch.equal(y[-tail:], m.si_moe_matmul(last, w[2:], int32(0, tail))) and not y[:-tail].any()
    gw = m.si_moe_matmul_grad_w(y, x, offsets)
    assert torch.equal(gw[2], m.si_moe_matmul_grad_w(y[-tail:].clone(), last, int32(0, tail))[0]) and not gw[:2].any()
    gx = m.si_moe_matmul(x, w.transpose(1, 2), offsets, out=y)
    assert torch.equal(gx[-tail:], m.si_moe_matmul(last, w[2:].transpose(1, 2), int32(0, tail)))


def test_matrices_beyond_32_bits():
    """2.2e9 values of w and of its gradient: the last expert's."""
    E, n, k = 66, 4104, 8200
    room(24 << 30)
    assert (E - 1) * n * k > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.zeros(E, n, k, dtype=torch.bfloat16, device="cuda")
    w[-1] = whole(g, n, k)
    for rows in (5, E * 20):                     # features on the lanes of one SM, of two
        x, gy = whole(g, rows, k), whole(g, rows, n)
        offsets = torch.full((E + 1,), 2, dtype=torch.int32, device="cuda")
        offsets[0], offsets[-1] = 0, rows
        one = int32(0, rows - 2)
        assert torch.equal(m.si_moe_matmul(x, w, offsets)[2:], m.si_moe_matmul(x[2:].clone(), w[-1:], one))
        gx, gw = m.si_moe_matmul_backward(gy, x, w, offsets)
        want = m.si_moe_matmul_backward(gy[2:].clone(), x[2:].clone(), w[-1:], one)
        assert torch.equal(gx[2:], want[0]) and torch.equal(gw[-1], want[1][0]) and not gw[1:-1].any()
        del gw


def test_activations_beyond_32_bits():
    """4.4e9 codes: the last rows equal the same rows alone."""
    R, I, tail = 1080000, 2056, 70
    room(60 << 30)
    assert R * 2 * I > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(3)
    gu = torch.zeros(R, 2 * I, dtype=torch.bfloat16, device="cuda")
    gu[-tail:] = torch.randn(tail, 2 * I, generator=g, device="cuda").to(torch.bfloat16)
    last = gu[-tail:].clone()
    h, kept = m.si_swiglu(gu, keep=True)
    want = m.si_swiglu(last, keep=True)
    assert torch.equal(h[-tail:], want[0]) and not h[:-tail].any()
    assert torch.equal(kept[0][-tail:], want[1][0]) and torch.equal(kept[1][-tail:], want[1][1])
    w = torch.randn(R, generator=g, device="cuda")
    back = m.si_swiglu_backward(h, kept, w)
    one = m.si_swiglu_backward(want[0], want[1], w[-tail:].clone())
    assert all(torch.equal(a[-tail:], b) for a, b in zip(back, one))
    del back, h
    codes, scales = m.si_quantize_mxint8(gu)
    want = m.si_quantize_mxint8(last)
    assert torch.equal(codes[-tail:], want[0]) and torch.equal(scales[-tail:], want[1])
    assert torch.equal(m.si_dequantize_mxint8(codes, scales, out=gu)[-tail:], m.si_dequantize_mxint8(*want))


# ---- many experts, one expert, long sums ------------------------------------------

@pytest.mark.parametrize("E,R", [(1024, 600), (1024, 20000), (1, 700), (1, 3)])
def test_numbers_of_experts(E, R):
    n, k = 24, 40
    g = torch.Generator(device="cuda").manual_seed(E + R)
    x, w, gy = whole(g, R, k), whole(g, E, n, k), whole(g, R, n)
    cut = torch.randint(0, R + 1, (E - 1,), generator=g, device="cuda").sort().values
    offsets = torch.cat([int32(0), cut.int(), int32(R)])
    e = torch.bucketize(torch.arange(R, device="cuda"), offsets[1:].long(), right=True)
    want = torch.einsum("rk,rnk->rn", x.double(), w.double()[e])
    assert torch.equal(m.si_moe_matmul(x, w, offsets), want.to(torch.bfloat16))
    gw = torch.zeros(E, n, k, dtype=torch.float64, device="cuda")
    gw.index_add_(0, e, gy.double()[:, :, None] * x.double()[:, None])
    assert torch.equal(m.si_moe_matmul_grad_w(gy, x, offsets, dtype=torch.float32), gw.float())


@pytest.mark.parametrize("rows", [9, 260])
def test_long_sums(rows):
    """65544 columns: 1025 stages, sums of whole numbers below 2^24."""
    n, k = 136, 65544
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w = whole(g, rows, k), whole(g, 2, n, k)
    offsets = int32(0, rows // 3, rows)
    want = torch.cat([x[:rows // 3].double() @ w[0].double().T, x[rows // 3:].double() @ w[1].double().T])
    for out in (torch.bfloat16, torch.float32):
        assert torch.equal(m.si_moe_matmul(x, w, offsets, dtype=out), want.to(out))
    wt = w.transpose(1, 2).contiguous()
    gw = m.si_moe_matmul_grad_w(wt[0], wt[0], int32(0, 40000, k), dtype=torch.float32)
    assert torch.equal(gw[1], (wt[0, 40000:].double().T @ wt[0, 40000:].double()).float())


# ---- streams, captures --------------------------------------------------------------

def test_two_streams_at_once():
    """Steps on two streams, many in flight, each with its own inputs: as alone."""
    def inputs(seed, T):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids = torch.randint(0, 9, (T, 2), generator=g, device="cuda", dtype=torch.int32)
        x, gate_up, down = whole(g, T, 136), whole(g, 8, 144, 136) / 8, whole(g, 8, 136, 72) / 8
        return [x, torch.rand(T, 2, generator=g, device="cuda"), gate_up, down], ids, whole(g, T, 136)

    def step(leaves, ids, gy, stream=None):
        leaves = [t.detach().requires_grad_() for t in leaves]
        y = m.si_moe_experts(leaves[0], ids, *leaves[1:], stream=stream)
        return [y.detach(), *torch.autograd.grad(y, leaves, gy)]

    sets = [inputs(1, 30), inputs(2, 600)]
    want = [step(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    for _ in range(10):
        for i, s in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(*s))
    torch.cuda.synchronize()
    for runs, w in zip(got, want):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(r, w))


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: nothing that a capture forbids
    happens in them."""
    code = """
import torch, moe_decode_ffn_gb300 as m
def step(T):
    x, ids, w, gu, dn, gy, off = sets[T]
    leaves = [t.detach().requires_grad_() for t in (x, w, gu, dn)]
    y = m.si_moe_experts(leaves[0], ids, *leaves[1:])
    o, p, f = m.si_moe_sort(ids, 4)
    xs = m.si_moe_gather(x, p, f)
    z = m.si_moe_matmul(xs, gu, f, dtype=torch.float32)
    h, kept = m.si_swiglu(z, keep=True)
    q = m.si_quantize_mxint8(h)
    return (y, *torch.autograd.grad(y, leaves, gy), *m.si_moe_matmul_backward(z.to(x.dtype), xs, gu, f),
            *m.si_swiglu_backward(h, kept, w, o), m.si_dequantize_mxint8(*q), m.si_moe_matmul_grad_w(z.to(x.dtype), xs, f, dtype=torch.float32))
sets = {}
for T in (8, 90):
    sets[T] = (torch.randn(T, 64, device="cuda").to(torch.bfloat16), torch.randint(0, 5, (T, 2), device="cuda", dtype=torch.int32),
               torch.rand(T, 2, device="cuda"), (torch.randn(4, 80, 64, device="cuda") * 0.1).to(torch.bfloat16),
               (torch.randn(4, 64, 40, device="cuda") * 0.1).to(torch.bfloat16), torch.randn(T, 64, device="cuda").to(torch.bfloat16), None)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = [step(T) for T in sets]
graph.replay()
torch.cuda.synchronize()
for T, o in zip(sets, out):
    assert all(torch.equal(a, b) for a, b in zip(o, step(T)))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


# ---- gradients as autograd hands them on ------------------------------------------------

def test_gradients_expanded_or_unaligned():
    """The sum's gradient is one expanded value; that of a part of a flat tensor starts at
    an odd place: the same as from rows of their own."""
    g = torch.Generator(device="cuda").manual_seed(5)
    T, H = 12, 72
    x, ids = whole(g, T, H), torch.randint(0, 3, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    w, gate_up, down = torch.rand(T, 2, generator=g, device="cuda"), whole(g, 3, 80, H) / 8, whole(g, 3, H, 40) / 8
    flat = whole(g, T * 80 + 1)
    offsets = int32(0, 3, 4, T)

    def run(loss, f):
        leaves = [t.clone().requires_grad_() for t in (x, w, gate_up, down)]
        return torch.autograd.grad(loss(f(leaves)), leaves, allow_unused=True)

    for f in (lambda v: m.si_moe_experts(v[0], ids, *v[1:]), lambda v: m.si_moe_matmul(v[0], v[2], offsets),
              lambda v: m.si_swiglu(v[0])):
        n = f((x, w, gate_up, down)).numel()
        parts = flat[:n + 1].clone()
        pairs = [(lambda y: y.sum(), lambda y: (y * torch.ones_like(y)).sum()),
                 (lambda y: (torch.cat([torch.zeros(1, device="cuda", dtype=y.dtype), y.reshape(-1)]) * parts).sum(),
                  lambda y: (y * parts[1:].reshape(y.shape).clone()).sum())]
        for odd, even in pairs:
            for a, b in zip(run(odd, f), run(even, f)):
                assert (a is None and b is None) or torch.equal(a, b)
