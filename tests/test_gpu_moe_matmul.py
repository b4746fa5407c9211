"""Products of sorted rows with their experts' matrices, and their gradients.

With integers from -2 to 2 every product and every partial sum is an integer below
2^24, exact in fp32 in any order: the results have to be the integers' product,
rounded once to the output's type. With normal values a sum of n terms is off by at
most n 2^-23 of the terms' magnitudes (an addition on the tensor cores may
truncate: a whole unit in the last place) and by half a unit of its type on top."""
import pytest
import torch

import moe_decode_ffn_gb300 as m

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# rows of every expert, rows before the first and behind the last expert's, n, k.
# Up to 16 rows an expert on average the features go on the lanes, else the rows.
CASES = [
    ([1], 0, 0, 8, 8),
    ([0, 0, 3, 0], 0, 0, 136, 72),
    ([1, 1, 0, 2], 2, 5, 256, 64),
    ([16, 17, 15, 0, 33], 0, 0, 264, 1448),
    ([40, 0, 1], 0, 1, 1000, 200),
    ([17], 0, 0, 8, 8),
    ([128], 0, 0, 256, 64),
    ([5, 130, 0, 257, 16], 0, 37, 520, 712),
    ([300, 1, 127, 129], 3, 300, 264, 136),
    ([0, 640], 0, 0, 1000, 1448),
    ([64] * 7, 0, 0, 128, 256),
]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def offsets_of(counts, head):
    at = [head]
    for c in counts:
        at.append(at[-1] + c)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def whole(g, *shape, dtype):
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dtype)


def reference(x, w, counts, head):
    """fp64, zero rows outside the experts'."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    at = head
    for e, c in enumerate(counts):
        y[at:at + c] = x[at:at + c].double() @ w[e].double().T
        at += c
    return y


def reference_grad(gy, x, counts, head):
    gw = torch.zeros(len(counts), gy.shape[1], x.shape[1], dtype=torch.float64, device="cuda")
    at = head
    for e, c in enumerate(counts):
        gw[e] = gy[at:at + c].double().T @ x[at:at + c].double()
        at += c
    return gw


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts,head,tail,n,k", CASES)
def test_products_of_integers_are_exact(counts, head, tail, n, k, kind):
    dtype, R = TYPES[kind], head + sum(counts) + tail
    g = torch.Generator(device="cuda").manual_seed(n + k + R)
    x, w = whole(g, R, k, dtype=dtype), whole(g, len(counts), n, k, dtype=dtype)
    offsets, want = offsets_of(counts, head), reference(x, w, counts, head)
    for out in (dtype, torch.float32):
        assert torch.equal(m.si_moe_matmul(x, w, offsets, dtype=out), want.to(out))
        columns = w.transpose(1, 2).contiguous().transpose(1, 2)
        assert torch.equal(m.si_moe_matmul(x, columns, offsets, dtype=out), want.to(out))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts,head,tail,n,k", CASES)
def test_gradients_of_integers_are_exact(counts, head, tail, n, k, kind):
    dtype, R = TYPES[kind], head + sum(counts) + tail
    g = torch.Generator(device="cuda").manual_seed(n + k + R)
    x, w, gy = whole(g, R, k, dtype=dtype), whole(g, len(counts), n, k, dtype=dtype), whole(g, R, n, dtype=dtype)
    offsets = offsets_of(counts, head)
    gx, gw = m.si_moe_matmul_backward(gy, x, w, offsets)
    assert torch.equal(gx, reference(gy, w.transpose(1, 2), counts, head).to(dtype))
    want = reference_grad(gy, x, counts, head)
    assert torch.equal(gw, want.to(dtype))
    assert torch.equal(m.si_moe_matmul_grad_w(gy, x, offsets, dtype=torch.float32), want.float())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts,head,tail,n,k", CASES)
def test_normal_values_against_64_bits(counts, head, tail, n, k, kind):
    dtype, R = TYPES[kind], head + sum(counts) + tail
    g = torch.Generator(device="cuda").manual_seed(R)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, w, gy, offsets = draw(R, k), draw(len(counts), n, k), draw(R, n), offsets_of(counts, head)

    def near(got, want, size, terms):
        half = torch.finfo(got.dtype).eps / 2
        bound = terms * 2.0 ** -23 * size * (1 + half) + half * want.abs() + torch.finfo(got.dtype).smallest_normal * half * 2
        assert bool(((got.double() - want).abs() <= bound).all())

    for out in (dtype, torch.float32):
        near(m.si_moe_matmul(x, w, offsets, dtype=out), reference(x, w, counts, head),
             reference(x.abs(), w.abs(), counts, head), k)
        near(m.si_moe_matmul_grad_w(gy, x, offsets, dtype=out), reference_grad(gy, x, counts, head),
             reference_grad(gy.abs(), x.abs(), counts, head), max(counts))


@pytest.mark.parametrize("counts", [[3, 2, 0, 5], [30, 47, 0, 129]])
def test_not_a_number_stays_where_it_belongs(counts):
    """Rows of no expert hold NaN and infinities and are not read; a NaN in a row or a
    matrix reaches that row's, that matrix' outputs alone."""
    head, tail, n, k = 2, 7, 264, 136
    R, offsets = head + sum(counts) + tail, offsets_of(counts, head)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w, gy = (whole(g, *s, dtype=torch.bfloat16) for s in ((R, k), (len(counts), n, k), (R, n)))
    want, want_x = reference(x, w, counts, head), reference(gy, w.transpose(1, 2), counts, head)
    want_w = reference_grad(gy, x, counts, head)
    for t in (x, gy):
        t[:head], t[R - tail:] = float("nan"), float("inf")
    gx, gw = m.si_moe_matmul_backward(gy, x, w, offsets)
    assert torch.equal(m.si_moe_matmul(x, w, offsets, dtype=torch.float32), want.float())
    assert torch.equal(gx, want_x.to(torch.bfloat16)) and torch.equal(gw, want_w.to(torch.bfloat16))
    row = head + counts[0]                       # the first row of expert 1
    x[row, 5], gy[row, 9] = float("nan"), float("inf")
    w[3, 17, 33] = float("nan")
    y, (gx, gw) = m.si_moe_matmul(x, w, offsets), m.si_moe_matmul_backward(gy, x, w, offsets)
    last = slice(head + sum(counts[:3]), head + sum(counts))
    bad = torch.zeros(R, n, dtype=torch.bool, device="cuda")
    bad[row], bad[last, 17] = True, True
    assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], want.to(y.dtype)[~bad])
    bad = torch.zeros(R, k, dtype=torch.bool, device="cuda")
    bad[row], bad[last, 33] = True, True
    assert bool(torch.isfinite(gx[~bad]).all()) and torch.equal(gx[~bad], want_x.to(gx.dtype)[~bad])
    assert not bool(torch.isfinite(gx[row]).any()) and bool(torch.isnan(gx[last, 33]).all())
    bad = torch.zeros(len(counts), n, k, dtype=torch.bool, device="cuda")
    bad[1, :, 5], bad[1, 9] = True, True
    assert not bool(torch.isfinite(gw[bad]).any()) and torch.equal(gw[~bad], want_w.to(gw.dtype)[~bad])


@pytest.mark.parametrize("counts", [[3, 2, 0, 5], [30, 47, 0, 129]])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_strided_rows_and_matrices(counts, out):
    R, n, k, E = sum(counts) + 3, 72, 200, len(counts)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = whole(g, R, k + 24, dtype=torch.bfloat16)[:, 8:8 + k]
    w = whole(g, E, 2 * n, k + 8, dtype=torch.bfloat16)[:, n:, :k]       # the up rows of a fused matrix
    offsets, want = offsets_of(counts, 0), reference(x, w, counts, 0)
    y = torch.full((R + 1, n + 16), 7.0, dtype=out, device="cuda")
    assert m.si_moe_matmul(x, w, offsets, out=y[:R, 8:8 + n]) is not None
    assert torch.equal(y[:R, 8:8 + n], want.to(out))
    y[:R, 8:8 + n] = 7.0
    assert bool((y == 7.0).all())                # nothing beside the rows was written
    gy = whole(g, R, n + 8, dtype=torch.bfloat16)[:, :n]
    gx, gw = m.si_moe_matmul_backward(gy, x, w, offsets)
    assert torch.equal(gx, reference(gy, w.transpose(1, 2), counts, 0).to(gx.dtype))
    assert torch.equal(gw, reference_grad(gy, x, counts, 0).to(gw.dtype))


def test_bounds_that_are_out_of_order_or_outside():
    """Clamped into the rows and to a running maximum: no access leaves the tensors."""
    R, n, k = 100, 64, 64
    g = torch.Generator(device="cuda").manual_seed(7)
    x, w, gy = (whole(g, *s, dtype=torch.bfloat16) for s in ((R, k), (4, n, k), (R, n)))
    odd = torch.tensor([-5, 30, 20, 2000000000, 90], dtype=torch.int32, device="cuda")
    even = torch.tensor([0, 30, 30, 100, 100], dtype=torch.int32, device="cuda")
    assert torch.equal(m.si_moe_matmul(x, w, odd), m.si_moe_matmul(x, w, even))
    assert torch.isfinite(m.si_moe_matmul_grad_w(gy, x, odd)).all()


def test_without_rows():
    w = torch.ones(3, 16, 24, dtype=torch.bfloat16, device="cuda")
    x, gy = (torch.empty(0, c, dtype=torch.bfloat16, device="cuda") for c in (24, 16))
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert m.si_moe_matmul(x, w, offsets).shape == (0, 16)
    gx, gw = m.si_moe_matmul_backward(gy, x, w, offsets)
    assert gx.shape == (0, 24) and gw.shape == (3, 16, 24) and not bool(gw.any())


@pytest.mark.parametrize("T", [4, 64])
def test_through_autograd(T):
    E, k, n, H = 6, 2, 40, 72
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(0, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)   # E: dropped
    _, position, offsets = m.si_moe_sort(ids, E)
    x, w = whole(g, T, H, dtype=torch.bfloat16), whole(g, E, n, H, dtype=torch.bfloat16)
    xs, gy = m.si_moe_gather(x, position, offsets), whole(g, T * k, n, dtype=torch.bfloat16)
    a, b = xs.clone().requires_grad_(), w.clone().requires_grad_()
    y = m.si_moe_matmul(a, b, offsets)
    assert torch.equal(y, m.si_moe_matmul(xs, w, offsets))
    y.backward(gy)
    gx, gw = m.si_moe_matmul_backward(gy, xs, w, offsets)
    assert torch.equal(a.grad, gx) and torch.equal(b.grad, gw)
    only = torch.autograd.grad(m.si_moe_matmul(xs, b, offsets, dtype=torch.float32), b, gy.float())[0]
    assert torch.equal(only, gw)
    with torch.no_grad():
        assert not m.si_moe_matmul(a, b, offsets).requires_grad
    with pytest.raises(ValueError):
        m.si_moe_matmul(a, b, offsets, out=torch.empty_like(gy))


def test_streams_graphs_and_the_status_word():
    counts, n, k = [20, 0, 300, 64], 264, 136
    R, offsets = sum(counts), offsets_of(counts, 0)
    g = torch.Generator(device="cuda").manual_seed(9)
    x, w, gy = (whole(g, *s, dtype=torch.bfloat16) for s in ((R, k), (4, n, k), (R, n)))
    want = m.si_moe_matmul(x, w, offsets), *m.si_moe_matmul_backward(gy, x, w, offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.si_moe_matmul(x, w, offsets, stream=side), *m.si_moe_matmul_backward(gy, x, w, offsets, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws, graph = m.workspace(m.moe_matmul_workspace_bytes()), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.si_moe_matmul(x, w, offsets, ws=ws), *m.si_moe_matmul_backward(gy, x, w, offsets, ws=ws)
    for seed in (1, 2):
        x.copy_(whole(g, R, k, dtype=torch.bfloat16))
        offsets.copy_(offsets_of([seed, 200, 100, 50], 0))
        graph.replay()
        want = m.si_moe_matmul(x, w, offsets), *m.si_moe_matmul_backward(gy, x, w, offsets)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert m.si_workspace_status(ws) == m.SI_OK


@pytest.mark.parametrize("call", ["moe", "mxfp4"])
def test_first_calls_of_a_new_thread(call):
    """A thread that has made no CUDA call has no current context yet."""
    import threading
    x, w = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 8, 64, dtype=torch.bfloat16, device="cuda")
    offsets, q = offsets_of([4], 0), m.si_quantize_mxfp4(x)
    torch.cuda.synchronize()
    got = []
    run = {"moe": lambda: m.si_moe_matmul(x, w, offsets), "mxfp4": lambda: m.si_mxfp4_matmul(*q, *q)}[call]
    t = threading.Thread(target=lambda: got.append(run()))
    t.start()
    t.join()
    assert len(got) == 1 and bool((got[0] == 64).all())
