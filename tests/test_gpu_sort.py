"""Tokens sorted by expert and back, and the gradients, against the fp64 oracle.

Tolerances: moved rows are exact; a sum of n fp32 terms is off by at most
n 2^-24 of the sum of their magnitudes, and a result by half a unit in the last
place of its type (finfo.eps / 2 relative) on top.
"""
import numpy as np
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxfp4 as X

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def routing(seed, T, k, E, outside=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    if outside:
        drop = torch.rand(T, k, generator=g) < outside
        ids = torch.where(drop, torch.where(torch.rand(T, k, generator=g) < 0.5, -1, E + 3), ids)
    return ids.to(torch.int32), torch.randn(T, k, generator=g)


CASES = [(1, 1, 1, 8, 0), (1, 8, 128, 2048, 0), (3, 2, 8, 1, 0), (17, 5, 100, 1000, 0.4), (64, 8, 128, 2048, 0),
         (64, 3, 1024, 36, 0.1), (513, 4, 7, 130, 0.5), (20, 8, 16, 64, 1.0), (2000, 7, 33, 72, 0.2), (40, 2, 4, 4104, 0)]


@pytest.mark.parametrize("T,k,E,H,outside", CASES)
def test_sort(T, k, E, H, outside):
    ids, _ = routing(T + E, T, k, E, outside)
    got = m.si_moe_sort(ids.cuda(), E)
    for a, b in zip(got, X.sort(ids.numpy(), E)):
        assert a.dtype == torch.int32 and np.array_equal(a.cpu().numpy(), b)


def test_sort_skewed_and_large():
    """All pairs on one expert; a batch of many thousand pairs."""
    ids = torch.full((300, 8), 5, dtype=torch.int32)
    order, position, offsets = m.si_moe_sort(ids.cuda(), 8)
    assert torch.equal(order.cpu(), torch.arange(2400, dtype=torch.int32))
    assert offsets.tolist() == [0] * 6 + [2400] * 3
    ids, _ = routing(1, 8192, 8, 256)
    order, position, offsets = m.si_moe_sort(ids.cuda(), 256)
    want = torch.sort(ids.reshape(-1), stable=True).indices.to(torch.int32)
    assert torch.equal(order.cpu(), want)
    assert torch.equal(position.reshape(-1)[order.long()].cpu(), torch.arange(65536, dtype=torch.int32))


@pytest.mark.parametrize("pairs", [2049, 4095, 4096, 4097, 64 * 1024 - 1, 64 * 1024 + 1, 64 * 2048 + 1, 300001])
@pytest.mark.parametrize("E", [1, 100, 1024])
def test_sort_at_the_borders_of_its_rounds(pairs, E):
    """One launch or two, chunks of one round or of several, the last one ragged."""
    ids, _ = routing(pairs + E, pairs, 1, E, 0.05)
    order, position, offsets = m.si_moe_sort(ids.cuda(), E)
    flat = ids.reshape(-1).long()
    keep = (flat >= 0) & (flat < E)
    key = torch.where(keep, flat, torch.full_like(flat, E))
    perm = torch.sort(key, stable=True).indices
    kept = int(keep.sum())
    assert torch.equal(order.cpu()[:kept].long(), perm[:kept]) and bool((order.cpu()[kept:] == -1).all())
    want = torch.full_like(flat, -1)
    want[perm[:kept]] = torch.arange(kept)
    assert torch.equal(position.cpu().reshape(-1).long(), want)
    assert torch.equal(offsets.cpu().long(), torch.searchsorted(key[perm], torch.arange(E + 1)))


def _inputs(T, k, E, H, outside, kind):
    ids, w = routing(T * 3 + H, T, k, E, outside)
    g = torch.Generator().manual_seed(T + H)
    make = lambda r: torch.randn(r, H, generator=g).to(TYPES[kind])  # noqa: E731
    return ids, w, make(T), make(T * k)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,k,E,H,outside", CASES)
def test_rows_and_gradients(T, k, E, H, outside, kind):
    ids, w, x, rows = _inputs(T, k, E, H, outside, kind)
    order, position, offsets = m.si_moe_sort(ids.cuda(), E)
    oo, op, of = X.sort(ids.numpy(), E)
    kept = int(of[-1])
    tok = oo[:kept] // k
    xd, rd, wd = x.double().numpy(), rows.double().numpy(), w.double().numpy()
    half = torch.finfo(TYPES[kind]).eps / 2

    xs = m.si_moe_gather(x.cuda(), position, offsets).cpu()
    assert torch.equal(xs[:kept], x[torch.from_numpy(tok).long()])
    assert not xs[kept:].any()

    def near(got, want, terms, n):
        tol = n * 2.0 ** -24 * terms
        err = np.abs(got.cpu().double().numpy() - want)
        assert got.dtype in (TYPES[kind], torch.float32)
        extra = half * (np.abs(want) + tol) if got.dtype == TYPES[kind] else 0
        tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0     # half the smallest subnormal step
        assert np.all(err <= tol + extra + tiny)

    y, gx = np.zeros((T, H)), np.zeros((T, H))
    ay, agx = np.zeros((T, H)), np.zeros((T, H))
    for p in range(kept):
        t, r = divmod(int(oo[p]), k)
        y[t] += wd[t, r] * rd[p]
        ay[t] += np.abs(wd[t, r] * rd[p])
        gx[t] += rd[p]
        agx[t] += np.abs(rd[p])
    near(m.si_moe_combine(rows.cuda(), position, w.cuda()), y, ay, k)
    near(m.si_moe_gather_backward(rows.cuda(), position), gx, agx, k)

    gys, gw = m.si_moe_combine_backward(x.cuda(), rows.cuda(), position, offsets, w.cuda())
    assert not gys.cpu()[kept:].any()
    flat = wd.reshape(-1)[oo[:kept]][:, None]
    near(gys[:kept], flat * xd[tok], np.abs(flat * xd[tok]), 1)
    want, terms = np.zeros(T * k), np.zeros(T * k)
    want[oo[:kept]] = (xd[tok] * rd[:kept]).sum(1)
    terms[oo[:kept]] = np.abs(xd[tok] * rd[:kept]).sum(1)
    err = np.abs(gw.cpu().double().numpy().reshape(-1) - want)
    assert gw.dtype == torch.float32 and np.all(err <= (H + 1) * 2.0 ** -24 * terms)


def test_gradients_against_differences():
    """L = <c, combine(ys, w)> is linear in ys and in w: its difference over a
    step of one equals the gradient, up to the fp32 rounding of L's terms."""
    T, k, E, H = 9, 3, 5, 40
    ids, w, c, ys = _inputs(T, k, E, H, 0.2, "f32")
    _, position, offsets = m.si_moe_sort(ids.cuda(), E)
    g = [t.cuda() for t in (c, ys, w)]
    L = lambda ys, w: float((m.si_moe_combine(ys, position, w).double() * g[0].double()).sum())  # noqa: E731
    gys, gw = m.si_moe_combine_backward(g[0], g[1], position, offsets, g[2])
    size = float(c.double().abs().sum() * (ys.double().abs().max() + 1) * (w.double().abs().max() + 1) * k)
    tol = 2 * (k + 2) * 2.0 ** -24 * size
    rng = np.random.default_rng(3)
    for _ in range(12):
        p, h, t, r = rng.integers(T * k), rng.integers(H), rng.integers(T), rng.integers(k)
        ys2, w2 = g[1].clone(), g[2].clone()
        ys2[p, h] += 1
        w2[t, r] += 1
        assert abs(L(ys2, g[2]) - L(g[1], g[2]) - float(gys[p, h])) <= tol
        assert abs(L(g[1], w2) - L(g[1], g[2]) - float(gw[t, r])) <= tol
    # the gather: <c, gather(x)> against its gradient
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).cuda()
    G = lambda x: float((m.si_moe_gather(x, position, offsets).double() * g[1].double()).sum())  # noqa: E731
    gx = m.si_moe_gather_backward(g[1], position)
    for _ in range(6):
        t, h = rng.integers(T), rng.integers(H)
        x2 = x.clone()
        x2[t, h] += 1
        assert abs(G(x2) - G(x) - float(gx[t, h])) <= tol


def test_values_of_dropped_pairs_do_not_leak():
    """Infinities and NaN in rows and weights that belong to no kept pair."""
    T, k, E, H = 6, 2, 4, 64
    ids = torch.tensor([[0, 1], [-1, 2], [9, -1], [3, 3], [1, 0], [2, 4]], dtype=torch.int32)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(2))
    drop = (ids < 0) | (ids >= E)
    w[drop] = float("nan")
    order, position, offsets = m.si_moe_sort(ids.cuda(), E)
    kept = int(offsets[-1])
    ys = torch.randn(T * k, H, generator=torch.Generator().manual_seed(3))
    ys[kept:] = float("inf")
    y = m.si_moe_combine(ys.cuda(), position, w.cuda()).cpu()
    assert torch.isfinite(y).all() and not y[2].any()
    gys, gw = m.si_moe_combine_backward(torch.ones(T, H).cuda(), ys.cuda(), position, offsets, w.cuda())
    assert torch.isfinite(gys).all() and torch.isfinite(gw).all()
    assert not gys[kept:].any() and not gw.cpu()[drop].any()
    assert torch.isfinite(m.si_moe_gather_backward(ys.cuda(), position)).all()


def test_unaligned_rows():
    """Rows whose base is not 16-byte aligned take the value-by-value path."""
    T, k, E, H = 11, 3, 6, 64
    ids, w, x, rows = _inputs(T, k, E, H, 0, "bf16")
    _, position, offsets = m.si_moe_sort(ids.cuda(), E)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)]).cuda()[1:].view(t.shape)  # noqa: E731
    assert off(x).data_ptr() % 16
    assert torch.equal(m.si_moe_gather(off(x), position, offsets), m.si_moe_gather(x.cuda(), position, offsets))
    assert torch.equal(m.si_moe_combine(off(rows), position, w.cuda()), m.si_moe_combine(rows.cuda(), position, w.cuda()))
    a = m.si_moe_combine_backward(off(x), off(rows), position, offsets, w.cuda())
    b = m.si_moe_combine_backward(x.cuda(), rows.cuda(), position, offsets, w.cuda())
    assert torch.equal(a[0], b[0]) and torch.allclose(a[1], b[1], rtol=0, atol=2 * H * 2.0 ** -24 * H * 16)


def test_places_outside_the_rows_count_as_dropped():
    T, k, E, H = 5, 2, 4, 32
    ids, w, x, rows = _inputs(T, k, E, H, 0, "f32")
    _, position, offsets = m.si_moe_sort(ids.cuda(), E)
    bad = position.clone()
    bad[2, 1], bad[4, 0] = 1 << 30, -5
    y = m.si_moe_combine(rows.cuda(), bad, w.cuda())
    zero = w.clone()
    zero[2, 1] = zero[4, 0] = 0
    assert torch.equal(y, m.si_moe_combine(rows.cuda(), position, zero.cuda()))


def test_run_together_in_a_graph_and_on_a_stream():
    """sort, gather, combine and the gradients as one training step uses them,
    captured once and replayed with other routing."""
    T, k, E, H = 48, 4, 12, 256
    ids, w, x, _ = _inputs(T, k, E, H, 0.1, "bf16")
    ids, w, x = ids.cuda(), w.cuda(), x.cuda()
    gy = torch.randn(T, H, device="cuda").to(torch.bfloat16)

    def step(stream=None):
        order, position, offsets = m.si_moe_sort(ids, E, stream=stream)
        xs = m.si_moe_gather(x, position, offsets, stream=stream)
        y = m.si_moe_combine(xs, position, w, stream=stream)
        gys, gw = m.si_moe_combine_backward(gy, xs, position, offsets, w, stream=stream)
        return order, xs, y, gys, gw, m.si_moe_gather_backward(gys, position, stream=stream)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in (1, 2):
        ids.copy_(routing(seed, T, k, E, 0.3)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        again = step(other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, again))
