"""Activations in 8 bits, SwiGLU and its gradients against the oracle in 64 bits.

Codes and scales have to be equal: a block's scale is a power of two, so x times its
inverse is exact and the rounding the same. What the codes stand for is exact in fp32
and rounded once to the output's type. SwiGLU and its gradients: the logistic
function is off by at most 2^-20 (1 + |g|) relative (the product of g and log2 e is
rounded, off by 2^-24 |g| 1.44 in the exponent, ex2 by 2 units in the last place, the
sum and the reciprocal by one each), every further product by 2^-24, and the result by
half a unit in the last place of its type."""
import numpy as np
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxint8 as Q

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SHAPES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 200), (4, 256), (7, 1000), (33, 264), (1, 2048)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def f64(t):
    return t.detach().double().cpu().numpy()


def values(g, rows, cols, kind):
    """Blocks of very different sizes, zero blocks, ties and large elements among them."""
    v = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, cols), generator=g).float() * 0.5)
    v[:, ::7] = torch.round(v[:, ::7] * 8) / 8
    if cols > 64:
        v[0, 32:64] = 0
    return v.to(TYPES[kind]).cuda()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_scales_and_values(rows, cols, kind):
    x = values(torch.Generator().manual_seed(rows * 100 + cols), rows, cols, kind)
    codes, scales = m.si_quantize_mxint8(x)
    want = Q.quantize(f64(x))
    assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
    exact = torch.from_numpy(Q.dequantize(*want))
    for dtype in TYPES.values():
        assert torch.equal(m.si_dequantize_mxint8(codes, scales, dtype).cpu(), exact.to(torch.float32).to(dtype))


@pytest.mark.parametrize("cols", [32, 40, 45])
def test_extremes(cols):
    """Subnormal numbers, the largest ones, infinities and NaN, in blocks of their own."""
    x = torch.zeros(8, cols)
    x[0, 3], x[0, 5] = 2.0 ** -149, -3 * 2.0 ** -140
    x[1, 0], x[1, 1] = torch.finfo(torch.float32).max, -2.0 ** 127
    x[2, 0], x[2, 9] = 2.0 ** -126, 2.0 ** -127
    x[3, 7] = float("inf")
    x[4, 7] = float("nan")
    x[5, 0], x[5, 1], x[5, 2] = 1.9999, -1.9999, 0.5 / 64      # beyond the last code; a tie to even
    x[6, 0], x[6, 1] = 2.0 ** -121, 1.5 / 64 * 2.0 ** -121
    x[7, 0] = -0.0
    codes, scales = m.si_quantize_mxint8(x.cuda())
    want = Q.quantize(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(scales.cpu().numpy(), want[1])
    got, exact = m.si_dequantize_mxint8(codes, scales, torch.float32).double().cpu().numpy(), Q.dequantize(*want)
    assert np.array_equal(np.isnan(got), np.isnan(exact)) and np.array_equal(got[~np.isnan(got)], exact[~np.isnan(exact)])
    assert np.isnan(got[3, :32]).all() and not np.isnan(got[3, 32:]).any()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("pad", [1, 8])
def test_strided_rows(kind, pad):
    rows, cols = 9, 72
    wide = values(torch.Generator().manual_seed(pad), rows, cols + 2 * pad, kind)
    x = wide[:, pad:pad + cols]
    codes, scales = m.si_quantize_mxint8(x)
    want = m.si_quantize_mxint8(x.contiguous())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    y = torch.full_like(wide, 5.0)
    m.si_dequantize_mxint8(codes, scales, out=y[:, pad:pad + cols])
    assert torch.equal(y[:, pad:pad + cols], m.si_dequantize_mxint8(codes, scales, TYPES[kind]))
    assert bool((y[:, :pad] == 5).all()) and bool((y[:, pad + cols:] == 5).all())


def test_without_rows():
    codes, scales = m.si_quantize_mxint8(torch.empty(0, 40, device="cuda"))
    assert codes.shape == (0, 40) and scales.shape == (0, 2)
    assert m.si_dequantize_mxint8(codes, scales).shape == (0, 40)
    h, kept = m.si_swiglu(torch.empty(0, 80, device="cuda"), keep=True)
    assert h.shape == (0, 40)
    assert m.si_swiglu_backward(h, kept)[0].shape == (0, 80)


def near(got, want, terms, size):
    """Within `terms` 2^-24 of `size`, and half a unit of got's type."""
    info = torch.finfo(got.dtype)
    got, half = f64(got), info.eps / 2
    bound = terms * 2.0 ** -24 * size + half * (np.abs(want) + terms * 2.0 ** -24 * size) + info.smallest_normal * info.eps
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], bound[bad][:3])


def silu_terms(g):
    """In units of 2^-24: the logistic function's 2^-20 (1 + |g|) and a few products."""
    return 16 * (1 + np.abs(g)) + 4


SWIGLU = [(1, 1), (1, 8), (3, 40), (2, 45), (5, 256), (9, 1000), (4, 2304), (130, 96)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,inter", SWIGLU)
def test_swiglu_and_its_gradients(rows, inter, kind):
    g_ = torch.Generator().manual_seed(rows + inter)
    gu = (torch.randn(rows, 2 * inter, generator=g_) * 4).to(TYPES[kind]).cuda()
    gh = torch.randn(rows, inter, generator=g_).to(TYPES[kind]).cuda()
    h, kept = m.si_swiglu(gu, keep=True)
    assert torch.equal(m.si_swiglu(gu), h)
    g, u = f64(gu[:, :inter]), f64(gu[:, inter:])
    near(h, Q.swiglu(g, u), silu_terms(g), np.abs(Q.swiglu(g, u)))
    parts = [Q.quantize(v) for v in (g, u)]
    assert np.array_equal(kept[0].cpu().numpy(), np.concatenate([p[0] for p in parts], 1))
    assert np.array_equal(kept[1].cpu().numpy(), np.concatenate([p[1] for p in parts], 1))
    qg, qu = (Q.dequantize(*p) for p in parts)
    w = torch.randn(rows, generator=g_).cuda()
    d, s = f64(gh), Q.logistic(qg)
    for c in (None, w):
        ggu, wh, gw = m.si_swiglu_backward(gh, kept, c)
        cc = np.ones(rows) if c is None else f64(c)
        gg, gu_, ch, gc = Q.swiglu_backward(qg, qu, d, cc)
        # 1 + g (1 - s) as two terms of their own size
        size = np.abs(cc[:, None] * d * qu * s) * (1 + np.abs(qg) * (1 - s))
        near(ggu[:, :inter], gg, silu_terms(qg), size)
        near(ggu[:, inter:], gu_, silu_terms(qg), np.abs(gu_))
        near(wh, ch, silu_terms(qg), np.abs(ch))
        if c is None:
            assert gw is None
        else:
            terms = np.abs(d * qg * s * qu)
            near(gw, gc, 1, ((silu_terms(qg) + inter) * terms).sum(1))


@pytest.mark.parametrize("kind", list(TYPES))
def test_weights_of_pairs(kind):
    """Rows in sorted order, weights and their gradient by (token, rank); dropped pairs."""
    T, k, E, inter = 37, 3, 5, 72
    g_ = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(0, E + 3, (T, k), generator=g_, device="cuda", dtype=torch.int32)
    order, position, offsets = m.si_moe_sort(ids, E)
    R, kept_rows = T * k, int(offsets[E])
    gu, gh = (torch.randn(R, c, generator=g_, device="cuda").to(TYPES[kind]) for c in (2 * inter, inter))
    gh[kept_rows:] = float("nan")                # rows of no pair are not read
    w = torch.randn(T, k, generator=g_, device="cuda")
    _, kept = m.si_swiglu(gu, keep=True)
    ggu, wh, gw = m.si_swiglu_backward(gh, kept, w, order)
    rows = w.reshape(-1)[order[:kept_rows].long()].contiguous()
    one = m.si_swiglu_backward(gh[:kept_rows].contiguous(), tuple(t[:kept_rows].contiguous() for t in kept), rows)
    assert torch.equal(ggu[:kept_rows], one[0]) and torch.equal(wh[:kept_rows], one[1])
    assert not bool(ggu[kept_rows:].any()) and not bool(wh[kept_rows:].any())
    want = torch.zeros(R, device="cuda")
    want[order[:kept_rows].long()] = one[2]
    assert gw.shape == w.shape and torch.equal(gw.reshape(-1), want)


def test_extreme_activations():
    """silu of far values: 0 or g, no NaN; a block with an infinity gives NaN gradients."""
    g = torch.tensor([[-1e4, -100.0, -0.0, 0.0, 100.0, 1e4, 88.5, -88.5]], device="cuda")
    u = torch.full_like(g, 2.0)
    h, kept = m.si_swiglu(torch.cat([g, u], 1), keep=True)
    want = 2 * g.double() * torch.sigmoid(g.double())
    assert torch.allclose(h.double(), want, rtol=1e-5, atol=1e-30)
    ggu, _, _ = m.si_swiglu_backward(torch.ones_like(g), kept)
    assert bool(torch.isfinite(ggu).all())
    g[0, 3] = float("inf")
    _, kept = m.si_swiglu(torch.cat([g, u], 1), keep=True)
    assert bool(torch.isnan(m.si_swiglu_backward(torch.ones_like(g), kept)[0]).all())


@pytest.mark.parametrize("kind", list(TYPES))
def test_through_autograd(kind):
    gu = torch.randn(6, 144, generator=torch.Generator().manual_seed(3)).to(TYPES[kind]).cuda()
    leaf = gu.clone().requires_grad_()
    h = m.si_swiglu(leaf)
    gh = torch.randn_like(h)
    h.backward(gh)
    plain, kept = m.si_swiglu(gu, keep=True)
    assert torch.equal(h, plain) and torch.equal(leaf.grad, m.si_swiglu_backward(gh, kept)[0])
    h2, kept2 = m.si_swiglu(leaf, keep=True)
    assert h2.requires_grad and torch.equal(kept2[0], kept[0]) and not kept2[0].requires_grad


def test_gradient_against_differences():
    """Central differences of <gh, silu(g) u> in 64 bits at the kept values."""
    gu = torch.randn(2, 64, generator=torch.Generator().manual_seed(8)).cuda()
    gh = torch.randn(2, 32, generator=torch.Generator().manual_seed(9)).cuda()
    _, (codes, scales) = m.si_swiglu(gu, keep=True)
    at = f64(m.si_dequantize_mxint8(codes, scales, torch.float32))
    got = f64(m.si_swiglu_backward(gh, (codes, scales))[0])
    f = lambda v: (f64(gh) * Q.swiglu(v[:, :32], v[:, 32:])).sum()  # noqa: E731
    eps = 2.0 ** -14                             # error of the difference: eps^2 f''' / 6 + 2^-53 |f| / eps < 1e-7
    for r, c in [(0, 0), (0, 31), (1, 5), (0, 32), (1, 63), (1, 40)]:
        up, down = at.copy(), at.copy()
        up[r, c] += eps
        down[r, c] -= eps
        assert abs((f(up) - f(down)) / (2 * eps) - got[r, c]) <= 1e-7 + 2.0 ** -18 * (1 + np.abs(at[r]).max()) * np.abs(f64(gh)).max() * 4
