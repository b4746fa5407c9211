"""The rows of the (token, rank) pairs stay fp32 between the experts' down product
and the weighted sum over the ranks: the expert FFN rounds once, at its end."""
import numpy as np
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxfp4 as X
from tests.test_gpu_mxfp4 import check_exact_sums

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def raw(seed, lo, hi, *shape):
    """Random codes and scale tiles with bytes in [lo, hi] of n matrices, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r, c = shape[-2:]
    codes = torch.randint(0, 256, (*shape[:-1], c // 2), generator=g, device="cuda", dtype=torch.uint8)
    tiles = torch.randint(lo, hi + 1, (*shape[:-2], *m.mxfp4_scale_shape(r, c)), generator=g, device="cuda", dtype=torch.uint8)
    return codes, tiles


def decode(codes, tiles):
    return X.decode(codes.cpu().numpy(), tiles.cpu().numpy())


@pytest.mark.parametrize("T,E,k,H,I", [(40, 8, 4, 256, 160), (300, 4, 2, 160, 96)])
def test_experts_equal_the_calls_that_they_are_made_of(T, E, k, H, I):
    """sort, gather, quantise, one product an expert and the combine by their own
    calls, SwiGLU in 64 bits. The kernel's h is within 2^-18 of it, so a code may
    lie on the other side of a border: the tolerance takes both sides, the fp32
    additions of down (at most I) and of the ranks, and a rounding of the result.
    The pair rows are fp32 in both."""
    parts = raw(E, 122, 123, E, I, H), raw(E + 1, 122, 123, E, I, H), raw(E + 2, 122, 123, E, H, I)
    experts = m.Mxfp4Experts(*parts)
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, H, generator=g)).to(torch.bfloat16).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    w = torch.randn(T, k, generator=g).cuda()
    y = m.si_moe_ffn_mxfp4(experts, x, ids, w)
    _, position, offsets = m.si_moe_sort(ids, E)
    xs, at = m.si_moe_gather(x, position, offsets), offsets.tolist()
    ys, dy = torch.zeros(T * k, H, device="cuda"), torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = at[e], at[e + 1]
        if a == b:
            continue
        mat = [(p[0][e], p[1][e]) for p in parts]
        q = m.si_quantize_mxfp4(xs[a:b].contiguous())
        check_exact_sums(decode(*q), np.concatenate([decode(*mat[0]), decode(*mat[1])]))
        z, u = (m.si_mxfp4_matmul(*q, *p, dtype=torch.float32).double() for p in mat[:2])
        assert float(z.abs().max()) < 32
        h = z * torch.sigmoid(z) * u
        mid, lo, hi = (m.si_quantize_mxfp4((h * (1 + d)).float()) for d in (0, -2.0 ** -18, 2.0 ** -18))
        ys[a:b] = m.si_mxfp4_matmul(*mid, *mat[2], dtype=torch.float32)
        val = lambda p: m.si_dequantize_mxfp4(*p, dtype=torch.float32).double()  # noqa: E731
        down = val(mat[2]).abs()
        dy[a:b] = (val(hi) - val(lo)).abs() @ down.T + 2 * I * 2.0 ** -23 * (val(mid).abs() @ down.T)
    want = m.si_moe_combine(ys, position, w).double()
    pos = position.long()
    aw = w.double().abs()[..., None]
    tol = (aw * (dy[pos] * 1.01 + 2 * k * 2.0 ** -24 * ys.double().abs()[pos])).sum(1)
    half = torch.finfo(torch.bfloat16).eps / 2
    # y is rounded to bf16, want is not
    err = (y.double() - want).abs()
    assert bool((err <= tol + half * (want.abs() + tol)).all()), float((err / (tol + half * want.abs() + 1e-30)).max())
