"""Scales come in tiles or as the flat bytes of the tiles. Scales that lie row by
row, as checkpoints hold them, have as many bytes where rows and columns are
multiples of 128, and are refused."""
import numpy as np
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxfp4 as X

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def matrix(seed, r, c):
    """(packed codes, scales row by row) on the host."""
    g = np.random.default_rng(seed)
    return X.pack(g.integers(0, 16, (r, c), dtype=np.uint8)), g.integers(125, 130, (r, c // 32), dtype=np.uint8)


def gpu(a):
    return torch.from_numpy(a).cuda()


def test_scales_row_by_row_are_refused():
    codes, s = matrix(1, 256, 384)
    tiles = X.tile(s)
    assert tiles.size == s.size                      # the number of bytes cannot tell them apart
    a, ok, bad = gpu(codes), gpu(tiles), gpu(s)
    x = torch.randn(256, 384, device="cuda")
    for f in (lambda q: m.si_dequantize_mxfp4(a, q), lambda q: m.si_mxfp4_matmul(a, q, a, ok),
              lambda q: m.si_mxfp4_matmul(a, ok, a, q), lambda q: m.si_quantize_mxfp4(x, scales=q)):
        f(ok)
        for q in (bad, ok.reshape(3, 2, 512), ok[None], ok.reshape(2, -1)):
            with pytest.raises(ValueError, match="scales"):
                f(q)


def test_experts_with_scales_row_by_row_are_refused():
    E, I, H = 3, 256, 128
    part = lambda seed, r, c: [np.stack(t) for t in zip(*(matrix(seed + e, r, c) for e in range(E)))]  # noqa: E731
    gate, up, down = part(1, I, H), part(11, I, H), part(21, H, I)
    tiled = [(gpu(c), gpu(np.stack([X.tile(q) for q in s]))) for c, s in (gate, up, down)]
    raw = [(gpu(c), gpu(s)) for c, s in (gate, up, down)]
    m.Mxfp4Experts(*tiled)
    for i in range(3):
        assert raw[i][1].numel() == tiled[i][1].numel()
        with pytest.raises(ValueError, match="scales"):
            m.Mxfp4Experts(*(raw[j] if j == i else tiled[j] for j in range(3)))


def test_flat_bytes_of_the_tiles_are_taken():
    codes, s = matrix(2, 130, 160)
    a, tiles = gpu(codes), gpu(X.tile(s))
    y = m.si_dequantize_mxfp4(a, tiles, dtype=torch.float32)
    assert torch.equal(y, m.si_dequantize_mxfp4(a, tiles.reshape(-1), dtype=torch.float32))
    assert np.array_equal(y.cpu().double().numpy(), X.decode(codes, X.tile(s)))
    z = m.si_mxfp4_matmul(a, tiles, a, tiles)
    assert torch.equal(z, m.si_mxfp4_matmul(a, tiles.reshape(-1), a, tiles.reshape(-1)))
    x = torch.randn(130, 160, device="cuda")
    flat = torch.empty(tiles.numel(), dtype=torch.uint8, device="cuda")
    c, q = m.si_quantize_mxfp4(x, scales=flat)
    assert q is flat and torch.equal(flat, m.si_quantize_mxfp4(x)[1].reshape(-1))
