"""Products and the expert FFN where their kernels loop: more tiles than SMs, more
columns than the ring of stages holds, more pairs than one launch sorts. Sums are
exact as in test_gpu_mxfp4.py (asserted), so products equal the 64-bit ones after
one rounding."""
import numpy as np
import pytest
import torch

import moe_decode_ffn_gb300 as m
from oracle import mxfp4 as X
from tests.test_gpu_mxfp4 import TYPES, ffn_oracle

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


class Decoded:
    """Expert e's matrix in 64 bits, decoded when it is asked for."""

    def __init__(self, pair):
        self.pair, self.kept = pair, {}

    def __getitem__(self, e):
        if e not in self.kept:
            self.kept[e] = decode(self.pair[0][e], self.pair[1][e])
        return self.kept[e]


# ---- products of few tokens, several tiles a block, k behind the ring ------------

@pytest.mark.parametrize("mm", [1, 16, 20, 33, 64])
@pytest.mark.parametrize("n,k", [(130 * 2 * 152 + 1, 160), (129 * 152 + 8, 2144)])
def test_few_tokens_and_more_tiles_than_sms(mm, n, k):
    assert -(-n // 128) > torch.cuda.get_device_properties(0).multi_processor_count
    a, w = raw(mm, 126, 128, mm, k), raw(n, 126, 128, n, k)
    ad, wd = decode(*a), m.si_dequantize_mxfp4(*w, dtype=torch.float32).double()
    assert np.abs(ad).max() * float(wd.abs().max()) * k * 16 < 2 ** 24     # values are multiples of 1/4
    want = torch.from_numpy(ad).cuda() @ wd.T
    ws = m.workspace(m.mxfp4_matmul_workspace_bytes(mm, n, k))
    for dtype in TYPES.values():
        y = torch.full((mm, n + 8), 5.0, dtype=dtype, device="cuda")
        m.si_mxfp4_matmul(*a, *w, out=y[:, :n], ws=ws)
        assert torch.equal(y[:, :n], want.to(dtype)) and bool((y[:, n:] == 5).all())
    assert m.si_workspace_status(ws) == m.SI_OK


def test_decoded_values_are_those_of_the_oracle():
    w = raw(3, 120, 130, 300, 416)
    assert np.array_equal(m.si_dequantize_mxfp4(*w, dtype=torch.float32).double().cpu().numpy(), decode(*w))


# ---- expert FFN ------------------------------------------------------------------

# tokens, experts, ranks, H, I, share of dropped pairs
# - 16 tokens a tile: about a thousand tiles; the ring of 6 stages wraps in gate/up,
#   in down; both
# - tokens on the lanes: two or three rounds of tiles, the ring of 4 wraps in both,
#   more than 1024 inner columns (down's other way to store), one launch and two of
#   the sort
LARGE = [(600, 1024, 8, 1696, 64, 0.05), (620, 1000, 7, 64, 1696, 0.0), (40, 200, 8, 1600, 1632, 0.0),
         (2100, 6, 2, 1120, 1312, 0.1), (2100, 6, 2, 1344, 640, 0.0), (2040, 5, 2, 2144, 672, 0.1), (4100, 300, 8, 64, 96, 0.02)]


@pytest.mark.parametrize("T,E,k,H,I,drop", LARGE)
def test_experts_of_large_batches(T, E, k, H, I, drop):
    """Sampled tokens against 64 bits; every token the same as in batches of 40
    (which sort in one launch, in tiles of 16)."""
    parts = raw(T, 122, 123, E, I, H), raw(T + 1, 122, 123, E, I, H), raw(T + 2, 122, 123, E, H, I)
    experts = m.Mxfp4Experts(*parts)
    g = torch.Generator().manual_seed(T + H)
    # sixteenths: |g| stays below the oracle's limit
    x = (torch.randn(T, H, generator=g) * min(1.0, 16 / H ** 0.5)).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(E - 1, generator=g)[:k] for _ in range(T)]).to(torch.int32)      # the last one stays empty
    lost = torch.rand(T, k, generator=g) < drop
    ids = torch.where(lost, torch.where(torch.rand(T, k, generator=g) < 0.5, -1, E), ids).to(torch.int32)
    ids[3] = -1
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    ws = m.workspace(m.ffn_mxfp4_workspace_bytes(experts, T, k))
    ws[256:].fill_(255)
    gx, gi, gw = x.cuda(), ids.cuda(), w.cuda()
    y = m.si_moe_ffn_mxfp4(experts, gx, gi, gw, ws=ws)
    assert torch.equal(y, m.si_moe_ffn_mxfp4(experts, gx, gi, gw, ws=ws))
    assert m.si_workspace_status(ws) == m.SI_OK
    for t in range(0, T, 40):
        assert torch.equal(y[t:t + 40], m.si_moe_ffn_mxfp4(experts, gx[t:t + 40], gi[t:t + 40], gw[t:t + 40])), t
    assert not y[3].any()
    some = torch.randperm(T, generator=g)[:10]
    want, tol = ffn_oracle([Decoded(p) for p in parts], x[some].double().numpy(), ids[some].numpy(), w[some].double().numpy(), E)
    assert np.all(np.abs(y.cpu()[some].double().numpy() - want) <= tol)
