"""Padded batches and values that are not finite in the experts' training step.

Tokens whose ids are all dropped hold NaN in x, gy and w and must reach nothing; a live
token's NaN reaches its own rows and its experts' gradients alone, so everything else keeps
its bits. Each in both forms of the products (few rows an expert, and more)."""
import pytest
import torch

import moe_decode_ffn_gb300 as m
from tests.test_gpu_moe_experts import TYPES, V, expected, inputs, near, silu_off

pytestmark = pytest.mark.gpu

# tokens, ranks, experts, hidden, inter: 2.5 rows an expert and 100; blocks of 8 values at a row's end
FORMS = [(10, 2, 8, 72, 40), (200, 2, 4, 136, 264)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


def step(x, ids, w, gate_up, down, gy):
    leaves = [t.clone().requires_grad_() for t in (x, w, gate_up, down)]
    y = m.si_moe_experts(leaves[0], ids, *leaves[1:])
    return y.detach(), *torch.autograd.grad(y, leaves, gy)


def same_bits(a, b):
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("all_of_them", [False, True])
def test_padding_reaches_nothing(form, kind, all_of_them):
    x, ids, w, gate_up, down, gy = inputs(*form, 0, kind, seed=11)
    T = x.shape[0]
    pad = torch.ones(T, dtype=torch.bool, device="cuda") if all_of_them else torch.arange(T, device="cuda") % 3 == 1
    ids[pad] = -1
    for t in (x, w, gy):
        t[pad] = float("nan")
    got = step(x, ids, w, gate_up, down, gy)
    for a in got[:3]:
        assert int(torch.count_nonzero(a[pad])) == 0
    for a, b, name in zip(got, expected(x, ids, w, gate_up, down, gy), ("y", "gx", "gw", "ggate_up", "gdown")):
        near(a, b, name)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("form", FORMS)
def test_a_tokens_nan_stays_with_it(form, kind):
    x, ids, w, gate_up, down, gy = inputs(*form, 0, kind, seed=12)
    T, E = x.shape[0], gate_up.shape[0]
    clean = step(x, ids, w, gate_up, down, gy)
    x[5] = float("nan")
    got = step(x, ids, w, gate_up, down, gy)
    tokens = torch.arange(T, device="cuda") != 5
    experts = torch.ones(E, dtype=torch.bool, device="cuda")
    experts[ids[5].long()] = False
    assert bool(experts.any())
    for a, b in zip(got[:3], clean[:3]):         # y, gx, gw
        assert bool(a[5].isnan().all()) and same_bits(a[tokens], b[tokens])
    for a, b in zip(got[3:], clean[3:]):         # ggate_up, gdown
        assert bool(a[~experts].isnan().all()) and same_bits(a[experts], b[experts])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_kept_blocks_that_are_not_finite(form, kind, bad):
    x, ids, _, gate_up, _, _ = inputs(*form, 0, kind, seed=13)
    _, position, offsets = m.si_moe_sort(ids, gate_up.shape[0])
    xs = m.si_moe_gather(x, position, offsets)
    h, (codes, scales) = m.si_moe_gateup(xs, gate_up, offsets, keep=True)
    xs[3, 17] = bad                              # every sum of the row: an infinity, or times 0 NaN
    h2, (codes2, scales2) = m.si_moe_gateup(xs, gate_up, offsets, keep=True)
    rows = torch.arange(xs.shape[0], device="cuda") != 3
    assert bool((scales2[3] == 255).all()) and int(torch.count_nonzero(codes2[3])) == 0
    assert same_bits(h2[rows], h[rows]) and torch.equal(codes2[rows], codes[rows]) and torch.equal(scales2[rows], scales[rows])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("H", [520, 1024, 1032, 1536, 2056])
@pytest.mark.parametrize("counts", [[3, 0, 9], [70, 0, 300]])
def test_gate_and_up_over_long_sums(counts, H, kind):
    """Whole numbers, exact in any order of the sums and in however many parts: every part once."""
    g = torch.Generator(device="cuda").manual_seed(H)
    dtype, R, I = TYPES[kind], sum(counts) + 2, 72
    xs = torch.randint(-2, 3, (R, H), generator=g, device="cuda").to(dtype)
    gate_up = torch.randint(-2, 3, (3, 2 * I, H), generator=g, device="cuda").to(dtype) / 64
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    gu = torch.zeros(R, 2 * I, dtype=torch.float64, device="cuda")
    for e in range(3):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        gu[rows] = xs[rows].double() @ gate_up[e].double().T
    h, (codes, scales) = m.si_moe_gateup(xs, gate_up, offsets, keep=True)
    assert torch.equal(h, m.si_moe_gateup(xs, gate_up, offsets))
    parts = [m.si_quantize_mxint8(v.float().contiguous()) for v in (gu[:, :I], gu[:, I:])]   # |sums| < 2^18 / 64: exact
    assert torch.equal(codes, torch.cat([p[0] for p in parts], 1)) and torch.equal(scales, torch.cat([p[1] for p in parts], 1))
    want = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    near(h, V(want, silu_off(gu[:, :I], want)).round(dtype), "h")
