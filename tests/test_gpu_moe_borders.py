"""The products and the fused forms where one form gives way to another and where a block
takes several tiles.

Up to 12 rows an expert on average (rows of no expert count too) a tile is one SM's, with 16
rows, else a pair's, with up to 256; the features lie on the lanes of tensor memory in both."""
import pytest
import torch

import moe_decode_ffn_gb300 as m
from tests import test_gpu_moe_experts as X
from tests import test_gpu_moe_matmul as P

pytestmark = pytest.mark.gpu
KINDS = list(X.TYPES)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    m.build()
    m.library()


# ---- 12 rows an expert, and one row more ---------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,head,tail", [([20, 0, 16], 0, 0), ([20, 1, 16], 0, 0), ([17, 0, 9], 3, 7), ([0, 0, 35], 0, 2)])
def test_products_at_the_border(counts, head, tail, kind):
    assert head + sum(counts) + tail in (12 * 3, 12 * 3 + 1)
    for test in (P.test_products_of_integers_are_exact, P.test_gradients_of_integers_are_exact, P.test_normal_values_against_64_bits):
        test(counts, head, tail, 264, 136, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows", [12 * 3, 12 * 3 + 1])
def test_fused_forms_at_the_border(rows, kind):
    """Beside the experts' rows the product has 1 + 3 of no expert, the gradient 2 + 3."""
    X.test_gate_and_up_product([20, 0, rows - 24], 72, 264, kind)
    X.test_gradient_behind_the_down_product([16, 0, rows - 21], 72, 264, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", [(18, 2, 3, 72, 40, 0.2), (37, 1, 3, 72, 40, 0.0)])
def test_experts_at_the_border(case, kind):
    X.test_against_64_bits(case, kind)


# ---- several tiles a block -------------------------------------------------------------

# 27 tiles of rows with those of no expert, in pairs of SMs; about 80 in one
WIDE = [300, 0, 1, 17, 33, 16, 31, 64, 2, 15] + [14] * 15
FEW = [7 * i % 23 for i in range(64)]


def test_which_form_these_take():
    assert sum(WIDE) > 12 * len(WIDE) and sum(FEW) + 5 <= 12 * len(FEW)


# 1032 features: 9 tiles of 128 and 5 of 256, so 243 and 135 for at most 76 pairs, more than 700 for 152 SMs. Summed
# widths within and beyond the first part of fp16's gate and up (1024 in pairs, 512 in one SM)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,H", [(WIDE, 136), (WIDE, 2056), (FEW, 136), (FEW, 1032)])
def test_gate_and_up_over_many_tiles(counts, H, kind):
    X.test_gate_and_up_product(counts, H, 1032, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts", [WIDE, FEW])
def test_gradient_behind_down_over_many_tiles(counts, kind):
    X.test_gradient_behind_the_down_product(counts, 200, 1032, kind)


# ---- bounds that decrease or lie outside the rows -----------------------------------------

def bounds(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# bounds, those that the products take them for, the rows that each expert's gradient sums up (100 rows; in one SM: 16 experts)
ODD = [([-5, 30, 20, 2000000000, 90], [0, 30, 30, 100, 100], [(0, 30), (0, 0), (20, 100), (0, 0)]),
       ([7, 2, 60, -1, 61] + [40] * 11 + [70], [7, 7, 60, 60, 61] + [61] * 11 + [70],
        [(0, 0), (2, 60), (0, 0), (0, 61), (0, 0)] + [(0, 0)] * 10 + [(40, 70)])]


@pytest.mark.parametrize("odd,even,own", ODD)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_odd_bounds_in_products_and_gradients(odd, even, own, out):
    R, E, n, k = 100, len(own), 264, 136
    assert len(odd) == len(even) == E + 1 and (E == 4) == (R > 12 * E)
    g = torch.Generator(device="cuda").manual_seed(E)
    x, w, gy = (P.whole(g, *s, dtype=torch.bfloat16) for s in ((R, k), (E, n, k), (R, n)))
    counts = [b - a for a, b in zip(even, even[1:])]
    want = P.reference(x, w, counts, even[0])
    assert torch.equal(m.si_moe_matmul(x, w, bounds(*odd), dtype=out), want.to(out))
    gw = m.si_moe_matmul_grad_w(gy, x, bounds(*odd), dtype=out)
    for e, (a, b) in enumerate(own):
        assert torch.equal(gw[e], (gy[a:b].double().T @ x[a:b].double()).to(out))


@pytest.mark.parametrize("odd,even,own", ODD)
def test_odd_bounds_in_the_fused_forms(odd, even, own):
    R, E, H, I = 100, len(own), 72, 136
    g = torch.Generator(device="cuda").manual_seed(E)
    x, gate_up, down, gy = (P.whole(g, *s, dtype=torch.bfloat16) for s in ((R, H), (E, 2 * I, H), (E, H, I), (R, H)))
    a, b = (m.si_moe_gateup(x, gate_up, bounds(*v), keep=True) for v in (odd, even))
    assert torch.equal(a[0], b[0]) and all(torch.equal(p, q) for p, q in zip(a[1], b[1])) and bool(a[0].any())
    w = torch.rand(R, generator=g, device="cuda")
    for p, q in zip(*(m.si_moe_down_backward(gy, down, a[1], bounds(*v), w) for v in (odd, even))):
        assert torch.equal(p, q) and bool(p.any())


# ---- the fused forms beyond 32-bit offsets ----------------------------------------------

def room(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < nbytes:
        pytest.skip(f"needs {nbytes >> 30} GB")


def test_fused_forms_of_many_rows():
    """2.2e9 values of h, 4.4e9 codes: the last rows, one expert's own, equal the same rows alone."""
    R, I, H, tail = 1080000, 2056, 40, 300
    room(60 << 30)
    assert R * I > 2 ** 31 and R * 2 * I > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(8)
    x, gy = (torch.zeros(R, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-tail:], gy[-tail:] = (P.whole(g, tail, H, dtype=torch.bfloat16) for _ in range(2))
    gate_up, down = P.whole(g, 3, 2 * I, H, dtype=torch.bfloat16) / 16, P.whole(g, 3, H, I, dtype=torch.bfloat16)
    offsets, w = bounds(0, 5, R - tail, R), torch.rand(R, generator=g, device="cuda")
    h, kept = m.si_moe_gateup(x, gate_up, offsets, keep=True)
    one, one_kept = m.si_moe_gateup(x[-tail:].clone(), gate_up[2:], bounds(0, tail), keep=True)
    assert torch.equal(h[-tail:], one) and not h[:-tail].any()
    assert all(torch.equal(a[-tail:], b) for a, b in zip(kept, one_kept)) and not kept[0][:-tail].any()
    del h
    got = m.si_moe_down_backward(gy, down, kept, offsets, w)
    want = m.si_moe_down_backward(gy[-tail:].clone(), down[2:], one_kept, bounds(0, tail), w[-tail:].clone())
    assert all(torch.equal(a[-tail:], b) and not a[:-tail].any() for a, b in zip(got, want))
    del got, kept
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [5, 66 * 30])
def test_fused_forms_of_large_matrices(rows):
    """2.2e9 values of gate_up and of down: the last expert's rows equal the same alone."""
    E, I, H = 66, 2056, 8200
    room(24 << 30)
    assert (E - 1) * 2 * I * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(rows)
    offsets = torch.full((E + 1,), 2, dtype=torch.int32, device="cuda")
    offsets[0], offsets[-1] = 0, rows
    one = bounds(0, rows - 2)
    x = P.whole(g, rows, H, dtype=torch.bfloat16)
    gate_up = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    gate_up[-1] = P.whole(g, 2 * I, H, dtype=torch.bfloat16) / 16
    h, kept = m.si_moe_gateup(x, gate_up, offsets, keep=True)
    want, want_kept = m.si_moe_gateup(x[2:].clone(), gate_up[-1:], one, keep=True)
    assert torch.equal(h[2:], want) and bool(want.any()) and all(torch.equal(a[2:], b) for a, b in zip(kept, want_kept))
    del gate_up
    assert (2 * E - 1) * H * I > 2 ** 31
    down = torch.zeros(2 * E, H, I, dtype=torch.bfloat16, device="cuda")
    down[-1] = P.whole(g, H, I, dtype=torch.bfloat16)
    offsets = torch.cat([offsets[:1].expand(E), offsets])
    got = m.si_moe_down_backward(x, down, kept, offsets)
    alone = m.si_moe_down_backward(x[2:].clone(), down[-1:], want_kept, one)
    assert all(torch.equal(a[2:], b) and bool(b.any()) for a, b in zip(got[:2], alone[:2]))
    del down
    torch.cuda.empty_cache()
