"""Calls that the documentation allows and no other test makes: offsets beyond 32
bits, calls on two streams at once, the gradient of weights on unaligned rows."""
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


def raw(seed, lo, hi, *shape):
    """Random codes and scale tiles with bytes in [lo, hi] of n matrices, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r, c = shape[-2:]
    codes = torch.randint(0, 256, (*shape[:-1], c // 2), generator=g, device="cuda", dtype=torch.uint8)
    tiles = torch.randint(lo, hi + 1, (*shape[:-2], *m.mxfp4_scale_shape(r, c)), generator=g, device="cuda", dtype=torch.uint8)
    return codes, tiles


def room(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < nbytes:
        pytest.skip(f"needs {nbytes >> 30} GB")


# ---- offsets beyond 2^31 values --------------------------------------------------

def test_quantiser_beyond_32_bits():
    """The last rows of 2.2e9 values equal the same rows alone; and decoded."""
    r, c = 128 * 8400, 2048
    room(24 << 30)
    x = torch.zeros(r, c, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(256, c, generator=g, device="cuda").to(torch.bfloat16)
    x[-256:] = tail
    codes, scales = m.si_quantize_mxfp4(x)
    want = m.si_quantize_mxfp4(tail)
    assert torch.equal(codes[-256:], want[0]) and torch.equal(scales[-2:], want[1])
    assert not codes[:-256].any() and not scales[:-2].any()
    y = m.si_dequantize_mxfp4(codes, scales, out=x)
    assert torch.equal(y[-256:], m.si_dequantize_mxfp4(*want)) and not y[:-256].any()


@pytest.mark.parametrize("mm,n", [(2 ** 31 // 40 + 4000, 40), (66000, 33000), (64, 2 ** 31 // 64 + 12800)])
def test_product_beyond_32_bits(mm, n):
    """2.2e9 outputs, tall, square and wide: the last rows and columns. Every sum
    of 32 terms is exact (scales of two bytes, products multiples of 2^-4 below
    2^24 of them), so parts equal the whole."""
    room(16 << 30)
    assert mm * n > 2 ** 31
    a, w = raw(2, 126, 127, mm, 32), raw(3, 126, 127, n, 32)
    y = m.si_mxfp4_matmul(*a, *w)
    r0, c0 = (max(0, (s - 1) // 128 * 128 - 128) for s in (mm, n))         # the last two tiles of scales
    part = lambda q, at: (q[0][at:].contiguous(), q[1][at // 128:].contiguous())  # noqa: E731
    want = m.si_mxfp4_matmul(*part(a, r0), *part(w, c0), dtype=torch.float32)
    va, vw = (m.si_dequantize_mxfp4(*p, dtype=torch.float32).double() for p in (part(a, r0), part(w, c0)))
    assert torch.equal(want.double(), va @ vw.T)
    assert torch.equal(y[r0:, c0:], want.to(torch.bfloat16))
    vw = m.si_dequantize_mxfp4(w[0][:256].contiguous(), w[1][:2].contiguous(), dtype=torch.float32).double()[:n]
    assert torch.equal(y[r0:, :256], (va @ vw.T).to(torch.bfloat16))


def test_rows_beyond_32_bits():
    """2.1e9 sorted values: gather, combine and their gradients on the last tokens."""
    T, k, E, H = 131080, 8, 16, 2056
    room(80 << 30)
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    _, position, offsets = m.si_moe_sort(ids, E)
    assert T * k * H > 2 ** 31 and int(position.max()) == T * k - 1
    xs = m.si_moe_gather(x, position, offsets)
    far = (position.long() == T * k - 1).any(1).nonzero()[0]         # the token of the last place
    some = torch.cat([far, torch.arange(T - 300, T, device="cuda")])
    p = position[some].long()
    assert torch.equal(xs[p], x[some][:, None].expand(-1, k, -1))
    # rows of one token are equal: exact in any order up to the rounding of the sums
    y = m.si_moe_combine(xs, position, w)[some].double()
    want = (w[some].double()[..., None] * x[some].double()[:, None]).sum(1)
    terms = (w[some].double()[..., None] * x[some].double()[:, None]).abs().sum(1)
    half = torch.finfo(torch.bfloat16).eps / 2
    tol = k * 2.0 ** -24 * terms
    assert bool(((y - want).abs() <= tol + half * (want.abs() + tol)).all())
    gx = m.si_moe_gather_backward(xs, position)[some].double()
    want = k * x[some].double()
    tol = k * 2.0 ** -24 * want.abs()
    assert bool(((gx - want).abs() <= tol + half * (want.abs() + tol)).all())
    gys, gw = m.si_moe_combine_backward(x, xs, position, offsets, w)
    want = (w[some][..., None] * x[some].float()[:, None]).to(torch.bfloat16)          # one product, one rounding
    assert torch.equal(gys[p], want)
    want = (x[some].double() ** 2).sum(1, keepdim=True).expand(-1, k)
    assert bool(((gw[some].double() - want).abs() <= (H + 1) * 2.0 ** -24 * want).all())


def test_experts_beyond_32_bits():
    """2.2e9 values in the rows of the pairs: the last tokens equal their own batch."""
    T, E, k, H, I = 270000, 16, 8, 1024, 32
    room(40 << 30)
    experts = m.Mxfp4Experts(raw(5, 122, 123, E, I, H), raw(6, 122, 123, E, I, H), raw(7, 122, 123, E, H, I))
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda")
    assert T * k * H > 2 ** 31
    ws = m.workspace(m.ffn_mxfp4_workspace_bytes(experts, T, k))
    y = m.si_moe_ffn_mxfp4(experts, x, ids, w, ws=ws)
    assert m.si_workspace_status(ws) == m.SI_OK
    for a, b in ((0, 50), (T // 2, T // 2 + 3000), (T - 50, T)):
        assert torch.equal(y[a:b], m.si_moe_ffn_mxfp4(experts, x[a:b], ids[a:b], w[a:b]))


def test_experts_of_the_most_pairs():
    """2^24 pairs are taken, one token more is refused."""
    T, E, k, H, I = 2 ** 21, 4, 8, 32, 32
    room(40 << 30)
    experts = m.Mxfp4Experts(raw(9, 122, 123, E, I, H), raw(10, 122, 123, E, I, H), raw(11, 122, 123, E, H, I))
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(T + 1, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T + 1, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand(T + 1, k, generator=g, device="cuda")
    y = m.si_moe_ffn_mxfp4(experts, x[:T], ids[:T], w[:T])
    for a, b in ((0, 100), (T - 100, T)):
        assert torch.equal(y[a:b], m.si_moe_ffn_mxfp4(experts, x[a:b], ids[a:b], w[a:b]))
    with pytest.raises((ValueError, m.SiError)):
        m.si_moe_ffn_mxfp4(experts, x, ids, w)


# ---- two streams -------------------------------------------------------------------

def test_experts_on_two_streams_at_once():
    """One set of experts, batches of both tile sizes, a workspace a stream."""
    E, k, H, I = 8, 2, 512, 384
    experts = m.Mxfp4Experts(raw(13, 122, 123, E, I, H), raw(14, 122, 123, E, I, H), raw(15, 122, 123, E, H, I))
    g = torch.Generator(device="cuda").manual_seed(16)
    calls = []
    for T in (1, 30, 500, 17, 2000, 3):
        ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.to(torch.int32)
        calls.append((torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16), ids, torch.rand(T, k, generator=g, device="cuda")))
    want = [m.si_moe_ffn_mxfp4(experts, *c) for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [m.workspace(max(m.ffn_mxfp4_workspace_bytes(experts, c[0].shape[0], k) for c in calls)) for _ in streams]
    torch.cuda.synchronize()
    got = [(i, m.si_moe_ffn_mxfp4(experts, *calls[i], ws=ws[s], stream=streams[s]))
           for r in range(4) for i in range(len(calls)) for s in ((i + r) % 2,)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)
    assert all(m.si_workspace_status(q) == m.SI_OK for q in ws)


# ---- rows that do not start on 16 bytes --------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_weights_gradient_of_unaligned_rows(dtype):
    """Both ways to read the rows are within (H + 1) 2^-24 of the terms' magnitudes."""
    T, k, E, H = 11, 3, 6, 64
    g = torch.Generator(device="cuda").manual_seed(17)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    gy, ys, w = (torch.randn(*s, generator=g, device="cuda") for s in ((T, H), (T * k, H), (T, k)))
    gy, ys = gy.to(dtype), ys.to(dtype)
    _, position, offsets = m.si_moe_sort(ids, E)
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    prod = gy.double()[:, None] * ys.double()[position.long()]
    for a, b in ((gy, ys), (off(gy), off(ys))):
        gw = m.si_moe_combine_backward(a, b, position, offsets, w)[1].double()
        assert bool(((gw - prod.sum(2)).abs() <= (H + 1) * 2.0 ** -24 * prod.abs().sum(2)).all())
