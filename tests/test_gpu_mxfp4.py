"""MXFP4 quantisation, products and the MXFP4 expert FFN against the fp64 oracle.

Tolerances. Quantisation is exact. Inputs of the products are chosen so that
every partial sum of every dot is a multiple of one quantum below 2^24 of them
(asserted on the host): the fp32 accumulators are then exact in any order, and
only the rounding to the output type is allowed for, half a unit in the last
place (finfo.eps / 2 relative).
"""
import os
import subprocess
import sys

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


def rows(seed, r, c, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(r, c, generator=g) * torch.exp2(torch.randint(-3, 4, (r, 1), generator=g) * spread / 2)
    return x.to(dtype)


def coded(seed, r, c, lo=125, hi=129):
    """Random codes and scales in [2^(lo-127), 2^(hi-127)]: (numpy codes, scale bytes)."""
    g = np.random.default_rng(seed)
    return g.integers(0, 16, (r, c), dtype=np.uint8), g.integers(lo, hi + 1, (r, c // 32), dtype=np.uint8)


def on_gpu(codes, s):
    return torch.from_numpy(X.pack(codes)).cuda(), torch.from_numpy(X.tile(s)).cuda()


def half_ulp(dtype):
    return torch.finfo(dtype).eps / 2


# ---- quantisation ------------------------------------------------------------

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("r,c", [(1, 32), (1, 2048), (3, 96), (127, 160), (128, 128), (130, 544), (257, 64)])
def test_quantize_bytes(kind, r, c):
    x = rows(r * 7 + c, r, c, TYPES[kind])
    codes, scales = m.si_quantize_mxfp4(x.cuda())
    oc, os = X.quantize(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), X.pack(oc))
    assert np.array_equal(scales.cpu().numpy(), X.tile(os))      # zeros outside the matrix among them
    for out in TYPES.values():
        y = m.si_dequantize_mxfp4(codes, scales, dtype=out)
        want = torch.from_numpy(X.values(oc, os)).to(out)
        assert torch.equal(y.cpu(), want)


def test_quantize_borders_and_ties():
    """Every border between two codes, each side of it, at several scales."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.999])
    v = np.concatenate([borders, np.nextafter(borders.astype(np.float32), np.float32(0)),
                        np.nextafter(borders.astype(np.float32), np.float32(9))])
    blk = np.zeros((2, 64))
    blk[0, :27], blk[1, :27] = v, -v
    blk[:, 31] = 7.9
    blk[0, 32:59], blk[1, 32:59], blk[:, 63] = -v, v, -7.5
    x = np.concatenate([np.ldexp(blk, e) for e in (0, -130, -147, 100, 124)]).astype(np.float32)
    codes, scales = m.si_quantize_mxfp4(torch.from_numpy(x).cuda())
    oc, os = X.quantize(x.astype(np.float64))
    assert np.array_equal(codes.cpu().numpy(), X.pack(oc))
    assert np.array_equal(scales.cpu().numpy(), X.tile(os))


def test_quantize_extremes():
    x = torch.zeros(8, 128)
    x[0, 5], x[1, 40], x[2, 70] = float("inf"), float("nan"), -float("inf")
    x[3] = torch.finfo(torch.float32).max
    x[4] = 2.0 ** -149
    x[5, ::2] = -0.0
    x[6] = 2.0 ** -126
    x[7, 32:64] = 65504.0
    codes, scales = m.si_quantize_mxfp4(x.cuda())
    oc, os = X.quantize(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), X.pack(oc))
    assert np.array_equal(scales.cpu().numpy(), X.tile(os))
    y = m.si_dequantize_mxfp4(codes, scales, dtype=torch.float32).cpu()
    assert torch.equal(torch.nan_to_num(y, nan=-1.5), torch.nan_to_num(torch.from_numpy(X.values(oc, os)).float(), nan=-1.5))
    # fp16 overflows to infinity where a value is beyond it
    assert torch.isinf(m.si_dequantize_mxfp4(codes, scales, dtype=torch.float16)[3]).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_quantize_strides_and_alignment(kind):
    """Rows and matrices at odd strides, a base that is not 16-byte aligned; the
    values between the rows are neither read into the result nor written."""
    big = rows(5, 3 * 70, 331, TYPES[kind]).cuda()
    view = big.view(3, 70, 331)[:, ::2, 3:3 + 96]
    assert view.stride(-1) == 1
    codes, scales = m.si_quantize_mxfp4(view)
    for i in range(3):
        oc, os = X.quantize(view[i].double().cpu().numpy())
        assert np.array_equal(codes[i].cpu().numpy(), X.pack(oc))
        assert np.array_equal(scales[i].cpu().numpy(), X.tile(os))
    out = torch.full((3, 70, 331), 7.0, dtype=TYPES[kind], device="cuda")
    m.si_dequantize_mxfp4(codes, scales, out=out[:, ::2, 3:3 + 96])
    assert torch.equal(out[:, ::2, 3:99].cpu(), m.si_dequantize_mxfp4(codes, scales, dtype=TYPES[kind]).cpu())
    out[:, ::2, 3:99] = 7.0
    assert bool((out == 7.0).all())
    # matrices whose rows lie in turn
    turn = big.view(70, 3, 331)[..., :96].transpose(0, 1)
    codes, scales = m.si_quantize_mxfp4(turn)
    want = m.si_quantize_mxfp4(turn.contiguous())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    with pytest.raises(m.SiError):      # rows that lie on one another
        m.si_quantize_mxfp4(big[:1, :96].expand(4, 96))


def test_quantize_empty():
    codes, scales = m.si_quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and scales.shape == (0, 1, 512)
    codes, scales = m.si_quantize_mxfp4(torch.empty(0, 4, 64, device="cuda"))
    assert codes.shape == (0, 4, 32)


# ---- product -----------------------------------------------------------------

def check_exact_sums(a, w):
    """Every partial sum is a multiple of q with fewer than 2^24 of them."""
    q = min(np.min(np.abs(v[v != 0])) for v in (a, w)) if a.any() and w.any() else 1.0
    qa, qw = (np.ldexp(1.0, int(np.floor(np.log2(np.min(np.abs(v[v != 0])))))) for v in (a, w))
    assert np.max(np.abs(a) @ np.abs(w).T) / (qa * qw / 4) < 2 ** 24, q


PRODUCTS = [(1, 1, 32), (1, 4096, 2048), (2, 130, 64), (16, 128, 96), (17, 257, 160), (32, 384, 256), (33, 64, 288),
            (64, 96, 512), (65, 129, 544), (128, 256, 1024), (129, 300, 1056), (300, 77, 320), (1000, 513, 512)]


@pytest.mark.parametrize("mm,n,k", PRODUCTS)
def test_matmul_exact(mm, n, k):
    ac, asc = coded(mm + n, mm, k, 126, 128)
    wc, wsc = coded(n + k, n, k, 126, 128)
    a, w = X.values(ac, asc), X.values(wc, wsc)
    check_exact_sums(a, w)
    want = a @ w.T
    ga, gw = on_gpu(ac, asc), on_gpu(wc, wsc)
    y = m.si_mxfp4_matmul(*ga, *gw, dtype=torch.float32)
    assert np.array_equal(y.cpu().double().numpy(), want)
    for kind in ("bf16", "f16"):
        y = m.si_mxfp4_matmul(*ga, *gw, dtype=TYPES[kind]).cpu()
        assert torch.equal(y, torch.from_numpy(want).to(TYPES[kind]))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("mm,n,k,pad", [(2500, 2088, 96, 0), (1290, 4356, 320, 0), (2600, 2056, 64, 24), (2049, 2500, 544, 4),
                                        (2500, 2088, 1024, 0), (2500, 2088, 1120, 0), (2600, 2056, 1056, 8), (2049, 2500, 1152, 4)])
def test_matmul_of_many_tokens(mm, n, k, pad, kind):
    """Enough tiles for the tokens to lie on the lanes: ragged in tokens, in the
    256 rows of a tile and (one tile of 128 left) in their halves, odd columns,
    rows of whole 16-byte words and others; up to 1024 columns, whose outputs go
    through shared memory, and more."""
    g = torch.Generator(device="cuda").manual_seed(mm + n)
    draw = lambda r, hi: torch.randint(0, hi, r, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    ac, asc = draw((mm, k), 16).cpu().numpy().astype(np.uint8), (126 + draw((mm, k // 32), 3)).cpu().numpy().astype(np.uint8)
    wc, wsc = draw((n, k), 16).cpu().numpy().astype(np.uint8), (126 + draw((n, k // 32), 3)).cpu().numpy().astype(np.uint8)
    a, w = X.values(ac, asc), X.values(wc, wsc)
    check_exact_sums(a, w)
    want = torch.from_numpy(a @ w.T).to(TYPES[kind])
    out = torch.full((mm, n + pad), 9.0, dtype=TYPES[kind], device="cuda")
    m.si_mxfp4_matmul(*on_gpu(ac, asc), *on_gpu(wc, wsc), out=out[:, :n])
    assert torch.equal(out[:, :n].cpu(), want)
    assert bool((out[:, n:] == 9.0).all())


def test_matmul_of_the_whole_code_range():
    """Scales far apart: the fp32 sum of k terms is off by at most
    k 2^-23 sum |a||w| (each addition rounds or truncates the running sum)."""
    mm, n, k = 40, 200, 512
    ac, asc = coded(1, mm, k, 90, 160)
    wc, wsc = coded(2, n, k, 90, 160)
    a, w = X.values(ac, asc), X.values(wc, wsc)
    y = m.si_mxfp4_matmul(*on_gpu(ac, asc), *on_gpu(wc, wsc), dtype=torch.float32).cpu().double().numpy()
    assert np.all(np.abs(y - a @ w.T) <= k * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T))


def test_matmul_nan_scales_stay_in_their_row():
    ac, asc = coded(3, 20, 128)
    wc, wsc = coded(4, 200, 128)
    asc[7, 2] = 255
    wsc[150, 0] = 255
    y = m.si_mxfp4_matmul(*on_gpu(ac, asc), *on_gpu(wc, wsc), dtype=torch.float32).cpu().numpy()
    bad = np.zeros((20, 200), dtype=bool)
    bad[7], bad[:, 150] = True, True
    assert np.array_equal(np.isnan(y), bad)


def test_matmul_into_strided_output():
    ac, asc = coded(5, 50, 96)
    wc, wsc = coded(6, 70, 96)
    out = torch.full((50, 101), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = m.workspace(m.mxfp4_matmul_workspace_bytes(50, 70, 96))
    m.si_mxfp4_matmul(*on_gpu(ac, asc), *on_gpu(wc, wsc), out=out[:, 5:75], ws=ws)
    assert m.si_workspace_status(ws) == m.SI_OK
    want = torch.from_numpy(X.values(ac, asc) @ X.values(wc, wsc).T).to(torch.bfloat16)
    assert torch.equal(out[:, 5:75].cpu(), want)
    out[:, 5:75] = 3.0
    assert bool((out == 3.0).all())


def test_matmul_graph_and_streams():
    """A captured product replays on new contents; calls on two streams at once."""
    ac, asc = coded(7, 24, 256)
    wc, wsc = coded(8, 300, 256)
    want = torch.from_numpy(X.values(ac, asc) @ X.values(wc, wsc).T).to(torch.bfloat16)
    (a, sa), (w, sw) = on_gpu(ac, asc), on_gpu(wc, wsc)
    ws, out = m.workspace(256), torch.zeros(24, 300, dtype=torch.bfloat16, device="cuda")
    m.si_mxfp4_matmul(a, sa, w, sw, out=out, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        m.si_mxfp4_matmul(a, sa, w, sw, out=out, ws=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    a.bitwise_xor_(0x88)                 # every sign flipped
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), -want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [m.si_mxfp4_matmul(a, sa, w, sw, stream=streams[i % 2]) for i in range(16)]
    torch.cuda.synchronize()
    assert all(torch.equal(y.cpu(), -want) for y in got)


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: nothing that a capture forbids
    happens in them."""
    code = """
import torch, moe_decode_ffn_gb300 as m
x = torch.randn(40, 256, device="cuda").to(torch.bfloat16)
ids = torch.randint(0, 4, (40, 2), device="cuda", dtype=torch.int32)
w = torch.rand(40, 2, device="cuda")
gate, up, down = (torch.randn(4, 128, 256, device="cuda"), torch.randn(4, 128, 256, device="cuda"), torch.randn(4, 256, 128, device="cuda"))
def step():
    e = m.Mxfp4Experts.quantize(gate, up, down)
    y = m.si_moe_ffn_mxfp4(e, x, ids, w)
    c, s = m.si_quantize_mxfp4(x)
    z = m.si_mxfp4_matmul(c, s, *m.si_quantize_mxfp4(gate[0]))
    o, p, f = m.si_moe_sort(ids, 4)
    xs = m.si_moe_gather(x, p, f)
    g = m.si_moe_combine_backward(x, xs, p, f, w)
    return y, z, m.si_moe_combine(xs, p, w), m.si_moe_gather_backward(xs, p), *g, m.si_dequantize_mxfp4(c, s), e
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out[:-1], step()[:-1]))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


# ---- expert FFN --------------------------------------------------------------

def make_experts(seed, E, H, I):
    parts = []
    for j, (r, c) in enumerate(((I, H), (I, H), (H, I))):
        # codes with scales near 2^-4 .. 2^-3: h of order one
        cs = [coded(seed * 97 + j * 31 + e, r, c, 122, 123) for e in range(E)]
        parts.append(cs)
    gpu = [tuple(torch.stack(t) for t in zip(*(on_gpu(*c) for c in p))) for p in parts]
    return [[X.values(*c) for c in p] for p in parts], m.Mxfp4Experts(*gpu)


def ffn_oracle(weights, x, ids, w, E):
    """(routed, tolerance) in fp64. h differs from the device's fp32 h by at
    most 2^-18 relative (the exponential, the division and two products, each a
    few 2^-23; |g| < 32 asserted), which may put a value on the other side of a
    border between two codes: the tolerance takes both sides. y is rounded to
    bf16, the sum over ranks is fp32 (8 terms), the result bf16."""
    gate, up, down = weights
    xq = X.round_trip(x)
    T, k = ids.shape
    out, tol = np.zeros(x.shape), np.zeros(x.shape)
    half = half_ulp(torch.bfloat16)
    for t in range(T):
        for r in range(k):
            e = int(ids[t, r])
            if not 0 <= e < E:
                continue
            check_exact_sums(xq[t:t + 1], np.concatenate([gate[e], up[e]]))
            g, u = gate[e] @ xq[t], up[e] @ xq[t]
            assert np.max(np.abs(g)) < 32
            h = X.silu(g) * u
            lo, hi = (X.round_trip((h * (1 + d))[None])[0] for d in (-2.0 ** -18, 2.0 ** -18))
            hq = X.round_trip(h[None])[0]
            # the additions of the down product: at most I of them
            s = np.abs(down[e]) @ np.abs(hq)
            y = down[e] @ hq
            dy = np.abs(down[e]) @ np.abs(hi - lo) + len(h) * 2.0 ** -23 * s + half * np.abs(y)
            out[t] += w[t, r] * y
            tol[t] += abs(w[t, r]) * (dy * (1 + half) + 8 * 2.0 ** -24 * np.abs(y))
    return out, tol + half * (np.abs(out) + tol)


# up to 32 pairs in one launch with the sort, then one or two launches of it; 16
# and 128 tokens a tile
FFN = [(32, 1, 1, 64, 64), (33, 1, 1, 64, 64), (16, 2, 2, 96, 64), (4, 1024, 8, 64, 32), (1, 8, 2, 256, 128), (1, 4, 1, 32, 32), (5, 8, 8, 96, 160), (16, 3, 2, 288, 96), (70, 4, 3, 128, 256),
       (40, 1, 1, 64, 416), (150, 2, 2, 160, 64), (200, 1, 1, 544, 32), (9, 40, 8, 256, 128)]


@pytest.mark.parametrize("T,E,k,H,I", FFN)
def test_ffn_against_oracle(T, E, k, H, I):
    weights, experts = make_experts(T + E, E, H, I)
    g = torch.Generator().manual_seed(T * 13 + E)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(max(E, k), generator=g)[:k] for _ in range(T)]).to(torch.int32)
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    ws = m.workspace(m.ffn_mxfp4_workspace_bytes(experts, T, k))
    y = m.si_moe_ffn_mxfp4(experts, x.cuda(), ids.cuda(), w.cuda(), ws=ws)
    assert m.si_workspace_status(ws) == m.SI_OK
    want, tol = ffn_oracle(weights, x.double().numpy(), ids.numpy(), w.double().numpy(), E)
    err = np.abs(y.cpu().double().numpy() - want)
    assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-30)))


def test_ffn_dropped_repeated_and_unused_experts():
    """Ids outside the experts, the same expert twice in a token, a token that
    keeps no pair, experts without tokens, a workspace used before."""
    E, H, I = 6, 128, 96
    weights, experts = make_experts(77, E, H, I)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(30, H, generator=g).to(torch.bfloat16)
    ids = torch.randint(0, 3, (30, 4), generator=g).to(torch.int32)
    ids[3] = -1
    ids[4] = torch.tensor([6, 1000, -7, 2])
    ids[5] = 2
    w = torch.rand(30, 4, generator=g)
    w[3, 0], w[4, 0] = float("nan"), float("inf")      # weights of dropped pairs
    ws = m.workspace(m.ffn_mxfp4_workspace_bytes(experts, 30, 4))
    ws[256:].fill_(255)                                # what an earlier call may have left
    clean = torch.where(torch.isfinite(w), w, torch.zeros_like(w))
    want, tol = ffn_oracle(weights, x.double().numpy(), ids.numpy(), clean.double().numpy(), E)
    for _ in range(2):
        y = m.si_moe_ffn_mxfp4(experts, x.cuda(), ids.cuda(), w.cuda(), ws=ws).cpu().double().numpy()
        assert np.all(np.abs(y - want) <= tol)
    assert not y[3].any()
    none = m.si_moe_ffn_mxfp4(experts, x.cuda(), torch.full_like(ids, -1).cuda(), w.cuda(), ws=ws)
    assert not none.cpu().any()


def test_ffn_nan_token_stays_in_its_row():
    E, H, I = 4, 64, 64
    _, experts = make_experts(78, E, H, I)
    g = torch.Generator().manual_seed(6)
    x = torch.randn(20, H, generator=g).to(torch.bfloat16)
    ids = torch.randint(0, E, (20, 2), generator=g).to(torch.int32).cuda()
    w = torch.rand(20, 2, generator=g).cuda()
    clean = m.si_moe_ffn_mxfp4(experts, x.cuda(), ids, w).cpu()
    x[11, 3] = float("inf")
    y = m.si_moe_ffn_mxfp4(experts, x.cuda(), ids, w).cpu()
    keep = torch.arange(20) != 11
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[11]).all()


def test_ffn_rows_do_not_depend_on_the_batch():
    """A token's result is the same alone and among others (any tile size), and
    equals the calls that the FFN is made of."""
    E, H, I, k = 4, 256, 128, 2
    _, experts = make_experts(79, E, H, I)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(400, H, generator=g).to(torch.bfloat16).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(400)]).to(torch.int32).cuda()
    w = torch.rand(400, k, generator=g).cuda()
    y = m.si_moe_ffn_mxfp4(experts, x, ids, w)
    for n in (1, 7, 33, 100, 170):
        assert torch.equal(m.si_moe_ffn_mxfp4(experts, x[:n].contiguous(), ids[:n].contiguous(), w[:n].contiguous()),
                           y[:n])


def test_ffn_graph_replay():
    E, H, I, k, T = 8, 256, 128, 2, 40
    _, experts = make_experts(80, E, H, I)
    g = torch.Generator().manual_seed(8)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    ws = m.workspace(m.ffn_mxfp4_workspace_bytes(experts, T, k))
    m.si_moe_ffn_mxfp4(experts, x, ids, w, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = m.si_moe_ffn_mxfp4(experts, x, ids, w, ws=ws)
    for seed in (9, 10):
        g.manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=g))
        ids.copy_(torch.randint(0, E, (T, k), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, m.si_moe_ffn_mxfp4(experts, x, ids, w))
    assert m.si_workspace_status(ws) == m.SI_OK


def test_ffn_marks_weights_as_used_by_the_given_stream():
    """Experts that are let go right after a call on another stream: their memory
    is not handed out again while that stream still has the call before it."""
    E, H, I, k, T = 8, 256, 128, 2, 5
    _, experts = make_experts(81, E, H, I)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    w = torch.rand(T, k, device="cuda")
    want = m.si_moe_ffn_mxfp4(experts, x, ids, w)
    ws = m.workspace(m.ffn_mxfp4_workspace_bytes(experts, T, k))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)      # about 0.1 s
    got = m.si_moe_ffn_mxfp4(experts, x, ids, w, ws=ws, stream=side)
    size = sum(t.numel() for t in (*experts.gate, *experts.up, *experts.down))
    stat = lambda name: torch.cuda.memory_stats()[name + "_bytes.all.current"]  # noqa: E731
    owned, busy = stat("allocated"), stat("active")
    del experts
    assert owned - stat("allocated") >= size        # let go ...
    assert stat("active") == busy                   # ... but not free for others
    assert not side.query()                         # the call still waits
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_layer_of_router_experts_and_norm():
    """A layer as a user builds it: the router, the MXFP4 experts, the residual
    norm; then the same rows through the sorted calls. Captured and replayed on
    other tokens, equal to the calls one by one, and the expert outputs near the
    same chain with fp32 products. There y and the result are rounded to bf16
    (2^-8 each, y in k = 4 terms whose norms add up to about twice the sum's: 3 *
    2^-8 = 0.012 of the norm) and a few h lie on a border between two codes."""
    E, H, I, T, k = 16, 256, 128, 24, 4
    g = torch.Generator(device="cuda").manual_seed(11)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    gate, up, down = draw(E, I, H) * 0.1, draw(E, I, H) * 0.1, draw(E, H, I) * 0.1
    experts = m.Mxfp4Experts.quantize(gate, up, down)
    wr, wn = draw(E, H).to(torch.bfloat16), torch.ones(H, dtype=torch.bfloat16, device="cuda")
    x = draw(T, H).to(torch.bfloat16)
    ws = m.workspace(m.ffn_mxfp4_workspace_bytes(experts, T, k))
    wsr = m.workspace(m.router_workspace_bytes(E, H, T))

    def layer():
        ids, w, _ = m.si_moe_router_topk(x, wr, k, ws=wsr)
        routed = m.si_moe_ffn_mxfp4(experts, x, ids, w, ws=ws)
        s, y, _ = m.si_add_rmsnorm3(routed, x, None, wn)
        order, position, offsets = m.si_moe_sort(ids, E)
        xs = m.si_moe_gather(x, position, offsets)
        return ids, w, routed, s, y, order, xs, m.si_moe_combine(xs, position, w)

    layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = layer()
    for _ in range(2):
        x.copy_(draw(T, H))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, layer()))
    ids, w, routed, s, y, order, xs, comb = got
    assert torch.equal(s, (routed + x))
    # the combine of a token's own rows is the token times the sum of its weights (one)
    assert torch.allclose(comb.float(), x.float(), rtol=2.0 ** -7, atol=2.0 ** -20)
    G, U, D = (m.si_dequantize_mxfp4(*p, dtype=torch.float32) for p in (experts.gate, experts.up, experts.down))
    xq = m.si_dequantize_mxfp4(*m.si_quantize_mxfp4(x), dtype=torch.float32)
    want = torch.zeros(T, H, device="cuda")
    for t in range(T):
        for r in range(k):
            e = int(ids[t, r])
            z = G[e] @ xq[t]
            h = m.si_dequantize_mxfp4(*m.si_quantize_mxfp4((z * torch.sigmoid(z) * (U[e] @ xq[t]))[None]), dtype=torch.float32)[0]
            want[t] += w[t, r] * (D[e] @ h)
    assert float((routed.float() - want).norm() / want.norm()) < 0.02
    assert m.si_workspace_status(ws) == m.SI_OK and m.si_workspace_status(wsr) == m.SI_OK
