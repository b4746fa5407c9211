"""Measured cases of the products grouped by expert and of the 8-bit activation
checkpoints, with their plain forms.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a
seed, ``run`` makes one pass over them: in elementary torch operations where
``own`` is false, through the framework's calls where it is true. ``exact`` gives
the same outputs from the definitions in 64 bits.

Sorted rows: the (token, rank) pairs ordered by expert, expert e at rows
offsets[e] .. offsets[e + 1]; rows behind the last expert's belong to none (pairs of
experts on another partition) and give zeros.

  product     y[r] = w[e(r)] x[r]
  gradients   gx[r] = w[e(r)]^T gy[r], gw[e] = sum over its rows of gy[r] x[r]^T

8-bit checkpoint (OCP MXINT8): 32 neighbours share X = 2^(s - 127), s the exponent
field of the largest magnitude; code = x / X * 64 rounded to nearest even, within
+-127; value = code * X / 64.

SwiGLU   h = silu(g) u, and backwards from the kept 8-bit g and u
  gg = c gh u s (1 + g (1 - s)), gu = c gh g s, ch = c g s u, gc = <gh, g s u>
with s the logistic function of g and c a row's routing weight.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token's gate and up rows over its 8 experts of 128: the latency of a decode step
        {"name": "product_1", "op": "product", "t": 1, "k": 8, "experts": 128, "rows": 1536, "cols": 2048, "type": "bf16", "out": "bf16", "local": False},
        # the down rows of a decode batch of 64 tokens
        {"name": "product_64", "op": "product", "t": 64, "k": 8, "experts": 128, "rows": 2048, "cols": 768, "type": "bf16", "out": "bf16", "local": False},
        # a partition that owns half of 100 experts: ragged, odd widths, half precision to fp32
        {"name": "product_part", "op": "product", "t": 201, "k": 5, "experts": 100, "rows": 1000, "cols": 1448, "type": "f16", "out": "f32", "local": True},
        # a prompt of 8192 tokens over 8 wide experts, top-2: bound by arithmetic
        {"name": "product_8192", "op": "product", "t": 8192, "k": 2, "experts": 8, "rows": 4096, "cols": 4096, "type": "bf16", "out": "bf16", "local": False},
        # both gradients of a training micro-batch of 4096 tokens
        {"name": "gradients_4096", "op": "gradients", "t": 4096, "k": 8, "experts": 128, "rows": 1536, "cols": 2048, "type": "bf16", "local": False},
        # both gradients on a small partition, half precision, odd widths
        {"name": "gradients_part", "op": "gradients", "t": 301, "k": 3, "experts": 20, "rows": 520, "cols": 712, "type": "f16", "local": True},
        # one row kept in 8 bits and read again
        {"name": "keep_1", "op": "keep", "rows": 1, "cols": 2048, "type": "bf16"},
        # the sorted rows of 4096 tokens, top-8, kept and read again
        {"name": "keep_32768", "op": "keep", "rows": 32768, "cols": 2048, "type": "bf16"},
        # SwiGLU of the same rows (expert width 768), kept in 8 bits, and its backward pass
        {"name": "swiglu_4096", "op": "swiglu", "t": 4096, "k": 8, "experts": 128, "inter": 768, "type": "bf16", "local": False},
        # the same on a partition: odd width, fp32
        {"name": "swiglu_part", "op": "swiglu", "t": 201, "k": 5, "experts": 100, "inter": 1000, "type": "f32", "local": True},
        # a training step through the experts of a layer: 64 tokens, and a micro-batch of 4096
        {"name": "train_64", "op": "train", "t": 64, "k": 8, "experts": 128, "hidden": 2048, "inter": 768, "type": "bf16"},
        {"name": "train_4096", "op": "train", "t": 4096, "k": 8, "experts": 128, "hidden": 2048, "inter": 768, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["product", "gradients", "keep", "swiglu", "train"])
    if op == "keep":
        cols = _log(rng, 8, 8192)
        rows = _log(rng, 1, max(1, min(32768, 32768 * 2048 // (2 * cols))))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "f16", "f32"])}
    k = rng.randint(1, 8)
    if op == "swiglu":
        inter = 8 * _log(rng, 4, 512)
        t = _log(rng, 1, max(1, min(8192, 4096 * 8 * 768 // (2 * k * inter))))
        return {"op": op, "t": t, "k": k, "experts": _log(rng, 8, 256), "inter": inter, "type": rng.choice(["bf16", "f16", "f32"]), "local": rng.random() < 0.3}
    experts = _log(rng, 8, 256)
    if op == "train":
        hidden, inter = 8 * _log(rng, 32, 512), 32 * _log(rng, 2, 32)
        experts = max(8, min(experts, 64 * 768 * 2048 // (hidden * inter)))
        return {"op": op, "t": _log(rng, 1, 2048), "k": k, "experts": experts, "hidden": hidden, "inter": inter, "type": rng.choice(["bf16", "f16"])}
    rows, cols = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512)
    experts = max(8, min(experts, 64 * 1536 * 2048 // (rows * cols)))
    t = _log(rng, 1, max(1, min(8192, 4096 * 8 * 1536 * 2048 // (2 * k * rows * cols))))
    case = {"op": op, "t": t, "k": k, "experts": experts, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "f16"]), "local": rng.random() < 0.3}
    return {**case, "out": rng.choice([case["type"], "f32"])} if op == "product" else case


# ---- inputs ----------------------------------------------------------------

def _activations(g, rows, cols, dtype):
    """Rows of unit normal values, each row at a scale of its own."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (x * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))).to(dtype)


def _routing(g, t, experts, k):
    """Distinct experts of every token in rank order and their softmax weights;
    some experts are in more demand than others."""
    logits = torch.randn(t, experts, generator=g, device="cuda") + 0.5 * torch.randn(experts, generator=g, device="cuda")
    top = torch.topk(logits, k, dim=1)
    return top.indices.to(torch.int32), torch.softmax(top.values, 1)


def _weights(g, experts, rows, cols, dtype):
    """Matrices of normal weights, filled one expert at a time."""
    w = torch.empty(experts, rows, cols, dtype=dtype, device="cuda")
    for e in range(experts):
        w[e] = torch.randn(rows, cols, generator=g, device="cuda") * 0.02
    return w


def _sort(ids, n):
    """Stable order of the (token, rank) pairs by expert: (order, position,
    offsets); pairs of experts outside [0, n) are dropped."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < n), flat, torch.full_like(flat, n))
    perm = torch.sort(key, stable=True).indices
    position = torch.empty_like(perm)
    position[perm] = torch.arange(flat.numel(), device=ids.device)
    offsets = torch.searchsorted(key[perm].contiguous(), torch.arange(n + 1, device=ids.device))
    position = torch.where(key < n, position, torch.full_like(position, -1)).reshape(ids.shape)
    order = torch.where(key[perm] < n, perm, torch.full_like(perm, -1))
    return order.to(torch.int32), position.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s, dtype = case["op"], dict(case), DTYPES[case["type"]]
    if op == "keep":
        s["x"] = _activations(g, case["rows"], case["cols"], dtype)
        return s
    t, k, experts = case["t"], case["k"], case["experts"]
    s["ids"], s["c"] = _routing(g, t, experts, k)
    # a partition that owns the first half of the experts drops the other pairs
    s["n"] = max(1, experts // 2) if case.get("local") else experts
    s["order"], s["position"], s["offsets"] = _sort(s["ids"], s["n"])
    s["most"] = max(1, int((s["offsets"][1:] - s["offsets"][:-1]).max()))   # rows of the longest expert, for padding
    pairs = t * k
    if op == "train":
        h, i = case["hidden"], case["inter"]
        s["x"], s["gy"] = _activations(g, t, h, dtype), _activations(g, t, h, dtype)
        s["c"] = s["c"].to(dtype)                # a router in the model's type
        s["gate_up"], s["down"] = _weights(g, experts, 2 * i, h, dtype), _weights(g, experts, h, i, dtype)
        s["leaves"] = [s[n].requires_grad_() for n in ("x", "c", "gate_up", "down")]
    elif op == "swiglu":
        s["gu"] = _activations(g, pairs, 2 * case["inter"], dtype)
        s["gh"] = torch.randn(pairs, case["inter"], generator=g, device="cuda").to(dtype)
    else:
        s["x"] = _activations(g, pairs, case["cols"], dtype)
        s["w"] = _weights(g, s["n"], case["rows"], case["cols"], dtype)
        if op == "gradients":
            s["gy"] = torch.randn(pairs, case["rows"], generator=g, device="cuda").to(dtype)
    return s


# ---- plain forms -----------------------------------------------------------

def _kept_values(x):
    """The values that the 8-bit codes of the rows of x stand for."""
    cols = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -cols % 32))
    v = v.reshape(*x.shape[:-1], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    s = (torch.frexp(top).exponent.to(torch.int32) - 1 + 127).clamp(0, 254)
    s = torch.where(top > 0, s, torch.zeros_like(s))
    up = torch.where(s == 254, torch.full_like(s, 1 << 22), (254 - s) << 23).view(torch.float32)   # 2^(127 - s)
    down = torch.where(s == 0, torch.full_like(s, 1 << 22), s << 23).view(torch.float32)           # 2^(s - 127)
    q = torch.round(v * up * 64).clamp(-127, 127) / 64 * down
    q = torch.where(torch.isfinite(top), q, torch.full_like(q, float("nan")))
    return q.reshape(*x.shape[:-1], -1)[..., :cols]


def _places(offsets, rows):
    """(expert, place among its rows, whether it has one) of every sorted row;
    rows of no expert are put behind the last one."""
    r = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long().contiguous(), r, right=True)
    return e, r - offsets[e.clamp(max=offsets.numel() - 1)].long(), e < offsets.numel() - 1


def _pad(v, e, slot, live, experts, most):
    """[experts, most, cols] with the sorted rows side by side, zeros elsewhere."""
    out = torch.zeros(experts + 1, most, v.shape[-1], device=v.device)
    out[e, torch.where(live, slot, torch.zeros_like(slot))] = v.float()
    return out[:experts]


def _unpad(v, e, slot, live):
    """The sorted rows of a padded batch, zeros for rows of no expert."""
    got = v[torch.where(live, e, torch.zeros_like(e)), torch.where(live, slot, torch.zeros_like(slot))]
    return torch.where(live[:, None], got, torch.zeros_like(got))


def _product(s, x, w):
    """Sorted rows x through their experts' matrices w [experts, rows, cols]."""
    e, slot, live = _places(s["offsets"], x.shape[0])
    if x.shape[0] <= 32:   # few rows: their experts' matrices alone
        y = (w[torch.where(live, e, torch.zeros_like(e))].float() @ x.float()[..., None])[..., 0]
        return torch.where(live[:, None], y, torch.zeros_like(y))
    return _unpad(_pad(x, e, slot, live, w.shape[0], s["most"]) @ w.float().transpose(1, 2), e, slot, live)


def _weights_gradient(s, gy, x, experts):
    e, slot, live = _places(s["offsets"], x.shape[0])
    put = lambda v: _pad(v, e, slot, live, experts, s["most"])  # noqa: E731
    return put(gy).transpose(1, 2) @ put(x)


def _swiglu(g, u):
    return g / (1 + torch.exp(-g)) * u


def _swiglu_back(g, u, gh, c):
    """(gg, gu, c h, gradient of c) of h = silu(g) u, c a column of row weights."""
    s = 1 / (1 + torch.exp(-g))
    h = g * s * u
    return c * gh * u * s * (1 + g * (1 - s)), c * gh * g * s, c * h, (gh * h).sum(1)


def _row_weights(s, c):
    """c [t, k] in sorted order, 0 for rows of no expert."""
    order = s["order"].long()
    got = c.float().reshape(-1)[order.clamp(min=0)]
    return torch.where(order >= 0, got, torch.zeros_like(got))[:, None]


def _by_pair(s, v):
    """Values of the sorted rows [t * k] back to [t, k], 0 for dropped pairs."""
    at = s["position"].long()
    got = v[at.clamp(min=0)]
    return torch.where((at >= 0).reshape(*at.shape, *[1] * (v.dim() - 1)), got, torch.zeros_like(got))


def _plain(s):
    op, dtype = s["op"], DTYPES[s["type"]]
    if op == "keep":
        return {"values": _kept_values(s["x"]).to(dtype)}
    if op == "product":
        return {"y": _product(s, s["x"], s["w"]).to(DTYPES[s["out"]])}
    if op == "gradients":
        gx = _product(s, s["gy"], s["w"].transpose(1, 2))
        return {"gx": gx.to(dtype), "gw": _weights_gradient(s, s["gy"], s["x"], s["n"]).to(dtype)}
    c, i = _row_weights(s, s["c"]), s["inter"]
    if op == "swiglu":
        gu = s["gu"].float()
        kept = [_kept_values(v) for v in (gu[:, :i], gu[:, i:])]
        gg, gu_, ch, gc = _swiglu_back(*kept, s["gh"].float(), c)
        return {"h": _swiglu(gu[:, :i], gu[:, i:]).to(dtype), "ggu": torch.cat([gg, gu_], 1).to(dtype), "ch": ch.to(dtype), "gc": _by_pair(s, gc)}
    k, x, gy, gate_up, down = s["k"], s["x"].detach().float(), s["gy"].float(), s["gate_up"].detach(), s["down"].detach()
    token = s["order"].long() // k             # every pair is kept
    gu = _product(s, x[token], gate_up)
    y = _product(s, _swiglu(gu[:, :i], gu[:, i:]), down)
    y = (_by_pair(s, y) * s["c"].detach().float()[..., None]).sum(1)
    gh = _product(s, gy[token], down.transpose(1, 2))
    gg, gu_, ch, gc = _swiglu_back(_kept_values(gu[:, :i]), _kept_values(gu[:, i:]), gh, c.detach())
    ggu = torch.cat([gg, gu_], 1)
    gx = _by_pair(s, _product(s, ggu, gate_up.transpose(1, 2))).sum(1)
    gw = _weights_gradient(s, ggu, x[token], s["n"]), _weights_gradient(s, gy[token], ch, s["n"])
    return {"y": y.to(dtype), "gx": gx.to(dtype), "gc": _by_pair(s, gc).to(dtype), "ggate_up": gw[0].to(dtype), "gdown": gw[1].to(dtype)}


# ---- the framework's calls -------------------------------------------------

def _framework(s):
    import moe_decode_ffn_gb300 as m
    op, dtype = s["op"], DTYPES[s["type"]]
    if op == "keep":
        return {"values": m.si_dequantize_mxint8(*m.si_quantize_mxint8(s["x"]), dtype=dtype)}
    if op == "product":
        return {"y": m.si_moe_matmul(s["x"], s["w"], s["offsets"], dtype=DTYPES[s["out"]])}
    if op == "gradients":
        gx, gw = m.si_moe_matmul_backward(s["gy"], s["x"], s["w"], s["offsets"])
        return {"gx": gx, "gw": gw}
    if op == "swiglu":
        h, kept = m.si_swiglu(s["gu"], keep=True)
        ggu, ch, gc = m.si_swiglu_backward(s["gh"], kept, s["c"], s["order"])
        return {"h": h, "ggu": ggu, "ch": ch, "gc": gc}
    x, c, gate_up, down = s["leaves"]
    y = m.si_moe_experts(x, s["ids"], c.float(), gate_up, down)
    grads = torch.autograd.grad(y, s["leaves"], s["gy"])
    return {"y": y.detach(), "gx": grads[0], "gc": grads[1], "ggate_up": grads[2], "gdown": grads[3]}


def run(state):
    return _framework(state) if own else _plain(state)


def work(case):
    op, size = case["op"], SIZE[case["type"]]
    if op == "keep":
        # the values are read, their codes and scales written, read, and the values written
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * size + 2 * 33 / 32), "flops": 4 * n}
    pairs = case["t"] * case["k"]
    kept = pairs / (2 if case.get("local") else 1)
    if op == "swiglu":
        # backwards: codes, scales and gh in, ggu and the weighted h out
        i = case["inter"]
        return {"bytes": i * (pairs * (6 * size + 2 * 33 / 32) + kept * (size + 2 * 33 / 32)), "flops": 30 * pairs * i}
    # the matrices of the experts that at least one token takes
    here = case["experts"] // 2 if case.get("local") else case["experts"]
    taken = here * (1 - (1 - case["k"] / case["experts"]) ** case["t"])
    if op == "train":
        t, h, i = case["t"], case["hidden"], case["inter"]
        # forward and backward read x, gy and the matrices, the codes go out and come
        # back; y, gx and the matrices' gradients (of every expert) are written
        acts = 6 * t * h * size + pairs * 4 * i * 33 / 32
        return {"bytes": acts + (2 * taken + case["experts"]) * 3 * h * i * size, "flops": 18 * pairs * h * i}
    n, k = case["rows"], case["cols"]
    if op == "product":
        return {"bytes": kept * k * size + taken * n * k * size + pairs * n * SIZE[case["out"]], "flops": 2 * kept * n * k}
    return {"bytes": (2 * kept * (n + k) + (pairs - kept) * k) * size + (taken + here) * n * k * size, "flops": 4 * kept * n * k}


# ---- the definitions in 64 bits ----------------------------------------------

def _pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _kept64(x):
    """x [rows, cols] after MXINT8, block by block of a row."""
    v, out = x.double(), []
    for b in range(0, v.shape[1], 32):
        p = v[:, b:b + 32]
        top = p.abs().amax(1, keepdim=True)
        e = torch.where(top > 0, torch.frexp(top).exponent.double() - 1, torch.full_like(top, -127)).clamp(min=-127)
        unit = _pow2(e - 6)
        out.append((torch.round(p / unit)).clamp(-127, 127) * unit)
    return torch.cat(out, 1)


def _sorted64(s):
    """Per expert: its places and its pairs, from the ids alone."""
    flat = s["ids"].reshape(-1).long()
    at, got = 0, []
    for e in range(s["n"]):
        pair = torch.nonzero(flat == e)[:, 0]
        got.append((slice(at, at + pair.numel()), pair))
        at += pair.numel()
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op, zeros = case["op"], lambda *n: torch.zeros(*n, dtype=torch.float64, device="cuda")
    if op == "keep":
        return {"values": _kept64(s["x"])}
    lists, pairs = _sorted64(s), case["t"] * case["k"]
    if op == "product":
        y = zeros(pairs, case["rows"])
        for e, (rows, _) in enumerate(lists):
            y[rows] = s["x"][rows].double() @ s["w"][e].double().T
        return {"y": y}
    if op == "gradients":
        gx, gw = zeros(pairs, case["cols"]), zeros(s["n"], case["rows"], case["cols"])
        for e, (rows, _) in enumerate(lists):
            gy = s["gy"][rows].double()
            gx[rows], gw[e] = gy @ s["w"][e].double(), gy.T @ s["x"][rows].double()
        return {"gx": gx, "gw": gw}
    i, c = case["inter"], s["c"].detach().double().reshape(-1)
    back = lambda g, u, gh, c: (c * gh * u * (torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)), c * gh * torch.nn.functional.silu(g))  # noqa: E731
    if op == "swiglu":
        gu, gh = s["gu"].double(), s["gh"].double()
        qg, qu = _kept64(s["gu"][:, :i]), _kept64(s["gu"][:, i:])
        row_c, gc, qh = zeros(pairs, 1), zeros(pairs), torch.nn.functional.silu(qg) * qu
        for rows, pair in lists:
            row_c[rows, 0] = c[pair]
            gc[pair] = (gh[rows] * qh[rows]).sum(1)
        return {"h": torch.nn.functional.silu(gu[:, :i]) * gu[:, i:], "ggu": torch.cat(back(qg, qu, gh, row_c), 1), "ch": row_c * qh, "gc": gc.reshape(case["t"], -1)}
    t, h, k = case["t"], case["hidden"], case["k"]
    x, gy = s["x"].detach().double(), s["gy"].double()
    y, gx, gc = zeros(t, h), zeros(t, h), zeros(pairs)
    ggate_up, gdown = zeros(s["n"], 2 * i, h), zeros(s["n"], h, i)
    for e, (_, pair) in enumerate(lists):
        up, down, tok, w = s["gate_up"][e].detach().double(), s["down"][e].detach().double(), pair // k, c[pair][:, None]
        gu = x[tok] @ up.T
        y.index_add_(0, tok, w * ((torch.nn.functional.silu(gu[:, :i]) * gu[:, i:]) @ down.T))
        qg, qu, gh = _kept64(gu[:, :i]), _kept64(gu[:, i:]), gy[tok] @ down
        qh = torch.nn.functional.silu(qg) * qu
        gc[pair] = (gh * qh).sum(1)
        ggu = torch.cat(back(qg, qu, gh, w), 1)
        gx.index_add_(0, tok, ggu @ up)
        ggate_up[e], gdown[e] = ggu.T @ x[tok], gy[tok].T @ (w * qh)
    return {"y": y, "gx": gx, "gc": gc.reshape(t, k), "ggate_up": ggate_up, "gdown": gdown}
