"""Measured cases of the operators around a stack of experts' matrices (`experts`
in this repository's package) and of the optimizer step for what is no matrix
(`optim`): tokens sorted by expert and back, with weights applied, and the
gradients; the experts' 8-bit products; a projection of all experts, forward and
backward; and an AdamW step over many tensors with 32-bit or 8-bit moments.
Each has a plain form here, made of elementary torch operations.

The sorted order: choice (i / K, i % K) of T tokens' K choices has the number i.
Expert e's rows begin at offsets[e] and hold its choices in the order of their
numbers; offsets[e + 1] is the next multiple of `align` behind them.  Rows without
a choice are zeros.  A choice outside 0 .. E - 1 is none.

8-bit matrices are held as (codes, scales): blocks of 128 values of a row share a
power-of-two scale, the smallest whose format holds the block's largest value.
8-bit moments hold m and the root of v that way, in e4m3, along a tensor's elements;
they are rounded up where a threshold between 0 and 1, made from the step, the
tensor's place in the list and the element's number, reaches what is left of the
code below, and the root always where it is below the smallest normal code.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
LR, BETA1, BETA2, EPS, DECAY, MAX_NORM = 3e-4, 0.9, 0.999, 1e-8, 0.1, 1.0
MASK = 0xFFFFFFFF


def listed():
    return [
        # norm weights and biases of a 24-layer model: many small tensors, latency
        {"name": "adamw: norms and biases", "op": "adamw", "large": 0, "size": 0, "small": 97, "width": 2048, "grad": "f32", "state": "fp32", "clip": False},
        # an embedding table and the norms of the 1.2B class, 16-bit gradients clipped by their norm over all tensors
        {"name": "adamw: embedding, clipped", "op": "adamw", "large": 1, "size": 50257 * 2048, "small": 49, "width": 2048, "grad": "bf16", "state": "fp32", "clip": True},
        # a d=1024 block's tensors of odd sizes, moments in 8 bits
        {"name": "adamw 8 bits: odd sizes", "op": "adamw", "large": 7, "size": 1023 * 2815, "small": 9, "width": 1023, "grad": "f16", "state": "8bit", "clip": True},
        # eight experts' gate projections of the 1.2B class, moments in 8 bits
        {"name": "adamw 8 bits: expert stack", "op": "adamw", "large": 1, "size": 8 * 5632 * 2048, "small": 0, "width": 0, "grad": "f32", "state": "8bit", "clip": False},
        # a decode step's few tokens to their experts' rows and back: latency
        {"name": "tokens: decode step", "op": "tokens", "tokens": 8, "each": 2, "experts": 8, "width": 4096, "align": 16, "type": "bf16", "dropped": False},
        # a training batch over many experts
        {"name": "tokens: training batch", "op": "tokens", "tokens": 8192, "each": 8, "experts": 64, "width": 2048, "align": 128, "type": "bf16", "dropped": False},
        # its way back
        {"name": "tokens gradient: training", "op": "tokens_grad", "tokens": 8192, "each": 8, "experts": 64, "width": 2048, "align": 128, "type": "bf16", "dropped": False},
        # a short batch of an odd width in fp32, some choices dropped by a capacity limit
        {"name": "tokens gradient: odd, fp32", "op": "tokens_grad", "tokens": 777, "each": 3, "experts": 10, "width": 1111, "align": 128, "type": "f32", "dropped": True},
        # a decode batch through the 6.5B-class up projections of eight experts: the weights' bytes bound it
        {"name": "product: decode batch", "op": "product", "tokens": 16, "each": 2, "experts": 8, "n": 11008, "k": 4096, "align": 16, "type": "bf16", "format": "e4m3"},
        # a ragged training batch forward through the d=1024 gate projections of many experts
        {"name": "product: forward, ragged", "op": "product", "tokens": 8191, "each": 4, "experts": 64, "n": 2816, "k": 1024, "align": 128, "type": "bf16", "format": "e4m3"},
        # the weight gradients of eight 1.2B-class gate projections: fp32, as the optimizer reads them
        {"name": "product: weight gradients", "op": "weight_grad", "tokens": 16384, "each": 2, "experts": 8, "n": 5632, "k": 2048, "align": 128, "type": "f32", "format": "e5m2"},
        # such a projection from tokens to tokens, forward and backward
        {"name": "layer: 1.2B class", "op": "layer", "tokens": 8192, "each": 2, "experts": 8, "n": 5632, "k": 2048, "align": 128, "format": "e5m2"},
    ]


def _between(rng, lo, hi):
    """A size spread over its logarithm; every second one is left as it falls, the others are multiples of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if v < 16 or rng.random() < 0.5 else v // 8 * 8


def draw(rng):
    """One more case, its tokens or sizes halved until it costs no more than the largest listed one of its kind."""
    c = _drawn(rng)
    if c["op"] == "adamw":
        while c["large"] * c["size"] > 8 * 5632 * 2048:
            c["size"] //= 2
        return c
    rows, wide = 65536, 65536 * 2048
    while c["tokens"] * c["each"] > rows or c["tokens"] * c["each"] * c.get("width", 1) > wide:
        c["tokens"] = max(1, c["tokens"] // 2)
    most = 16384 * 5632 * 2048 if c["op"] == "layer" else 32768 * 5632 * 2048
    while c["tokens"] * c["each"] * c.get("n", 1) * c.get("k", 1) > most:
        c["tokens"] = max(1, c["tokens"] // 2)
    while c.get("n", 1) * c.get("k", 1) * c["experts"] > 8 * 11008 * 4096:
        c["experts"] //= 2
    c["each"] = min(c["each"], c["experts"])
    return c


def _drawn(rng):
    op = rng.choice(("adamw", "adamw", "tokens", "tokens_grad", "product", "product", "weight_grad", "layer"))
    if op == "adamw":
        return {"op": op, "large": rng.randint(1, 8), "size": _between(rng, 1000, 5632 * 2048), "small": rng.randint(0, 100), "width": _between(rng, 1, 8192),
                "grad": rng.choice(("f32", "bf16", "f16")), "state": rng.choice(("fp32", "8bit", "8bit")), "clip": rng.random() < 0.5}
    experts = _between(rng, 2, 128)
    c = {"op": op, "tokens": _between(rng, 1, 16384), "each": rng.randint(1, min(8, experts)), "experts": experts, "align": 128}
    if op in ("tokens", "tokens_grad"):
        c |= {"width": _between(rng, 16, 8192), "type": rng.choice(("bf16", "bf16", "f16", "f32")), "dropped": rng.random() < 0.3}
        c["align"] = 128 if op == "tokens_grad" else rng.choice((16, 128))
        return c
    fmt = rng.choice(("e4m3", "e4m3", "e5m2"))
    if op == "product":
        return c | {"n": _between(rng, 64, 8192), "k": _between(rng, 64, 8192), "align": rng.choice((16, 128)), "type": rng.choice(("bf16", "bf16", "f16", "f32")), "format": fmt}
    if op == "weight_grad":
        return c | {"n": _between(rng, 64, 5632), "k": _between(rng, 64, 5632), "type": "f32", "format": fmt}
    return c | {"tokens": _between(rng, 16, 8192), "n": _between(rng, 128, 5632), "k": _between(rng, 128, 4096), "format": fmt}


# ---------------------------------------------------------------------------
# The plain form: the sorted order
# ---------------------------------------------------------------------------
def _up(v, n):
    return -(-v // n) * n


def _capacity(c):
    """Rows of the sorted order: as many as any choices of these sizes need."""
    pairs = c["tokens"] * c["each"]
    return (pairs + min(c["experts"], pairs) * (c["align"] - 1)) // c["align"] * c["align"]


def _plan(choice, c):
    """(row of each choice or -1, choice of each row or -1, offsets, counts)."""
    e, flat = c["experts"], choice.reshape(-1)
    flat = torch.where((flat < 0) | (flat >= e), e, flat)               # dropped choices behind the last expert
    counts = torch.bincount(flat, minlength=e + 1)[:e]
    room = (counts + c["align"] - 1) // c["align"] * c["align"]
    offsets = torch.cat([room.new_zeros(1), room.cumsum(0)])
    order = torch.argsort(flat, stable=True)
    expert = flat[order]
    place = torch.arange(flat.numel(), device=flat.device) - torch.cat([counts.new_zeros(1), counts.cumsum(0)])[expert]
    row = torch.where(expert < e, offsets[expert] + place, -1)
    rows = torch.empty_like(flat).scatter_(0, order, row)
    pairs = torch.full((_capacity(c) + 1,), -1, dtype=flat.dtype, device=flat.device)
    pairs = pairs.scatter_(0, torch.where(row < 0, _capacity(c), row), torch.where(row < 0, -1, order))[:-1]
    return rows.int().reshape(choice.shape), pairs.int(), offsets.int(), counts.int()


def _gathered(x, pairs, each):
    """x's rows in the sorted order, zeros in rows without a choice."""
    return torch.where((pairs < 0)[:, None], torch.zeros((), dtype=x.dtype, device=x.device), x[pairs.clamp_min(0) // each])


def _combined(ys, rows, weights):
    """Each token's sum over its choices' rows, in fp32, rounded once."""
    taken = torch.where((rows < 0)[..., None], 0.0, ys[rows.clamp_min(0).reshape(-1)].float().reshape(*rows.shape, -1))
    return (taken if weights is None else taken * torch.where(rows < 0, 0.0, weights.float())[..., None]).sum(1).to(ys.dtype)


def _combine_grads(dy, ys, rows, pairs, weights):
    """The gradients of the rows and of the weights."""
    each = rows.shape[1]
    w = weights.reshape(-1)[pairs.clamp_min(0)].float()[:, None]
    dys = torch.where((pairs < 0)[:, None], 0.0, dy[pairs.clamp_min(0) // each].float() * w).to(ys.dtype)
    taken = ys[rows.clamp_min(0).reshape(-1)].float().reshape(*rows.shape, -1)
    return dys, torch.where(rows < 0, 0.0, (taken * dy.float()[:, None]).sum(2)).to(weights.dtype)


# ---------------------------------------------------------------------------
# The plain form: 8-bit matrices and the experts' products
# ---------------------------------------------------------------------------
def _power(e):
    """2^e in fp32 of an int32 e in [-127, 127], from its bits: 2^-127 is a subnormal."""
    return torch.where(e == -127, 1 << 22, (e + 127) << 23).int().view(torch.float32)


def _exponent(top, fmt):
    """The exponent of the smallest power-of-two scale whose format holds `top`."""
    frac, ex = torch.frexp(top)                                   # top = frac 2^ex, frac in [1/2, 1)
    e = ex - (9 if fmt == "e4m3" else 16) + (frac > 0.875).int()  # F = 0.875 2^9 or 0.875 2^16
    return torch.where(top == 0, 0, e.clamp_min(-127))


def _quantised(v, fmt):
    """(codes, scales) of the fp32 matrix v."""
    rows, cols = v.shape
    blocks = -(-cols // 128)
    w = torch.nn.functional.pad(v, (0, blocks * 128 - cols)).reshape(rows, blocks, 128)
    e = _exponent(w.abs().amax(2), fmt)
    codes = (w * _power(-e)[:, :, None]).to(F8[fmt]).reshape(rows, blocks * 128)
    scales = torch.full((blocks, _up(rows, 16)), 127, dtype=torch.uint8, device=v.device)
    scales[:, :rows] = (e + 127).T.to(torch.uint8)
    return codes, scales.view(torch.float8_e8m0fnu)


def _values(held, rows, cols):
    """The fp32 matrix that codes and scales stand for."""
    codes, scales = held
    e = scales.view(torch.uint8)[:, :rows].T.int() - 127
    return (codes.float().reshape(rows, -1, 128) * _power(e)[:, :, None]).reshape(rows, -1)[:, :cols]


def _products(a, b, starts, ends, dtype):
    """Rows starts[e] .. ends[e] of a times b[e]'s transpose, zeros elsewhere."""
    out = torch.zeros(a.shape[0], b.shape[1], dtype=dtype, device=a.device)
    for e, (i, j) in enumerate(zip(starts, ends)):
        if j > i:
            out[i:j] = (a[i:j] @ b[e].T).to(dtype)
    return out


def _weight_products(a, b, starts, ends):
    """For each expert a's columns times b's, over its rows."""
    out = torch.zeros(len(starts), a.shape[0], b.shape[0], device=a.device)
    for e, (i, j) in enumerate(zip(starts, ends)):
        if j > i:
            out[e] = a[:, i:j] @ b[:, i:j].T
    return out


# ---------------------------------------------------------------------------
# The plain form: AdamW
# ---------------------------------------------------------------------------
def _key(t, j):
    return (t * 0x6A09E667 + j * 0xBB67AE85) & MASK


def _thresholds(key, n, device):
    """Two numbers in [0, 1) for each of n elements, sixteen bits each of one 32-bit mixture."""
    i = torch.arange(n, dtype=torch.int64, device=device)
    x = ((i & MASK) * 0x9E3779B9 + (i >> 32) * 0x3C6EF372 + key) & MASK
    x = ((x ^ (x >> 16)) * 0x6A09E667) & MASK
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & MASK
    x = x ^ (x >> 16)
    return (x & 0xFFFF).float() / 65536, (x >> 16).float() / 65536


def _rounded8(v, u, up):
    """(codes, scale bytes) of the fp32 vector v in e4m3, rounded by the thresholds u; below the smallest normal code always up where `up` says so."""
    n = v.numel()
    blocks = -(-n // 128)
    w, u = (torch.nn.functional.pad(x, (0, blocks * 128 - n)).reshape(blocks, 128) for x in (v, u))
    e = _exponent(w.abs().amax(1), "e4m3")
    a = w.abs() * _power(-e)[:, None]
    size = (torch.frexp(a)[1] - 1).clamp_min(-6)                  # the exponent, no lower than the smallest normal code's
    y = a * _power(3 - size)
    k = torch.floor(y + u)
    if up:
        k = torch.where(a < 2.0 ** -6, torch.ceil(y), k)
    r = torch.copysign((k * _power(size - 3)).clamp_max(448.0), w)
    return r.to(torch.float8_e4m3fn).reshape(-1)[:n], (e + 127).to(torch.uint8)


def _held8(codes, scales):
    n = codes.numel()
    e = (scales.view(torch.uint8).int() - 127).repeat_interleave(128)[:n]
    return codes.float() * _power(e)


def _norm(grads):
    return torch.stack([g.double().square().sum() for g in grads]).sum().sqrt().float()


def _adamw(p, g, m, v, scales, t, j, factor):
    """One tensor's step, in place; m and v (in 8 bits its root) with scales, or without."""
    r1, r2 = 1 - BETA1, 1 - BETA2
    g = g.float() if factor is None else g.float() * factor
    if scales is not None:
        old_m, old_s = _held8(m, scales[0]), _held8(v, scales[1])
        new_m, new_v = BETA1 * old_m + r1 * g, BETA2 * (old_s * old_s) + r2 * g * g
    else:
        new_m, new_v = BETA1 * m + r1 * g, BETA2 * v + r2 * g * g
    s = new_v.double().sqrt().float()
    p.copy_(p * (1 - LR * DECAY) - (LR / (1 - BETA1 ** t)) * (new_m / (s * (1 - BETA2 ** t) ** -0.5 + EPS)))
    if scales is None:
        m.copy_(new_m)
        v.copy_(new_v)
        return
    u, w = _thresholds(_key(t, j), p.numel(), p.device)
    for held, scale, (codes, e) in ((m, scales[0], _rounded8(new_m, u, False)), (v, scales[1], _rounded8(s, w, True))):
        held.view(torch.uint8).copy_(codes.view(torch.uint8))
        scale.view(torch.uint8).copy_(e)


# ---------------------------------------------------------------------------
# States
# ---------------------------------------------------------------------------
def _stream(g, m, k, scale=1.0):
    """Rows as a residual stream has them: their sizes differ, and a few channels are much larger than the others."""
    v = torch.randn(m, k, generator=g, device="cuda")
    v *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda")) * scale
    v *= 1 + 15 * (torch.rand(1, k, generator=g, device="cuda") < 0.005)
    return v


def _choices(g, c):
    """Choices and weights as a router gives them: the best `each` of skewed scores, so that some experts get few tokens or none."""
    scores = torch.randn(c["tokens"], c["experts"], generator=g, device="cuda") + torch.randn(c["experts"], generator=g, device="cuda")
    best, choice = scores.topk(c["each"], dim=1)
    if c.get("dropped"):
        choice = torch.where(torch.rand(choice.shape, generator=g, device="cuda") < 0.1, -1, choice)
    return choice, torch.softmax(best, 1)


def _sizes(c):
    return [c["size"]] * c["large"] + [c["width"]] * c["small"]


def _pieces(flat, sizes, room):
    """One tensor of each size out of a flat buffer, each at a multiple of 128 elements (or of `room` elements for 128 of them)."""
    at, out = 0, []
    for n in sizes:
        out.append(flat[at: at + (n if room == 128 else -(-n // 128) * room)])
        at += -(-n // 128) * room
    return out


def _adamw_state(c, g):
    sizes = _sizes(c)
    blocks = sum(-(-n // 128) for n in sizes)
    s = {"t": 9}
    s["flat"] = 0.02 * torch.randn(blocks * 128, generator=g, device="cuda")
    s["p"] = _pieces(s["flat"], sizes, 128)
    s["g"] = [(1e-3 * torch.randn(n, generator=g, device="cuda") * torch.exp(torch.randn(n, generator=g, device="cuda"))).to(FLOATS[c["grad"]]) for n in sizes]
    m = [3e-4 * torch.randn(n, generator=g, device="cuda") for n in sizes]
    v = [3e-6 * torch.exp(torch.randn(n, generator=g, device="cuda")) for n in sizes]
    if c["state"] == "fp32":
        s["flat_m"], s["flat_v"] = (torch.zeros(blocks * 128, device="cuda") for _ in range(2))
        s["scales"] = [None] * len(sizes)
    else:
        s["flat_m"], s["flat_v"] = (torch.zeros(blocks * 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
        s["flat_scales"] = torch.zeros(blocks * 2, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        s["scales"] = [x.view(2, -1) for x in _pieces(s["flat_scales"], sizes, 2)]
    s["m"], s["v"] = _pieces(s["flat_m"], sizes, 128), _pieces(s["flat_v"], sizes, 128)
    for j, n in enumerate(sizes):
        if c["state"] == "fp32":
            s["m"][j].copy_(m[j])
            s["v"][j].copy_(v[j])
            continue
        half = torch.full((n,), 0.5, device="cuda")
        for held, scale, x, up in ((s["m"][j], s["scales"][j][0], m[j], False), (s["v"][j], s["scales"][j][1], v[j].sqrt(), True)):
            codes, e = _rounded8(x, half, up)
            held.view(torch.uint8).copy_(codes.view(torch.uint8))
            scale.view(torch.uint8).copy_(e)
    return s


@torch.no_grad()
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, op = case, case["op"]
    if op == "adamw":
        return {"case": case, **_adamw_state(c, g)}
    s = {"case": case}
    s["choice"], weights = _choices(g, c)
    s["plan"] = _plan(s["choice"], c)
    starts, counts = s["plan"][2].tolist()[:-1], s["plan"][3].tolist()
    s["spans"] = (starts, [i + n for i, n in zip(starts, counts)])
    rows, t, e = _capacity(c), c["tokens"], c["experts"]
    if op in ("tokens", "tokens_grad"):
        s["weights"] = weights.to(FLOATS[c["type"]]).requires_grad_(op == "tokens_grad")
        s["x"] = _stream(g, t, c["width"]).to(FLOATS[c["type"]])
    if op == "tokens_grad":
        s["ys"] = _gathered(_stream(g, t * c["each"], c["width"]).to(FLOATS[c["type"]]), s["plan"][1], 1).requires_grad_()
        s["dy"] = _stream(g, t, c["width"], 1e-2).to(FLOATS[c["type"]])
        s["dxs"] = _gathered(_stream(g, t * c["each"], c["width"], 1e-2).to(FLOATS[c["type"]]), s["plan"][1], 1)
        s["x"].requires_grad_()
    elif op == "product":
        s["a"] = _quantised(_gathered(_stream(g, t, c["k"], 0.5), s["plan"][1], c["each"]), c["format"])
        # each expert's rows begin at a multiple of 16
        stack = torch.nn.functional.pad(0.02 * torch.randn(e, c["n"], c["k"], generator=g, device="cuda"), (0, 0, 0, -c["n"] % 16))
        s["b"] = _quantised(stack.reshape(-1, c["k"]), "e4m3")
    elif op == "weight_grad":
        s["a"] = _quantised(_gathered(_stream(g, t * c["each"], c["n"], 1e-2), s["plan"][1], 1).T.contiguous(), c["format"])
        s["b"] = _quantised(_gathered(_stream(g, t, c["k"], 0.5), s["plan"][1], c["each"]).T.contiguous(), "e4m3")
    elif op == "layer":
        s["x"] = _stream(g, t, c["k"], 0.5).bfloat16().requires_grad_()
        s["weights"] = weights.bfloat16().requires_grad_()
        s["W"] = (0.02 * torch.randn(e, c["n"], c["k"], generator=g, device="cuda")).requires_grad_()
        s["dy"] = _stream(g, t, c["n"], 1e-2).bfloat16()
    assert rows == s["plan"][1].numel()
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from kronecker_factored_second_amd import experts, linear, optim
    c = s["case"]
    op = c["op"]
    if op == "adamw":
        s["t"] += 1
        norm = optim.grad_norm(s["g"]) if c["clip"] else None
        moments = [optim.Moments(*x) for x in zip(s["m"], s["v"], s["scales"])]
        optim.adamw(s["p"], s["g"], moments, s["t"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, norm=norm, max_norm=MAX_NORM)
        return _adamw_outputs(s, norm)
    if op == "tokens":
        plan = experts.plan(s["choice"], c["experts"], align=c["align"])
        xs = experts.gather(s["x"], plan)
        return [plan.rows, plan.pairs, plan.offsets, plan.counts, xs, experts.combine(xs, s["weights"], plan)]
    if op == "layer":
        plan = experts.plan(s["choice"], c["experts"], align=c["align"])
        ys = experts.token_linear(s["x"], s["W"], plan, grad_dtype=F8[c["format"]])
        y = experts.combine(ys, s["weights"], plan)
        return [y.detach(), *torch.autograd.grad(y, (s["x"], s["W"], s["weights"]), s["dy"])]
    plan = experts.Plan(*s["plan"], align=c["align"])
    rows, e = _capacity(c), c["experts"]
    if op == "tokens_grad":
        xs, y = experts.gather(s["x"], plan), experts.combine(s["ys"], s["weights"], plan)
        return list(torch.autograd.grad((xs, y), (s["x"], s["ys"], s["weights"]), (s["dxs"], s["dy"])))
    if op == "product":
        a, b = linear.Blocked(*s["a"], (rows, c["k"])), experts.Stack(*s["b"], (e, c["n"], c["k"]))
        return experts.matmul(a, b, plan, dtype=FLOATS[c["type"]])
    a, b = linear.Blocked(*s["a"], (c["n"], rows)), linear.Blocked(*s["b"], (c["k"], rows))
    return experts.weight_grad(a, b, plan, dtype=FLOATS[c["type"]])


def _adamw_outputs(s, norm):
    return [s["flat"], s["flat_m"], s["flat_v"], *([s["flat_scales"]] if s["case"]["state"] == "8bit" else []), *([norm] if norm is not None else [])]


@torch.no_grad()
def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "adamw":
        s["t"] += 1
        norm = _norm(s["g"]) if c["clip"] else None
        factor = None if norm is None else (MAX_NORM / (norm.double() + 1e-6)).clamp_max(1.0).float()
        for j, (p, g, m, v, scales) in enumerate(zip(s["p"], s["g"], s["m"], s["v"], s["scales"])):
            _adamw(p, g, m, v, scales, s["t"], j, factor)
        return _adamw_outputs(s, norm)
    if op == "tokens":
        plan = _plan(s["choice"], c)
        xs = _gathered(s["x"], plan[1], c["each"])
        return [*plan, xs, _combined(xs, plan[0], s["weights"])]
    e, n, k, rows = c["experts"], c.get("n"), c.get("k"), _capacity(c)
    if op == "tokens_grad":
        xs, y = _gathered(s["x"], s["plan"][1], c["each"]), _combined(s["ys"], s["plan"][0], s["weights"])
        return [_combined(s["dxs"], s["plan"][0], None), *_combine_grads(s["dy"], s["ys"], *s["plan"][:2], s["weights"])]
    if op == "product":
        return _products(_values(s["a"], rows, k), _values(s["b"], e * _up(n, 16), k).reshape(e, -1, k)[:, :n], *s["spans"], FLOATS[c["type"]])
    if op == "weight_grad":
        return _weight_products(_values(s["a"], n, rows), _values(s["b"], k, rows), *s["spans"])
    plan = _plan(s["choice"], c)
    xs, W = _gathered(s["x"], plan[1], c["each"]).float(), s["W"]
    w = _values(_quantised(W.reshape(e * n, k), "e4m3"), e * n, k).reshape(e, n, k)
    wt = _values(_quantised(W.transpose(1, 2).reshape(e * k, n), "e4m3"), e * k, n).reshape(e, k, n)
    ys = _products(_values(_quantised(xs, "e4m3"), rows, k), w, *s["spans"], torch.bfloat16)
    y = _combined(ys, plan[0], s["weights"])
    dys, dweights = _combine_grads(s["dy"], ys, *plan[:2], s["weights"])
    dys = dys.float()
    dxs = _products(_values(_quantised(dys, c["format"]), rows, n), wt, *s["spans"], torch.bfloat16)
    dW = _weight_products(_values(_quantised(dys.T, c["format"]), n, rows), _values(_quantised(xs.T, "e4m3"), k, rows), *s["spans"])
    return [y, _combined(dxs, plan[0], None), dW, dweights]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def _held(rows, cols):
    """Bytes of a matrix in 8 bits: its codes and a scale byte for each block of 128."""
    return rows * cols + rows * -(-cols // 128)


def work(case):
    c, op = case, case["op"]
    if op == "adamw":  # the parameter and its moments in and out, the gradient in
        n = sum(_sizes(c))
        return {"bytes": n * (8 + SIZE[c["grad"]]) + (16 * n if c["state"] == "fp32" else 2 * (2 * n + 2 * -(-n // 128))), "flops": 14 * n}
    pairs, rows, t, e = c["tokens"] * c["each"], _capacity(c), c["tokens"], c["experts"]
    b = SIZE[c.get("type", "bf16")]
    if op == "tokens":  # choices and tokens in; the order, the sorted rows and the tokens' sums out
        return {"bytes": 12 * pairs + 4 * rows + (2 * t + rows) * c["width"] * b + pairs * b, "flops": 2 * pairs * c["width"]}
    if op == "tokens_grad":  # both ways' gradients in and out, and the rows that the weights' gradients need
        return {"bytes": 8 * pairs + (2 * pairs + rows + 2 * t) * c["width"] * b + 2 * pairs * b, "flops": 5 * pairs * c["width"]}
    n, k = c["n"], c["k"]
    if op == "product":  # at least as many experts' weights as can have no token left over; rows out
        return {"bytes": _held(pairs, k) + min(e, pairs) * _held(n, k) + rows * n * b, "flops": 2 * pairs * n * k}
    if op == "weight_grad":
        return {"bytes": _held(n, pairs) + _held(k, pairs) + 4 * e * n * k, "flops": 2 * pairs * n * k}
    # tokens and their gradients in and out in 16 bits; W in and its gradient out in 32
    return {"bytes": 4 * t * (k + n) + 8 * e * n * k, "flops": 6 * pairs * n * k}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _pow2(e):
    """2^e in float64 of whole e, from its bits: pow is not exact on every device."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _floor_log2(x):
    e = x.log2().floor()
    e = torch.where(_pow2(e) > x, e - 1, e)
    return torch.where(_pow2(e + 1) <= x, e + 1, e)


def _scale_exponent(top, fmt):
    e = (top.clamp_min(2.0 ** -200) / TOP[fmt]).log2().ceil()
    e = torch.where(top > TOP[fmt] * _pow2(e), e + 1, e)
    e = torch.where(top <= TOP[fmt] * _pow2(e - 1), e - 1, e).clamp_min(-127)
    return torch.where(top == 0, torch.zeros_like(e), e)


def _exact_held(v, fmt):
    """v (float64) through its 8-bit form: each block's scale by comparison, the rounding as a multiple of the step at each value's size."""
    out = torch.empty_like(v)
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    for b in range(0, v.shape[1], 128):
        part = v[:, b: b + 128]
        sc = _pow2(_scale_exponent(part.abs().amax(1), fmt))[:, None]
        step = _pow2(_floor_log2((part / sc).abs().clamp_min(2.0 ** low)) - bits)
        out[:, b: b + 128] = torch.round(part / sc / step) * step * sc
    return out


def _exact_rows(choice, c):
    """Each expert's choices in their order, and the row of its first one, in plain Python."""
    flat, mine = choice.reshape(-1).tolist(), [[] for _ in range(c["experts"])]
    for i, e in enumerate(flat):
        if 0 <= e < c["experts"]:
            mine[e].append(i)
    at, starts = 0, []
    for m in mine:
        starts.append(at)
        at += -(-len(m) // c["align"]) * c["align"]
    return mine, starts + [at]


def _exact_layout(s):
    """For each expert with tokens: (its number, its choices' numbers, its first row)."""
    mine, starts = _exact_rows(s["choice"], s["case"])
    return [(e, torch.tensor(m, device="cuda"), starts[e]) for e, m in enumerate(mine) if m]


def _exact_moment(x, u, up):
    """(codes' values, scales' values) of x by the definition of the rounding by thresholds."""
    n = x.numel()
    w = torch.nn.functional.pad(x, (0, -n % 128)).view(-1, 128)
    e = _scale_exponent(w.abs().amax(1), "e4m3")
    a = (w / _pow2(e)[:, None]).reshape(-1)[:n]
    step = _pow2(_floor_log2(a.abs().clamp_min(2.0 ** -6)) - 3)
    k = torch.floor(a.abs() / step + u)
    if up:
        k = torch.where(a.abs() < 2.0 ** -6, torch.ceil(a.abs() / step), k)
    return torch.sign(a) * (k * step).clamp_max(448.0), _pow2(e)


def _exact_adamw(s):
    c, t = s["case"], s["t"] + 1
    sizes = _sizes(c)
    total = sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["g"]) ** 0.5
    factor = min(1.0, MAX_NORM / (total + 1e-6)) if c["clip"] else 1.0
    flat, fm, fv = (torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda") for _ in range(3))
    flat.copy_(s["flat"])
    fs = torch.zeros(s["flat_scales"].numel(), dtype=torch.float64, device="cuda") if c["state"] == "8bit" else None
    at = 0
    for j, n in enumerate(sizes):
        room = -(-n // 128) * 128
        g, p, m, v = (x[j].double() for x in (s["g"], s["p"], s["m"], s["v"]))
        if fs is not None:
            by = s["scales"][j].view(torch.uint8).int() - 127
            m, v = m * _pow2(by[0]).repeat_interleave(128)[:n], (v * _pow2(by[1]).repeat_interleave(128)[:n]) ** 2
        m, v = m + (1 - BETA1) * (factor * g - m), v + (1 - BETA2) * ((factor * g) ** 2 - v)
        hat = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        flat[at: at + n] = p - LR * (DECAY * p + hat)
        if fs is None:
            fm[at: at + n], fv[at: at + n] = m, v
        else:
            u = _thresholds(_key(t, j), n, p.device)
            half = at // 128 * 2
            for q, (x, to) in enumerate(((m, fm), (v.sqrt(), fv))):
                to[at: at + n], sc = _exact_moment(x, u[q].double(), q == 1)
                fs[half + q * (room // 128): half + (q + 1) * (room // 128)] = sc
        at += room
    return [flat, fm, fv, *([fs] if fs is not None else []), *([torch.tensor(total, dtype=torch.float64)] if c["clip"] else [])]


@torch.no_grad()
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "adamw":
        return _exact_adamw(s)
    rows, each, lay = _capacity(c), c["each"], _exact_layout(s)
    if op == "tokens":
        x, w = s["x"].double(), s["weights"].double().reshape(-1)
        xs, y = torch.zeros(rows, c["width"], dtype=torch.float64, device="cuda"), torch.zeros_like(x)
        for _, m, at in lay:
            xs[at: at + len(m)] = x[m // each]
            y.index_add_(0, m // each, x[m // each] * w[m][:, None])
        return [None, None, None, None, xs, y]
    if op == "tokens_grad":
        dx, dys, dw = (torch.zeros(v.shape, dtype=torch.float64, device="cuda") for v in (s["x"], s["ys"], s["weights"]))
        dy, ys, w = s["dy"].double(), s["ys"].double(), s["weights"].double().reshape(-1)
        for _, m, at in lay:
            dx.index_add_(0, m // each, s["dxs"][at: at + len(m)].double())
            dys[at: at + len(m)] = dy[m // each] * w[m][:, None]
            dw.view(-1)[m] = torch.einsum("mk,mk->m", dy[m // each], ys[at: at + len(m)])
        return [dx, dys, dw]
    e, n, k = c["experts"], c["n"], c["k"]

    def held(pair, r, cols):
        return pair[0][:, :cols].double() * pair[1][:, :r].double().T.repeat_interleave(128, 1)[:, :cols]

    if op == "product":
        step = s["b"][0].shape[0] // e
        a, b = held(s["a"], rows, k), held(s["b"], e * step, k)
        out = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
        for q, m, at in lay:
            out[at: at + len(m)] = a[at: at + len(m)].mm(b[q * step: q * step + n].T)
        return out
    if op == "weight_grad":
        a, b = held(s["a"], n, rows), held(s["b"], k, rows)
        out = torch.zeros(e, n, k, dtype=torch.float64, device="cuda")
        for q, m, at in lay:
            out[q] = a[:, at: at + len(m)].mm(b[:, at: at + len(m)].T)
        return out
    x, w, dy = s["x"].double(), s["weights"].reshape(-1), s["dy"]
    y, dx = torch.zeros(c["tokens"], n, dtype=torch.float64, device="cuda"), torch.zeros_like(x)
    dW, dw = torch.zeros(e, n, k, dtype=torch.float64, device="cuda"), torch.zeros(w.shape, dtype=torch.float64, device="cuda")
    for q, m, at in lay:
        t, W, wm = m // each, s["W"][q].double(), w[m].double()[:, None]
        out = _exact_held(x[t], "e4m3").mm(_exact_held(W, "e4m3").T)
        y.index_add_(0, t, out * wm)
        dw[m] = torch.einsum("mk,mk->m", out, dy[t].double())
        d = (dy[t].double() * wm).bfloat16().double()        # the rows' gradient has their type
        dx.index_add_(0, t, _exact_held(d, c["format"]).mm(_exact_held(W.T.contiguous(), "e4m3").T))
        # blocks of 128 rows from the expert's first one on
        dW[q] = _exact_held(d.T.contiguous(), c["format"]).mm(_exact_held(x[t].T.contiguous(), "e4m3").T)
    return [y, dx, dW, dw.view(s["weights"].shape)]
