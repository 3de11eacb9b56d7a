"""Measured cases of the 8-bit linear layer's operators (`linear` in this
repository's package): the root-mean-square norm with the residual's addition
and an 8-bit output, its gradient, the block quantisation, the block-scaled
8-bit matrix product, and a normed linear layer's training pass over all of
them.  Each has a plain form here, made of elementary torch operations.

The 8-bit form of a matrix: along its columns (the axis a product sums over)
every block of 128 values of a row shares one power-of-two scale 2^e, e the
smallest integer >= -127 with max|v| <= F 2^e over the block's finite values
(F = 448 for e4m3, 57344 for e5m2; a block of zeros has e = 0), and holds
v 2^-e rounded to nearest even.  Codes are (rows, 128 B) with zeros past the
last column, B the number of blocks; scales are (B, rows) as e + 127 in a byte,
their rows padded to a multiple of 16.
"""
import math

import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
MANTISSA = {"e4m3": 3, "e5m2": 2}
LOWEST = {"e4m3": -6, "e5m2": -14}          # exponent of the smallest normal number
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def listed():
    return [
        # one token of a decode step through the norm before a 6.5B-class block's projections: latency
        {"name": "norm: one token", "op": "norm", "m": 1, "k": 4096, "type": "bf16", "format": "e4m3", "residual": True},
        # a training batch's residual stream at the 1.2B-class width
        {"name": "norm: training batch", "op": "norm", "m": 16384, "k": 2048, "type": "bf16", "format": "e4m3", "residual": True},
        # the same stream's way back, the residual's gradient joining in
        {"name": "norm gradient: training batch", "op": "norm_grad", "m": 16384, "k": 2048, "type": "bf16", "residual": True},
        # a short ragged batch of an odd width in fp32
        {"name": "norm gradient: odd, fp32", "op": "norm_grad", "m": 777, "k": 5121, "type": "f32", "residual": False},
        # the gradient of a gate projection's output, in the two forms its two products read
        {"name": "quantise: output gradient", "op": "quantize", "m": 16384, "k": 5632, "type": "bf16", "format": "e5m2"},
        # a 6.5B-class up projection's fp32 master weight, requantised after an optimizer step
        {"name": "quantise: master weight", "op": "quantize", "m": 11008, "k": 4096, "type": "f32", "format": "e4m3"},
        # one token through that projection: the weight's bytes bound it
        {"name": "product: one token", "op": "matmul", "m": 1, "n": 11008, "k": 4096, "type": "bf16", "format": "e4m3"},
        # a decode batch through a 13B-class down projection
        {"name": "product: decode batch", "op": "matmul", "m": 48, "n": 5120, "k": 13824, "type": "bf16", "format": "e4m3"},
        # a ragged training batch forward through a 1.2B-class gate projection
        {"name": "product: forward, ragged", "op": "matmul", "m": 8191, "n": 5632, "k": 2048, "type": "bf16", "format": "e4m3"},
        # the weight gradient of a 6.5B-class up projection: fp32, as the optimizer reads it
        {"name": "product: weight gradient", "op": "matmul", "m": 11008, "n": 4096, "k": 16384, "type": "f32", "format": "e5m2"},
        # a normed projection of the d=1024 block, forward and backward, on a short ragged batch
        {"name": "layer: d=1024, short", "op": "layer", "m": 333, "k": 1024, "n": 2816, "format": "e4m3"},
        # the 1.2B-class one on a full batch
        {"name": "layer: 1.2B class", "op": "layer", "m": 8192, "k": 2048, "n": 5632, "format": "e5m2"},
    ]


def _between(rng, lo, hi):
    """A size spread over its logarithm; every second one is left as it falls, the others are multiples of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v if v < 16 or rng.random() < 0.5 else v // 8 * 8


def draw(rng):
    """One more case, its rows halved until it costs no more than the largest listed one of its kind."""
    c = _drawn(rng)
    n, most = c.get("n", 1), {"matmul": 11008 * 4096 * 16384, "layer": 8192 * 2048 * 5632}.get(c["op"], 16384 * 5632)
    while c["m"] * c["k"] * n > most:
        c["m"] //= 2
    return c


def _drawn(rng):
    op = rng.choice(("norm", "norm_grad", "quantize", "matmul", "matmul", "layer"))
    kind = rng.choice(("bf16", "bf16", "f16", "f32"))
    fmt = rng.choice(("e4m3", "e4m3", "e5m2"))
    if op == "norm":
        return {"op": op, "m": _between(rng, 1, 16384), "k": _between(rng, 64, 16384), "type": kind, "format": fmt, "residual": rng.random() < 0.7}
    if op == "norm_grad":
        return {"op": op, "m": _between(rng, 1, 16384), "k": _between(rng, 64, 16384), "type": kind, "residual": rng.random() < 0.7}
    if op == "quantize":
        return {"op": op, "m": _between(rng, 1, 16384), "k": _between(rng, 64, 13824), "type": kind, "format": fmt}
    if op == "matmul":
        m = _between(rng, 1, 64) if rng.random() < 0.4 else _between(rng, 64, 8192)
        return {"op": op, "m": m, "n": _between(rng, 128, 13824), "k": _between(rng, 128, 11008), "type": kind, "format": fmt}
    return {"op": op, "m": _between(rng, 16, 8192), "k": _between(rng, 256, 5120), "n": _between(rng, 256, 5632), "format": fmt}


# ---------------------------------------------------------------------------
# The plain form
# ---------------------------------------------------------------------------
def _power(e):
    """2^e in fp32 of an int32 e in [-127, 127], from its bits: 2^-127 is a subnormal."""
    return torch.where(e == -127, 1 << 22, (e + 127) << 23).int().view(torch.float32)


def _quantised(v, fmt):
    """(codes, scales) of the fp32 matrix v."""
    rows, cols = v.shape
    blocks = -(-cols // 128)
    w = torch.nn.functional.pad(v, (0, blocks * 128 - cols)).reshape(rows, blocks, 128)
    top = torch.where(torch.isfinite(w), w.abs(), 0.0).amax(2)
    frac, ex = torch.frexp(top)                                   # top = frac 2^ex, frac in [1/2, 1)
    e = ex - (9 if fmt == "e4m3" else 16) + (frac > 0.875).int()  # F = 0.875 2^9 or 0.875 2^16
    e = torch.where(top == 0, 0, e.clamp_min(-127))
    codes = (w * _power(-e)[:, :, None]).to(F8[fmt]).reshape(rows, blocks * 128)
    scales = torch.full((blocks, -(-rows // 16) * 16), 127, dtype=torch.uint8, device=v.device)
    scales[:, :rows] = (e + 127).T.to(torch.uint8)
    return codes, scales.view(torch.float8_e8m0fnu)


def _values(codes, scales, rows, cols):
    """The fp32 matrix that codes and scales stand for."""
    e = scales.view(torch.uint8)[:, :rows].T.int() - 127
    return (codes.float().reshape(rows, -1, 128) * _power(e)[:, :, None]).reshape(rows, -1)[:, :cols]


def _outputs(codes, scales, rows, cols):
    return codes[:, :cols], scales[:, :rows]


def _norm(x, r, w):
    """(normed values in fp32, residual stream, 1 / rms): the mean square in 64 bits and one rounding, so that the 8-bit codes do not hang on its order of summation."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    return h.float() * rstd[:, None] * w.float(), h, rstd


def _norm_grad(dy, h, rstd, w, dh):
    g, hat = dy.float() * w.float(), h.float() * rstd[:, None]
    dx = rstd[:, None] * (g - hat * (g * hat).mean(1, keepdim=True))
    dx = dx if dh is None else dx + dh.float()
    return dx.to(h.dtype), (dy.float() * hat).sum(0, dtype=torch.float64).to(w.dtype)


# ---------------------------------------------------------------------------
# States
# ---------------------------------------------------------------------------
def _stream(g, m, k, kind, scale=1.0):
    """Rows as a residual stream has them: their sizes differ, and a few channels are much larger than the others."""
    v = torch.randn(m, k, generator=g, device="cuda")
    v *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda")) * scale
    v *= 1 + 15 * (torch.rand(1, k, generator=g, device="cuda") < 0.005)
    return v.to(FLOATS[kind])


def _gain(g, k, kind):
    return (1 + 0.2 * torch.randn(k, generator=g, device="cuda")).to(FLOATS[kind])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    s = {"case": case}
    if op == "norm":
        s["x"], s["w"] = _stream(g, m, k, case["type"], 0.3), _gain(g, k, case["type"])
        s["r"] = _stream(g, m, k, case["type"]) if case["residual"] else None
    elif op == "norm_grad":
        s["h"], s["w"] = _stream(g, m, k, case["type"]), _gain(g, k, case["type"])
        s["rstd"] = (s["h"].double().square().mean(1) + EPS).rsqrt().float()
        s["dy"] = _stream(g, m, k, case["type"], 1e-2)
        s["dh"] = _stream(g, m, k, case["type"], 1e-2) if case["residual"] else None
    elif op == "quantize":
        s["x"] = _stream(g, m, k, case["type"], 1e-2)
    elif op == "matmul":
        s["a"] = _quantised(_stream(g, m, k, "bf16", 0.5).float(), case["format"])
        s["b"] = _quantised(_stream(g, case["n"], k, "bf16", 0.02).float(), "e4m3")
    else:
        s["x"], s["r"] = _stream(g, m, k, "bf16", 0.3).requires_grad_(), _stream(g, m, k, "bf16")
        s["w"] = _gain(g, k, "bf16").requires_grad_()
        s["W"] = (0.02 * torch.randn(case["n"], k, generator=g, device="cuda")).requires_grad_()
        s["dy"], s["dh"] = _stream(g, m, case["n"], "bf16", 1e-2), _stream(g, m, k, "bf16", 1e-2)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from kronecker_factored_second_amd import linear
    c = s["case"]
    op, m, k = c["op"], c["m"], c["k"]
    if op == "norm":
        q, h, rstd = linear.rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, dtype=F8[c["format"]])
        return [*_outputs(q.codes, q.scales, m, k), h, rstd]
    if op == "norm_grad":
        return list(linear.rms_norm_backward(s["dy"], s["h"], s["rstd"], s["w"], dh=s["dh"]))
    if op == "quantize":
        q, t = linear.quantize_both(s["x"], dtype=F8[c["format"]])
        return [*_outputs(q.codes, q.scales, m, k), *_outputs(t.codes, t.scales, k, m)]
    if op == "matmul":
        return linear.matmul(linear.Blocked(*s["a"], (m, k)), linear.Blocked(*s["b"], (c["n"], k)), dtype=FLOATS[c["type"]])
    y, h = linear.rms_norm_linear(s["x"], s["w"], s["W"], residual=s["r"], eps=EPS, grad_dtype=F8[c["format"]])
    dx, dw, dW = torch.autograd.grad((y, h), (s["x"], s["w"], s["W"]), (s["dy"], s["dh"]))
    return [y.detach(), h.detach(), dx, dw, dW]


@torch.no_grad()
def _run_plain(s):
    c = s["case"]
    op, m, k = c["op"], c["m"], c["k"]
    if op == "norm":
        y, h, rstd = _norm(s["x"], s["r"], s["w"])
        return [*_outputs(*_quantised(y, c["format"]), m, k), h, rstd]
    if op == "norm_grad":
        return list(_norm_grad(s["dy"], s["h"], s["rstd"], s["w"], s["dh"]))
    if op == "quantize":
        v = s["x"].float()
        return [*_outputs(*_quantised(v, c["format"]), m, k), *_outputs(*_quantised(v.T, c["format"]), k, m)]
    if op == "matmul":
        return (_values(*s["a"], m, k) @ _values(*s["b"], c["n"], k).T).to(FLOATS[c["type"]])
    n = c["n"]
    v, h, rstd = _norm(s["x"], s["r"], s["w"])
    y = (_values(*_quantised(v, "e4m3"), m, k) @ _values(*_quantised(s["W"], "e4m3"), n, k).T).bfloat16()
    dy = s["dy"].float()
    dv = (_values(*_quantised(dy, c["format"]), m, n) @ _values(*_quantised(s["W"].T, "e4m3"), k, n).T).bfloat16()
    dW = _values(*_quantised(dy.T, c["format"]), n, m) @ _values(*_quantised(v.T, "e4m3"), k, m).T
    dx, dw = _norm_grad(dv, h, rstd, s["w"], s["dh"])
    return [y, h, dx, dw, dW]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def _held(rows, cols):
    """Bytes of a matrix in 8 bits: its codes and a scale byte for each block of 128."""
    return rows * cols + rows * -(-cols // 128)


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    b = SIZE[case.get("type", "bf16")]
    if op == "norm":  # x (and the residual) in; the sum, where there is one, the codes and 1/rms out
        return {"bytes": m * k * b * (3 if case["residual"] else 1) + _held(m, k) + k * b + 4 * m, "flops": 6 * m * k}
    if op == "norm_grad":
        return {"bytes": m * k * b * (4 if case["residual"] else 3) + 2 * k * b + 4 * m, "flops": 12 * m * k}
    if op == "quantize":
        return {"bytes": m * k * b + _held(m, k) + _held(k, m), "flops": 4 * m * k}
    n = case["n"]
    if op == "matmul":
        return {"bytes": _held(m, k) + _held(n, k) + m * n * b, "flops": 2 * m * n * k}
    # x, r, dy and dh in, y, h and dx out in 16 bits; W in and its gradient out in 32
    return {"bytes": 2 * (5 * m * k + 2 * m * n) + 8 * n * k, "flops": 6 * m * n * k}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _pow2(e):
    """2^e in float64 of whole e, from its bits: pow is not exact on every device."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _size(u, fmt):
    """The exponent of each |u|, no lower than the format's smallest normal number's."""
    u = u.abs().clamp_min(2.0 ** LOWEST[fmt])
    e = u.log2().floor()
    e = torch.where(_pow2(e) > u, e - 1, e)
    return torch.where(_pow2(e + 1) <= u, e + 1, e)


def _exact_blocks(v, fmt):
    """The codes' values and scales' values (both float64) of v by the definition: a logarithm's guess at e made right by comparison, and the rounding as a multiple of the step at each value's size."""
    rows, cols = v.shape
    v = v.double()
    q, sc = torch.empty_like(v), torch.empty(-(-cols // 128), rows, dtype=torch.float64, device=v.device)
    for b in range(sc.shape[0]):
        part = v[:, 128 * b: 128 * b + 128]
        top = part.abs().masked_fill(~part.isfinite(), 0).max(1).values
        e = (top.clamp_min(2.0 ** -200) / TOP[fmt]).log2().ceil()
        e = torch.where(top > TOP[fmt] * _pow2(e), e + 1, e)
        e = torch.where(top <= TOP[fmt] * _pow2(e - 1), e - 1, e).clamp_min(-127)
        sc[b] = _pow2(torch.where(top == 0, torch.zeros_like(e), e))
        u = part / sc[b][:, None]
        step = _pow2(_size(u, fmt) - MANTISSA[fmt])
        q[:, 128 * b: 128 * b + 128] = torch.round(u / step) * step
    return q, sc


def _exact_held(v, fmt):
    q, sc = _exact_blocks(v, fmt)
    return q * sc.T.repeat_interleave(128, 1)[:, : v.shape[1]]


def _exact_normed(h, w):
    """1/rms from 64 bits, and the normed values as the operator defines them: 1/rms and the two products each rounded once to 32 bits."""
    d = h.double()
    rstd = (1 / torch.sqrt(torch.linalg.vector_norm(d, dim=1) ** 2 / h.shape[1] + EPS))
    return rstd, ((d * rstd.float().double()[:, None]).float().double() * w.double()).float()


def _exact_grads(dy, h, rstd, w, dh):
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    along = torch.einsum("mk,mk->m", dy * w, h)[:, None]
    dx = rstd * dy * w - h * rstd ** 3 * along / h.shape[1]
    return (dx if dh is None else dx + dh.double()), torch.einsum("mk,mk->k", dy * rstd, h)


@torch.no_grad()
def exact(case, seed):
    s = prepare(case, seed)
    op, m, k, fmt = case["op"], case["m"], case["k"], case.get("format")
    if op in ("norm", "layer"):
        h = s["x"].detach() if s["r"] is None else (s["x"].double() + s["r"].double()).to(s["x"].dtype)
        rstd, v = _exact_normed(h, s["w"])
    if op == "norm":
        return [*_exact_blocks(v, fmt), h.double(), rstd]
    if op == "norm_grad":
        return list(_exact_grads(s["dy"], s["h"], s["rstd"], s["w"], s["dh"]))
    if op == "quantize":
        return [*_exact_blocks(s["x"], fmt), *_exact_blocks(s["x"].T, fmt)]
    if op == "matmul":
        def held(pair, rows):
            return pair[0][:, :k].double() * pair[1][:, :rows].double().T.repeat_interleave(128, 1)[:, :k]
        return held(s["a"], m).mm(held(s["b"], case["n"]).T)
    W, dy = s["W"].detach(), s["dy"]
    y = _exact_held(v, "e4m3").mm(_exact_held(W, "e4m3").T)
    dv = _exact_held(dy, fmt).mm(_exact_held(W.T.contiguous(), "e4m3").T).bfloat16()
    dW = _exact_held(dy.T.contiguous(), fmt).mm(_exact_held(v.T.contiguous(), "e4m3").T)
    dx, dw = _exact_grads(dv, h, rstd.float(), s["w"], s["dh"])
    return [y, h.double(), dx, dw, dW]
