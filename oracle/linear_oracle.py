"""Plain fp64 forms of the 8-bit linear-layer operators, in numpy, written from
their definitions (include/okls_linear.h).  Test infrastructure: nothing on the
product path uses it.

The 8-bit form is returned as two fp64 arrays: the codes' values (rows, cols) and
the scales' values (ceil(cols / 128), rows)."""
import numpy as np

BLOCK = 128
# largest finite value, bits of the significand's fraction, exponent of the smallest normal number
FORMATS = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}


def round8(u, fmt):
    """u to the nearest value of the format, ties to the even code; |u| <= its largest value."""
    top, frac, low = FORMATS[fmt]
    u = np.asarray(u, dtype=np.float64)
    fin = np.isfinite(u)
    a = np.where(fin, u, 0.0)
    _, ex = np.frexp(np.maximum(np.abs(a), np.ldexp(1.0, low)))     # |a| = f 2^ex, f in [1/2, 1)
    step = np.ldexp(1.0, ex - 1 - frac)
    r = np.copysign(np.rint(np.abs(a) / step) * step, a)
    assert (np.abs(r) <= top).all()
    bad = np.full_like(r, np.nan) if fmt == "e4m3" else u           # e4m3 has no infinity
    return np.where(fin, r, np.where(np.isnan(u), np.nan, bad))


def scale_exponent(top, fmt):
    """The smallest e >= -127 with top <= F 2^e; 0 for top = 0."""
    big = FORMATS[fmt][0]
    if top == 0:
        return 0
    e = -127
    while top > np.ldexp(big, e):
        e += 1
    return e


def quantize(v, fmt):
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    codes, scales = np.zeros((rows, cols)), np.ones((nb, rows))
    for b in range(nb):
        sl = slice(b * BLOCK, min(cols, (b + 1) * BLOCK))
        for r in range(rows):
            part = v[r, sl]
            fin = np.abs(part[np.isfinite(part)])
            e = scale_exponent(fin.max() if fin.size else 0.0, fmt)
            scales[b, r] = np.ldexp(1.0, e)
            codes[r, sl] = round8(np.ldexp(part, -e), fmt)
    return codes, scales


def dequantize(codes, scales):
    return codes * np.repeat(scales.T, BLOCK, axis=1)[:, :codes.shape[1]]


def rms(h, eps):
    h = np.asarray(h, dtype=np.float64)
    return 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)


def normed32(h, rstd32, w):
    """fl32(fl32(h rstd) w) of exact inputs: each product of two fp32 values is exact in fp64 and rounded once."""
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        p = (np.asarray(h, np.float64) * np.asarray(rstd32, np.float64)[:, None]).astype(np.float32)
        return (p.astype(np.float64) * np.asarray(w, np.float64)).astype(np.float32)


def norm_value(x, w, eps):
    x = np.asarray(x, np.float64)
    return x * rms(x, eps)[:, None] * w


def norm_backward(dy, h, rstd, w, dh=None):
    """(dx, dweight, and a bound's ingredients: |rstd g|, rstd |hat| mean|g hat|, sum |dy hat|)."""
    dy, h, w, rstd = (np.asarray(t, np.float64) for t in (dy, h, w, rstd))
    g, hat = dy * w, h * rstd[:, None]
    dx = rstd[:, None] * (g - hat * np.mean(g * hat, axis=1, keepdims=True))
    if dh is not None:
        dx = dx + dh
    sizes = (np.abs(rstd[:, None] * g), np.abs(rstd[:, None] * hat) * np.mean(np.abs(g * hat), axis=1, keepdims=True),
             np.sum(np.abs(dy * hat), axis=0))
    return dx, np.sum(dy * hat, axis=0), sizes
