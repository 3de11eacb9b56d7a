"""Plain forms of the many-tensor optimizer step, in numpy, written from its
definition (include/okls_optim.h).  Test infrastructure: nothing on the product
path uses it.

Two forms of the step: `step64`, the formulas in fp64; and `step32`, whose products
and sums are fp32 ones in the order that the definition gives, so that moments, also
those held in 8 bits, are the same bits."""
import numpy as np

from oracle import linear_oracle as L

F = np.float32
LOW = 2.0 ** -6         # e4m3's smallest normal number


def thresholds(t, place, n, first=0):
    """(u for m, u for the root) of elements first .. first + n - 1."""
    i = np.arange(first, first + n, dtype=np.uint64)
    mask = np.uint64(0xFFFFFFFF)
    key = np.uint64((t * 0x6A09E667 + place * 0xBB67AE85) & 0xFFFFFFFF)
    x = ((i & mask) * np.uint64(0x9E3779B9) + (i >> np.uint64(32)) * np.uint64(0x3C6EF372) + key) & mask
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x6A09E667)) & mask
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xBB67AE85)) & mask
    x = x ^ (x >> np.uint64(16))
    return (x & np.uint64(0xFFFF)).astype(np.float64) / 65536, (x >> np.uint64(16)).astype(np.float64) / 65536


def hold(x, u, up):
    """(codes' values, scales' values) of the fp32 vector x in blocks of 128."""
    x = np.asarray(x, F).astype(np.float64)
    n = x.size
    blocks = -(-n // 128)
    values, scales = np.zeros(n), np.ones(blocks)
    for b in range(blocks):
        part = x[b * 128: b * 128 + 128]
        fin = np.isfinite(part)
        scale = np.ldexp(1.0, L.scale_exponent(np.abs(part[fin]).max() if fin.any() else 0.0, "e4m3"))
        a = np.where(fin, np.abs(part) / scale, 0.0)
        _, ex = np.frexp(np.maximum(a, LOW))
        step = np.ldexp(1.0, ex - 1 - 3)
        k = np.floor((a / step + u[b * 128: b * 128 + 128]).astype(F))
        if up:
            k = np.where(a < LOW, np.ceil(a / step), k)
        r = np.copysign(np.minimum(k * step, 448.0), part)
        values[b * 128: b * 128 + 128] = np.where(fin, r, np.nan)
        scales[b] = scale
    return values, scales


def held(values, scales):
    return values * np.repeat(scales, 128)[: values.size]


def factor(norm, max_norm):
    """What a gradient is scaled by, in fp32."""
    return F(min(1.0, max_norm / (float(F(norm)) + 1e-6)))


def norm(grads):
    return np.sqrt(sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads))


def step64(p, g, m, v, t, lr, beta1, beta2, eps, weight_decay, scale=1.0):
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    g = g * scale
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    hat = (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return (1 - lr * weight_decay) * p - lr * hat, m, v


def step32(p, g, m, v, t, lr, beta1, beta2, eps, weight_decay, scale=None):
    """(p, m, v, v's root) in fp32 as the definition rounds them."""
    p, g, m, v = (np.asarray(x, F) for x in (p, g, m, v))
    with np.errstate(all="ignore"):
        g = g if scale is None else g * F(scale)
        m = F(beta1) * m + F(1 - beta1) * g
        v = F(beta2) * v + F(1 - beta2) * g * g
        s = np.sqrt(v)
        p = p * F(1 - lr * weight_decay) - F(lr / (1 - beta1 ** t)) * (m / (s * F((1 - beta2 ** t) ** -0.5) + F(eps)))
    return p, m, v, s


def step8(p, g, m, s, t, place, first=0, **hyper):
    """One step with moments held in 8 bits: m and s are (values, scales); (p, m, s) after it."""
    old_m, old_s = (held(*x).astype(F) for x in (m, s))
    p, new_m, _, new_s = step32(p, g, old_m, old_s * old_s, t, **hyper)
    u, w = thresholds(t, place, np.asarray(p).size, first)
    return p, hold(new_m, u, False), hold(new_s, w, True)
