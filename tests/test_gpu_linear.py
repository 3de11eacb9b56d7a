"""8-bit linear-layer operators on the GPU against the fp64 oracle.

Tolerances are derived from the roundings the operators make: the 8-bit form is
compared exactly (a power-of-two scale and one rounding leave one right answer);
a sum of k fp32 terms is off by at most k 2^-23 of the sum of their sizes (one
unit in the last place an addition); a result's type rounds by half its eps."""
import numpy as np
import pytest

from oracle import linear_oracle as L

torch = pytest.importorskip("torch")
from kronecker_factored_second_amd import linear, okls  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = 2.0 ** -23


def _rng(*key):
    return np.random.default_rng([hash_ % (1 << 31) for hash_ in key])


def _t(a, kind="f32"):
    return torch.tensor(np.asarray(a, np.float32)).to(FLOATS[kind]).cuda()


def _n(t):
    return t.detach().cpu().double().numpy()


def _padded(t, pad, offset=0):
    """The same matrix inside a wider one: row stride cols + pad, first element `offset` elements in."""
    rows, cols = t.shape
    base = torch.full((rows * (cols + pad) + offset,), 7.0, dtype=t.dtype, device=t.device)
    v = base[offset:].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def _half(kind):
    return torch.finfo(FLOATS[kind]).eps / 2


def _tiny(kind):
    """Half the smallest step of the type."""
    return {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}[kind]


def _check_blocked(q, v, fmt):
    codes, scales = L.quantize(v, fmt)
    rows, cols = v.shape
    assert np.array_equal(_n(q.scales)[:, :rows], scales)
    assert np.array_equal(_n(q.codes)[:, :cols], codes, equal_nan=True)
    end = -(-cols // 128) * 128
    assert not q.codes[:, cols:end].view(torch.uint8).any()       # the last block's rest is zeros


def _values(rng, m, k):
    v = rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)))
    v[:, rng.random(k) < 0.02] *= 20
    return v


# ---------------------------------------------------------------------------
# quantize
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 128), (3, 127), (17, 129), (128, 128), (130, 257), (129, 1000), (300, 72)])
def test_quantize(m, k, kind, fmt):
    x = _t(_values(_rng(m, k), m, k), kind)
    q, t = linear.quantize_both(x, dtype=F8[fmt])
    _check_blocked(q, _n(x), fmt)
    _check_blocked(t, _n(x).T, fmt)
    one, other = linear.quantize(x, dtype=F8[fmt]), linear.quantize(x, dtype=F8[fmt], transpose=True)
    for a, b in ((one, q), (other, t)):
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
        assert torch.equal(a.scales.view(torch.uint8)[:, :a.shape[0]], b.scales.view(torch.uint8)[:, :a.shape[0]])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (3, 1), (0, 1), (0, 3)])
def test_quantize_strides_and_alignment(kind, pad, offset):
    x = _padded(_t(_values(_rng(5), 140, 200), kind), pad, offset)
    q, t = linear.quantize_both(x)
    _check_blocked(q, _n(x), "e4m3")
    _check_blocked(t, _n(x).T, "e4m3")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_borders(fmt):
    """Block maxima at and next to F 2^e, every rounding midpoint, zeros, subnormals, the largest floats, infinities and NaN."""
    top, frac, low = L.FORMATS[fmt]
    x = np.zeros((40, 256), np.float32)
    x[0, 0], x[1, 0], x[2, 0] = top, np.nextafter(np.float32(top), np.float32(np.inf)), np.nextafter(np.float32(top), np.float32(0))
    for i, e in enumerate((-140, -127, -120, -100, -1, 60, 110)):
        x[3 + i, 5] = np.ldexp(np.float32(1.75), e)
        x[3 + i, 130] = np.nextafter(np.ldexp(np.float32(1.75), e), np.float32(np.inf))
    x[10, 3], x[10, 4] = 2.0 ** -149, -2.0 ** -149
    x[11, 7], x[11, 200] = 3.4e38, -3.4e38
    x[12, :] = np.inf
    x[13, 9], x[13, 10], x[13, 11], x[13, 12] = np.inf, -np.inf, np.nan, 3.0
    x[14, 200] = np.nan
    codes = torch.arange(128, dtype=torch.uint8).view(F8[fmt]).double().numpy()
    fin = np.unique(codes[np.isfinite(codes)])
    mid = (fin[1:] + fin[:-1]) / 2
    for r, vals in ((15, mid), (16, np.nextafter(mid.astype(np.float32), np.float32(np.inf))), (17, np.nextafter(mid.astype(np.float32), np.float32(0)))):
        x[r, 0] = top                                   # the block's scale is 1
        x[r, 1:1 + len(vals[:127])] = vals[:127]
        x[r, 128] = -top
        x[r, 129:129 + len(vals[:127])] = -vals[:127]
    g = torch.tensor(x, device="cuda")
    q, t = linear.quantize_both(g, dtype=F8[fmt])
    _check_blocked(q, x.astype(np.float64), fmt)
    _check_blocked(t, x.astype(np.float64).T, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_two_formats_and_factors(fmt):
    rng = _rng(9)
    h, w = _t(_values(rng, 200, 150), "bf16"), _t(1 + 0.2 * rng.standard_normal(150), "bf16")
    rstd = _t(np.exp(rng.standard_normal(200)))
    q, t = linear.quantize_both(h, dtype=F8[fmt], row_factor=rstd, col_factor=w)
    v = L.normed32(_n(h), _n(rstd), _n(w)).astype(np.float64)
    _check_blocked(q, v, fmt)
    _check_blocked(t, v.T, fmt)
    # one call, another format for each orientation
    a, b = linear.Blocked.empty(200, 150, F8["e4m3"], h.device), linear.Blocked.empty(150, 200, F8["e5m2"], h.device)
    linear._quantize(h, a, b, None, None)
    _check_blocked(a, _n(h), "e4m3")
    _check_blocked(b, _n(h).T, "e5m2")


def test_quantize_nothing():
    for shape in ((0, 300), (5, 0)):
        q, t = linear.quantize_both(torch.zeros(shape, device="cuda"))
        assert q.shape == shape and t.shape == shape[::-1]


# ---------------------------------------------------------------------------
# matmul
# ---------------------------------------------------------------------------
def _held(q):
    rows, cols = q.shape
    return L.dequantize(_n(q.codes)[:, :cols], _n(q.scales)[:, :rows])


def _check_product(c, a, b, kind, base=None):
    """c against a b^T (+ base) of the held values.

    fp32 results come from bf16 products, whose sums round as fp32's.  16-bit
    results come from the 8-bit matrix instructions, which line up each eight
    products on the largest and cut what is below 2^-13 of it: a group loses less
    than 8 2^-13 of its largest, so no more than 2^-10 of its sum of sizes.  The
    cut parts have their products' signs, so over k products of signs of their
    own they add up to sqrt(k) 2^-13 times a group's largest, at most sqrt(8)
    times a product's root mean square: 2^-11.5 of the result in norm."""
    x, y = _held(a), _held(b)
    want, size = x @ y.T, np.abs(x) @ np.abs(y).T
    cut = 0.0 if kind == "f32" else size * 2.0 ** -10
    if base is not None:
        want, size = want + base, size + np.abs(base)
    k = x.shape[1]
    got, most = _n(c), size * (k + 1) * ULP + cut
    if kind == "f16":       # a result that rounds past 65504 is an infinity of its sign
        over = np.isinf(got)
        assert (np.abs(want) + most >= 65520)[over].all() and (np.sign(got) == np.sign(want))[over].all()
        got = np.where(over, want, got)
    off = np.abs(got - want)
    assert (off <= np.abs(want) * _half(kind) + most + _tiny(kind)).all()
    if kind != "f32" and want.size >= 1000:
        assert np.linalg.norm(off) <= (_half(kind) + 2.0 ** -11.5) * np.linalg.norm(want)


def _operands(m, n, k, fa="e4m3", fb="e4m3", key=0):
    rng = _rng(m, n, k, key)
    return (linear.quantize(_t(_values(rng, m, k)), dtype=F8[fa]), linear.quantize(_t(_values(rng, n, k)), dtype=F8[fb]))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 128), (1, 100, 1000), (2, 513, 129), (15, 17, 255), (16, 256, 640), (17, 130, 384),
                                   (33, 64, 512), (64, 1000, 2000), (65, 127, 300), (128, 128, 128), (129, 255, 1100),
                                   (256, 256, 256), (300, 520, 130), (511, 257, 896), (1000, 700, 1500)])
def test_matmul(m, n, k, kind):
    a, b = _operands(m, n, k)
    _check_product(linear.matmul(a, b, dtype=FLOATS[kind]), a, b, kind)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", [(5, 300, 700), (200, 150, 300), (600, 600, 400)])
def test_matmul_formats(fa, fb, m, n, k):
    a, b = _operands(m, n, k, fa, fb)
    _check_product(linear.matmul(a, b, dtype=torch.float32), a, b, "f32")


@pytest.mark.parametrize("m,n,k", [(3, 200, 5000), (1, 64, 16384), (48, 128, 11008), (100, 200, 9000), (260, 300, 20000), (2000, 1030, 640)])
def test_matmul_long_and_tall(m, n, k):
    a, b = _operands(m, n, k)
    c = linear.matmul(a, b, dtype=torch.float32)
    _check_product(c, a, b, "f32")
    assert torch.equal(c, linear.matmul(a, b, dtype=torch.float32))     # equal bits every time


def test_matmul_every_scale():
    """Each row of a and b at its own power of two, over all that a block can have next to the other's."""
    rng = _rng(11)
    x, y = rng.standard_normal((253, 128)), rng.standard_normal((64, 128))
    x = np.ldexp(x, (np.arange(253) - 130)[:, None])
    y = np.ldexp(y, np.where(np.arange(64) % 2, 3, -20)[:, None])
    a, b = linear.quantize(_t(x)), linear.quantize(_t(y))
    c = _n(linear.matmul(a, b, dtype=torch.float32))
    p, q = _held(a), _held(b)
    want, size = p @ q.T, np.abs(p) @ np.abs(q).T
    normal = (np.abs(p).max(1)[:, None] * np.abs(q).max(1)[None, :] > 2.0 ** -100) & (size < 2.0 ** 126)
    assert normal.sum() > 8000
    assert (np.abs(c - want) <= size * 129 * ULP + np.abs(want) * 2.0 ** -24)[normal].all()
    # below: no more than a product of subnormal operands leaves
    assert (np.abs(c - want) <= 2.0 ** -99)[~normal & (size < 2.0 ** -90)].all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 70, 300), (40, 200, 5000), (130, 250, 300), (513, 260, 300)])
def test_matmul_accumulate_and_strided_output(m, n, k, kind):
    a, b = _operands(m, n, k)
    base = _t(_rng(3).standard_normal((m, n)) * 10, kind)
    for pad, offset in ((0, 0), (1, 0), (8, 0), (5, 3)):
        out = _padded(base, pad, offset)
        whole = out.storage_offset(), out.untyped_storage().size()
        linear.matmul(a, b, out=out, accumulate=True)
        _check_product(out, a, b, kind, _n(base))
        flat = torch.as_strided(out, (m * (n + pad),), (1,), whole[0])
        assert (flat.view(m, n + pad)[:, n:] == 7.0).all()          # nothing past a row's end is written
        assert (torch.as_strided(out, (offset,), (1,), 0) == 7.0).all()


def test_matmul_nan_stays_in_its_row():
    x = _values(_rng(4), 70, 400)
    x[3, 200], x[69, 399] = np.nan, np.inf
    a, b = linear.quantize(_t(x)), linear.quantize(_t(_values(_rng(5), 300, 400)))
    c = linear.matmul(a, b)
    bad = torch.zeros(70, dtype=torch.bool)
    bad[[3, 69]] = True
    assert c[bad.cuda()].isnan().all() and c[~bad.cuda()].isfinite().all()


def test_matmul_nothing_to_sum_or_give():
    a, b = linear.quantize(torch.zeros(5, 0, device="cuda")), linear.quantize(torch.zeros(7, 0, device="cuda"))
    assert torch.equal(linear.matmul(a, b), torch.zeros(5, 7, dtype=torch.bfloat16, device="cuda"))
    out = torch.ones(5, 7, device="cuda")
    assert torch.equal(linear.matmul(a, b, out=out, accumulate=True), torch.ones(5, 7, device="cuda"))
    e = linear.quantize(torch.zeros(0, 300, device="cuda"))
    f = linear.quantize(torch.ones(4, 300, device="cuda"))
    assert linear.matmul(e, f).shape == (0, 4) and linear.matmul(f, e).shape == (4, 0)


def test_matmul_wide_strided_operand():
    """Operands whose code rows and scale rows are longer than the matrix."""
    a, b = _operands(40, 50, 300)
    codes = torch.full((40, 640), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((5, 64), 255, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    codes.view(torch.uint8)[:, :384] = a.codes.view(torch.uint8)
    scales.view(torch.uint8)[:3, :48] = a.scales.view(torch.uint8)
    wide = linear.Blocked(codes, scales[:3], (40, 300))
    assert torch.equal(linear.matmul(wide, b), linear.matmul(a, b))


def test_matmul_refusals():
    a, b = _operands(4, 5, 200)
    with pytest.raises(ValueError):
        linear.matmul(a, _operands(4, 5, 201)[1])
    with pytest.raises(ValueError):
        linear.matmul(a, b, dtype=torch.float64)
    with pytest.raises(ValueError):
        linear.matmul(a, b, accumulate=True)
    for out in (torch.empty(4, 6, device="cuda"), torch.empty(5, 4, device="cuda").T, torch.empty(4, 5, dtype=torch.int32, device="cuda"), torch.empty(4, 5)):
        with pytest.raises(ValueError):
            linear.matmul(a, b, out=out)
    with pytest.raises(ValueError):     # codes that do not hold the shape
        linear.matmul(linear.Blocked(a.codes, a.scales, (4, 300)), b)
    with pytest.raises(ValueError):
        linear.matmul(linear.Blocked(a.codes.view(torch.uint8), a.scales, (4, 200)), b)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
NORM_SIZES = [(1, 1), (1, 128), (2, 127), (5, 129), (1, 4096), (7, 1000), (33, 2048), (9, 2816), (130, 384), (3, 5121), (2, 16384), (2, 16391), (1, 40000)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k", NORM_SIZES)
def test_rms_norm(m, k, kind):
    rng = _rng(m, k, 1)
    x, r, w = _t(_values(rng, m, k), kind), _t(_values(rng, m, k), kind), _t(1 + 0.2 * rng.standard_normal(k), kind)
    for res, fmt in ((None, "e4m3"), (r, "e4m3"), (r, "e5m2")):
        q, h, rstd = linear.rms_norm(x, w, residual=res, eps=1e-5, dtype=F8[fmt])
        if res is None:
            assert h is x
        else:
            assert torch.equal(h, (x.float() + r.float()).to(x.dtype))
        want = L.rms(_n(h), np.float64(np.float32(1e-5)))
        # one rounding to fp32; the fp64 sums' own are 2^-29 of it
        assert (np.abs(_n(rstd) - want) <= want * 2.0 ** -24 * (1 + 2.0 ** -20)).all()
        _check_blocked(q, L.normed32(_n(h), _n(rstd), _n(w)).astype(np.float64), fmt)


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (3, 1), (0, 1)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rms_norm_strides(kind, pad, offset):
    rng = _rng(21)
    x, r, w = _t(_values(rng, 9, 700), kind), _t(_values(rng, 9, 700), kind), _t(1 + 0.2 * rng.standard_normal(701), "bf16")[1:]
    a = linear.rms_norm(_padded(x, pad, offset), w, residual=_padded(r, 2 * pad, offset))
    b = linear.rms_norm(x, w.clone(), residual=r)
    assert torch.equal(a.h, b.h) and torch.equal(a.rstd, b.rstd)
    assert torch.equal(a.q.codes.view(torch.uint8), b.q.codes.view(torch.uint8))
    assert torch.equal(a.q.scales.view(torch.uint8)[:, :9], b.q.scales.view(torch.uint8)[:, :9])


def test_rms_norm_rows_of_zeros_and_extremes():
    x = np.zeros((6, 300), np.float32)
    x[1, 5] = 1e30          # its square is beyond fp32
    x[2] = 1e-30            # and this one's below it
    x[3, 7] = np.inf
    x[4, 8] = np.nan
    x[5] = 1.0
    w = np.ones(300, np.float32)
    q, h, rstd = linear.rms_norm(_t(x), _t(w), eps=1e-6)
    with np.errstate(invalid="ignore"):
        want = L.rms(x, np.float64(np.float32(1e-6))).astype(np.float32)
    assert np.array_equal(rstd.cpu().numpy(), want, equal_nan=True)
    _check_blocked(q, L.normed32(x, want, w).astype(np.float64), "e4m3")
    e = linear.rms_norm(torch.zeros(0, 300, device="cuda"), _t(w), residual=torch.zeros(0, 300, device="cuda"))
    assert e.q.shape == (0, 300) and e.h.shape == (0, 300) and e.rstd.shape == (0,)


def _check_norm_grads(dx, dw, dy, h, rstd, w, dh, kind, wkind):
    k, m = h.shape[1], h.shape[0]
    want, wantw, (s1, s2, s3) = L.norm_backward(_n(dy), _n(h), _n(rstd), _n(w), None if dh is None else _n(dh))
    size = s1 + s2 + (0 if dh is None else np.abs(_n(dh)))
    assert (np.abs(_n(dx) - want) <= np.abs(want) * _half(kind) + 8 * ULP * size + s2 * (k + 8) * ULP + _tiny(kind)).all()
    assert (np.abs(_n(dw) - wantw) <= np.abs(wantw) * _half(wkind) + s3 * (m + 8) * ULP + _tiny(wkind)).all()


@pytest.mark.parametrize("kind,wkind", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("m,k", NORM_SIZES + [(1500, 512), (600, 257), (2100, 64)])
def test_rms_norm_backward(m, k, kind, wkind):
    rng = _rng(m, k, 2)
    h, dy, dh = (_t(_values(rng, m, k), kind) for _ in range(3))
    w = _t(1 + 0.2 * rng.standard_normal(k), wkind)
    rstd = _t(L.rms(_n(h), 1e-6))
    for d in (None, dh):
        dx, dw = linear.rms_norm_backward(dy, h, rstd, w, dh=d)
        assert dx.dtype == h.dtype and dw.dtype == w.dtype
        _check_norm_grads(dx, dw, dy, h, rstd, w, d, kind, wkind)
        again = linear.rms_norm_backward(dy, h, rstd, w, dh=d)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 1)])
def test_rms_norm_backward_strides(pad, offset):
    rng = _rng(31)
    h, dy, dh = (_t(_values(rng, 50, 333), "bf16") for _ in range(3))
    w, rstd = _t(1 + 0.2 * rng.standard_normal(333)), _t(L.rms(_n(h), 1e-6))
    a = linear.rms_norm_backward(_padded(dy, pad, offset), _padded(h, pad, offset), rstd, w, dh=_padded(dh, pad, offset))
    b = linear.rms_norm_backward(dy, h, rstd, w, dh=dh)
    _check_norm_grads(*a, dy, h, rstd, w, dh, "bf16", "f32")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rms_norm_backward_nothing_and_refusals():
    w = torch.ones(40, device="cuda")
    z = torch.zeros(0, 40, device="cuda")
    dx, dw = linear.rms_norm_backward(z, z, torch.zeros(0, device="cuda"), w)
    assert dx.shape == (0, 40) and torch.equal(dw, torch.zeros(40, device="cuda"))
    h, r = torch.ones(4, 40, device="cuda"), torch.ones(4, device="cuda")
    for bad in (dict(dy=h[:3]), dict(dy=h.bfloat16()), dict(rstd=r[:3]), dict(rstd=r.double()), dict(rstd=r.half()), dict(weight=w[:39]),
                dict(dh=h.half()), dict(dy=torch.ones(40, 4, device="cuda").T), dict(dy=h[:1].expand(4, 40))):
        with pytest.raises(ValueError):
            linear.rms_norm_backward(**{**dict(dy=h, h=h, rstd=r, weight=w), **bad})
    for bad in (dict(weight=w[:39]), dict(residual=h[:3]), dict(residual=h.half()), dict(dtype=torch.float16), dict(x=h.double()), dict(x=h[0])):
        with pytest.raises(ValueError):
            linear.rms_norm(**{**dict(x=h, weight=w), **bad})
    with pytest.raises(okls.OKLSError):
        linear.rms_norm(h, w, eps=-1.0)
    for bad in (dict(row_factor=r), dict(row_factor=r[:3], col_factor=w), dict(row_factor=r.half(), col_factor=w), dict(row_factor=r, col_factor=w[1:])):
        with pytest.raises(ValueError):
            linear.quantize(h, **bad)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,k,n,grad", [(40, 200, 300, "e4m3"), (130, 256, 128, "e5m2"), (1, 128, 257, "e4m3")])
@pytest.mark.parametrize("residual", [True, False])
def test_layer_gradients(m, k, n, grad, residual):
    """rms_norm_linear's outputs and gradients: each against the formula on what the step before it gave."""
    rng = _rng(m, k, n)
    x, r = _t(_values(rng, m, k), "bf16").requires_grad_(), _t(_values(rng, m, k), "bf16").requires_grad_()
    nw, W = _t(1 + 0.2 * rng.standard_normal(k)).requires_grad_(), _t(0.05 * rng.standard_normal((n, k))).requires_grad_()
    dy, dh = _t(rng.standard_normal((m, n)), "bf16"), _t(rng.standard_normal((m, k)), "bf16")
    y, h = linear.rms_norm_linear(x, nw, W, residual=r if residual else None, grad_dtype=F8[grad])
    leaves = (x, r, nw, W) if residual else (x, nw, W)
    grads = torch.autograd.grad((y, h), leaves, (dy, dh))
    q, hh, rstd = linear.rms_norm(x.detach(), nw.detach(), residual=r.detach() if residual else None)
    assert torch.equal(h, hh)
    w, wt = linear.quantize_both(W.detach())
    _check_product(y, q, w, "bf16")
    dq, dt = linear.quantize_both(dy, dtype=F8[grad])
    v = L.normed32(_n(hh), _n(rstd), _n(nw)).astype(np.float64)
    vt = linear.quantize(hh, transpose=True, row_factor=rstd, col_factor=nw.detach())
    _check_blocked(vt, v.T, "e4m3")
    _check_product(grads[-1], dt, vt, "f32")
    assert grads[-1].dtype == torch.float32
    dv = linear.matmul(dq, wt)
    _check_product(dv, dq, wt, "bf16")
    dx, dw = linear.rms_norm_backward(dv, hh, rstd, nw.detach(), dh=dh if residual else None)
    if residual:
        assert torch.equal(grads[0], dx) and torch.equal(grads[1], dx)
    else:       # the stream's gradient joins outside, rounded to its type there
        assert torch.equal(grads[0], dx + dh)
    assert torch.equal(grads[-2], dw)


def test_layer_gradient_near_the_unrounded_layers():
    """Against the layer in fp64 without 8 bits: the roundings are off by 2^-4 of each value at most, independent over a sum, so the sums' own relative error stays below it."""
    rng = _rng(77)
    x, nw, W = _t(rng.standard_normal((256, 512))), _t(1 + 0.2 * rng.standard_normal(512)), _t(0.05 * rng.standard_normal((384, 512)))
    dy = _t(rng.standard_normal((256, 384)))
    for t in (x, nw, W):
        t.requires_grad_()
    y, _ = linear.rms_norm_linear(x, nw, W)
    got = torch.autograd.grad(y, (x, nw, W), dy)
    X, N, V = (t.detach().cpu().double().requires_grad_() for t in (x, nw, W))
    ref = (X * torch.rsqrt(X.square().mean(1, keepdim=True) + 1e-6) * N) @ V.T
    want = torch.autograd.grad(ref, (X, N, V), dy.cpu().double())
    for a, b in zip((y, *got), (ref, *want)):
        assert (a.detach().cpu().double() - b.detach()).norm() < 2.0 ** -4 * b.norm()


def test_scaled_linear_and_partial_gradients():
    rng = _rng(88)
    x, W, dy = _t(_values(rng, 70, 300), "bf16"), _t(0.05 * rng.standard_normal((140, 300))), _t(rng.standard_normal((70, 140)), "bf16")
    (q, t), (w, wt), (dq, dt) = linear.quantize_both(x), linear.quantize_both(W), linear.quantize_both(dy)
    for nx, nw in ((True, True), (True, False), (False, True)):
        a, b = x.clone().requires_grad_(nx), W.clone().requires_grad_(nw)
        y = linear.scaled_linear(a, b)
        assert torch.equal(y, linear.matmul(q, w))
        y.backward(dy)
        assert (a.grad is not None) == nx and (b.grad is not None) == nw
        if nx:
            assert torch.equal(a.grad, linear.matmul(dq, wt))
        if nw:
            assert torch.equal(b.grad, linear.matmul(dt, t, dtype=torch.float32))
    # an expanded gradient, as a sum's backward hands it over
    a = x.clone().requires_grad_()
    linear.scaled_linear(a, W).sum().backward()
    assert torch.equal(a.grad, linear.matmul(linear.quantize(torch.ones_like(dy)), wt))
    # only the residual stream went on
    a, r = x.clone().requires_grad_(), x.clone().requires_grad_()
    _, h = linear.rms_norm_linear(a, torch.ones(300, device="cuda"), W, residual=r)
    h.sum().backward()
    assert (a.grad == 1).all() and (r.grad == 1).all() and a.grad.data_ptr() != r.grad.data_ptr()


def test_other_stream():
    rng = _rng(99)
    x, w, W = _t(_values(rng, 500, 700), "bf16"), _t(np.ones(700)), _t(rng.standard_normal((300, 700)))
    want = linear.matmul(linear.rms_norm(x, w).q, linear.quantize(W))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = linear.matmul(linear.rms_norm(x, w).q, linear.quantize(W))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_graph_replays():
    """Forward and backward calls captured once and replayed, with eager work and new inputs between."""
    rng = _rng(111)
    x, w, W = _t(_values(rng, 300, 640), "bf16"), _t(1 + 0.1 * rng.standard_normal(640)), _t(0.05 * rng.standard_normal((520, 640)))
    dy = _t(rng.standard_normal((300, 520)), "bf16")

    def step():
        q, h, rstd = linear.rms_norm(x, w, residual=x)
        a, at = linear.quantize_both(W)
        y = linear.matmul(q, a)
        dq, dt = linear.quantize_both(dy)
        dW = linear.matmul(dt, linear.quantize(h, transpose=True, row_factor=rstd, col_factor=w), dtype=torch.float32)
        return (y, dW, *linear.rms_norm_backward(linear.matmul(dq, at), h, rstd, w, dh=h))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(4):
        x.copy_(_t(_values(_rng(i), 300, 640), "bf16"))
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_with_the_optimizer():
    """A layer's weight gradient goes into the optimizer's step as it comes."""
    rng = _rng(123)
    x, nw, W = _t(_values(rng, 200, 96), "bf16"), _t(np.ones(96)), _t(0.05 * rng.standard_normal((160, 96))).requires_grad_()
    twin = W.detach().clone()
    opt, other = okls.OKLS([W]), okls.OKLS([twin])
    for _ in range(2):
        y, _ = linear.rms_norm_linear(x, nw, W)
        y.float().square().mean().backward()
        g = W.grad.clone()
        with torch.no_grad():
            opt.step()
        other.step(grads=[g])
        opt.zero_grad()
    assert torch.equal(W.detach(), twin)


# ---------------------------------------------------------------------------
# Every way through the product and the norm that sizes choose
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(2569, 4101, 200), (2600, 4352, 130), (8300, 1300, 1), (1409, 1921, 300), (1280, 2048, 385),
                                   (40, 2101, 4101), (17, 4096, 2200), (63, 9000, 1000), (65, 130, 8000), (100, 100, 3333), (700, 701, 640)])
def test_matmul_tiles(m, n, k, kind):
    """256 and 128 tiles whole and with ragged ends, narrow tiles with the sum whole and split."""
    a, b = _operands(m, n, k, "e5m2" if k % 2 else "e4m3", "e4m3", key=5)
    _check_product(linear.matmul(a, b, dtype=FLOATS[kind]), a, b, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(2569, 4101, 140), (1409, 1921, 140), (40, 2101, 4101)])
def test_matmul_tiles_accumulate_and_strided_output(m, n, k, kind):
    a, b = _operands(m, n, k, key=6)
    base = _t(_rng(8).standard_normal((m, n)) * 10, kind)
    for pad, offset in ((0, 0), (3, 1)):
        out = _padded(base, pad, offset)
        whole = out.storage_offset()
        linear.matmul(a, b, out=out, accumulate=True)
        _check_product(out, a, b, kind, _n(base))
        flat = torch.as_strided(out, (m * (n + pad),), (1,), whole)
        assert (flat.view(m, n + pad)[:, n:] == 7.0).all()
        assert (torch.as_strided(out, (offset,), (1,), 0) == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_matmul_far_rows(kind):
    """Rows of codes 2^24 bytes apart: offsets inside a tile pass 32 bits."""
    a, b = _operands(130, 70, 300, key=9)
    codes = torch.empty((130, 1 << 24), dtype=torch.uint8, device="cuda")
    codes[:, :384] = a.codes.view(torch.uint8)
    far = linear.Blocked(codes.view(torch.float8_e4m3fn), a.scales, (130, 300))
    c = linear.matmul(far, b, dtype=FLOATS[kind])
    _check_product(c, a, b, kind)
    _check_product(linear.matmul(b, far, dtype=FLOATS[kind]), b, a, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m", [3, 70, 1300])
def test_matmul_ends_of_the_scales(m, kind):
    """Blocks at the lowest scale, 2^-127, and at the highest, times ones that bring them back."""
    n = 2000 if m == 1300 else 100
    rng = _rng(m, 17)
    low = np.ldexp(rng.integers(1, 16, (m, 128)).astype(np.float64), -124)       # normal floats; 15 2^-124 <= 448 2^-127
    high = np.ldexp(rng.integers(1, 8, (n, 128)).astype(np.float64), 120)
    a, b = linear.quantize(_t(low)), linear.quantize(_t(high))
    assert (a.scales.view(torch.uint8)[:, :m] < 8).all()
    _check_product(linear.matmul(a, b, dtype=FLOATS[kind]), a, b, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("k", [512, 513, 600, 1024, 1025, 1500, 2049, 6000, 8192, 8193, 9001, 16385])
def test_norm_widths(k, kind):
    """Each layout of a row over waves, and the widths around where it changes."""
    m = 37
    rng = _rng(k, 41)
    x, r, dy, dh = (_t(_values(rng, m, k), kind) for _ in range(4))
    w = _t(1 + 0.2 * rng.standard_normal(k), kind)
    q, h, rstd = linear.rms_norm(x, w, residual=r)
    want = L.rms(_n(h), np.float64(np.float32(1e-6)))
    assert (np.abs(_n(rstd) - want) <= want * 2.0 ** -24 * (1 + 2.0 ** -20)).all()
    _check_blocked(q, L.normed32(_n(h), _n(rstd), _n(w)).astype(np.float64), "e4m3")
    _check_norm_grads(*linear.rms_norm_backward(dy, h, rstd, w, dh=dh), dy, h, rstd, w, dh, kind, kind)


def test_norm_backward_in_place():
    """dx may be dy or dh, through the C entry: every row is read before it is written."""
    lib = linear.load()
    rng = _rng(51)
    for m, k in ((300, 700), (40, 3000), (9, 20000)):
        h, dy, dh = (_t(_values(rng, m, k), "bf16") for _ in range(3))
        w, rstd = _t(1 + 0.2 * rng.standard_normal(k)), _t(L.rms(_n(h), 1e-6))
        want, wantw = linear.rms_norm_backward(dy, h, rstd, w, dh=dh)
        need = lib.okls_rms_norm_backward_workspace_size(m, k)
        for which in range(2):
            ins = [dy.clone(), dh.clone()]
            dw, ws = torch.empty_like(w), torch.empty(need, dtype=torch.uint8, device="cuda")
            st = lib.okls_rms_norm_backward(ins[0].data_ptr(), k, h.data_ptr(), k, rstd.data_ptr(), w.data_ptr(), okls.OKLS_F32, ins[1].data_ptr(), k,
                                            okls.OKLS_BF16, m, k, ins[which].data_ptr(), k, dw.data_ptr(), ws.data_ptr(), need,
                                            torch.cuda.current_stream().cuda_stream)
            assert st == 0 and torch.equal(dw, wantw)
            assert torch.equal(ins[which], want)


def test_example_learns():
    """The example's stack comes nearer its teacher, by the same losses every time."""
    from examples import train_8bit_mlp
    losses = train_8bit_mlp.train(steps=12, blocks=2, d=128, f=192, tokens=200)
    assert np.isfinite(losses).all() and np.mean(losses[-3:]) < np.mean(losses[:3])
    assert losses == train_8bit_mlp.train(steps=12, blocks=2, d=128, f=192, tokens=200)


def test_no_second_derivative():
    """A gradient of a gradient is refused, not taken as zero."""
    x, W = torch.randn(8, 128, device="cuda").requires_grad_(), torch.randn(16, 128, device="cuda").requires_grad_()
    (g,) = torch.autograd.grad(linear.scaled_linear(x, W).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), W)


def test_matmul_more_columns_than_a_launch():
    """2^24 columns are more 16-column groups than one launch of the few-rows kernel takes."""
    n = (1 << 24) + 40
    a = linear.quantize(_t(_rng(61).integers(1, 8, (1, 8))))
    b = linear.Blocked.empty(n, 8, torch.float8_e4m3fn, "cuda")
    b.scales.view(torch.uint8).fill_(127)
    b.codes.view(torch.uint8).zero_()
    b.codes[:, 0] = (torch.arange(n, device="cuda") % 13).float().to(torch.float8_e4m3fn)
    c = linear.matmul(a, b, dtype=torch.float32)
    want = a.dequantize()[0, 0] * (torch.arange(n, device="cuda") % 13).float()
    assert torch.equal(c[0], want)          # small whole numbers: nothing rounds


@pytest.mark.parametrize("m", [1, 5, 70])
def test_gradient_of_one_column(m):
    """A layer of one output column (a value or reward head), and a stream of one: gradients that a sum's backward expands have a row stride of zero."""
    rng = _rng(m, 89)
    x, W, nw = _t(_values(rng, m, 300), "bf16"), _t(0.05 * rng.standard_normal((1, 300))), _t(1 + 0.2 * rng.standard_normal(300))
    for f in (lambda a, b: linear.scaled_linear(a, b), lambda a, b: linear.rms_norm_linear(a, nw, b)[0],
              lambda a, b: linear.rms_norm_linear(a, nw, b, residual=x)[0]):
        got, want = [], []
        for grads, back in ((got, lambda y: y.sum().backward()), (want, lambda y: y.backward(torch.ones_like(y)))):
            a, b = x.clone().requires_grad_(), W.clone().requires_grad_()
            back(f(a, b))
            grads += [a.grad, b.grad]
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    # a residual stream of one column, its gradient expanded as well
    s, w1, V = _t(_values(rng, m, 1), "bf16"), _t([1.5]), _t(rng.standard_normal((20, 1)))

    def grads(back):
        a, r = s.clone().requires_grad_(), s.clone().requires_grad_()
        back(linear.rms_norm_linear(a, w1, V, residual=r))
        return a.grad, r.grad

    got = grads(lambda yh: torch.autograd.backward(yh, (torch.ones_like(yh[0]), torch.ones(1, dtype=torch.bfloat16, device="cuda").expand(m, 1))))
    want = grads(lambda yh: torch.autograd.backward(yh, [torch.ones_like(t) for t in yh]))
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def _bits(q):
    return q.codes.view(torch.uint8), q.scales.view(torch.uint8)[:, :q.shape[0]]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m,k", [(9, 700), (5, 1000), (5, 4096), (3, 16384), (3, 16385), (3, 16391), (2, 40000)])
def test_rms_norm_in_place(m, k, kind):
    """h may be x or the residual, through the C entry: rows that are read once and rows that are read again."""
    lib = linear.load()
    rng = _rng(m, k, 52)
    x, r, w = _t(_values(rng, m, k), kind), _t(_values(rng, m, k), kind), _t(1 + 0.2 * rng.standard_normal(k))
    want = linear.rms_norm(x, w, residual=r)
    for which in range(2):
        ins = [x.clone(), r.clone()]
        q, rstd = linear.Blocked.empty(m, k, F8["e4m3"], x.device), torch.empty(m, device="cuda")
        dt = linear.DTYPES[x.dtype]
        st = lib.okls_rms_norm(ins[0].data_ptr(), k, ins[1].data_ptr(), k, dt, m, k, w.data_ptr(), okls.OKLS_F32, 1e-6, ins[which].data_ptr(), k,
                               rstd.data_ptr(), q.struct(), torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(ins[which], want.h) and torch.equal(rstd, want.rstd)
        assert all(torch.equal(p, o) for p, o in zip(_bits(q), _bits(want.q)))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("m", [8, 70, 300])
def test_out_is_seen_by_autograd(m, accumulate):
    """A buffer that a graph keeps and a product then overwrites: the graph's backward raises, as after torch's own writes."""
    a, b = linear.quantize(torch.ones(m, 128, device="cuda")), linear.quantize(torch.ones(16, 128, device="cuda"))
    out, x = torch.ones(m, 16, device="cuda"), torch.ones(m, 16, device="cuda").requires_grad_()
    y = (x * out).sum()                             # keeps out for x's gradient
    view = out[:, :8]
    linear.matmul(a, b, out=out, accumulate=accumulate)
    assert out._version > 0 and view._version == out._version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    fresh = (x * out).sum()                         # what is kept after the write is right
    fresh.backward()
    assert torch.equal(x.grad, out)


def test_out_that_requires_a_gradient():
    """Refused where autograd records, as torch does for out=; taken where it does not."""
    a, b = linear.quantize(torch.ones(8, 128, device="cuda")), linear.quantize(torch.ones(16, 128, device="cuda"))
    leaf = torch.zeros(8, 16, device="cuda").requires_grad_()
    for out in (leaf, leaf * 2):
        before = out.detach().clone()
        with pytest.raises(ValueError, match="no_grad"):
            linear.matmul(a, b, out=out)
        assert torch.equal(out.detach(), before)
        with torch.no_grad():
            linear.matmul(a, b, out=out, accumulate=True)
        assert torch.equal(out.detach(), before + 128)
    with torch.inference_mode():                    # its tensors have no version
        out = torch.empty(8, 16, device="cuda")
        assert (linear.matmul(a, b, out=out) == 128).all()


@pytest.mark.parametrize("which", ["codes", "scales"])
def test_blocked_tensor_moved_in_place(which):
    """A product reads an operand's tensors where they are at the call, after .data or set_ too."""
    a, b = _operands(20, 30, 300, key=12)
    want = linear.matmul(a, b, dtype=torch.float32)
    t = getattr(a, which)
    old = t.detach()                                    # the former memory stays allocated
    fresh = torch.zeros_like(t.view(torch.uint8))       # zero codes, or scales of 2^-127
    t.data = fresh.view(t.dtype)
    now = linear.matmul(a, b, dtype=torch.float32)
    assert not torch.equal(now, want)
    _check_product(now, a, b, "f32")
    t.set_(old)
    assert torch.equal(linear.matmul(a, b, dtype=torch.float32), want)
    t.set_(old[:1].clone())                             # and checked there: too few rows
    with pytest.raises(ValueError):
        linear.matmul(a, b)


@pytest.mark.parametrize("m,n", [(3, 200), (40, 500), (40, 4096), (300, 520), (1300, 2100)])
def test_matmul_sums_that_cancel(m, n):
    """What is left when a row's large products cancel: whole in a float32 result and its cast, within the stated bound in a 16-bit one."""
    rng = _rng(m, n, 71)
    # large products of one sign in the first half of k and of the other in the second, small ones between them: whole
    # numbers whose partial sums stay below 2^24, so that fp32 sums them exactly in any order
    x, y = np.repeat(rng.integers(1, 4, (m, 1)), 256, 1).astype(np.float64), np.repeat(rng.integers(1, 4, (n, 1)), 256, 1).astype(np.float64)
    x[:, ::8], y[:, ::8] = 448, 448
    x[:, 128::8] = -448
    # and random products in cancelling pairs, on small ones of random signs
    u, v = rng.standard_normal((m, 1024)), rng.standard_normal((n, 1024))
    u[:, 1:896:2], v[:, 1:896:2] = -u[:, 0:896:2], v[:, 0:896:2]
    u[:, 896:] *= 2.0 ** -7
    for p, q, whole_numbers in ((x, y, True), (u, v, False)):
        a, b = linear.quantize(_t(p)), linear.quantize(_t(q))
        p, q = _held(a), _held(b)
        k, want, size = p.shape[1], p @ q.T, np.abs(p) @ np.abs(q).T
        assert np.linalg.norm(want) < 2.0 ** -6 * np.linalg.norm(size)
        whole, half = linear.matmul(a, b, dtype=torch.float32), linear.matmul(a, b)
        sums = 0.0 if whole_numbers else size * (k + 1) * ULP
        assert (np.abs(_n(whole) - want) <= sums).all()
        assert (np.abs(_n(whole.bfloat16()) - want) <= np.abs(want) * _half("bf16") + sums * (1 + _half("bf16"))).all()
        most = size * ((k + 1) * ULP + 2.0 ** -10)
        assert (np.abs(_n(half) - want) <= np.abs(want) * _half("bf16") + most * (1 + _half("bf16"))).all()


def test_matmul_value_past_fp32():
    """An input next to fp32's largest rounds to 2^128 in 8 bits: an infinity in a float32 result, a factor like any other in a 16-bit one."""
    for m in (3, 70, 300):
        x = torch.zeros(m, 256, device="cuda")
        x[1, 7] = 3.4e38
        for fmt in F8.values():
            a, b = linear.quantize(x, dtype=fmt), linear.quantize(torch.full((40, 256), 2.0 ** -30, device="cuda"))
            c = linear.matmul(a, b, dtype=torch.float32)
            assert c[1].isposinf().all() and (c[[0, *range(2, m)]] == 0).all()
            assert (linear.matmul(a, b)[1] == 2.0 ** 98).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(17, 41100, 260), (100, 41000, 130), (128, 41217, 129), (129, 41000, 130), (20500, 3, 300), (41000, 1, 130),
                                   (41100, 128, 257), (41000, 129, 130)])
def test_matmul_few_rows_through_many_columns(m, n, k, kind):
    """Vocabulary-wide products of a decode batch, and many tokens into few columns, on both sides of where the tile changes."""
    a, b = _operands(m, n, k, key=13)
    _check_product(linear.matmul(a, b, dtype=FLOATS[kind]), a, b, kind)


def test_side_stream_in_order():
    """Every operator, forward and backward, runs on the current stream: behind a side stream's own queued work, whose results it reads.
    Launched on another stream it would read the values from before."""
    rng = _rng(100)
    m, k, n = 300, 700, 260

    def inputs(key):
        g = _rng(key)
        return [_t(_values(g, m, k), "bf16"), _t(_values(g, m, k), "bf16"), _t(1 + 0.2 * g.standard_normal(k)), _t(0.05 * g.standard_normal((n, k))),
                _t(g.standard_normal((m, n)), "bf16")]

    def calls(x, r, w, W, dy):
        q, h, rstd = linear.rms_norm(x, w, residual=r)
        a, at = linear.quantize_both(W)
        out = linear.matmul(q, a)
        dq, dt = linear.quantize_both(dy)
        single = (q.codes.view(torch.uint8), h, rstd, out, linear.matmul(dt, linear.quantize(h, transpose=True, row_factor=rstd, col_factor=w), dtype=torch.float32),
                  *linear.rms_norm_backward(linear.matmul(dq, at), h, rstd, w, dh=h))
        leaves = [t.detach().requires_grad_() for t in (x, r, w, W)]
        y, s = linear.rms_norm_linear(leaves[0], leaves[2], leaves[3], residual=leaves[1])
        z = linear.scaled_linear(s, leaves[3])
        return (*single, y.detach(), z.detach(), *torch.autograd.grad((y, s, z), leaves, (dy, h, dy)))

    before, after = inputs(1), inputs(2)
    old, want = calls(*before), calls(*after)
    assert not any(torch.equal(a, b) for a, b in zip(old, want))        # the values from before would be told apart
    heavy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):                         # some milliseconds ahead of the inputs' new values
            heavy = torch.mm(heavy, heavy) * 1e-2
        for t, v in zip(before, after):
            t.copy_(v)
        got = calls(*before)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("m,k", [((1 << 20) + 101, 2048), (54000, 40000)])
def test_more_elements_than_32_bits_count(m, k):
    """More than 2^31 elements in each tensor: the last rows come as they do from a matrix of their own."""
    def stream(seed):
        return torch.randn(m, k, dtype=torch.bfloat16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    x, r = stream(1), stream(2)
    assert x.numel() > 1 << 31
    w = _t(1 + 0.2 * _rng(14).standard_normal(k))
    start = (m - 64) // 128 * 128                   # a block of the transposed form begins there
    tail = slice(start, m)

    def tails(q):
        return q.codes.view(torch.uint8)[tail], q.scales.view(torch.uint8)[:, tail]

    q, h, rstd = linear.rms_norm(x, w, residual=r)
    small = linear.rms_norm(x[tail], w, residual=r[tail])
    assert torch.equal(h[tail], small.h) and torch.equal(rstd[tail], small.rstd)
    assert all(torch.equal(a, b) for a, b in zip(tails(q), _bits(small.q)))
    # a product that reads the last rows of such a matrix
    b = linear.quantize(_t(_rng(15).standard_normal((20, k))))
    _check_product(linear.matmul(q, b)[tail], small.q, b, "bf16")
    del q
    # gradients, r as dy and x as what reaches h
    dx, dw = linear.rms_norm_backward(r, h, rstd, w, dh=x)
    part, _ = linear.rms_norm_backward(r[tail], h[tail], rstd[tail], w, dh=x[tail])
    assert torch.equal(dx[tail], part)
    want, size = torch.zeros(k, dtype=torch.float64, device="cuda"), torch.zeros(k, dtype=torch.float64, device="cuda")
    for i in range(0, m, 16384):
        p = r[i:i + 16384].double() * (h[i:i + 16384].double() * rstd[i:i + 16384].double()[:, None])
        want += p.sum(0)
        size += p.abs().sum(0)
    # a workgroup sums every 256th row at the most in fp32, the workgroups' sums are added in fp64
    assert ((dw.double() - want).abs() <= want.abs() * 2.0 ** -24 + size * (-(-m // 256) + 8) * ULP).all()
    del dx, r, rstd
    q, t = linear.quantize_both(h)
    one, other = linear.quantize_both(h[tail])
    assert all(torch.equal(a, b) for a, b in zip(tails(q), _bits(one)))
    assert torch.equal(t.codes.view(torch.uint8)[:, start:m], other.codes.view(torch.uint8)[:, :m - start])
    assert torch.equal(t.scales.view(torch.uint8)[start // 128:, :k], other.scales.view(torch.uint8)[:, :k])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_matmul_result_of_more_elements_than_32_bits_count(kind):
    """Whole numbers, which every order of summation adds exactly: the last rows as from operands of their own."""
    m, n, k = 65700, 32800, 128
    rng = _rng(16)
    x, y = _t(rng.integers(-4, 5, (m, k))), _t(rng.integers(-4, 5, (n, k)))
    a, b = linear.quantize(x), linear.quantize(y)
    c = linear.matmul(a, b, dtype=FLOATS[kind])
    assert c.numel() > 1 << 31
    assert torch.equal(c[-300:], linear.matmul(linear.quantize(x[-300:]), b, dtype=FLOATS[kind]))
    assert torch.equal(c[:300], (x[:300] @ y.T).to(FLOATS[kind]))
    assert torch.equal(c[-300:], (x[-300:] @ y.T).to(FLOATS[kind]))
    once = x[-300:] @ y.T
    assert torch.equal(linear.matmul(a, b, out=c, accumulate=True)[-300:], (once.to(c.dtype).float() + once).to(c.dtype))


def test_layer_pass_in_a_graph():
    """A layer's forward and backward captured once and replayed on new inputs, with eager passes over other leaves between the replays."""
    m, k, n = 300, 640, 520

    def inputs(i):
        g = _rng(i, 113)
        return [_t(_values(g, m, k), "bf16"), _t(_values(g, m, k), "bf16"), _t(1 + 0.1 * g.standard_normal(k)), _t(0.05 * g.standard_normal((n, k))), _t(g.standard_normal((m, n)), "bf16")]

    def layer(x, r, w, W, dy):
        y, h = linear.rms_norm_linear(x, w, W, residual=r)
        z = linear.scaled_linear(h, W)
        return (y.detach(), h.detach(), z.detach(), *torch.autograd.grad((y, z, h), (x, r, w, W), (dy, dy, x.detach())))

    held = inputs(0)
    leaves = [t.requires_grad_() for t in held[:4]] + held[4:]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*leaves)                              # its graph is gone before the capture begins
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = layer(*leaves)
    for i in range(4):
        new = inputs(i)
        with torch.no_grad():
            for t, v in zip(held, new):
                t.copy_(v)
        want = layer(*[t.requires_grad_() for t in new[:4]], new[4])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("m", [1, 5, 70, 400])
def test_forward_without_gradients(m):
    """Serving: the operators under no_grad and inference_mode, and the single calls on a weight quantised once, give a training forward's bits."""
    rng = _rng(m, 114)
    x, r, nw = _t(_values(rng, m, 300), "bf16"), _t(_values(rng, m, 300), "bf16"), _t(1 + 0.2 * rng.standard_normal(300)).requires_grad_()
    W = _t(0.05 * rng.standard_normal((500, 300))).requires_grad_()
    y, h = linear.rms_norm_linear(x, nw, W, residual=r)
    z = linear.scaled_linear(h, W)
    assert y.requires_grad and z.requires_grad
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            a, s = linear.rms_norm_linear(x, nw, W, residual=r)
            b = linear.scaled_linear(s, W)
            assert not a.requires_grad and not b.requires_grad
            kept = linear.quantize(W)
            q, t, _ = linear.rms_norm(x, nw, residual=r)
            for got, want in ((a, y), (s, h), (b, z), (t, h), (linear.matmul(q, kept), y), (linear.matmul(linear.quantize(t), kept), z)):
                assert torch.equal(got, want)
