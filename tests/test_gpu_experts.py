"""The experts' operators on the GPU against the oracle.

Orders and 8-bit forms are compared exactly; sums of k fp32 terms are off by at
most k 2^-23 of the sum of their sizes (one unit in the last place an addition), products
on the 8-bit instructions also by what those drop (as tests/test_gpu_linear.py
derives it), and a result's type rounds by half its eps."""
import numpy as np
import pytest

from oracle import experts_oracle as E
from oracle import linear_oracle as L

torch = pytest.importorskip("torch")
from kronecker_factored_second_amd import experts, linear, okls, optim  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ULP = 2.0 ** -23


def _rng(*key):
    return np.random.default_rng([k % (1 << 31) for k in key])


def _t(a, kind="f32"):
    return torch.tensor(np.asarray(a, np.float32)).to(FLOATS[kind]).cuda()


def _n(t):
    return t.detach().cpu().double().numpy()


def _half(kind):
    return torch.finfo(FLOATS[kind]).eps / 2


def _tiny(kind):
    """Half the smallest step of the type."""
    return {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}[kind]


def _padded(t, pad, offset=0):
    """The same matrix inside a wider one: row stride cols + pad, first element `offset` elements in."""
    rows, cols = t.shape
    base = torch.full((rows * (cols + pad) + offset,), 7.0, dtype=t.dtype, device=t.device)
    v = base[offset:].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def _choices(rng, tokens, each, n, dropped=0.1, skew=1.0):
    """Distinct experts of each token by skewed scores, some of them dropped."""
    scores = rng.standard_normal((tokens, n)) + skew * rng.standard_normal(n)
    c = np.argsort(-scores, axis=1)[:, :each]
    return np.where(rng.random(c.shape) < dropped, rng.choice([-1, n, n + 7, -(1 << 31)], c.shape), c)


def _case(key, tokens, each, n, align=128, dropped=0.1, skew=1.0, dtype=torch.int64):
    rng = _rng(key, tokens, each, n)
    choice = _choices(rng, tokens, each, n, dropped, skew)
    return rng, choice, E.plan(choice, n, align), experts.plan(torch.tensor(choice).to(dtype).cuda(), n, align=align)


def _check_plan(got, want):
    rows, pairs, offsets, counts = want
    assert np.array_equal(got.rows.cpu().numpy(), rows) and np.array_equal(got.pairs.cpu().numpy(), pairs)
    assert np.array_equal(got.offsets.cpu().numpy(), offsets) and np.array_equal(got.counts.cpu().numpy(), counts)


# ---------------------------------------------------------------------------
# The order
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("align", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens,each,n", [(1, 1, 1), (1, 1, 512), (1, 8, 8), (5, 2, 3), (63, 1, 64), (64, 1, 65), (65, 3, 7), (100, 2, 1 + 1), (2048, 2, 8), (2049, 2, 8), (4097, 1, 64), (1500, 8, 512)])
def test_plan(tokens, each, n, align):
    for dtype in (torch.int64, torch.int32):
        _, _, want, got = _case(1, tokens, each, n, align, dtype=dtype)
        _check_plan(got, want)


@pytest.mark.parametrize("tokens,each,n", [(30000, 3, 60), (131072, 2, 8), (100000, 3, 130), (270001, 1, 512)])
def test_plan_of_many(tokens, each, n):
    """Many workgroups, and from 64 x 4096 choices on several groups in each; sorted here by numpy."""
    rng = _rng(tokens)
    choice = rng.integers(-2, n + 1, (tokens, each))
    got = experts.plan(torch.tensor(choice).cuda(), n)
    flat = choice.reshape(-1)
    counts = np.bincount(flat[(flat >= 0) & (flat < n)], minlength=n)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // 128) * 128)])
    order = np.argsort(np.where((flat < 0) | (flat >= n), n, flat), kind="stable")[: counts.sum()]
    rows, pairs = np.full(flat.size, -1), np.full(got.capacity, -1)
    rows[order] = offsets[flat[order]] + np.arange(order.size) - np.repeat(np.cumsum(counts) - counts, counts)
    pairs[rows[order]] = order
    _check_plan(got, (rows.reshape(choice.shape), pairs, offsets, counts))


def test_plan_one_expert_takes_all_or_none():
    for fill, n in ((0, 5), (4, 5), (-1, 5), (511, 512)):
        choice = np.full((700, 2), fill)
        _check_plan(experts.plan(torch.tensor(choice).cuda(), n), E.plan(choice, n, 128))


def test_plan_of_nothing():
    p = experts.plan(torch.zeros(0, 2, dtype=torch.int64, device="cuda"), 5)
    assert p.capacity == 0 and p.offsets.tolist() == [0] * 6 and p.counts.tolist() == [0] * 5
    x = torch.zeros(0, 40, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.zeros(0, 2, device="cuda", requires_grad=True)
    W = torch.randn(5, 24, 40, device="cuda", requires_grad=True)
    y = experts.combine(experts.token_linear(x, W, p), w, p)
    assert y.shape == (0, 24)
    y.sum().backward()
    assert x.grad.shape == (0, 40) and w.grad.shape == (0, 2) and not W.grad.any()


def test_plan_of_a_strided_choice():
    choice = torch.randint(0, 6, (50, 4), device="cuda")
    a, b = experts.plan(choice[:, ::2], 6), experts.plan(choice[:, ::2].contiguous(), 6)
    assert torch.equal(a.rows, b.rows) and torch.equal(a.pairs, b.pairs)


# ---------------------------------------------------------------------------
# Rows there and back
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 1, 1), (1, 8, 8, 4096), (3, 2, 5, 7), (9, 2, 5, 8), (50, 3, 10, 511), (50, 4, 10, 512), (50, 5, 10, 513), (33, 1, 4, 1024), (33, 9, 20, 1025), (40, 2, 70, 4100), (7, 65, 80, 100), (3, 130, 140, 600), (1000, 2, 8, 40)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,each,n,cols", SHAPES)
def test_gather(tokens, each, n, cols, kind):
    rng, _, (_, pairs, _, _), p = _case(2, tokens, each, n, 16 if tokens % 2 else 128)
    x = _t(rng.standard_normal((tokens, cols)), kind)
    want = E.gather(_n(x), pairs, each)
    assert np.array_equal(_n(experts.gather(x, p)), want)
    if cols > 1:
        for pad, offset in ((1, 0), (8, 3)):
            assert np.array_equal(_n(experts.gather(_padded(x, pad, offset), p)), want)


def _check_combine(got, y, rows, weights, kind):
    want, size = E.combine(y, rows, weights)
    assert (np.abs(_n(got) - want) <= np.abs(want) * _half(kind) + size * (rows.shape[1] + 1) * ULP + _tiny(kind)).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,each,n,cols", SHAPES)
def test_combine(tokens, each, n, cols, kind):
    """With weights of each type and without; rows without a choice and weights without a row hold NaN, which reaches nothing."""
    rng, choice, (rows, pairs, _, _), p = _case(3, tokens, each, n, 16 if tokens % 2 else 128)
    y = _t(rng.standard_normal((p.capacity, cols)), kind)
    y[torch.tensor(pairs < 0).cuda()] = float("nan")
    held = np.where(pairs[:, None] < 0, 0.0, _n(y))
    for wkind in ("f32", "bf16", "f16"):
        w = _t(rng.random((tokens, each)), wkind)
        w[torch.tensor(rows < 0).cuda()] = float("nan")
        out = experts.combine(y, w, p)
        _check_combine(out, held, rows, np.where(rows < 0, 0.0, _n(w)), kind)
        assert torch.equal(out, experts.combine(_padded(y, 8, 1), w, p))
    _check_combine(experts.combine(y, None, p), held, rows, None, kind)


@pytest.mark.parametrize("kind,wkind", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,each,n,cols", SHAPES)
def test_gradients(tokens, each, n, cols, kind, wkind):
    rng, choice, (rows, pairs, _, _), p = _case(4, tokens, each, n)
    x = _t(rng.standard_normal((tokens, cols)), kind).requires_grad_()
    y = _t(E.gather(rng.standard_normal((tokens * each, cols)), pairs, 1), kind)
    y[torch.tensor(pairs < 0).cuda()] = float("nan")
    y.requires_grad_()
    w = _t(rng.random((tokens, each)), wkind).requires_grad_()
    dxs, dout = _t(rng.standard_normal((p.capacity, cols)), kind), _t(rng.standard_normal((tokens, cols)), kind)
    dx, dy, dw = torch.autograd.grad((experts.gather(x, p), experts.combine(y, w, p)), (x, y, w), (dxs, dout))
    _check_combine(dx, _n(dxs), rows, None, kind)
    held = np.where(pairs[:, None] < 0, 0.0, _n(y))
    want_y, want_w, size = E.combine_backward(_n(dout), held, rows, pairs, _n(w))
    assert dy.dtype == y.dtype and dw.dtype == w.dtype
    # one product in fp32, rounded once to the type
    assert (np.abs(_n(dy) - want_y) <= np.abs(want_y) * (_half(kind) + 2.0 ** -24) + _tiny(kind)).all()
    assert (np.abs(_n(dw) - want_w) <= np.abs(want_w) * _half(wkind) + size * (cols + 1) * ULP + _tiny(wkind)).all()
    again = torch.autograd.grad((experts.gather(x, p), experts.combine(y, w, p)), (x, y, w), (_padded(dxs, 8, 1), _padded(dout, 8, 1)))
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dy, dw)))


def test_gradients_as_autograd_hands_them_over():
    """Expanded and transposed gradients, and leaves that want none."""
    rng, _, (rows, pairs, _, _), p = _case(5, 30, 2, 4)
    x, y, w = _t(rng.standard_normal((30, 24))), _t(rng.standard_normal((p.capacity, 24))), _t(rng.random((30, 2)))
    a = x.clone().requires_grad_()
    experts.gather(a, p).sum().backward()
    assert np.array_equal(_n(a.grad), np.repeat((rows >= 0).sum(1)[:, None], 24, 1).astype(float))
    d = _t(rng.standard_normal((24, 30)))
    for ny, nw in ((True, False), (False, True)):
        b, c = y.clone().requires_grad_(ny), w.clone().requires_grad_(nw)
        experts.combine(b, c, p).backward(d.T)
        e, f = y.clone().requires_grad_(), w.clone().requires_grad_()
        experts.combine(e, f, p).backward(d.T.contiguous())
        assert (b.grad is None) != ny and (c.grad is None) != nw
        assert torch.equal(b.grad, e.grad) if ny else torch.equal(c.grad, f.grad)
    b = y.clone().requires_grad_()
    experts.combine(b, None, p).backward(d.T)
    assert torch.equal(b.grad, experts.gather(d.T.contiguous(), p))
    with pytest.raises(RuntimeError):       # no second derivative
        a = x.clone().requires_grad_()
        g, = torch.autograd.grad(experts.gather(a, p).square().sum(), a, create_graph=True)
        g.sum().backward()


# ---------------------------------------------------------------------------
# 8-bit forms
# ---------------------------------------------------------------------------
def _check_blocked(q, v, fmt, rows=None):
    codes, scales = L.quantize(v, fmt)
    rows = slice(0, v.shape[0]) if rows is None else rows
    assert np.array_equal(_n(q.scales)[:, rows], scales) and np.array_equal(_n(q.codes)[rows, : v.shape[1]], codes)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,each,n,cols", [(1, 1, 1, 1), (40, 2, 5, 300), (200, 3, 7, 129)])
def test_quantize_rows(tokens, each, n, cols, kind, fmt):
    """Both ways and forms; what rows without a choice hold (NaN here) reaches no code and no scale."""
    rng, _, (_, pairs, _, _), p = _case(6, tokens, each, n)
    x = _t(rng.standard_normal((tokens, cols)), kind)
    want = E.gather(_n(x), pairs, each)
    xs = experts.gather(x, p)
    xs[torch.tensor(pairs < 0).cuda()] = float("nan")
    for src, gathered in ((x, True), (xs, False), (_padded(x, 3, 1), True), (_padded(xs, 3, 1), False)):
        q, t = experts.quantize_rows_both(src, p, dtype=F8[fmt], gathered=gathered)
        _check_blocked(q, want, fmt)
        _check_blocked(t, want.T, fmt)
    one = experts.quantize_rows(x, p, dtype=F8[fmt], gathered=True)
    two = experts.quantize_rows(x, p, dtype=F8[fmt], gathered=True, transpose=True)
    assert torch.equal(one.codes.view(torch.uint8), q.codes.view(torch.uint8)) and torch.equal(two.codes.view(torch.uint8), t.codes.view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("e,n,k", [(1, 1, 1), (3, 17, 130), (5, 128, 256), (70, 33, 40), (512, 3, 20)])
def test_quantize_stack(e, n, k, kind):
    W = _t(_rng(e, n, k).standard_normal((e, n, k)), kind)
    wide = torch.full((e, n + 2, k + 5), 9.0, dtype=W.dtype, device="cuda")
    wide[:, :n, :k] = W
    for src in (W, wide[:, :n, :k], W.transpose(1, 2).contiguous().transpose(1, 2)):
        q, t = experts.quantize_stack_both(src)
        for i in range(0, e, max(1, e // 5)):
            _check_blocked(q.blocked, _n(W[i]), "e4m3", slice(i * -(-n // 16) * 16, i * -(-n // 16) * 16 + n))
            _check_blocked(t.blocked, _n(W[i]).T, "e4m3", slice(i * -(-k // 16) * 16, i * -(-k // 16) * 16 + k))
    assert q.shape == (e, n, k) and t.shape == (e, k, n)
    assert torch.equal(experts.quantize_stack(W, transpose=True).dequantize(), t.dequantize())
    assert torch.equal(experts.quantize_stack(W).dequantize(), q.dequantize())


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------
def _held(q, rows=None):
    r, c = q.shape
    return L.dequantize(_n(q.codes)[:, :c], _n(q.scales)[:, :r])


def _check_sums(got, want, size, terms, kind):
    """As _check_product of the plain product's tests derives it."""
    most = size * (terms + 1) * ULP + (0.0 if kind == "f32" else size * 2.0 ** -10)
    got = _n(got)
    if kind == "f16":
        over = np.isinf(got)
        assert (np.abs(want) + most >= 65520)[over].all() and (np.sign(got) == np.sign(want))[over].all()
        got = np.where(over, want, got)
    off = np.abs(got - want)
    assert (off <= np.abs(want) * _half(kind) + most + _tiny(kind)).all()
    if kind != "f32" and want.size >= 1000:
        assert np.linalg.norm(off) <= (_half(kind) + 2.0 ** -11.5) * np.linalg.norm(want)


def _product(key, tokens, each, e, n, k, kind, align=128, fa="e4m3", fb="e4m3", dropped=0.1, skew=1.0):
    rng, choice, (_, pairs, _, _), p = _case(key, tokens, each, e, align, dropped, skew)
    a = experts.quantize_rows(_t(rng.standard_normal((tokens, k)) * np.exp(rng.standard_normal((tokens, 1)))), p, dtype=F8[fa], gathered=True)
    W = _t(0.1 * rng.standard_normal((e, n, k)))
    b = experts.quantize_stack(W, dtype=F8[fb])
    c = experts.matmul(a, b, p, dtype=FLOATS[kind])
    want, size = E.matmul(_held(a), _n(b.dequantize()), pairs, choice)
    _check_sums(c, want, size, k, kind)
    assert not c[torch.tensor(pairs < 0).cuda()].any()
    assert torch.equal(c, experts.matmul(a, b, p, dtype=FLOATS[kind]))      # equal bits every time


# few rows an expert (a stream), up to 64 (narrow tiles), up to 128 and few tiles (small ones), many (large ones)
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,each,e,n,k", [
    (1, 1, 1, 1, 1), (1, 2, 8, 300, 1000), (8, 2, 8, 513, 129), (20, 2, 5, 64, 4000), (17, 1, 3, 65, 128), (60, 2, 70, 200, 300), (9, 8, 512, 40, 200),
    (150, 2, 7, 300, 500), (50, 3, 4, 129, 260), (500, 8, 70, 100, 300),
    (400, 1, 4, 300, 640), (300, 2, 6, 129, 200), (600, 8, 70, 200, 130), (1, 1, 1, 500, 100),
    (1000, 2, 8, 4000, 200), (1400, 8, 70, 900, 129), (2000, 1, 2, 5000, 128)])
def test_matmul(tokens, each, e, n, k, kind):
    _product(7, tokens, each, e, n, k, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,each,e,n,align", [(1700, 1, 5, 8000, 128), (1700, 1, 5, 6100, 16), (2000, 1, 4, 8192, 128), (2300, 1, 6, 7000, 128)])
def test_matmul_long_sums(tokens, each, e, n, align, kind):
    """From 4096 of the summed axis on, what whole rounds of large tiles leave goes to small ones: rests of less and of more than half a round."""
    _product(22, tokens, each, e, n, 4096 + 130, kind, align=align, dropped=0.02)


@pytest.mark.parametrize("align", [16, 32, 64])
@pytest.mark.parametrize("tokens,each,e,n,k", [(8, 2, 8, 300, 700), (150, 2, 7, 300, 500), (400, 2, 6, 300, 256), (1400, 4, 20, 2500, 130)])
def test_matmul_close_rows(tokens, each, e, n, k, align):
    """Experts that begin at multiples of 16: tiles that end inside the next one's rows."""
    for kind in ("bf16", "f32"):
        _product(8, tokens, each, e, n, k, kind, align=align)


@pytest.mark.parametrize("fa,fb", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("tokens,each,e,n,k", [(8, 2, 8, 200, 500), (150, 2, 7, 300, 300), (400, 2, 6, 300, 256), (1000, 2, 8, 4000, 130)])
def test_matmul_formats(fa, fb, tokens, each, e, n, k):
    _product(9, tokens, each, e, n, k, "f32", fa=fa, fb=fb)
    _product(9, tokens, each, e, n, k, "bf16", fa=fa, fb=fb)


@pytest.mark.parametrize("tokens,each,e,n,k", [(30, 1, 8, 300, 700), (300, 1, 8, 200, 300), (1500, 1, 12, 3300, 130)])
def test_matmul_uneven(tokens, each, e, n, k):
    """Nearly all tokens to one expert, several without any; and every choice dropped."""
    _product(10, tokens, each, e, n, k, "bf16", skew=6.0)
    _product(10, tokens, each, e, n, k, "f32", dropped=1.0)
    _product(10, tokens, each, e, n, k, "bf16", align=16, skew=6.0, dropped=0.0)


def test_matmul_nan_stays_with_its_token_or_expert():
    rng, choice, (rows, pairs, _, _), p = _case(11, 60, 2, 5)
    x, W = _t(rng.standard_normal((60, 300)), "bf16"), _t(rng.standard_normal((5, 200, 300)))
    x[7, 3] = float("nan")
    W[2, 5, 7] = float("inf")
    c = experts.matmul(experts.quantize_rows(x, p, gathered=True), experts.quantize_stack(W), p)
    of = E.expert_of(pairs, choice)
    token = np.where(pairs >= 0, pairs // 2, -1)
    bad = np.zeros(tuple(c.shape), bool)
    bad[token == 7] = True
    bad[of == 2, 5] = True
    got = np.isnan(_n(c))
    assert np.array_equal(got[pairs >= 0], bad[pairs >= 0])
    assert (_n(c)[:, 6:][(pairs < 0)] == 0).all()


def test_matmul_nothing_to_sum():
    _, _, (_, pairs, _, _), p = _case(12, 30, 2, 4)
    a = experts.quantize_rows(torch.zeros(30, 0, device="cuda"), p, gathered=True)
    b = experts.quantize_stack(torch.zeros(4, 20, 0, device="cuda"))
    assert torch.equal(experts.matmul(a, b, p), torch.zeros(p.capacity, 20, dtype=torch.bfloat16, device="cuda"))
    c = experts.quantize_stack(torch.zeros(4, 0, 50, device="cuda"))
    assert experts.matmul(experts.quantize_rows(torch.zeros(30, 50, device="cuda"), p, gathered=True), c, p).shape == (p.capacity, 0)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,each,e,n,k", [(1, 1, 1, 1, 1), (1, 1, 3, 5, 7), (60, 2, 5, 70, 200), (500, 2, 6, 129, 130), (300, 3, 70, 300, 260), (900, 1, 20, 700, 900), (50, 8, 512, 20, 30)])
def test_weight_grad(tokens, each, e, n, k, kind):
    """Small and large tiles, more experts than a wave has lanes, experts without tokens (zeros)."""
    for fa in ("e4m3", "e5m2"):
        rng, choice, (_, pairs, _, counts), p = _case(13, tokens, each, e)
        dy, x = _t(rng.standard_normal((tokens * each, n))), _t(rng.standard_normal((tokens, k)))
        dys = torch.zeros(p.capacity, n, device="cuda")
        dys[p.pairs >= 0] = dy[p.pairs[p.pairs >= 0].long()]
        a = experts.quantize_rows(dys, p, dtype=F8[fa], transpose=True)
        b = experts.quantize_rows(x, p, gathered=True, transpose=True)
        c = experts.weight_grad(a, b, p, dtype=FLOATS[kind])
        want, size = E.weight_grad(_held(a), _held(b), pairs, choice, e)
        _check_sums(c, want, size, int(counts.max()) if counts.size else 0, kind)
        assert c.shape == (e, n, k) and not c[torch.tensor(counts == 0).cuda()].any()
        assert torch.equal(c, experts.weight_grad(a, b, p, dtype=FLOATS[kind]))


def test_weight_grad_one_expert_has_all():
    rng, choice, (_, pairs, _, _), p = _case(14, 700, 1, 9, skew=50.0, dropped=0.0)
    a = experts.quantize_rows(_t(rng.standard_normal((700, 300))), p, gathered=True, transpose=True)
    b = experts.quantize_rows(_t(rng.standard_normal((700, 520))), p, gathered=True, transpose=True)
    want, size = E.weight_grad(_held(a), _held(b), pairs, choice, 9)
    _check_sums(experts.weight_grad(a, b, p), want, size, 700, "f32")


# ---------------------------------------------------------------------------
# Layers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,each,e,k,n,grad", [(1, 1, 2, 128, 64, "e4m3"), (40, 2, 5, 200, 300, "e5m2"), (300, 2, 6, 129, 130, "e4m3"), (500, 4, 70, 64, 96, "e5m2")])
def test_layer(tokens, each, e, k, n, grad):
    """token_linear and linear with their gradients: each against the single operators on what the step before it gave, and those are checked above."""
    rng, choice, (_, pairs, _, _), p = _case(15, tokens, each, e)
    x, W = _t(rng.standard_normal((tokens, k)), "bf16").requires_grad_(), _t(0.1 * rng.standard_normal((e, n, k))).requires_grad_()
    dy = _t(rng.standard_normal((p.capacity, n)), "bf16")
    dy[p.pairs < 0] = float("nan")       # no gradient of a row without a choice counts
    y = experts.token_linear(x, W, p, grad_dtype=F8[grad])
    dx, dW = torch.autograd.grad(y, (x, W), dy)
    (q, t), (w, wt) = experts.quantize_rows_both(x.detach(), p, gathered=True), experts.quantize_stack_both(W.detach())
    dq, dt = experts.quantize_rows_both(dy, p, dtype=F8[grad])
    assert torch.equal(y, experts.matmul(q, w, p))
    assert torch.equal(dW, experts.weight_grad(dt, t, p)) and dW.dtype == torch.float32
    dxs = experts.matmul(dq, wt, p)
    assert torch.equal(dx, experts.combine(dxs, None, p))
    xs = experts.gather(x.detach(), p).requires_grad_()
    z = experts.linear(xs, W, p, grad_dtype=F8[grad])
    assert torch.equal(y, z)
    both = torch.autograd.grad(z, (xs, W), dy)
    assert torch.equal(both[0], dxs) and torch.equal(both[1], dW)
    for nx, nw in ((True, False), (False, True)):
        a, b = x.detach().clone().requires_grad_(nx), W.detach().clone().requires_grad_(nw)
        experts.token_linear(a, b, p, grad_dtype=F8[grad]).backward(dy)
        assert torch.equal(a.grad, dx) if nx else a.grad is None
        assert torch.equal(b.grad, dW) if nw else b.grad is None


def test_layer_gradient_near_the_unrounded_layers():
    """A gated layer of experts, there and back, in fp64 without 8 bits: the roundings are off by 2^-4 of each value at most, independent over a sum, two layers deep."""
    rng, choice, (rows, pairs, _, _), p = _case(16, 256, 2, 4, dropped=0.05)
    x, wts = _t(rng.standard_normal((256, 192))), _t(rng.random((256, 2)))
    up, down = _t(0.1 * rng.standard_normal((4, 128, 192))), _t(0.1 * rng.standard_normal((4, 192, 128)))
    dout = _t(rng.standard_normal((256, 192)))
    leaves = [t.requires_grad_() for t in (x, up, down, wts)]
    h = torch.tanh(experts.token_linear(x, up, p))
    out = experts.combine(experts.linear(h, down, p), wts, p)
    got = torch.autograd.grad(out, leaves, dout)
    X, U, D, V = (t.detach().cpu().double().requires_grad_() for t in leaves)
    ref = 0
    for k in range(2):
        ok = torch.tensor(rows[:, k] >= 0)
        c = torch.tensor(np.where(rows[:, k] >= 0, choice[:, k], 0))
        y = torch.tanh((U[c] @ X[:, :, None])[..., 0])
        ref = ref + ((D[c] @ y[:, :, None])[..., 0] * V[:, k: k + 1]).masked_fill(~ok[:, None], 0)
    want = torch.autograd.grad(ref, (X, U, D, V), dout.cpu().double())
    for a, b in zip((out, *got), (ref, *want)):
        assert (a.detach().cpu().double() - b.detach()).norm() < 2.0 ** -3 * b.norm()


def test_forward_without_gradients():
    """Serving: one token at a time through weights brought to 8 bits once gives a training forward's rows."""
    rng, choice, _, p = _case(17, 12, 2, 6, dropped=0.0)
    x, W, w = _t(rng.standard_normal((12, 300)), "bf16"), _t(0.1 * rng.standard_normal((6, 200, 300))).requires_grad_(), _t(rng.random((12, 2)))
    y = experts.combine(experts.token_linear(x, W, p), w, p)
    kept = experts.quantize_stack(W.detach())
    with torch.inference_mode():
        assert torch.equal(y, experts.combine(experts.token_linear(x, W, p), w, p))
        for t in range(12):
            one = experts.plan(torch.tensor(choice[t: t + 1]).cuda(), 6, align=16)
            ys = experts.matmul(experts.quantize_rows(x[t: t + 1], one, gathered=True), kept, one)
            assert torch.equal(experts.combine(ys, w[t: t + 1], one), y[t: t + 1])


@pytest.mark.parametrize("gathered", [False, True])
def test_no_grad_forward_is_the_training_forward(gathered):
    """Under no_grad nothing is kept for a gradient, and a plan of close rows will do for weights that ask for one elsewhere."""
    _, choice, _, p = _case(26, 40, 2, 6)
    rng, close = _rng(27, 40, 6), experts.plan(torch.tensor(choice).cuda(), 6, align=32)
    x, W = _t(rng.standard_normal((40, 300)), "bf16"), _t(0.1 * rng.standard_normal((6, 200, 300))).requires_grad_()
    run = lambda order: (experts.token_linear(x, W, order) if gathered else experts.linear(experts.gather(x, order), W, order))  # noqa: E731
    y = run(p)
    with torch.no_grad():
        same, near = run(p), run(close)
        assert torch.equal(experts.combine(near, None, close), experts.combine(y, None, p))
    assert y.requires_grad and not same.requires_grad and torch.equal(same, y)


def test_refusals():
    _, _, _, p = _case(18, 30, 2, 4)
    _, _, _, close = _case(18, 30, 2, 4, align=16)
    x, xs, W = torch.zeros(30, 40, device="cuda"), torch.zeros(p.capacity, 40, device="cuda"), torch.zeros(4, 24, 40, device="cuda")
    q, s, w = experts.quantize_rows(x, p, gathered=True), experts.quantize_stack(W), torch.zeros(30, 2, device="cuda")
    t = experts.quantize_rows(x, p, gathered=True, transpose=True)
    for bad in (lambda: experts.gather(xs, p), lambda: experts.gather(x[0], p), lambda: experts.gather(x.double(), p), lambda: experts.gather(x.cpu(), p),
                lambda: experts.gather(x.T.contiguous().T, p), lambda: experts.combine(x, w, p), lambda: experts.combine(xs, w[:, :1], p),
                lambda: experts.combine(xs, w.long(), p), lambda: experts.combine(xs, w.cpu(), p), lambda: experts.quantize_rows(xs, p, gathered=True),
                lambda: experts.quantize_rows(x, p), lambda: experts.quantize_rows(x, p, gathered=True, dtype=torch.float16), lambda: experts.quantize_stack(W[0]),
                lambda: experts.quantize_stack(W.double()), lambda: experts.matmul(q, s, close), lambda: experts.matmul(t, s, p), lambda: experts.matmul(q, s, p, dtype=torch.float64),
                lambda: experts.matmul(q, experts.quantize_stack(W[:3]), p), lambda: experts.weight_grad(q, t, p), lambda: experts.weight_grad(t, t, close),
                lambda: experts.weight_grad(t, t, p, dtype=torch.int32), lambda: experts.linear(xs, W[:3], p), lambda: experts.linear(xs, W[:, :, :39], p),
                lambda: experts.linear(x, W, p), lambda: experts.token_linear(xs, W, p), lambda: experts.token_linear(x, W.clone().requires_grad_(), close),
                lambda: experts.Plan(p.rows, p.pairs[1:], p.offsets, p.counts), lambda: experts.Plan(p.rows, p.pairs, p.offsets[1:], p.counts),
                lambda: experts.Plan(p.rows.long(), p.pairs, p.offsets, p.counts), lambda: experts.Plan(p.rows, p.pairs.cpu(), p.offsets, p.counts),
                lambda: experts.Plan(p.rows, p.pairs, p.offsets, p.counts, align=16)):
        with pytest.raises(ValueError):
            bad()
    same = experts.Plan(p.rows.clone(), p.pairs.clone(), p.offsets.clone(), p.counts.clone())
    assert torch.equal(experts.gather(x + 1, same), experts.gather(x + 1, p))
    # without the weights' gradient a plan of close rows will do
    assert experts.token_linear(x.clone().requires_grad_(), W, close).shape == (close.capacity, 24)


def test_other_stream():
    rng, _, _, p = _case(19, 300, 2, 6)
    x, W, w = _t(rng.standard_normal((300, 256)), "bf16"), _t(rng.standard_normal((6, 200, 256))), _t(rng.random((300, 2)))
    choice = torch.where(p.rows >= 0, torch.searchsorted(p.offsets[1:], p.rows, right=True), -1)
    want = experts.combine(experts.token_linear(x, W, p), w, p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        order = experts.plan(choice, 6)
        got = experts.combine(experts.token_linear(x, W, order), w, order)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


@pytest.mark.parametrize("tokens", [6, 3000])
def test_layer_in_a_graph(tokens):
    """Sorting, the layer forward and backward captured once and replayed on new inputs and choices, with eager passes over other leaves between: the host learns nothing of the choices."""
    e, k, n = 6, 130, 200

    def inputs(i):
        rng = _rng(i, tokens, 20)
        return [_t(rng.standard_normal((tokens, k)), "bf16"), _t(0.1 * rng.standard_normal((e, n, k))), _t(rng.random((tokens, 2))),
                torch.tensor(_choices(rng, tokens, 2, e, skew=float(i))).cuda(), _t(rng.standard_normal((tokens, n)), "bf16")]

    def layer(x, W, w, choice, dout):
        p = experts.plan(choice, e)
        y = experts.combine(experts.token_linear(x, W, p), w, p)
        return (y.detach(), p.rows, p.pairs, *torch.autograd.grad(y, (x, W, w), dout))

    held = inputs(0)
    leaves = [t.requires_grad_() for t in held[:3]] + held[3:]
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
        new = inputs(i + 1)
        with torch.no_grad():
            for t, v in zip(held, new):
                t.copy_(v)
        want = layer(*[t.requires_grad_() for t in new[:3]], *new[3:])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i


def test_a_plan_whose_entries_are_out_of_range():
    """Entries of a plan of one's own that point nowhere count as none: nothing outside the tensors is read or written."""
    _, _, _, p = _case(21, 40, 2, 4)
    wild = torch.tensor([-5, 1 << 30, -(1 << 31), (1 << 31) - 1], dtype=torch.int32, device="cuda")
    rows, pairs = p.rows.clone(), p.pairs.clone()
    rows.view(-1)[:4] = wild
    pairs[:4] = wild
    odd = experts.Plan(rows, pairs, p.offsets, p.counts)
    x, w = torch.randn(40, 72, device="cuda"), torch.rand(40, 2, device="cuda")
    ys = torch.randn(p.capacity, 72, device="cuda")
    none = experts.Plan(torch.where((rows < 0) | (rows >= p.capacity), -1, rows), torch.where((pairs < 0) | (pairs >= 80), -1, pairs), p.offsets, p.counts)
    assert torch.equal(experts.combine(ys, w, odd), experts.combine(ys, w, none))
    a, b = experts.quantize_rows(x, odd, gathered=True), experts.quantize_rows(x, none, gathered=True)
    assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
    W = experts.quantize_stack(torch.randn(4, 64, 72, device="cuda"))
    for offsets in (torch.full_like(p.offsets, 1 << 30), torch.full_like(p.offsets, -7), torch.flip(p.offsets, (0,))):
        bent = experts.Plan(p.rows, p.pairs, offsets.contiguous(), p.counts)
        assert experts.matmul(b, W, bent).shape == (p.capacity, 64)
        experts.weight_grad(experts.quantize_rows(x, p, gathered=True, transpose=True), experts.quantize_rows(x, p, gathered=True, transpose=True), bent)
        experts.gather(x, bent)
    torch.cuda.synchronize()


@pytest.mark.timeout(600)
def test_more_elements_than_32_bits_count():
    """Sorted rows of more than 2^31 elements: the last rows come and go like the first."""
    tokens, each, cols = 140000, 4, 4096
    choice = torch.arange(tokens * each, device="cuda").view(tokens, each) % 3
    p = experts.plan(choice, 3)
    assert p.capacity * cols > 1 << 31
    x = torch.randn(tokens, cols, device="cuda").bfloat16()
    xs = experts.gather(x, p)
    for r in (0, 1, p.capacity // 2, int(p.rows.max())):
        i = int(p.pairs[r])
        assert torch.equal(xs[r], x[i // each] if i >= 0 else torch.zeros_like(x[0]))
    w = torch.full((tokens, each), 0.25, device="cuda")
    assert torch.equal(experts.combine(xs, w, p), x)            # exact: a quarter of the same four
    W = torch.randn(3, 64, cols, device="cuda")
    q, s = experts.quantize_rows(xs, p), experts.quantize_stack(W)
    y = experts.matmul(q, s, p)
    last = int(p.offsets[3]) - 128
    held = _held(linear.quantize(xs[last: last + 128])), _held(linear.quantize(W[2]))
    _check_sums(y[last: last + 128], held[0] @ held[1].T, np.abs(held[0]) @ np.abs(held[1]).T, cols, "bf16")


def test_training_steps_together():
    """A run as it is used: router, experts' layers, the stacks' 3-D gradients into the matrix step, the rest into AdamW, clipped by one norm."""
    torch.manual_seed(3)
    e, d, f, tokens = 4, 64, 96, 200
    router = (torch.randn(e, d, device="cuda") / 8).requires_grad_()
    norm = torch.ones(d, device="cuda", requires_grad=True)
    gate_up, down = ((torch.randn(*s, device="cuda") / 8).requires_grad_() for s in ((e, 2 * f, d), (e, d, f)))
    matrices, rest = okls.OKLS([gate_up, down], mode="muon"), optim.AdamW([router, norm], moments="8bit")
    start = [t.detach().clone() for t in (gate_up, down, router, norm)]
    for _ in range(3):
        x = torch.randn(tokens, d, device="cuda")
        h = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * norm
        best, choice = (h @ router.T).topk(2)
        order = experts.plan(choice, e)
        gate, up = experts.token_linear(h.bfloat16(), gate_up, order).chunk(2, dim=1)
        y = experts.linear(torch.nn.functional.silu(gate) * up, down, order)
        out = experts.combine(y, best.softmax(1), order)
        (out.float() - x).square().mean().backward()
        assert gate_up.grad.shape == gate_up.shape and gate_up.grad.dtype == torch.float32
        total = optim.grad_norm([t.grad for t in (gate_up, down, router, norm)])
        with torch.no_grad():
            matrices.step()
        rest.step(norm=total, max_norm=1.0)
        matrices.zero_grad()
        rest.zero_grad()
        assert all(t.isfinite().all() for t in (total, gate_up, down, router, norm))
    assert all(not torch.equal(t.detach(), s) for t, s in zip((gate_up, down, router, norm), start))


def test_example_runs():
    """The example's steps run, and its stack's gradients are the formula's: against the same blocks in fp32 without 8 bits, whose roundings are off by 2^-4 of each value at most."""
    from examples import train_experts
    losses = train_experts.train(steps=3, blocks=1, n_experts=4, d=64, f=64, tokens=200)
    assert len(losses) == 3 and all(np.isfinite(losses))
    gen = torch.Generator(device="cuda").manual_seed(4)
    (norm, router, gate_up, down), = train_experts.make(1, 4, 64, 64, gen, "cuda")
    leaves = [t.requires_grad_() for t in (gate_up, down)]
    x, dout = torch.randn(200, 64, generator=gen, device="cuda"), torch.randn(200, 64, generator=gen, device="cuda")
    got = torch.autograd.grad(train_experts.forward([(norm, router, gate_up, down)], x, 2), leaves, dout)
    U, D = (t.detach().double().cpu().requires_grad_() for t in leaves)
    h = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * norm
    best, choice = (h @ router.T).topk(2)
    H, V, C = h.double().cpu(), best.softmax(1).double().cpu(), choice.cpu()
    ref = x.double().cpu()
    for k in range(2):
        gate, up = (U[C[:, k]] @ H[:, :, None])[..., 0].chunk(2, dim=1)
        ref = ref + (D[C[:, k]] @ (torch.nn.functional.silu(gate) * up)[:, :, None])[..., 0] * V[:, k: k + 1]
    want = torch.autograd.grad(ref, (U, D), dout.double().cpu())
    for a, b in zip(got, want):
        # products of two rounded factors, two layers deep, and the output's gradient in two bits of fraction
        assert (a.double().cpu() - b).norm() < 2.0 ** -2 * b.norm()


def test_forward_mode_is_refused():
    """With a tangent nothing comes back; without one, the same calls under a dual level do."""
    rng, _, _, p = _case(28, 30, 2, 4)
    x, W, w = _t(rng.standard_normal((30, 40))), _t(rng.standard_normal((4, 24, 40))), _t(rng.random((30, 2)))
    want = experts.combine(experts.token_linear(x, W, p), w, p)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual
        for bad in (lambda: experts.gather(dual(x, x), p), lambda: experts.token_linear(x, dual(W, W), p), lambda: experts.combine(experts.token_linear(x, W, p), dual(w, w), p)):
            with pytest.raises(NotImplementedError):
                bad()
        assert torch.equal(experts.combine(experts.token_linear(x, W, p), w, p), want)


def test_a_plan_written_to_between_the_passes():
    """The backward pass of a plan over buffers that were filled again raises; a pass of its own on them gives their gradients."""
    _, _, _, a = _case(29, 60, 2, 5)
    _, _, _, b = _case(30, 60, 2, 5)
    held = experts.Plan(*[getattr(a, n).clone() for n in ("rows", "pairs", "offsets", "counts")])
    x, dxs = torch.randn(60, 72, device="cuda").requires_grad_(), torch.randn(a.capacity, 72, device="cuda")
    want = [torch.autograd.grad(experts.gather(x, p), x, dxs)[0] for p in (a, b)]
    assert torch.equal(torch.autograd.grad(experts.gather(x, held), x, dxs)[0], want[0])
    y = experts.gather(x, held)
    for n in ("rows", "pairs", "offsets", "counts"):
        getattr(held, n).copy_(getattr(b, n))
    with pytest.raises(RuntimeError, match="modified in place"):
        torch.autograd.grad(y, x, dxs)
    assert torch.equal(torch.autograd.grad(experts.gather(x, held), x, dxs)[0], want[1])


@pytest.mark.parametrize("tokens,each,e,n", [(9, 2, 5, 70), (150, 2, 7, 300), (1000, 2, 8, 4000)])
def test_rows_without_a_choice_multiply_as_they_are(tokens, each, e, n):
    """An operand of one's own may hold anything in an expert's rows without a choice; behind the last expert's rows there are zeros whatever it holds."""
    rng, choice, (_, pairs, offsets, _), p = _case(31, tokens, each, e)
    a = linear.quantize(_t(rng.standard_normal((p.capacity, 200))))
    b = experts.quantize_stack(_t(0.1 * rng.standard_normal((e, n, 200))))
    c = experts.matmul(a, b, p, dtype=torch.float32)
    A, B = _held(a), _n(b.dequantize())
    for i in range(e):
        rows = slice(int(offsets[i]), int(offsets[i + 1]))
        _check_sums(c[rows], A[rows] @ B[i].T, np.abs(A[rows]) @ np.abs(B[i]).T, 200, "f32")
    assert not c[int(offsets[-1]):].any()
