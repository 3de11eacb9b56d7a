"""The many-tensor optimizer step on the GPU against the oracle.

The definition rounds every product and sum of the moments by itself, so moments,
in 32 and in 8 bits, are compared exactly; the parameter takes ten more roundings
of 2^-24 of its parts' sizes."""
import numpy as np
import pytest

from oracle import optim_oracle as A

torch = pytest.importorskip("torch")
from kronecker_factored_second_amd import linear, okls, optim  # noqa: E402

pytestmark = pytest.mark.gpu

FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _n(t):
    return t.detach().cpu().double().numpy()


def _gradient(rng, shape, kind):
    return torch.tensor((rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape))).astype(np.float32)).to(FLOATS[kind]).cuda()


def _values(held):
    return _n(held.m).ravel(), _n(held.scales[0]), _n(held.v).ravel(), _n(held.scales[1])


def _check_p(got, p, m, s, t, hyper):
    """The parameter against the formula in fp64 on the fp32 moments: its two factors, the update's two products, sum, quotient and three constants, and the difference, each off by 2^-24 of itself."""
    update = hyper["lr"] / (1 - hyper["beta1"] ** t) * np.abs(m) / (s / (1 - hyper["beta2"] ** t) ** 0.5 + hyper["eps"])
    kept = (1 - hyper["lr"] * hyper["weight_decay"]) * p
    want = kept - np.sign(m) * update
    off = np.abs(got.astype(np.float64) - want)
    assert (off <= 2.0 ** -24 * (2 * np.abs(kept) + np.abs(want) + 8 * update) + 2.0 ** -149).all()


def _run(sizes, kinds, moments, steps=3, norm=None, max_norm=None, seed=0, shapes=None):
    """Steps of both sides from zero moments; every step starts from the GPU's own state."""
    rng = np.random.default_rng(seed)
    ps = [torch.tensor(rng.standard_normal(s).astype(np.float32)).cuda() for s in sizes]
    held = [optim.new_moments(p, moments) for p in ps]
    for t in range(1, steps + 1):
        gs = [_gradient(rng, s, kinds[i % len(kinds)]) for i, s in enumerate(sizes)]
        before = [(_n(p), None if m.scales is None else _values(m), _n(m.m), _n(m.v)) for p, m in zip(ps, held)]
        scale = None if norm is None else A.factor(float(norm), max_norm)
        optim.adamw(ps, gs, held, t, norm=norm, max_norm=max_norm, **HYPER)
        for j, (p, g, m, (p0, v8, m0, v0)) in enumerate(zip(ps, gs, held, before)):
            if p.numel() == 0:
                continue
            if moments == "8bit":
                old_m, old_s = (A.held(*x).astype(np.float32) for x in (v8[:2], v8[2:]))
                old_v = old_s * old_s
            else:
                old_m, old_v = m0.ravel().astype(np.float32), v0.ravel().astype(np.float32)
            _, m32, v32, s32 = A.step32(p0.ravel(), _n(g).ravel(), old_m, old_v, t, scale=scale, **HYPER)
            if moments == "8bit":
                u, w = A.thresholds(t, j, p.numel())
                for got, want in zip(_values(m), (*A.hold(m32, u, False), *A.hold(s32, w, True))):
                    assert np.array_equal(got, want), (j, t)
            else:
                assert np.array_equal(_n(m.m).ravel().astype(np.float32), m32) and np.array_equal(_n(m.v).ravel().astype(np.float32), v32), (j, t)
            _check_p(_n(p).ravel().astype(np.float32), p0.ravel(), m32.astype(np.float64), s32.astype(np.float64), t, HYPER)


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [1, 7, 8, 127, 128, 129, 1023, 2047, 2048, 2049, 40001])
def test_one_tensor(n, kind, moments):
    _run([n], [kind], moments)


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
@pytest.mark.parametrize("count", [2, 63, 64, 65, 127, 128, 129, 200])
def test_many_tensors(count, moments):
    """More tensors than a launch takes, of mixed sizes (0 among them), shapes and gradient types."""
    rng = np.random.default_rng(count)
    sizes = [int(v) for v in rng.integers(0, 400, count)]
    sizes[count // 2] = 5000
    sizes[0] = 0
    _run([(s,) if i % 3 else (s, 1) for i, s in enumerate(sizes)], ["f32", "bf16", "f16"], moments, steps=2)


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_no_element_at_an_even_place(moments):
    """Views that begin at every element: nothing but the element's own alignment is needed, and nothing next to them is written."""
    rng = np.random.default_rng(5)
    for offset in range(1, 9):
        n = 300 + offset
        base = {k: torch.full((n + 32,), 3, dtype=d, device="cuda") for k, d in (("p", torch.float32), ("g", torch.bfloat16))}
        kind = torch.uint8 if moments == "8bit" else torch.float32
        base |= {k: torch.full((n + 32,), 5, dtype=kind, device="cuda") for k in ("m", "v")}
        p, g, m, v = (base[k][offset: offset + n] for k in ("p", "g", "m", "v"))
        x, y = torch.tensor(rng.standard_normal(n).astype(np.float32)).cuda(), _gradient(rng, n, "bf16")
        p.copy_(x), g.copy_(y), m.zero_(), v.zero_()
        scales = torch.full((2, -(-n // 128)), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu) if moments == "8bit" else None
        e = torch.float8_e4m3fn
        held = optim.Moments(m.view(e), v.view(e), scales) if moments == "8bit" else optim.Moments(m, v)
        optim.adamw([p], [g], [held], 1, **HYPER)
        twin = optim.new_moments(x, moments)
        optim.adamw([x], [y], [twin], 1, **HYPER)
        assert torch.equal(p, x) and all(torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8)) for a, b in zip(held, twin) if a is not None)
        for k, fill in (("p", 3), ("m", 5), ("v", 5)):
            assert (base[k][:offset] == fill).all() and (base[k][offset + n:] == fill).all()


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
@pytest.mark.parametrize("value", [1e-3, 0.5, 7.0, 1e20, 0.0])
def test_clipped(value, moments):
    _run([700, 33], ["f32", "bf16"], moments, norm=torch.tensor(value, device="cuda"), max_norm=0.75)


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_no_step_where_the_norm_is_no_number(value, moments):
    p, g = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
    held = optim.new_moments(p, moments)
    optim.adamw([p], [g], [held], 1, **HYPER)
    before = [x.clone() for x in (p, *held) if x is not None]
    optim.adamw([p], [g], [held], 2, norm=torch.tensor(value, device="cuda"), max_norm=1.0, **HYPER)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, [x for x in (p, *held) if x is not None]))


def test_8_bits_at_the_ends():
    """Infinities and NaN stay in their element and do not reach the block's scale; zeros, subnormals and fp32's ends are held as the definition says."""
    n = 512
    g = torch.randn(n, device="cuda")
    g[3], g[200], g[201] = float("inf"), float("nan"), -float("inf")
    g[256:384] = 0
    g[384:] *= 1e-30
    g[385], g[386] = 3e38, 1e-38
    p = torch.randn(n, device="cuda")
    held, p0 = optim.new_moments(p, "8bit"), _n(p)
    for t in (1, 2):
        before = _values(held)
        optim.adamw([p], [g], [held], t, **HYPER)
        old_m, old_s = (A.held(*x).astype(np.float32) for x in (before[:2], before[2:]))
        with np.errstate(all="ignore"):
            _, m32, _, s32 = A.step32(p0, _n(g), old_m, old_s * old_s, t, **HYPER)
        u, w = A.thresholds(t, 0, n)
        for got, want in zip(_values(held), (*A.hold(m32, u, False), *A.hold(s32, w, True))):
            assert np.array_equal(got, want, equal_nan=True)
    # 3e38 squared is an infinity, so that its root is held as NaN and its update is none
    bad = np.zeros(n, bool)
    bad[[3, 200, 201, 385]] = True
    assert np.array_equal(np.isnan(_values(held)[2]), bad) and np.isfinite(_n(p)[256:384]).all()
    assert (_values(held)[0][256:384] == 0).all() and (_values(held)[2][256:384] == 0).all()


@pytest.mark.timeout(600)
def test_more_elements_than_32_bits_count():
    """2^32 + 1000 elements of one tensor: the last ones against the oracle, with the upper half of their number in the thresholds."""
    n, tail = (1 << 32) + 1000, 2048
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    held = optim.new_moments(p, "8bit")
    rng = np.random.default_rng(9)
    last = _gradient(rng, tail, "bf16")
    g[-tail:] = last
    optim.adamw([p], [g], [held], 5, **HYPER)
    lead = (n - tail) % 128                       # the first block of the tail holds zeros from before it
    x = np.concatenate([np.zeros(lead), _n(last)])
    first = n - tail - lead
    _, m32, _, s32 = A.step32(np.zeros(x.size), x, np.zeros(x.size), np.zeros(x.size), 5, **HYPER)
    u, w = A.thresholds(5, 0, x.size, first=first)
    for got, want, sc, k in ((held.m, m32, held.scales[0], (u, False)), (held.v, s32, held.scales[1], (w, True))):
        values, scales = A.hold(want, *k)
        assert np.array_equal(_n(got[first:]), values) and np.array_equal(_n(sc[first // 128:]), scales)
    assert (p[-tail:] != 0).any() and not held.m[: 1 << 20].view(torch.uint8).any()
    norm = optim.grad_norm([g])
    assert abs(float(norm) - np.linalg.norm(_n(last))) <= 2.0 ** -23 * float(norm)


# ---------------------------------------------------------------------------
# The norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("count", [1, 5, 64, 65, 128, 129, 300])
def test_grad_norm(count):
    """Squares are exact in fp64 and their sum is off by 2^-53 each: what is left is the result's own rounding."""
    rng = np.random.default_rng(count)
    kinds = ["f32", "bf16", "f16"]
    gs = [_gradient(rng, int(s), kinds[i % 3]) for i, s in enumerate(rng.integers(0, 3000, count))]
    gs[0] = _gradient(rng, (70, 1001), "bf16")
    want = A.norm([_n(g) for g in gs])
    got = optim.grad_norm(gs)
    assert got.shape == () and got.dtype == torch.float32
    assert abs(float(got) - want) <= want * (2.0 ** -24 + 2.0 ** -30)
    assert torch.equal(got, optim.grad_norm(gs))


@pytest.mark.parametrize("n", [1, 8191, 8192, 8193, 32767, 32768, 32769, 1000003])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_grad_norm_sizes_and_places(n, kind):
    g = _gradient(np.random.default_rng(n), n + 3, kind)
    for offset in (0, 1, 3):
        v = g[offset: offset + n]
        want = A.norm([_n(v)])
        assert abs(float(optim.grad_norm([v])) - want) <= want * (2.0 ** -24 + 2.0 ** -30)


def test_grad_norm_ends():
    """Sizes whose squares leave fp32, nothing to sum, and values that are no numbers."""
    assert float(optim.grad_norm([torch.full((9,), 1e30, device="cuda")])) == pytest.approx(3e30, rel=1e-6)
    assert float(optim.grad_norm([torch.full((9,), 1e-30, device="cuda")])) == pytest.approx(3e-30, rel=1e-6)
    assert float(optim.grad_norm([torch.zeros(0, device="cuda"), torch.zeros(0, 5, device="cuda")])) == 0
    for bad in (float("inf"), float("nan")):
        g = torch.ones(5000, device="cuda")
        g[4321] = bad
        assert not torch.isfinite(optim.grad_norm([g]))
    t = torch.randn(30, 40, device="cuda")
    assert abs(float(optim.grad_norm([t.T])) - float(optim.grad_norm([t]))) <= 1e-6 * float(optim.grad_norm([t]))


# ---------------------------------------------------------------------------
# As it is used
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_class_and_checkpoint(moments):
    """The class is the function's steps; it reads p.grad; a checkpoint goes on as if nothing had happened; autograd sees the writes."""
    torch.manual_seed(0)
    ps = [torch.randn(s, device="cuda", requires_grad=True) for s in ((70, 30), (5,), (1,))]
    qs = [p.detach().clone() for p in ps]
    opt, held = optim.AdamW(ps, moments=moments, **HYPER), [optim.new_moments(q, moments) for q in qs]
    for t in (1, 2, 3):
        gs = [torch.randn_like(q) for q in qs]
        for p, g in zip(ps, gs):
            p.grad = g.clone()
        norm = optim.grad_norm(gs)
        version = ps[0]._version
        opt.step(norm=norm, max_norm=0.5, lr=1e-2 / t)
        assert ps[0]._version > version
        optim.adamw(qs, gs, held, t, norm=norm, max_norm=0.5, **{**HYPER, "lr": 1e-2 / t})
        opt.zero_grad()
        assert ps[0].grad is None and opt.t == t
    assert all(torch.equal(p.detach(), q) for p, q in zip(ps, qs))
    sd = opt.state_dict()
    twin = optim.AdamW([p.detach().clone() for p in ps], moments=moments, **HYPER)
    twin.load_state_dict(sd)
    gs = [torch.randn_like(q) for q in qs]
    opt.step(grads=gs)
    twin.step(grads=gs)
    assert all(torch.equal(p.detach(), q) for p, q in zip(ps, twin.params))
    with pytest.raises(ValueError, match="gradient 0"):
        opt.step()
    assert opt.t == 4


def test_transposed_gradient():
    p, q = torch.randn(30, 40, device="cuda"), torch.randn(30, 40, device="cuda")
    q.copy_(p)
    g = torch.randn(40, 30, device="cuda")
    optim.adamw([p], [g.T], [optim.new_moments(p)], 1, **HYPER)
    optim.adamw([q], [g.T.contiguous()], [optim.new_moments(q)], 1, **HYPER)
    assert torch.equal(p, q)


def test_refusals():
    p, g = torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda")
    m, e = optim.new_moments(p), optim.new_moments(p, "8bit")
    for bad in (dict(params=[p.double()]), dict(params=[p.view(20, 15).T]), dict(grads=[g[:299]]), dict(grads=[g.view(20, 15)]), dict(grads=[None]),
                dict(grads=[g.cpu()]), dict(grads=[g.double()]), dict(moments=[optim.Moments(m.m, m.v[:299])]), dict(moments=[optim.Moments(m.m.half(), m.v)]),
                dict(moments=[optim.Moments(e.m, e.v)]), dict(moments=[optim.Moments(m.m, m.v, e.scales)]), dict(moments=[optim.Moments(e.m, e.v, e.scales[:1])]),
                dict(moments=[optim.Moments(e.m, e.v, e.scales.view(torch.uint8))]), dict(params=[p, p], grads=[g, g], moments=[m, optim.new_moments(p)]),
                dict(params=[p, g], grads=[g, g], moments=[m, e]), dict(params=[p, g], grads=[g, g], moments=[m, m]), dict(moments=[optim.Moments(m.m, m.m)]), dict(norm=torch.ones(2, device="cuda"), max_norm=1.0), dict(norm=torch.ones(1), max_norm=1.0),
                dict(norm=torch.ones((), device="cuda"))):
        with pytest.raises(ValueError):
            optim.adamw(**{**dict(params=[p], grads=[g], moments=[m], t=1), **bad})
    for bad in (dict(t=0), dict(lr=-1.0), dict(beta1=1.0), dict(norm=torch.ones((), device="cuda"), max_norm=0.0)):
        with pytest.raises(okls.OKLSError):
            optim.adamw(**{**dict(params=[p], grads=[g], moments=[m], t=1), **bad})
    assert not p.any() and not m.m.any()
    with pytest.raises(ValueError):
        optim.grad_norm([g, g.cpu()])


def test_other_stream():
    """Work of a side stream in order: the gradient, its norm and the step."""
    p, q = torch.randn(100000, device="cuda"), torch.zeros(100000, device="cuda")
    q.copy_(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    base = torch.randn(100000, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = base
        for _ in range(20):
            g = g * 1.01
        optim.adamw([q], [g], [optim.new_moments(q, "8bit")], 1, norm=optim.grad_norm([g]), max_norm=1.0, **HYPER)
    torch.cuda.current_stream().wait_stream(s)
    optim.adamw([p], [g], [optim.new_moments(p, "8bit")], 1, norm=optim.grad_norm([g]), max_norm=1.0, **HYPER)
    assert torch.equal(p, q)


@pytest.mark.parametrize("moments", ["fp32", "8bit"])
def test_graph_replays(moments):
    """The norm and the step captured once (70 tensors: two launches) and replayed on new gradients, with eager steps of another set between."""
    torch.manual_seed(1)
    sizes = [1 + 37 * i for i in range(70)]
    ps = [torch.randn(n, device="cuda") for n in sizes]
    qs = [p.clone() for p in ps]
    gs = [torch.randn(n, device="cuda") for n in sizes]
    mp, mq = ([optim.new_moments(p, moments) for p in ps] for _ in range(2))

    def step(a, g, m):
        optim.adamw(a, g, m, 3, norm=optim.grad_norm(g), max_norm=1.0, **HYPER)

    step([p.clone() for p in ps], gs, [optim.new_moments(p, moments) for p in ps])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ps, gs, mp)
    for i in range(4):
        for g in gs:
            g.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(qs, [g.clone() for g in gs], mq)
        assert all(torch.equal(a, b) for a, b in zip(ps, qs)), i
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for a, b in zip(mp, mq) for x, y in zip(a, b) if x is not None)


def test_beside_the_matrix_step():
    """What a model's step takes: the matrix by okls, the norm's weight by AdamW, from one backward pass of the 8-bit layer."""
    torch.manual_seed(2)
    x = torch.randn(200, 96, device="cuda").bfloat16()
    w, W = torch.ones(96, device="cuda", requires_grad=True), (0.05 * torch.randn(160, 96, device="cuda")).requires_grad_()
    matrices, rest = okls.OKLS([W], mode="muon"), optim.AdamW([w], moments="8bit")
    start = w.detach().clone(), W.detach().clone()
    for _ in range(2):
        y, _ = linear.rms_norm_linear(x, w, W)
        y.float().square().mean().backward()
        norm = optim.grad_norm([w.grad, W.grad])
        assert float(norm) == pytest.approx(float((w.grad.double().square().sum() + W.grad.double().square().sum()).sqrt()), rel=1e-6)
        with torch.no_grad():
            matrices.step()
        rest.step(norm=norm, max_norm=1.0)
        matrices.zero_grad()
        rest.zero_grad()
    assert not torch.equal(w.detach(), start[0]) and not torch.equal(W.detach(), start[1]) and w.isfinite().all()
