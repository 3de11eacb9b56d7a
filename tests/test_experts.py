"""The experts' operators on the CPU: the oracle's own pins, and every refusal of
the C ABI and of the binding (all return before a launch)."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from kronecker_factored_second_amd import experts, linear, okls
from oracle import experts_oracle as E

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _lib():
    if not os.path.exists(okls.LIB_PATH):
        pytest.skip("libokls.so not built")
    return experts.load()


def _choices(rng, tokens, each, n, dropped=0.1):
    c = np.stack([rng.permutation(n)[:each] for _ in range(tokens)]) if tokens else np.zeros((0, each), np.int64)
    return np.where(rng.random(c.shape) < dropped, rng.choice([-1, n, 1 << 30], c.shape), c)


# ---------------------------------------------------------------------------
# Oracle
# ---------------------------------------------------------------------------
def test_a_plan_by_hand():
    rows, pairs, offsets, counts = E.plan(np.array([[2, 0], [0, 7], [2, 2], [-1, 0]]), 3, 16)
    assert rows.tolist() == [[16, 0], [1, -1], [17, 18], [-1, 2]]
    assert offsets.tolist() == [0, 16, 16, 32] and counts.tolist() == [3, 0, 3]
    assert pairs[:4].tolist() == [1, 2, 7, -1] and pairs[16:20].tolist() == [0, 4, 5, -1] and pairs.size == 48


@pytest.mark.parametrize("align", [16, 128])
def test_the_capacity_is_enough_and_is_reached(align):
    rng = np.random.default_rng(0)
    for tokens, each, n in ((1, 1, 1), (3, 2, 8), (40, 2, 5), (7, 3, 30), (200, 1, 3)):
        room = E.capacity(tokens, each, n, align)
        assert room == experts.capacity(tokens, each, n, align)
        for _ in range(5):
            assert E.plan(_choices(rng, tokens, each, n, 0), n, align)[2][-1] <= room
        # one choice of every expert but the last that gets any, which takes the rest
        worst = np.minimum(np.arange(tokens * each), min(n, tokens * each) - 1).reshape(tokens, each)
        assert E.plan(worst, n, align)[2][-1] > room - align * min(n, tokens * each)


def test_gradients_against_differences():
    """combine's and the products' gradients as the formulas give them, against central differences of the forward formulas in fp64 (linear in each argument: exact but for rounding)."""
    rng = np.random.default_rng(1)
    choice = _choices(rng, 9, 3, 5)
    rows, pairs, _, _ = E.plan(choice, 5, 16)
    y, w, dout = rng.standard_normal((pairs.size, 4)), rng.standard_normal((9, 3)), rng.standard_normal((9, 4))
    dy, dw, _ = E.combine_backward(dout, y, rows, pairs, w)

    def slope(f, at):
        g = np.zeros_like(at)
        for i in np.ndindex(at.shape):
            up, down = at.copy(), at.copy()
            up[i] += 0.5
            down[i] -= 0.5
            g[i] = f(up) - f(down)
        return g
    np.testing.assert_allclose(dy, slope(lambda v: (E.combine(v, rows, w)[0] * dout).sum(), y), atol=1e-12)
    np.testing.assert_allclose(dw, slope(lambda v: (E.combine(y, rows, v)[0] * dout).sum(), w), atol=1e-12)
    x, dxs = rng.standard_normal((9, 4)), rng.standard_normal((pairs.size, 4))
    np.testing.assert_allclose(E.combine(dxs, rows, None)[0], slope(lambda v: (E.gather(v, pairs, 3) * dxs).sum(), x), atol=1e-12)
    xs, W, dys = E.gather(x, pairs, 3), rng.standard_normal((5, 6, 4)), rng.standard_normal((pairs.size, 6))
    dys[pairs < 0] = 0
    np.testing.assert_allclose(E.weight_grad(dys.T, xs.T, pairs, choice, 5)[0], slope(lambda v: (E.matmul(xs, v, pairs, choice)[0] * dys).sum(), W), atol=1e-11)
    np.testing.assert_allclose(E.matmul(dys, W.transpose(0, 2, 1), pairs, choice)[0], slope(lambda v: (E.matmul(v, W, pairs, choice)[0] * dys).sum(), xs), atol=1e-11)


# ---------------------------------------------------------------------------
# ABI
# ---------------------------------------------------------------------------
def test_header_symbols_and_struct(tmp_path):
    lib = _lib()
    header = open(os.path.join(ROOT, "include", "okls_experts.h")).read()
    assert set(re.findall(r"\b(okls_[a-z_]+)\s*\(", header)) - {"okls_expert_plan"} == set(experts.EXPORTED)
    assert int(re.search(r"OKLS_MAX_EXPERTS (\d+)", header).group(1)) == experts.MAX_EXPERTS
    for name in experts.EXPORTED:
        assert hasattr(lib, name)
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [n for n, _ in experts.PlanStruct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "okls_experts.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu ", offsetof(okls_expert_plan, {n}));\n' for n in names)
                   + '  printf("%zu", sizeof(okls_expert_plan));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(experts.PlanStruct, n).offset for n in names] + [ctypes.sizeof(experts.PlanStruct)]


P = 0x1000   # a pointer that is never read: every call here is refused
INVALID, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -7


def _plan(**over):
    d = dict(rows=P, pairs=P, offsets=P, counts=P, tokens=100, each=2, capacity=E.capacity(100, 2, 4, 128), n_experts=4, align=128)
    d.update(over)
    return experts.PlanStruct(**d)


def _blk(rows, cols, **over):
    d = dict(codes=P, scales=P, rows=rows, cols=cols, ld=-(-cols // 128) * 128, ld_scale=-(-rows // 16) * 16, format=0)
    d.update(over)
    return linear.BlockedStruct(**d)


ROOM = E.capacity(100, 2, 4, 128)
PLANS = [(None, INVALID), (dict(tokens=-1), SHAPE), (dict(each=0), SHAPE), (dict(tokens=1 << 28, each=2), SHAPE), (dict(n_experts=0), SHAPE),
         (dict(n_experts=513), SHAPE), (dict(align=8), SHAPE), (dict(align=256), SHAPE), (dict(capacity=ROOM - 128), SHAPE), (dict(capacity=ROOM + 128), SHAPE),
         (dict(offsets=None), INVALID), (dict(counts=P + 2), INVALID), (dict(rows=None), INVALID), (dict(pairs=P + 1), INVALID)]


@pytest.mark.parametrize("over,status", PLANS)
def test_plan_refusals_everywhere(over, status):
    lib = _lib()
    p = None if over is None else ctypes.byref(_plan(**over))
    assert lib.okls_experts_plan(P, 64, p, P, 1 << 20, None) == status
    assert lib.okls_experts_gather(p, P, 8, 0, 8, P, 8, None) == status
    assert lib.okls_experts_combine(p, P, 8, 0, 8, None, 0, P, 8, None) == status
    assert lib.okls_experts_combine_backward(p, P, 8, P, 8, 0, 8, P, 0, P, 8, P, None) == status
    assert lib.okls_experts_quantize_rows(p, P, 8, 0, 8, 0, _blk(ROOM, 8), None, None) == status
    assert lib.okls_experts_matmul(p, _blk(ROOM, 8), _blk(64, 8), 16, P, 0, 16, None) == status
    assert lib.okls_experts_weight_grad(p, _blk(16, ROOM), _blk(8, ROOM), P, 0, 8, None) == status


def test_other_refusals():
    lib, p = _lib(), ctypes.byref(_plan())
    assert lib.okls_experts_capacity(100, 2, 4, 128) == ROOM and lib.okls_experts_capacity(-1, 2, 4, 128) == -1
    assert lib.okls_experts_plan_workspace_size(1 << 20, 1, 512) > 0 and lib.okls_experts_plan_workspace_size(1, 1, 513) == 0
    assert lib.okls_experts_plan(None, 64, p, P, 1 << 20, None) == INVALID
    assert lib.okls_experts_plan(P + 4, 64, p, P, 1 << 20, None) == INVALID
    assert lib.okls_experts_plan(P, 16, p, P, 1 << 20, None) == DTYPE
    big = ctypes.byref(_plan(tokens=100000, capacity=E.capacity(100000, 2, 4, 128)))
    assert lib.okls_experts_plan(P, 64, big, None, 1 << 20, None) == WORKSPACE
    assert lib.okls_experts_plan(P, 64, big, P + 8, 1 << 20, None) == WORKSPACE
    assert lib.okls_experts_plan(P, 64, big, P, 16, None) == WORKSPACE

    for dtype in (-1, 3):
        assert lib.okls_experts_gather(p, P, 8, dtype, 8, P, 8, None) == DTYPE
        assert lib.okls_experts_combine(p, P, 8, dtype, 8, None, 0, P, 8, None) == DTYPE
        assert lib.okls_experts_combine(p, P, 8, 0, 8, P, dtype, P, 8, None) == DTYPE
        assert lib.okls_experts_combine_backward(p, P, 8, P, 8, 0, 8, P, dtype, P, 8, P, None) == DTYPE
        assert lib.okls_experts_quantize_rows(p, P, 8, dtype, 8, 0, _blk(ROOM, 8), None, None) == DTYPE
        assert lib.okls_experts_quantize_stack(P, dtype, 4, 128, 16, 8, 8, _blk(64, 8), None, None) == DTYPE
        assert lib.okls_experts_matmul(p, _blk(ROOM, 8), _blk(64, 8), 16, P, dtype, 16, None) == DTYPE
        assert lib.okls_experts_weight_grad(p, _blk(16, ROOM), _blk(8, ROOM), P, dtype, 8, None) == DTYPE
    gather = lambda x=P, ldx=8, cols=8, out=P, ldo=8: lib.okls_experts_gather(p, x, ldx, 0, cols, out, ldo, None)  # noqa: E731
    assert gather(x=None) == INVALID and gather(x=P + 2) == INVALID and gather(ldx=7) == INVALID and gather(out=None) == INVALID and gather(ldo=7) == INVALID
    assert gather(cols=-1) == SHAPE and gather(cols=0, x=None, out=None) == 0
    combine = lambda y=P, ldy=8, w=P, out=P, ldo=8: lib.okls_experts_combine(p, y, ldy, 0, 8, w, 1, out, ldo, None)  # noqa: E731
    assert combine(y=None) == INVALID and combine(ldy=7) == INVALID and combine(w=P + 1) == INVALID and combine(out=P + 2) == INVALID and combine(ldo=1) == INVALID
    back = lambda d=P, y=P, w=P, dy=P, dw=P, ld=8: lib.okls_experts_combine_backward(p, d, ld, y, 8, 0, 8, w, 0, dy, 8, dw, None)  # noqa: E731
    assert back(d=None) == INVALID and back(y=None) == INVALID and back(w=None) == INVALID and back(dy=None) == INVALID and back(dw=None) == INVALID and back(ld=7) == INVALID
    rows = lambda a=None, b=None, g=0, x=P: lib.okls_experts_quantize_rows(p, x, 300, 0, 300, g, a, b, None)  # noqa: E731
    assert rows() == INVALID and rows(a=_blk(ROOM, 300), g=2) == INVALID and rows(a=_blk(ROOM, 300), x=None) == INVALID
    assert rows(a=_blk(ROOM + 1, 300)) == SHAPE and rows(b=_blk(ROOM, 300)) == SHAPE and rows(a=_blk(ROOM, 300, ld=256)) == SHAPE
    assert rows(a=_blk(ROOM, 300, format=2)) == DTYPE and rows(a=_blk(ROOM, 300, codes=None)) == INVALID
    stack = lambda a=None, b=None, e=4, stride=4800, n=16, x=P: lib.okls_experts_quantize_stack(x, 0, e, stride, n, 300, 300, a, b, None)  # noqa: E731
    assert stack() == INVALID and stack(a=_blk(64, 300), x=None) == INVALID and stack(a=_blk(64, 300), stride=-1) == INVALID
    assert stack(a=_blk(64, 300), e=0) == SHAPE and stack(a=_blk(64, 300), e=513) == SHAPE and stack(a=_blk(65, 300)) == SHAPE
    assert stack(a=_blk(4 * 16, 300), n=17) == SHAPE and stack(b=_blk(4 * 300, 16)) == SHAPE       # 17 rows take 32, 300 take 304
    mm = lambda a=None, b=None, n=16, c=P, ldc=16: lib.okls_experts_matmul(p, a or _blk(ROOM, 300), b or _blk(64, 300), n, c, 0, ldc, None)  # noqa: E731
    assert lib.okls_experts_matmul(p, None, _blk(64, 300), 16, P, 0, 16, None) == INVALID
    assert mm(a=_blk(ROOM, 301)) == SHAPE and mm(a=_blk(ROOM - 128, 300)) == SHAPE and mm(b=_blk(63, 300)) == SHAPE and mm(n=17) == SHAPE and mm(n=-1) == SHAPE
    assert mm(c=None) == INVALID and mm(ldc=15) == INVALID and mm(c=P + 2) == INVALID and mm(b=_blk(64, 300, format=7)) == DTYPE
    assert mm(a=_blk(ROOM, 300, ld=1 << 24)) == SHAPE                   # rows of codes too far apart
    assert mm(n=1 << 30, b=_blk(4 << 30, 300)) == SHAPE
    wg = lambda a=None, b=None, c=P, ldc=8, plan=p: lib.okls_experts_weight_grad(plan, a or _blk(16, ROOM), b or _blk(8, ROOM), c, 0, ldc, None)  # noqa: E731
    assert wg(a=_blk(16, ROOM + 128)) == SHAPE and wg(b=_blk(8, ROOM - 128)) == SHAPE and wg(c=None) == INVALID and wg(ldc=7) == INVALID
    assert wg(b=_blk(1 << 28, ROOM), ldc=1 << 28, a=_blk(1 << 10, ROOM)) == SHAPE
    small = E.capacity(100, 2, 4, 64)
    assert wg(plan=ctypes.byref(_plan(align=64, capacity=small)), a=_blk(16, small), b=_blk(8, small)) == UNSUPPORTED


# ---------------------------------------------------------------------------
# Binding
# ---------------------------------------------------------------------------
def test_binding_refuses_on_the_cpu():
    choice = torch.zeros(4, 2, dtype=torch.int64)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for bad in (lambda: experts.plan(choice, 3), lambda: experts.plan(choice[0], 3), lambda: experts.plan(choice.float(), 3), lambda: experts.plan(choice, 0),
                lambda: experts.plan(choice, 513), lambda: experts.plan(choice, 3, align=8), lambda: experts.plan(choice[:, :0], 3),
                lambda: experts.capacity(-1, 1, 1), lambda: experts.capacity(1 << 28, 2, 1),
                lambda: experts.Plan(i32(4, 2), i32(8), i32(4), i32(3)), lambda: experts.Plan(i32(4), i32(8), i32(4), i32(3)),
                lambda: experts.quantize_stack(torch.zeros(2, 3, 4)), lambda: experts.quantize_stack(torch.zeros(3, 4))):
        with pytest.raises(ValueError):
            bad()


def test_stack_dequantizes():
    """Each expert's rows begin at a multiple of 16; what lies between is no part of the stack."""
    e, n, k = 3, 5, 130
    s = experts.Stack.empty((e, n, k), torch.float8_e4m3fn, torch.device("cpu"))
    assert s.blocked.shape == (48, k)
    s.blocked.codes.view(torch.uint8).random_(0, 100)
    s.blocked.scales.view(torch.uint8).fill_(127)
    v = s.dequantize()
    assert v.shape == (e, n, k) and torch.equal(v[1, 2], s.blocked.codes[18, :k].float())


def test_a_plan_keeps_its_tensors():
    """A plan's tensors cannot be replaced, and ones that changed their sizes are refused before anything is launched."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    room = experts.capacity(4, 2, 3)
    p = experts.Plan.__new__(experts.Plan)
    p._set(i32(4, 2), i32(room), i32(4), i32(3), 128, room, 4, 2, 3)
    struct = experts.PlanStruct.from_address(p.address())
    assert (struct.rows, struct.pairs, struct.offsets, struct.counts) == tuple(t.data_ptr() for t in (p.rows, p.pairs, p.offsets, p.counts))
    for name in ("rows", "pairs", "offsets", "counts"):
        with pytest.raises(AttributeError):
            setattr(p, name, i32(1))
    for t in (p.rows, p.pairs, p.offsets, p.counts):
        kept, n = t.clone(), t.numel()
        t.set_(i32(n - 1))
        with pytest.raises(ValueError):
            p.address()
        t.set_(kept)
        assert p.address()


# ---------------------------------------------------------------------------
# Autograd
# ---------------------------------------------------------------------------
def _cpu_plan(tokens=4, each=2, n=3):
    """A plan whose tensors lie on the CPU, for what happens before a launch."""
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    room = experts.capacity(tokens, each, n)
    p = experts.Plan.__new__(experts.Plan)
    p._set(i32(tokens, each), i32(room), i32(n + 1), i32(n), 128, room, tokens, each, n)
    return p


def _no_launch(monkeypatch):
    """Every step that would launch something fails the test instead."""
    def launched(*args, **kwargs):
        raise AssertionError("a launch")
    for name in ("_call", "_gather", "_combine", "_quantize_rows", "_quantize_stack", "matmul"):
        monkeypatch.setattr(experts, name, launched)


@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(monkeypatch, grad):
    """A dual tensor does not require a gradient, and a result without a tangent would count as a constant: refused before anything is launched, under no_grad too, which leaves forward mode on."""
    _no_launch(monkeypatch)
    p = _cpu_plan()
    x, xs, w, W = torch.randn(4, 8), torch.randn(p.capacity, 8), torch.rand(4, 2), torch.randn(3, 5, 8)
    with torch.autograd.forward_ad.dual_level(), torch.set_grad_enabled(grad):
        dual = lambda t: torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for bad in (lambda: experts.gather(dual(x), p), lambda: experts.combine(dual(xs), w, p), lambda: experts.combine(xs, dual(w), p),
                    lambda: experts.combine(dual(xs), None, p), lambda: experts.linear(dual(xs), W, p), lambda: experts.linear(xs, dual(W), p),
                    lambda: experts.token_linear(dual(x), W, p), lambda: experts.token_linear(x, dual(W), p),
                    lambda: experts.gather(dual(x).requires_grad_(), p)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                bad()
        with pytest.raises(AssertionError, match="a launch"):      # a level alone refuses nothing
            experts.gather(x, p)


def _stubs(monkeypatch):
    """The operators' launches as plain tensors of the right sizes on the CPU."""
    monkeypatch.setattr(experts, "_gather", lambda x, p: x.new_zeros(p.capacity, x.shape[1]))
    monkeypatch.setattr(experts, "_combine", lambda y, w, p: y.new_zeros(p.tokens, y.shape[1]))
    monkeypatch.setattr(experts, "_call", lambda *args: None)
    monkeypatch.setattr(experts, "_matrix", lambda name, t: t.shape[1])
    monkeypatch.setattr(linear.Blocked, "address", lambda self: 0)
    monkeypatch.setattr(experts, "_quantize_stack", lambda W, dtype, along, across: (
        experts.Stack.empty(W.shape, dtype, W.device) if along else None, experts.Stack.empty((W.shape[0], W.shape[2], W.shape[1]), dtype, W.device) if across else None))


def _passes(p):
    """(forward pass of one leaf, the leaf) of every operator, and of combine with and without weights."""
    x, xs, w, W = torch.randn(4, 8), torch.randn(p.capacity, 8), torch.rand(4, 2), torch.randn(3, 5, 8)
    for f, leaf in ((lambda t: experts.gather(t, p), x), (lambda t: experts.combine(t, None, p), xs), (lambda t: experts.combine(t, w, p), xs),
                    (lambda t: experts.combine(xs, t, p), w), (lambda t: experts.linear(t, W, p), xs), (lambda t: experts.linear(xs, t, p), W),
                    (lambda t: experts.token_linear(t, W, p), x), (lambda t: experts.token_linear(x, t, p), W)):
        yield f, leaf.clone().requires_grad_()


def test_a_plan_written_to_between_the_passes_is_noticed(monkeypatch):
    """Gradients follow the forward pass's rows: a plan whose tensors torch wrote to in between makes the backward pass raise, one that is as it was does not."""
    _stubs(monkeypatch)
    for name in ("rows", "pairs", "offsets", "counts"):
        p = _cpu_plan()
        for f, leaf in _passes(p):
            f(leaf).sum().backward()
            assert leaf.grad.shape == leaf.shape
            y = f(leaf).sum()
            getattr(p, name).zero_()
            with pytest.raises(RuntimeError, match="modified in place"):
                y.backward()
            f(leaf).sum().backward()        # a pass after the write has its own


def test_a_plan_of_inference_tensors_trains(monkeypatch):
    """A plan made under inference_mode has no count of writes, and autograd refuses to save its tensors: the operators take it all the same."""
    _stubs(monkeypatch)
    with torch.inference_mode():
        p = _cpu_plan()
    assert p.rows.is_inference()
    for f, leaf in _passes(p):
        f(leaf).sum().backward()
        assert leaf.grad.shape == leaf.shape


@pytest.mark.parametrize("grad", [True, False])
def test_a_layer_refuses_before_anything_is_launched(monkeypatch, grad):
    """Wrong types and devices of the weight and the gradient's 8-bit type, which only the backward pass uses, as well."""
    _no_launch(monkeypatch)
    monkeypatch.setattr(experts, "_matrix", lambda name, t: t.shape[1])
    p = _cpu_plan()
    x, xs, W = torch.randn(4, 8).requires_grad_(grad), torch.randn(p.capacity, 8).requires_grad_(grad), torch.randn(3, 5, 8)
    for W_bad, kw in ((W.double(), {}), (W.to("meta"), {}), (W.long(), {}), (W, dict(grad_dtype=torch.float16)), (W, dict(grad_dtype=None)), (W, dict(grad_dtype=torch.float8_e8m0fnu))):
        for run, rows in ((experts.token_linear, x), (experts.linear, xs)):
            with pytest.raises(ValueError):
                run(rows, W_bad, p, **kw)
    for run, rows in ((experts.token_linear, xs), (experts.linear, x), (experts.linear, xs.detach().to("meta"))):
        with pytest.raises(ValueError):
            run(rows, W, p)
    with pytest.raises(AssertionError, match="a launch"):
        experts.linear(xs, W, p, grad_dtype=torch.float8_e5m2)


def test_a_layer_refuses_sums_that_only_its_gradients_cannot_take(monkeypatch):
    """Rows of codes 2^24 bytes apart are refused by the products, those of the gradients too: here before the forward pass, and only where a gradient needs them."""
    _no_launch(monkeypatch)
    monkeypatch.setattr(experts, "_matrix", lambda name, t: t.shape[1])
    meta = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    i32 = lambda *s: meta(*s, dtype=torch.int32)  # noqa: E731

    def runs(tokens, n, k, need_x, need_w):
        room = experts.capacity(tokens, 1, 2)
        p = experts.Plan.__new__(experts.Plan)
        p._set(i32(tokens, 1), i32(room), i32(3), i32(2), 128, room, tokens, 1, 2)
        with pytest.raises((ValueError, AssertionError)) as e:
            experts.token_linear(meta(tokens, k).requires_grad_(need_x), meta(2, n, k).requires_grad_(need_w), p)
        return e.type is AssertionError         # it went on to a launch
    most = (1 << 24) - 128
    assert experts.MAX_SUMMED == most
    fits = most - 2 * 127           # tokens of whose choices any leave at most `most` rows
    for need_x, need_w in ((False, False), (True, False), (False, True), (True, True)):
        assert runs(4, 8, most, need_x, need_w) and not runs(4, 8, most + 1, need_x, need_w)
        assert runs(4, most, 8, need_x, need_w) and runs(4, most + 1, 8, need_x, need_w) == (not need_x)
        assert runs(fits, 8, 8, need_x, need_w) and runs(1 << 24, 8, 8, need_x, need_w) == (not need_w)


def test_a_gradient_with_a_tangent_is_refused(monkeypatch):
    """Forward mode over a backward pass: the gradient that comes in carries a tangent, and what goes on would carry none."""
    _stubs(monkeypatch)
    for f, leaf in _passes(_cpu_plan()):
        with torch.autograd.forward_ad.dual_level():
            y = f(leaf)
            d = torch.autograd.forward_ad.make_dual(torch.ones_like(y), torch.ones_like(y))
            with pytest.raises(NotImplementedError, match="forward-mode"):
                torch.autograd.grad(y, leaf, d)
            assert torch.autograd.grad(f(leaf), leaf, torch.ones_like(y))[0].shape == leaf.shape
