"""The many-tensor optimizer step on the CPU: the oracle's own pins, and every
refusal of the C ABI and of the binding (all return before a launch)."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from kronecker_factored_second_amd import okls, optim
from oracle import optim_oracle as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _lib():
    if not os.path.exists(okls.LIB_PATH):
        pytest.skip("libokls.so not built")
    return optim.load()


# ---------------------------------------------------------------------------
# Oracle
# ---------------------------------------------------------------------------
def test_formula_is_torchs():
    """Ten steps of the fp64 formula against torch's AdamW in fp64: the same to the last few bits."""
    rng = np.random.default_rng(0)
    p, m, v = rng.standard_normal(50), np.zeros(50), np.zeros(50)
    q = torch.tensor(p, requires_grad=True)
    opt = torch.optim.AdamW([q], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    for t in range(1, 11):
        g = rng.standard_normal(50)
        p, m, v = A.step64(p, g, m, v, t, **HYPER)
        q.grad = torch.tensor(g)
        opt.step()
        np.testing.assert_allclose(p, q.detach().numpy(), rtol=1e-13)


def test_formula_in_32_bits_is_near():
    """Each product and sum rounds by 2^-24 of itself: four of them (and a constant's rounding) make m, five v, ten the update."""
    rng = np.random.default_rng(1)
    p, g, m, v = rng.standard_normal(4000), rng.standard_normal(4000), rng.standard_normal(4000), rng.random(4000)
    p, g, m, v = (x.astype(np.float32) for x in (p, g, m, v))
    want, got = A.step64(p, g, m, v, 7, **HYPER), A.step32(p, g, m, v, 7, **HYPER)
    size = np.abs(0.9 * m) + np.abs(0.1 * g)
    assert (np.abs(got[1] - want[1]) <= 4 * 2.0 ** -24 * size).all()
    assert (np.abs(got[2] - want[2]) <= 5 * 2.0 ** -24 * want[2]).all()
    update = size / np.sqrt(want[2]) * 1e-2 / (1 - 0.9 ** 7)
    assert (np.abs(got[0] - want[0]) <= 2.0 ** -24 * (2 * np.abs(p) + np.abs(want[0]) + 16 * update)).all()


def test_holding_is_in_proportion():
    """Over all thresholds a value is held as itself on average (a threshold is a multiple of 2^-16), by less than a step each time, and exactly where a code has it."""
    u = np.arange(65536) / 65536
    for x in (1.0, 0.7, 1.3e-3, 0.02, 1.0 / 3):
        block = np.zeros(128)
        block[0], block[1] = 1.0, x
        got = []
        for shift in range(0, 65536, 257):
            w = np.full(128, u[shift])
            values, scales = A.hold(block, w, False)
            got.append(A.held(values, scales)[1])
        step = max(np.ldexp(1.0, np.frexp(np.float32(x) * 256)[1] - 1 - 3), 2.0 ** -9) / 256
        assert max(abs(v - np.float32(x)) for v in got) < step
        assert abs(np.mean(got) - np.float32(x)) < step / 100
    values, scales = A.hold(np.array([1.0, 0.5, -0.25]), np.full(3, 65535 / 65536), False)
    assert list(A.held(values, scales)) == [1.0, 0.5, -0.25]


def test_small_roots_round_up():
    """A root below the smallest normal code is never held smaller than it is, so an update never divides by less than its own root's share."""
    rng = np.random.default_rng(2)
    x = np.exp(rng.uniform(-30, 0, 128))
    x[0] = 1.0
    values, scales = A.hold(x, np.zeros(128), True)
    a = x.astype(np.float32) / scales[0]
    small = a < A.LOW
    assert small.sum() > 20 and (values[small] >= a[small]).all() and (values > 0).all()
    assert A.hold(np.zeros(5), np.full(5, 0.99), True)[0].max() == 0


def test_decay_without_gradients():
    """Roots held in 8 bits and a beta2 of 0.999: without gradients v falls as 0.999^t, which to nearest it never would.  A step's rounding error has a variance of at most p of a step squared, p the part of a step that the root moves by (0.0005 s in steps of s / 16 to s / 8: at most 1 / 125); their sum over 1000 steps, root 8 steps, divided by the root of 4096 elements, is an eighth of a step, 1.6 % of s at most."""
    n = 4096
    s = (np.ones(n), np.ones(n // 128))
    m = (np.zeros(n), np.ones(n // 128))
    for t in range(1, 1001):
        _, m, s = A.step8(np.zeros(n), np.zeros(n), m, s, t, 0, lr=0.0, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    assert abs(A.held(*s).mean() / 0.999 ** 500 - 1) < 5 * 0.016
    nearest = np.float32(np.sqrt(np.float32(0.999)))
    assert A.hold(np.full(128, nearest), np.full(128, 0.5), True)[0][0] * A.hold(np.full(128, nearest), np.full(128, 0.5), True)[1][0] == 1.0


def test_roots_far_below_their_block_stay():
    """A root below the smallest normal code (2^-6 of 448, 3.5e-5 of its block's largest) always rounds up: while the largest stays where it is, so does the small one, and does not fall as 0.999^t makes the formula's."""
    start = np.full(128, 2e-5)
    start[0] = 1.0
    m, s = (np.zeros(128), np.ones(1)), A.hold(start, np.full(128, 0.5), True)
    first = A.held(*s)[1:]
    g = np.zeros(128)
    g[0] = 1.0
    for t in range(1, 301):
        _, m, s = A.step8(np.zeros(128), g, m, s, t, 0, lr=0.0, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    assert A.held(*s)[0] == 1.0 and np.array_equal(A.held(*s)[1:], first) and (first >= 2e-5).all() and (first < 2e-5 + 2.0 ** -17).all()


def test_roots_scatter_in_steady_state():
    """Gradients of one size each.  A step moves the root s by 0.0005 s |z^2 - 1|, 0.968 of 0.0005 s on average, and rounds with a variance of that times a code's step, 0.0902 s on average over the logarithm from s / 16 to s / 8: 4.37e-5 s^2.  What is off falls by a thousandth a step, so the variance settles at 4.37e-5 / 0.002 and the deviation at 0.148.  The drift, 0.0005 (v / s - s), is zero on average where the mean of 1 / s, (1 + 0.022) over s's, is s's over v: a mean of 1.011, and of the square 1.044.  2000 steps reach 0.98 of the variance.  1024 elements give the deviation within 0.148 / 45 and the means within 0.148 / 32 and twice that; v's own deviation, 1.6 % of the root, moves s with it for the most part."""
    rng = np.random.default_rng(3)
    n, hyper = 1024, dict(lr=0.0, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    size = np.exp(rng.standard_normal(n))
    m, s, v = (np.zeros(n), np.ones(n // 128)), A.hold(size, np.full(n, 0.5), True), size ** 2
    for t in range(1000, 3000):
        g = size * rng.standard_normal(n)
        _, m, s = A.step8(np.zeros(n), g, m, s, t, 0, **hyper)
        v = 0.999 * v + 0.001 * g * g
    ratio = A.held(*s) / np.sqrt(v)
    assert abs(ratio.std() - 0.148) < 5 * 0.148 / 45 + 0.01 * 0.148 + 0.0016      # five deviations; the variance's last 2 %; a tenth of v's own
    assert abs(ratio.mean() - 1.011) < 5 * 0.148 / 32
    assert abs((ratio ** 2).mean() - 1.044) < 5 * 2 * 0.148 / 32


def test_thresholds_are_spread():
    """65536 elements: a mean of 1/2 within 5 of its standard deviations (0.289 / 256), different for steps and places, and the element's upper 32 bits count."""
    u, w = A.thresholds(3, 1, 65536)
    for x in (u, w):
        assert x.min() >= 0 and x.max() < 1 and abs(x.mean() - 0.5) < 5 * 0.289 / 256
    assert abs(np.corrcoef(u, w)[0, 1]) < 5 / 256
    for other in (A.thresholds(4, 1, 65536), A.thresholds(3, 2, 65536), A.thresholds(3, 1, 65536, first=1 << 32)):
        assert abs(np.corrcoef(u, other[0])[0, 1]) < 5 / 256
    a, b = A.thresholds(3, 1, 100, first=(1 << 32) - 50), A.thresholds(3, 1, 50, first=1 << 32)
    assert np.array_equal(a[0][50:], b[0])


# ---------------------------------------------------------------------------
# ABI
# ---------------------------------------------------------------------------
def test_header_symbols_and_structs(tmp_path):
    lib = _lib()
    header = open(os.path.join(ROOT, "include", "okls_optim.h")).read()
    assert set(re.findall(r"\b(okls_[a-z_]+)\s*\(", header)) == set(optim.EXPORTED)
    for name in optim.EXPORTED:
        assert hasattr(lib, name)
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"okls_gradient": optim.GradientStruct, "okls_adamw_tensor": optim.TensorStruct, "okls_adamw_config": optim.ConfigStruct}
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "okls_optim.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu ", offsetof({c}, {n}));\n' for c, s in structs.items() for n, _ in s._fields_)
                   + "".join(f'  printf("%zu ", sizeof({c}));\n' for c in structs) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(s, n).offset for s in structs.values() for n, _ in s._fields_] + [ctypes.sizeof(s) for s in structs.values()]
    # the binding fills both tables as rows of 64-bit words
    assert ctypes.sizeof(optim.GradientStruct) == 3 * 8 and ctypes.sizeof(optim.TensorStruct) == 7 * 8


P = 0x1000   # a pointer that is never read: every call here is refused
INVALID, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -4


def test_grad_norm_refusals():
    lib = _lib()

    def call(n=1, data=P, count=100, dtype=0, norm=P, ws=P, size=1 << 20, table=True):
        t = (optim.GradientStruct * 1)(optim.GradientStruct(data, count, dtype))
        return lib.okls_grad_norm(n, t if table else None, norm, ws, size, None)
    assert call(n=-1) == INVALID
    assert call(table=False) == INVALID
    assert call(data=None) == INVALID
    assert call(data=P + 2) == INVALID and call(data=P + 1, dtype=1) == INVALID
    assert call(dtype=3) == DTYPE and call(dtype=-1) == DTYPE
    assert call(count=-1) == SHAPE and call(count=(1 << 34) + 1) == SHAPE
    assert call(norm=None) == INVALID and call(norm=P + 1) == INVALID
    assert call(ws=None) == WORKSPACE and call(ws=P + 4) == WORKSPACE and call(size=7) == WORKSPACE
    t = (optim.GradientStruct * 2)(optim.GradientStruct(P, 1, 0), optim.GradientStruct(None, 0, 0))
    assert lib.okls_grad_norm_workspace_size(2, t) == 8
    assert lib.okls_grad_norm_workspace_size(0, None) == 0 and lib.okls_grad_norm_workspace_size(-1, None) == 0


def test_adamw_refusals():
    lib = _lib()

    def call(n=1, t=1, bits=32, norm=None, max_norm=1.0, table=True, config=True, lr=0.1, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1, **over):
        c = optim.ConfigStruct(lr, beta1, beta2, eps, wd, max_norm, bits)
        d = dict(p=P, g=P, m=P, v=P, scales=P if bits == 8 else None, n=100, g_dtype=0)
        d.update(over)
        x = (optim.TensorStruct * 1)(optim.TensorStruct(**d))
        return lib.okls_adamw(ctypes.byref(c) if config else None, t, n, x if table else None, norm, None)
    assert call(config=False) == INVALID and call(table=False) == INVALID and call(n=-1) == INVALID
    assert call(t=0) == INVALID and call(t=-3) == INVALID
    assert call(bits=16) == DTYPE and call(g_dtype=5) == DTYPE
    inf, nan = float("inf"), float("nan")
    for bad in (dict(lr=-1.0), dict(lr=inf), dict(lr=nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta1=nan), dict(beta2=1.0), dict(beta2=nan),
                dict(eps=-1.0), dict(eps=inf), dict(wd=-1.0), dict(wd=nan)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=inf), dict(max_norm=nan)):
        assert call(norm=P, **bad) == INVALID, bad
    assert call(norm=P + 2) == INVALID
    for name in ("p", "g", "m", "v"):
        assert call(**{name: None}) == INVALID and call(**{name: P + 2}) == INVALID
    assert call(g=P + 1, g_dtype=1) == INVALID
    assert call(bits=8, m=None) == INVALID and call(bits=8, scales=None) == INVALID and call(scales=P) == INVALID
    assert call(n=1, **{"bits": 8, "v": None}) == INVALID
    d = dict(p=P, g=P, m=P, v=P, scales=None, g_dtype=0)
    for count in (-1, (1 << 34) + 1):
        x = (optim.TensorStruct * 1)(optim.TensorStruct(n=count, **d))
        assert lib.okls_adamw(ctypes.byref(optim.ConfigStruct(0.1, 0.9, 0.99, 1e-8, 0.1, 0.0, 32)), 1, 1, x, None, None) == SHAPE
    # nothing to do: accepted without a launch
    x = (optim.TensorStruct * 1)(optim.TensorStruct(n=0, p=None, g=None, m=None, v=None, scales=None, g_dtype=0))
    assert lib.okls_adamw(ctypes.byref(optim.ConfigStruct(0.1, 0.9, 0.99, 1e-8, 0.1, 0.0, 32)), 1, 1, x, None, None) == 0
    assert lib.okls_adamw(ctypes.byref(optim.ConfigStruct(0.1, 0.9, 0.99, 1e-8, 0.1, 0.0, 8)), 1, 0, None, None, None) == 0


# ---------------------------------------------------------------------------
# Binding
# ---------------------------------------------------------------------------
def test_binding_refuses_on_the_cpu():
    p, g = torch.zeros(4), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        optim.adamw([p], [g], [optim.new_moments(p)], 1)
    with pytest.raises(ValueError, match="GPU"):
        optim.grad_norm([g])
    with pytest.raises(ValueError, match="must be float32, bfloat16 or float16"):
        optim.grad_norm([g.double()])
    for bad in (lambda: optim.grad_norm([]), lambda: optim.adamw([], [], [], 1), lambda: optim.adamw([p], [], [optim.new_moments(p)], 1),
                lambda: optim.AdamW([]), lambda: optim.AdamW([p.double()]), lambda: optim.AdamW([torch.zeros(4, 6).T]),
                lambda: optim.AdamW([p], moments="4bit")):
        with pytest.raises(ValueError):
            bad()


def test_new_moments_and_checkpoints():
    """Zero moments of both kinds; a checkpoint that does not fit leaves the optimizer as it was."""
    p = torch.zeros(3, 100)
    m = optim.new_moments(p, "8bit")
    assert m.m.dtype == torch.float8_e4m3fn and m.scales.shape == (2, 3) and (m.m.float() == 0).all() and (m.scales.float() == 1).all()
    a, b = optim.AdamW([p, torch.zeros(5)], moments="8bit"), optim.AdamW([p, torch.zeros(5)], moments="8bit")
    a.state[0].m.view(torch.uint8).random_(0, 100)
    a.t, a.lr = 7, 0.5
    sd = a.state_dict()
    b.load_state_dict(sd)
    assert b.t == 7 and b.lr == 0.5 and torch.equal(b.state[0].m.view(torch.uint8), a.state[0].m.view(torch.uint8))
    for wrong in (optim.AdamW([p], moments="8bit"), optim.AdamW([p, torch.zeros(5)]), optim.AdamW([p, torch.zeros(6)], moments="8bit")):
        before = [[x.clone() for x in s if x is not None] for s in wrong.state]
        with pytest.raises(ValueError):
            wrong.load_state_dict(sd)
        assert wrong.t == 0 and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for s, o in zip(wrong.state, before)
                                    for x, y in zip([x for x in s if x is not None], o))
