"""8-bit linear-layer operators on the CPU: the oracle's own pins, and every
refusal of the C ABI and of the binding (all return before a launch)."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from kronecker_factored_second_amd import linear, okls
from oracle import linear_oracle as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _lib():
    if not os.path.exists(okls.LIB_PATH):
        pytest.skip("libokls.so not built")
    return linear.load()


# ---------------------------------------------------------------------------
# Oracle
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_rounding_is_the_formats(fmt):
    """Every representable value stays, midpoints go to the even code, and torch's cast agrees."""
    codes = torch.arange(256, dtype=torch.uint8).view(F8[fmt]).double().numpy()
    fin = np.unique(codes[np.isfinite(codes)])
    assert np.array_equal(L.round8(fin, fmt), fin)
    mid = (fin[1:] + fin[:-1]) / 2
    near = np.concatenate([mid, np.nextafter(mid, np.inf), np.nextafter(mid, -np.inf)]).astype(np.float32)
    want = torch.from_numpy(near).to(F8[fmt]).double().numpy()
    assert np.array_equal(L.round8(near, fmt), want)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scale_is_the_smallest_that_holds_the_block(fmt):
    big = L.FORMATS[fmt][0]
    for top in (1.0, big, np.nextafter(big, np.inf), 1.75, 1.7500001, 3.4e38, 2.0 ** -149, 2.0 ** -100):
        e = L.scale_exponent(top, fmt)
        assert top <= np.ldexp(big, e) and (e == -127 or top > np.ldexp(big, e - 1))
    assert L.scale_exponent(0.0, fmt) == 0


def test_held_values_are_near():
    """A rounding is off by half a step at most: eps / 2 of the value, or half the smallest step of its block."""
    rng = np.random.default_rng(0)
    v = rng.standard_normal((7, 300)) * np.exp(2 * rng.standard_normal((7, 1)))
    for fmt, (_, frac, low) in L.FORMATS.items():
        codes, scales = L.quantize(v, fmt)
        held = L.dequantize(codes, scales)
        step = np.repeat(scales.T, 128, 1)[:, :300] * 2.0 ** (low - frac)
        assert (np.abs(held - v) <= np.maximum(np.abs(v) * 2.0 ** -(frac + 1), step / 2)).all()


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, w, dy = rng.standard_normal((3, 17)), rng.standard_normal(17), rng.standard_normal((3, 17))
    eps = 1e-3
    dx, dw, _ = L.norm_backward(dy, x, L.rms(x, eps), w)
    d = 1e-6
    for i in range(3):
        for j in range(17):
            e = np.zeros_like(x)
            e[i, j] = d
            num = np.sum(dy * (L.norm_value(x + e, w, eps) - L.norm_value(x - e, w, eps))) / (2 * d)
            # central differences: rounding 1e-16 / d and curvature d^2, of values of order 10
            assert abs(num - dx[i, j]) < 1e-8
    for j in range(17):
        e = np.zeros_like(w)
        e[j] = d
        num = np.sum(dy * (L.norm_value(x, w + e, eps) - L.norm_value(x, w - e, eps))) / (2 * d)
        assert abs(num - dw[j]) < 1e-8


# ---------------------------------------------------------------------------
# ABI
# ---------------------------------------------------------------------------
def test_header_symbols_and_struct(tmp_path):
    lib = _lib()
    header = open(os.path.join(ROOT, "include", "okls_linear.h")).read()
    declared = set(re.findall(r"\b(okls_[a-z_]+)\s*\(", header))
    assert declared - {"okls_blocked"} == set(linear.EXPORTED)
    for name in linear.EXPORTED:
        assert hasattr(lib, name)
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [n for n, _ in linear.BlockedStruct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "okls_linear.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu ", offsetof(okls_blocked, {n}));\n' for n in names)
                   + '  printf("%zu", sizeof(okls_blocked));\n  return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(linear.BlockedStruct, n).offset for n in names] + [ctypes.sizeof(linear.BlockedStruct)]


P = 0x1000   # a pointer that is never read: every call here is refused


def _blk(rows, cols, **over):
    d = dict(codes=P, scales=P, rows=rows, cols=cols, ld=-(-cols // 128) * 128, ld_scale=-(-rows // 16) * 16, format=0)
    d.update(over)
    return linear.BlockedStruct(**d)


INVALID, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -4


@pytest.mark.parametrize("over,status", [
    (dict(format=2), DTYPE), (dict(format=-1), DTYPE), (dict(rows=9), SHAPE), (dict(cols=301), SHAPE),
    (dict(ld=256), SHAPE), (dict(ld=392), SHAPE), (dict(ld_scale=8), SHAPE), (dict(ld_scale=24), SHAPE),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(codes=P + 8), INVALID), (dict(scales=P + 1), INVALID)])
def test_blocked_refusals(over, status):
    lib = _lib()
    q = _blk(**{"rows": 8, "cols": 300, **over})
    assert lib.okls_quantize(P, 0, 8, 300, 300, None, None, 0, q, None, None) == status
    assert lib.okls_rms_norm(P, 300, None, 0, 0, 8, 300, P, 0, 1e-6, None, 0, P, q, None) == status
    if "rows" not in over and "cols" not in over:      # a product takes its sizes from the operands
        assert lib.okls_scaled_matmul(q, _blk(4, 300), P, 0, 4, 0, None, 0, None) == status


def test_quantize_refusals():
    lib, q = _lib(), _blk(8, 300)
    call = lambda x=P, dt=0, rows=8, cols=300, ld=300, rf=None, cf=None, cdt=0, a=q, b=None: \
        lib.okls_quantize(x, dt, rows, cols, ld, rf, cf, cdt, a, b, None)  # noqa: E731
    assert call(a=None) == INVALID
    assert call(x=None) == INVALID
    assert call(x=P + 2) == INVALID               # a float at an odd place
    assert call(ld=299) == INVALID                # rows overlap
    assert call(dt=3) == DTYPE
    assert call(rows=-1) == SHAPE
    assert call(rows=(1 << 30) + 1) == SHAPE
    assert call(rf=P) == INVALID and call(cf=P) == INVALID
    assert call(rf=P, cf=P, cdt=7) == DTYPE
    assert call(rf=P + 1, cf=P) == INVALID
    assert call(a=None, b=q) == SHAPE             # the transposed form is 300 x 8
    # nothing to do: accepted without a launch
    assert call(rows=0, a=_blk(0, 300), x=None) == 0


def test_matmul_refusals():
    lib = _lib()
    a, b = _blk(8, 300), _blk(20, 300)
    call = lambda a=a, b=b, c=P, dt=0, ld=20, acc=0, ws=None, n=0: lib.okls_scaled_matmul(a, b, c, dt, ld, acc, ws, n, None)  # noqa: E731
    assert call(a=None) == INVALID and call(b=None) == INVALID
    assert call(b=_blk(20, 301)) == SHAPE
    assert call(c=None) == INVALID
    assert call(c=P + 2) == INVALID
    assert call(ld=19) == INVALID
    assert call(dt=5) == DTYPE
    assert call(acc=2) == INVALID
    big = 1 << 20
    assert call(a=_blk(big, 300), b=_blk(big, 300), ld=big) == SHAPE    # 2^40 outputs
    assert call(a=_blk(0, 300)) == 0 and call(b=_blk(0, 300)) == 0
    for m, n, k in ((8, 20, 300), (1, 4096, 16384), (300, 300, 100000)):
        need = lib.okls_scaled_matmul_workspace_size(m, n, k)
        if need:
            x, y = _blk(m, k), _blk(n, k)
            assert call(a=x, b=y, ld=n) == WORKSPACE
            assert call(a=x, b=y, ld=n, ws=P, n=need - 1) == WORKSPACE
            assert call(a=x, b=y, ld=n, ws=P + 4, n=need) == WORKSPACE
    assert lib.okls_scaled_matmul_workspace_size(-1, 1, 1) == 0


def test_rms_norm_refusals():
    lib, q = _lib(), _blk(8, 300)
    call = lambda x=P, ldx=300, r=None, ldr=300, dt=0, rows=8, cols=300, w=P, wdt=0, eps=1e-6, h=None, ldh=300, rs=P, o=q: \
        lib.okls_rms_norm(x, ldx, r, ldr, dt, rows, cols, w, wdt, eps, h, ldh, rs, o, None)  # noqa: E731
    assert call(o=None) == INVALID
    assert call(x=None) == INVALID and call(w=None) == INVALID and call(rs=None) == INVALID
    assert call(h=P) == INVALID                   # no residual: h is x
    assert call(r=P) == INVALID                   # a residual needs h
    assert call(r=P, h=P, ldr=299) == INVALID and call(r=P, h=P, ldh=299) == INVALID
    assert call(ldx=299) == INVALID and call(x=P + 2) == INVALID
    assert call(dt=4) == DTYPE and call(wdt=4) == DTYPE
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(cols=0) == SHAPE and call(rows=-1) == SHAPE
    assert call(rows=0, o=_blk(0, 300), x=None) == 0


def test_rms_norm_backward_refusals():
    lib = _lib()
    need = lib.okls_rms_norm_backward_workspace_size(8, 300)
    call = lambda dy=P, ldy=300, h=P, ldh=300, rs=P, w=P, wdt=0, dh=None, ldd=300, dt=0, rows=8, cols=300, dx=P, ldx=300, dw=P, ws=P, n=need: \
        lib.okls_rms_norm_backward(dy, ldy, h, ldh, rs, w, wdt, dh, ldd, dt, rows, cols, dx, ldx, dw, ws, n, None)  # noqa: E731
    for k in ("dy", "h", "rs", "w", "dx", "dw"):
        assert call(**{k: None}) == INVALID, k
    for k in ("ldy", "ldh", "ldx"):
        assert call(**{k: 299}) == INVALID, k
    assert call(dh=P, ldd=299) == INVALID and call(dh=P + 2) == INVALID
    assert call(dt=3) == DTYPE and call(wdt=-1) == DTYPE
    assert call(rows=-1) == SHAPE and call(cols=0) == SHAPE
    if need:
        assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE and call(ws=P + 4) == WORKSPACE


# ---------------------------------------------------------------------------
# Binding
# ---------------------------------------------------------------------------
def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 128)
    w = torch.ones(128)
    for f in (lambda: linear.quantize(x), lambda: linear.quantize_both(x), lambda: linear.rms_norm(x, w),
              lambda: linear.rms_norm_backward(x, x, torch.ones(4), w), lambda: linear.quantize(x.double()),
              lambda: linear.quantize(x[0]), lambda: linear.quantize(x, dtype=torch.int8)):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("codes,scales,shape", [
    (torch.zeros(4, 128), torch.zeros(1, 16, dtype=torch.uint8), (4, 128)),
    (torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.ones(1, 16).to(torch.float8_e8m0fnu), (4, 128)),   # on the CPU
])
def test_blocked_struct_refuses(codes, scales, shape):
    with pytest.raises(ValueError):
        linear.Blocked(codes, scales, shape).struct()


def test_empty_blocked_and_dequantize():
    q = linear.Blocked.empty(5, 300, torch.float8_e5m2, "cpu")
    assert tuple(q.codes.shape) == (5, 384) and tuple(q.scales.shape) == (3, 16)
    with pytest.raises(ValueError):
        linear.Blocked.empty(5, 300, torch.float16, "cpu")
    v = np.random.default_rng(2).standard_normal((5, 300))
    codes, scales = L.quantize(v, "e5m2")
    q.codes.zero_()
    q.codes[:, :300] = torch.from_numpy(codes).to(torch.float8_e5m2)
    q.scales[:, :5] = torch.from_numpy(scales).to(torch.float8_e8m0fnu)
    assert np.array_equal(q.dequantize(torch.float64).numpy(), L.dequantize(codes, scales))


@pytest.mark.parametrize("m,n", [(1, 1), (5, 1), (0, 1), (1, 4), (5, 4), (5, 0)])
def test_gradients_reach_the_kernels_as_rows(m, n):
    """Any layout in which autograd hands a gradient over: expanded, transposed, strided, as it lies; one column is no exception."""
    base = torch.arange(2.0 * (m + 1) * (n + 3)).reshape(2 * (m + 1), n + 3)
    for t in (torch.ones(1).expand(m, n), base[:m, :n], base[:2 * m:2, :n], base.T[:n, :m].T, base[:1, :n].expand(m, n),
              torch.ones(m, 1).expand(m, n)):
        got = linear._rows(t)
        assert torch.equal(got, t)
        assert (n <= 1 or got.stride(1) == 1) and (m <= 1 or got.stride(0) >= n)
    whole = torch.zeros(m, n + 3)[:, :n]
    assert linear._rows(whole) is whole and linear._rows(None) is None      # nothing is copied that need not be


def test_blocked_is_fixed():
    """Its tensors and shape cannot be replaced under the C view that is kept of them, nor changed through the caller's list."""
    shape = [5, 300]
    q = linear.Blocked(torch.zeros(5, 384).to(torch.float8_e4m3fn), torch.ones(3, 16).to(torch.float8_e8m0fnu), shape)
    for name, other in (("codes", q.codes.clone()), ("scales", q.scales.clone()), ("shape", (4, 300))):
        with pytest.raises(AttributeError):
            setattr(q, name, other)
    shape[0] = 500
    assert q.shape == (5, 300)
    with pytest.raises(TypeError):
        linear.Blocked(q.codes, q.scales, (5, 300.5))


def test_blocked_view_follows_its_tensors():
    """A tensor that was moved in place (set_, .data) is checked again and read where it is.  The first view is set as the kernels' outputs have it."""
    q = linear.Blocked.empty(5, 300, torch.float8_e4m3fn, "cpu")
    q._view(q.codes.data_ptr(), q.scales.data_ptr(), 384, 16, 0)
    first = q.struct()
    assert q.struct() is first and q.address() == ctypes.addressof(first)
    q.codes.data = q.codes.clone()
    with pytest.raises(ValueError, match="GPU"):        # checked anew: these tensors are on the CPU
        q.struct()
    with pytest.raises(ValueError, match="GPU"):
        q.address()
