"""8-bit linear layers around the optimizer: what turns activations and fp32
master weights into a layer's output, and the output's gradient into the
gradient that `okls.OKLS.step` reads.

Binding of the entry points declared in include/okls_linear.h, with the same
rules as `okls`: argument checks and marshalling only, every operator runs in
the HIP library on the current stream, and there is no fallback.

    q, h, rstd = rms_norm(x, norm_weight, residual=r)      # h = x + r; q: normed, in 8 bits
    w, wt = quantize_both(weight)                           # the weight's two 8-bit forms
    y = matmul(q, w)                                        # q w^T
    dq, dt = quantize_both(dy)
    dv = matmul(dq, wt)                                     # the normed values' gradient
    dW = matmul(dt, quantize(h, transpose=True, row_factor=rstd, col_factor=norm_weight),
                dtype=torch.float32)                        # the optimizer's G
    dx, dnorm = rms_norm_backward(dv, h, rstd, norm_weight, dh=dh)

`rms_norm_linear` and `scaled_linear` are these calls as autograd operators, of
first derivatives backward; forward-mode ones are refused.  The single calls record nothing: their results carry no gradient back to inputs that
require one.
"""
from __future__ import annotations

import ctypes
import functools
import operator
from typing import NamedTuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import okls

BLOCK = 128
FORMATS = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
DTYPES = {torch.float32: okls.OKLS_F32, torch.bfloat16: okls.OKLS_BF16, torch.float16: okls.OKLS_F16}
EXPORTED = ("okls_quantize", "okls_scaled_matmul", "okls_scaled_matmul_workspace_size", "okls_rms_norm",
            "okls_rms_norm_backward", "okls_rms_norm_backward_workspace_size")


class BlockedStruct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld", ctypes.c_int64), ("ld_scale", ctypes.c_int64),
                ("format", ctypes.c_int32)]


_lib = None
# The same entry points with plain pointer arguments: what the calls below pass
# is checked by then, and a converted structure pointer costs more than the call.
_fast = {}


def load():
    """The library with this module's entry points declared; raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    lib = okls.load()
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    blk = ctypes.POINTER(BlockedStruct)
    lib.okls_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, blk, blk, vp]
    lib.okls_scaled_matmul.argtypes = [blk, blk, vp, i32, i64, i32, vp, sz, vp]
    lib.okls_scaled_matmul_workspace_size.argtypes = [i64, i64, i64]
    lib.okls_scaled_matmul_workspace_size.restype = sz
    lib.okls_rms_norm.argtypes = [vp, i64, vp, i64, i32, i64, i64, vp, i32, f32, vp, i64, vp, blk, vp]
    lib.okls_rms_norm_backward.argtypes = [vp, i64, vp, i64, vp, vp, i32, vp, i64, i32, i64, i64, vp, i64, vp, vp, sz, vp]
    lib.okls_rms_norm_backward_workspace_size.argtypes = [i64, i64]
    lib.okls_rms_norm_backward_workspace_size.restype = sz
    for name in ("okls_quantize", "okls_scaled_matmul", "okls_rms_norm", "okls_rms_norm_backward"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        _fast[name] = ctypes.CFUNCTYPE(ctypes.c_int, *[vp if t is blk else t for t in fn.argtypes])((name, lib))
    _matmul_workspace.cache_clear()
    _norm_workspace.cache_clear()
    _lib = lib
    return lib


def _up(v, n):
    return (v + n - 1) // n * n


class Blocked:
    """The 8-bit form of a (rows, cols) matrix: along its columns every block of
    128 values of a row shares a power-of-two scale.

    codes:  (rows, ld) float8_e4m3fn or float8_e5m2, ld >= cols rounded up to 128;
            zeros from cols to the end of the last block.
    scales: (ceil(cols / 128), ld_scale) float8_e8m0fnu, [b, r] the scale of block
            b of row r; ld_scale >= rows rounded up to 16 (entries past rows are unused).
    """
    __slots__ = ("_codes", "_scales", "_shape", "_struct", "_address", "_at")

    def __init__(self, codes, scales, shape):
        rows, cols = shape
        self._codes, self._scales, self._shape = codes, scales, (operator.index(rows), operator.index(cols))
        self._struct = self._address = self._at = None

    # read-only: another tensor or shape is another Blocked
    codes = property(operator.attrgetter("_codes"))
    scales = property(operator.attrgetter("_scales"))
    shape = property(operator.attrgetter("_shape"))

    @staticmethod
    def empty(rows, cols, dtype, device):
        if dtype not in FORMATS:
            raise ValueError(f"8-bit dtype must be float8_e4m3fn or float8_e5m2, got {dtype}")
        blocks, ld_scale = -(-cols // BLOCK), (rows + 15) // 16 * 16
        q = Blocked(torch.empty((rows, blocks * BLOCK), dtype=dtype, device=device),
                    torch.empty((blocks, ld_scale), dtype=torch.float8_e8m0fnu, device=device), (rows, cols))
        if q._codes.is_cuda:    # nothing to check in what was laid out here
            q._view(q._codes.data_ptr(), q._scales.data_ptr(), blocks * BLOCK, ld_scale, FORMATS[dtype])
        return q

    def _view(self, codes, scales, ld, ld_scale, fmt):
        self._struct = BlockedStruct(codes, scales, *self._shape, ld, ld_scale, fmt)
        self._address, self._at = ctypes.addressof(self._struct), (codes, scales)

    def struct(self):
        """The checked C view, kept for as long as both tensors stay where they are."""
        c, e = self._codes, self._scales
        codes, scales = c.data_ptr(), e.data_ptr()
        if self._at != (codes, scales):
            rows, cols = self._shape
            fmt = FORMATS.get(c.dtype)
            if fmt is None or e.dtype != torch.float8_e8m0fnu:
                raise ValueError(f"codes must be float8_e4m3fn or float8_e5m2 and scales float8_e8m0fnu, got {c.dtype} and {e.dtype}")
            if not c.is_cuda or c.device != e.device:
                raise ValueError(f"codes on {c.device} and scales on {e.device}: both must be on one GPU")
            cs, es, blocks = c.shape, e.shape, -(-cols // BLOCK)
            if len(cs) != 2 or len(es) != 2 or cs[0] != rows or cs[1] < blocks * BLOCK or es[0] != blocks or es[1] < _up(rows, 16):
                raise ValueError(f"codes {tuple(cs)} and scales {tuple(es)} do not hold a matrix of {rows} x {cols}")
            (ld, inner), (ld_scale, inner_scale) = c.stride(), e.stride()
            if (inner != 1 and rows and cs[1]) or (inner_scale != 1 and blocks and es[1]):
                raise ValueError("codes and scales must be contiguous along their last axis")
            ld = ld if rows > 1 and cs[1] else cs[1]
            ld_scale = ld_scale if blocks > 1 and es[1] else es[1]
            if (ld | ld_scale | codes | scales) % 16:
                raise ValueError("rows of codes and scales must be 16-byte aligned")
            self._view(codes, scales, ld, ld_scale, fmt)
        return self._struct

    def address(self):
        """The address of the checked C view."""
        self.struct()
        return self._address

    def dequantize(self, dtype=torch.float32):
        """The matrix that codes and scales stand for, in torch operations."""
        rows, cols = self.shape
        blocks = -(-cols // BLOCK)
        v = self.codes[:, :blocks * BLOCK].to(torch.float32).reshape(rows, blocks, BLOCK)
        return (v * self.scales[:, :rows].to(torch.float32).T[:, :, None]).reshape(rows, blocks * BLOCK)[:, :cols].to(dtype)


class NormOutput(NamedTuple):
    q: Blocked              # the normed values in 8 bits
    h: torch.Tensor         # x + residual (x itself without one)
    rstd: torch.Tensor      # (rows,) fp32


def _matrix(name, t, like=None):
    """The row stride of a 2-D GPU tensor of a float dtype, contiguous along its rows."""
    if t.dtype not in DTYPES:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if like is not None and (shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} is {tuple(shape)} {t.dtype} on {t.device}, expected {tuple(like.shape)} {like.dtype} on {like.device}")
    rows, cols = shape
    ld, inner = t.stride()
    if cols > 1 and rows and inner != 1:
        raise ValueError(f"{name} must be contiguous along its last axis, strides {t.stride()}")
    if rows <= 1:
        return max(cols, 1)
    if ld < cols:
        raise ValueError(f"{name}'s rows overlap: strides {t.stride()}")
    return ld


def _vector(name, t, n, device):
    if t.dtype not in DTYPES or t.shape != (n,) or t.device != device or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous float vector of {n} on {device}, got {tuple(t.shape)} {t.dtype} on {t.device}")


_raw_stream = torch._C._cuda_getCurrentRawStream     # current_stream(device).cuda_stream without the Stream object
_written = torch.autograd.graph.increment_version    # tells autograd of a write that went through data_ptr


@functools.lru_cache(maxsize=4096)
def _matmul_workspace(m, n, k):
    return load().okls_scaled_matmul_workspace_size(m, n, k)


@functools.lru_cache(maxsize=4096)
def _norm_workspace(rows, cols):
    return load().okls_rms_norm_backward_workspace_size(rows, cols)


def _call(name, device, *args):
    """One library call on the current stream of `device`."""
    if _lib is None:
        load()
    fn, index = _fast[name], device.index
    if index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st != okls.OKLS_OK:
        raise okls.OKLSError(name, st)


def _quantize(x, along_cols, along_rows, row_factor, col_factor, ldx=None):
    if ldx is None:
        ldx = _matrix("x", x)
    rows, cols = x.shape
    if (row_factor is None) != (col_factor is None):
        raise ValueError("row_factor and col_factor come together")
    rf = cf = None
    cdt = 0
    if row_factor is not None:
        _vector("row_factor", row_factor, rows, x.device)
        _vector("col_factor", col_factor, cols, x.device)
        if row_factor.dtype != torch.float32:
            raise ValueError(f"row_factor must be float32, got {row_factor.dtype}")
        rf, cf, cdt = row_factor.data_ptr(), col_factor.data_ptr(), DTYPES[col_factor.dtype]
    _call("okls_quantize", x.device, x.data_ptr(), DTYPES[x.dtype], rows, cols, ldx, rf, cf, cdt,
          along_cols.address() if along_cols is not None else None,
          along_rows.address() if along_rows is not None else None)


def quantize(x, dtype=torch.float8_e4m3fn, transpose=False, row_factor=None, col_factor=None) -> Blocked:
    """The 8-bit form of the matrix x, or of its transpose (blocks of 128 along
    x's rows).  With row_factor (rows, float32) and col_factor (cols), of
    fl32(fl32(x row_factor) col_factor): a norm's output formed again from h,
    rstd and the norm's weight."""
    ldx = _matrix("x", x)
    rows, cols = x.shape
    q = Blocked.empty(cols, rows, dtype, x.device) if transpose else Blocked.empty(rows, cols, dtype, x.device)
    _quantize(x, None if transpose else q, q if transpose else None, row_factor, col_factor, ldx)
    return q


def quantize_both(x, dtype=torch.float8_e4m3fn, row_factor=None, col_factor=None):
    """The 8-bit forms of x and of its transpose, from one read of x."""
    ldx = _matrix("x", x)
    rows, cols = x.shape
    q, t = Blocked.empty(rows, cols, dtype, x.device), Blocked.empty(cols, rows, dtype, x.device)
    _quantize(x, q, t, row_factor, col_factor, ldx)
    return q, t


def matmul(a: Blocked, b: Blocked, dtype=torch.bfloat16, out=None, accumulate=False):
    """a b^T for a (m, k) and b (n, k) in 8 bits: (m, n) of `dtype`, or into
    `out` (of its own dtype); accumulate=True adds to what `out` holds.  Autograd
    sees the write; an `out` that requires a gradient is refused while it records.

    A float32 result sums the exact products in fp32.  A 16-bit result is summed
    in fp32 and rounded once, but from each eight products the 8-bit matrix
    instructions drop what lies below 2^-13 of the largest of them: about 1.6e-5
    of a result in norm, up to 2^-10 of the sum of the products' sizes in an
    element whose large products cancel.  Where that counts, take a float32
    result and cast it."""
    pa, pb = a.address(), b.address()
    (m, k), (n, kb) = a.shape, b.shape
    device = a.codes.device
    if kb != k:
        raise ValueError(f"a is {a.shape} and b is {b.shape}: the second sizes must be equal")
    if b.codes.device != device:
        raise ValueError(f"a is on {device}, b on {b.codes.device}")
    given = out is not None
    if not given:
        if accumulate:
            raise ValueError("accumulate needs out")
        if dtype not in DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        out = torch.empty((m, n), dtype=dtype, device=device)
        ldc = n
    else:
        ldc = _matrix("out", out)
        if tuple(out.shape) != (m, n) or out.device != device:
            raise ValueError(f"out is {tuple(out.shape)} on {out.device}, the product is {(m, n)} on {device}")
        if out.requires_grad and torch.is_grad_enabled():
            raise ValueError("out requires a gradient, and this product has none: write to it under torch.no_grad()")
    need = _matmul_workspace(m, n, k)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call("okls_scaled_matmul", device, pa, pb, out.data_ptr(), DTYPES[out.dtype], ldc, 1 if accumulate else 0,
          ws.data_ptr() if need else None, need)
    if given:       # a graph that kept it has to know, as of torch's own writes
        _written((out,))
    return out


def rms_norm(x, weight, residual=None, eps=1e-6, dtype=torch.float8_e4m3fn) -> NormOutput:
    """Root-mean-square norm of h = x + residual over the last axis, times
    `weight`, in 8 bits; with h and 1/rms for the way back."""
    ldx = _matrix("x", x)
    rows, cols = x.shape
    _vector("weight", weight, cols, x.device)
    h, ldr, ldh = x, 0, 0
    if residual is not None:
        ldr = _matrix("residual", residual, x)
        h = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
        ldh = cols
    q = Blocked.empty(rows, cols, dtype, x.device)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    _call("okls_rms_norm", x.device, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
          DTYPES[x.dtype], rows, cols, weight.data_ptr(), DTYPES[weight.dtype], eps,
          None if residual is None else h.data_ptr(), ldh, rstd.data_ptr(), q.address())
    return NormOutput(q, h, rstd)


def rms_norm_backward(dy, h, rstd, weight, dh=None):
    """(dx, dweight) of the norm: dy the gradient of its output, dh that of h
    itself.  dx is the gradient of x and of the residual alike, in h's dtype;
    dweight has weight's dtype."""
    ldh = _matrix("h", h)
    lddy = _matrix("dy", dy, h)
    rows, cols = h.shape
    _vector("weight", weight, cols, h.device)
    _vector("rstd", rstd, rows, h.device)
    if rstd.dtype != torch.float32:
        raise ValueError(f"rstd must be float32, got {rstd.dtype}")
    lddh = _matrix("dh", dh, h) if dh is not None else 0
    dx = torch.empty((rows, cols), dtype=h.dtype, device=h.device)
    dweight = torch.empty(cols, dtype=weight.dtype, device=h.device)
    need = _norm_workspace(rows, cols)
    ws = torch.empty(need, dtype=torch.uint8, device=h.device) if need else None
    _call("okls_rms_norm_backward", h.device, dy.data_ptr(), lddy, h.data_ptr(), ldh, rstd.data_ptr(),
          weight.data_ptr(), DTYPES[weight.dtype], None if dh is None else dh.data_ptr(), lddh, DTYPES[h.dtype],
          rows, cols, dx.data_ptr(), cols, dweight.data_ptr(), ws.data_ptr() if need else None, need)
    return dx, dweight


# --------------------------------------------------------------------------
# Autograd
# --------------------------------------------------------------------------
def _no_tangents(*tensors):
    """Refuses forward-mode derivatives, which no operator of the library has: a tensor that carries
    a tangent need not require a gradient, and a result without one would count as a constant."""
    if forward_ad._current_level >= 0 and any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError("this operator has no forward-mode derivative")


class _NormLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, norm_weight, weight, eps, grad_dtype):
        q, h, rstd = rms_norm(x, norm_weight, residual=residual, eps=eps)
        w, wt = quantize_both(weight)
        y = matmul(q, w, dtype=x.dtype)
        ctx.save_for_backward(h, rstd, norm_weight, wt.codes, wt.scales)
        ctx.wt_shape, ctx.weight_dtype, ctx.grad_dtype, ctx.joined = wt.shape, weight.dtype, grad_dtype, residual is not None
        ctx.set_materialize_grads(False)
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable     # the kernels below have no gradients of their own
    def backward(ctx, dy, dh=None):
        h, rstd, norm_weight, wt_codes, wt_scales = ctx.saved_tensors
        need_x, need_r, need_n, need_w = ctx.needs_input_grad[:4]
        if dy is None:      # only the residual stream went on
            return dh if need_x else None, dh if need_r else None, None, None, None, None
        _no_tangents(dy, dh)
        dy = _rows(dy)
        dx = dnorm = dweight = None
        if need_w:
            dq, dt = quantize_both(dy, dtype=ctx.grad_dtype)
            v = quantize(h, transpose=True, row_factor=rstd, col_factor=norm_weight)
            dweight = matmul(dt, v, dtype=ctx.weight_dtype)
        else:
            dq = quantize(dy, dtype=ctx.grad_dtype)
        if need_x or need_r or need_n:
            dv = matmul(dq, Blocked(wt_codes, wt_scales, ctx.wt_shape), dtype=h.dtype)
            dx, dnorm = rms_norm_backward(dv, h, rstd, norm_weight, dh=_rows(dh))
        return dx if need_x else None, dx if need_r else None, dnorm if need_n else None, dweight, None, None


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, grad_dtype):
        need_x, need_w = ctx.needs_input_grad[:2]
        q, t = quantize_both(x) if need_w else (quantize(x), None)
        w, wt = quantize_both(weight) if need_x else (quantize(weight), None)
        kept = [b for b in (t, wt) if b is not None]
        ctx.save_for_backward(*[s for b in kept for s in (b.codes, b.scales)])
        ctx.shapes, ctx.dtypes, ctx.grad_dtype = [b.shape for b in kept], (x.dtype, weight.dtype), grad_dtype
        return matmul(q, w, dtype=x.dtype)

    @staticmethod
    @once_differentiable     # the kernels below have no gradients of their own
    def backward(ctx, dy):
        _no_tangents(dy)
        need_x, need_w = ctx.needs_input_grad[:2]
        saved = ctx.saved_tensors
        kept = [Blocked(saved[2 * i], saved[2 * i + 1], s) for i, s in enumerate(ctx.shapes)]
        dy, dx, dweight = _rows(dy), None, None
        if need_x and need_w:
            dq, dt = quantize_both(dy, dtype=ctx.grad_dtype)
        else:
            dq = dt = quantize(dy, dtype=ctx.grad_dtype, transpose=need_w)
        if need_w:
            dweight = matmul(dt, kept[0], dtype=ctx.dtypes[1])
        if need_x:
            dx = matmul(dq, kept[-1], dtype=ctx.dtypes[0])
        return dx, dweight, None


def _rows(t):
    """A gradient as autograd hands it over may be expanded or transposed; the kernels read rows."""
    if t is None:
        return t
    rows, cols = t.shape
    if (cols <= 1 or t.stride(1) == 1) and (rows <= 1 or t.stride(0) >= cols):
        return t
    return t.contiguous()


def rms_norm_linear(x, norm_weight, weight, residual=None, eps=1e-6, grad_dtype=torch.float8_e4m3fn):
    """(y, h): h = x + residual (x without one) and y = rms_norm(h) weight^T for x
    (tokens, k) and weight (n, k), y in x's dtype.  The products run in 8 bits
    (e4m3; the output's gradient in grad_dtype); gradients pass the rounding
    straight through, and weight's comes in weight's dtype: the G of its
    optimizer step.  y, and the gradient that goes back through the norm, are
    summed as `matmul` sums x's dtype: what 16-bit results drop there also
    reaches the gradients of x, of the residual and of norm_weight."""
    if residual is None:
        return _NormLinear.apply(x, None, norm_weight, weight, eps, grad_dtype), x
    return _NormLinear.apply(x, residual, norm_weight, weight, eps, grad_dtype)


def scaled_linear(x, weight, grad_dtype=torch.float8_e4m3fn):
    """x weight^T for x (tokens, k) and weight (n, k) in 8-bit products, in x's
    dtype, with the gradients of both.  The result and x's gradient are summed as
    `matmul` sums x's dtype, weight's gradient as it sums weight's.  weight is
    brought to 8 bits in every call; to serve, keep `quantize(weight)` and call
    `matmul`."""
    return _Linear.apply(x, weight, grad_dtype)
