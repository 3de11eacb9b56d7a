"""Operators around a stack of experts' matrices: tokens sorted by the experts that
they chose and back, with weights applied, and the experts' 8-bit products, whose
weight gradient is the 3-D gradient that `okls.OKLS.step` reads.

Binding of the entry points declared in include/okls_experts.h, with the same
rules as `okls` and `linear`: argument checks and marshalling only, every operator
runs in the HIP library on the current stream, nothing waits for the device, and
there is no fallback.

    best, choice = router(x).topk(2)                        # (tokens, 2)
    order = plan(choice, n_experts)
    h = token_linear(x, gate_up, order)                     # (order.capacity, n), gate_up (n_experts, n, k)
    y = linear(act(h), down, order)
    out = combine(y, best.softmax(1), order)                # (tokens, k)

`gather`, `combine`, `linear` and `token_linear` are autograd operators, of first
derivatives backward; forward-mode ones are refused.  To serve,
keep `quantize_stack(weight)` and call `plan` with align=16, `quantize_rows` and
`matmul`, which record no gradient.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import linear as _dense
from . import okls
from .linear import Blocked, BlockedStruct, DTYPES, _matrix, _no_tangents, _rows, _up

EXPORTED = ("okls_experts_capacity", "okls_experts_plan_workspace_size", "okls_experts_plan", "okls_experts_gather",
            "okls_experts_combine", "okls_experts_combine_backward", "okls_experts_quantize_rows",
            "okls_experts_quantize_stack", "okls_experts_matmul", "okls_experts_weight_grad")
MAX_EXPERTS = 512
ALIGNS = (16, 32, 64, 128)
MAX_SUMMED = (1 << 24) - 128    # of a product's axis: its rows of codes lie less than 2^24 bytes apart


class PlanStruct(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("pairs", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("tokens", ctypes.c_int64), ("each", ctypes.c_int64), ("capacity", ctypes.c_int64),
                ("n_experts", ctypes.c_int32), ("align", ctypes.c_int32)]


_lib = None
_fast = {}


def load():
    """The library with this module's entry points declared; raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    lib = okls.load()
    _dense.load()
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    plan, blk = ctypes.POINTER(PlanStruct), ctypes.POINTER(BlockedStruct)
    lib.okls_experts_capacity.argtypes = [i64, i64, i32, i32]
    lib.okls_experts_capacity.restype = i64
    lib.okls_experts_plan_workspace_size.argtypes = [i64, i64, i32]
    lib.okls_experts_plan_workspace_size.restype = sz
    lib.okls_experts_plan.argtypes = [vp, i32, plan, vp, sz, vp]
    lib.okls_experts_gather.argtypes = [plan, vp, i64, i32, i64, vp, i64, vp]
    lib.okls_experts_combine.argtypes = [plan, vp, i64, i32, i64, vp, i32, vp, i64, vp]
    lib.okls_experts_combine_backward.argtypes = [plan, vp, i64, vp, i64, i32, i64, vp, i32, vp, i64, vp, vp]
    lib.okls_experts_quantize_rows.argtypes = [plan, vp, i64, i32, i64, i32, blk, blk, vp]
    lib.okls_experts_quantize_stack.argtypes = [vp, i32, i32, i64, i64, i64, i64, blk, blk, vp]
    lib.okls_experts_matmul.argtypes = [plan, blk, blk, i64, vp, i32, i64, vp]
    lib.okls_experts_weight_grad.argtypes = [plan, blk, blk, vp, i32, i64, vp]
    for name in EXPORTED[2:]:
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        _fast[name] = ctypes.CFUNCTYPE(ctypes.c_int, *[vp if t in (plan, blk) else t for t in fn.argtypes])((name, lib))
    _lib = lib
    return lib


def _call(name, device, *args):
    """One library call on the current stream of `device`."""
    if _lib is None:
        load()
    fn, index = _fast[name], device.index
    if index == torch.cuda.current_device():
        st = fn(*args, _dense._raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _dense._raw_stream(index))
    if st != okls.OKLS_OK:
        raise okls.OKLSError(name, st)


def capacity(tokens, each, n_experts, align=128) -> int:
    """The rows of the sorted order of tokens * each choices: enough for any of them."""
    if align not in ALIGNS:
        raise ValueError(f"align must be one of {ALIGNS}, got {align}")
    if not 1 <= n_experts <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, got {n_experts}")
    if tokens < 0 or each < 1 or tokens > 1 << 28 or each > 1 << 28 or tokens * each > 1 << 28:
        raise ValueError(f"at most 2^28 choices, at least one a token, got {tokens} x {each}")
    pairs = tokens * each
    return (pairs + min(pairs, n_experts) * (align - 1)) // align * align


class Plan:
    """The sorted order of tokens' choices.

    rows (tokens, each) int32: the row of each choice, -1 for a dropped one.
    pairs (capacity) int32: the choice t * each + k of each row, -1 for a row without one.
    offsets (n_experts + 1) int32: each expert's first row, multiples of `align`.
    counts (n_experts) int32: each expert's choices; its other rows hold zeros.

    Autograd's operators keep the plan, not copies: a torch operation that writes into its
    tensors between a forward and its backward pass makes the second raise.  A captured
    graph's replay is not seen: its plan belongs to that graph's own backward pass.
    """
    __slots__ = ("_tensors", "_counted", "_at", "align", "capacity", "tokens", "each", "n_experts", "device", "_struct", "_address")

    rows = property(lambda self: self._tensors[0])
    pairs = property(lambda self: self._tensors[1])
    offsets = property(lambda self: self._tensors[2])
    counts = property(lambda self: self._tensors[3])

    def __init__(self, rows, pairs, offsets, counts, align=128):
        if rows.dim() != 2 or pairs.dim() != 1 or offsets.dim() != 1 or counts.dim() != 1:
            raise ValueError(f"rows {tuple(rows.shape)} must be 2-D, pairs {tuple(pairs.shape)}, offsets {tuple(offsets.shape)} "
                             f"and counts {tuple(counts.shape)} 1-D")
        for name, t in (("rows", rows), ("pairs", pairs), ("offsets", offsets), ("counts", counts)):
            if t.dtype != torch.int32 or not t.is_cuda or t.device != rows.device or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous int32 on one GPU, got {t.dtype} on {t.device}")
        tokens, each = rows.shape
        n_experts = counts.shape[0]
        room = capacity(tokens, each, n_experts, align)
        if pairs.shape[0] != room or offsets.shape[0] != n_experts + 1:
            raise ValueError(f"pairs {tuple(pairs.shape)} and offsets {tuple(offsets.shape)} do not hold the order of {tokens} x {each} "
                             f"choices of {n_experts} experts: {room} rows")
        self._set(rows, pairs, offsets, counts, align, room, tokens, each, n_experts)

    def _set(self, rows, pairs, offsets, counts, align, room, tokens, each, n_experts):
        self._tensors = rows, pairs, offsets, counts
        self._counted = [t for t in self._tensors if not t.is_inference()]       # those hold no count of writes
        self._at = rows.data_ptr(), pairs.data_ptr(), offsets.data_ptr(), counts.data_ptr()
        self.align, self.capacity, self.tokens, self.each, self.n_experts, self.device = align, room, tokens, each, n_experts, rows.device
        self._struct = PlanStruct(*self._at, tokens, each, room, n_experts, align)
        self._address = ctypes.addressof(self._struct)

    def address(self):
        """The address of the C view, of the tensors as they lie now."""
        rows, pairs, offsets, counts = self._tensors
        at = rows.data_ptr(), pairs.data_ptr(), offsets.data_ptr(), counts.data_ptr()
        if at != self._at:
            if (rows.numel(), pairs.numel(), offsets.numel(), counts.numel()) != (self.tokens * self.each, self.capacity, self.n_experts + 1, self.n_experts):
                raise ValueError(f"the plan's tensors changed their sizes: rows {tuple(rows.shape)}, pairs {tuple(pairs.shape)}, "
                                 f"offsets {tuple(offsets.shape)}, counts {tuple(counts.shape)}")
            s, self._at = self._struct, at
            s.rows, s.pairs, s.offsets, s.counts = at
        return self._address

    def _versions(self):
        """How often torch has written to each tensor in place."""
        return [t._version for t in self._counted]


def plan(choice, n_experts, align=128) -> Plan:
    """The sorted order of choice (tokens, each), integers of which those outside
    0 .. n_experts - 1 are dropped.  align=128 for everything; align=16, 32 or 64
    leaves fewer rows empty where no weight gradient is wanted."""
    if choice.dim() != 2 or choice.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"choice must be 2-D int32 or int64, got {tuple(choice.shape)} {choice.dtype}")
    tokens, each = choice.shape
    room = capacity(tokens, each, n_experts, align)
    if not choice.is_cuda:
        raise ValueError(f"choice must be on a GPU, got {choice.device}")
    choice, device = choice.contiguous(), choice.device
    pairs = tokens * each
    # one allocation: rows, pairs, offsets, counts
    held = torch.empty(pairs + room + 2 * n_experts + 1, dtype=torch.int32, device=device)
    rows, by_row, offsets, counts = held.split((pairs, room, n_experts + 1, n_experts))
    p = Plan.__new__(Plan)
    p._set(rows.view(tokens, each), by_row, offsets, counts, align, room, tokens, each, n_experts)
    need = (_lib or load()).okls_experts_plan_workspace_size(tokens, each, n_experts)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _call("okls_experts_plan", device, choice.data_ptr(), 32 if choice.dtype == torch.int32 else 64, p._address,
          ws.data_ptr() if need else None, need)
    return p


class Stack:
    """The 8-bit form of n_experts matrices (n, k): one `linear.Blocked` of
    n_experts * (n rounded up to 16) rows, expert e's from row e * (n rounded up to 16) on."""
    __slots__ = ("blocked", "shape")

    def __init__(self, codes, scales, shape):
        e, n, k = (int(v) for v in shape)
        self.shape = (e, n, k)
        self.blocked = Blocked(codes, scales, (e * _up(n, 16), k))

    @staticmethod
    def empty(shape, dtype, device):
        e, n, k = shape
        b = Blocked.empty(e * _up(n, 16), k, dtype, device)
        s = Stack.__new__(Stack)
        s.blocked, s.shape = b, (e, n, k)
        return s

    def dequantize(self, dtype=torch.float32):
        """The matrices that codes and scales stand for, in torch operations."""
        e, n, k = self.shape
        return self.blocked.dequantize(dtype).view(e, _up(n, 16), k)[:, :n]


def _sorted(name, t, order, rows):
    """The row stride of a tensor of `rows` rows on the plan's device."""
    ld = _matrix(name, t)
    if t.shape[0] != rows or t.device != order.device:
        raise ValueError(f"{name} is {tuple(t.shape)} on {t.device}, the plan has {rows} rows on {order.device}")
    return ld


def _weights(weights, order):
    if weights.dtype not in DTYPES or tuple(weights.shape) != (order.tokens, order.each) or weights.device != order.device:
        raise ValueError(f"weights must be float {(order.tokens, order.each)} on {order.device}, got {tuple(weights.shape)} {weights.dtype} on {weights.device}")
    return weights.contiguous()


def _gather(x, order):
    ldx = _sorted("x", x, order, order.tokens)
    cols = x.shape[1]
    out = torch.empty((order.capacity, cols), dtype=x.dtype, device=x.device)
    _call("okls_experts_gather", x.device, order.address(), x.data_ptr(), ldx, DTYPES[x.dtype], cols, out.data_ptr(), max(cols, 1))
    return out


def _combine(y, weights, order):
    ldy = _sorted("y", y, order, order.capacity)
    cols = y.shape[1]
    out = torch.empty((order.tokens, cols), dtype=y.dtype, device=y.device)
    _call("okls_experts_combine", y.device, order.address(), y.data_ptr(), ldy, DTYPES[y.dtype], cols,
          None if weights is None else weights.data_ptr(), 0 if weights is None else DTYPES[weights.dtype], out.data_ptr(), max(cols, 1))
    return out


def quantize_rows(x, order, dtype=torch.float8_e4m3fn, gathered=False, transpose=False) -> Blocked:
    """The 8-bit form of sorted rows x (capacity, k), or with gathered=True of the
    tokens x (tokens, k) in the sorted order; of the transpose with transpose=True.
    Rows without a choice are zeros, whatever x holds there."""
    q, t = _quantize_rows(x, order, dtype, gathered, not transpose, transpose)
    return t if transpose else q


def quantize_rows_both(x, order, dtype=torch.float8_e4m3fn, gathered=False):
    """Both forms of `quantize_rows` from one read of x."""
    return _quantize_rows(x, order, dtype, gathered, True, True)


def _quantize_rows(x, order, dtype, gathered, along, across):
    ldx = _sorted("x", x, order, order.tokens if gathered else order.capacity)
    rows, cols = order.capacity, x.shape[1]
    q = Blocked.empty(rows, cols, dtype, x.device) if along else None
    t = Blocked.empty(cols, rows, dtype, x.device) if across else None
    _call("okls_experts_quantize_rows", x.device, order.address(), x.data_ptr(), ldx, DTYPES[x.dtype], cols, 1 if gathered else 0,
          q.address() if along else None, t.address() if across else None)
    return q, t


def quantize_stack(weight, dtype=torch.float8_e4m3fn, transpose=False) -> Stack:
    """The 8-bit form of weight (n_experts, n, k), or of its matrices' transposes."""
    q, t = _quantize_stack(weight, dtype, not transpose, transpose)
    return t if transpose else q


def quantize_stack_both(weight, dtype=torch.float8_e4m3fn):
    """The 8-bit forms of weight (n_experts, n, k) and of its matrices' transposes from one read."""
    return _quantize_stack(weight, dtype, True, True)


def _quantize_stack(weight, dtype, along, across):
    if weight.dim() != 3 or weight.dtype not in DTYPES or not weight.is_cuda:
        raise ValueError(f"weight must be 3-D float32, bfloat16 or float16 on a GPU, got {tuple(weight.shape)} {weight.dtype} on {weight.device}")
    e, n, k = weight.shape
    if not 1 <= e <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, got {e}")
    if not (weight.stride(2) == 1 or k <= 1) or not (weight.stride(1) >= k or n <= 1):
        weight = weight.contiguous()
    q = Stack.empty((e, n, k), dtype, weight.device) if along else None
    t = Stack.empty((e, k, n), dtype, weight.device) if across else None
    _call("okls_experts_quantize_stack", weight.device, weight.data_ptr(), DTYPES[weight.dtype], e, weight.stride(0), n, k,
          weight.stride(1) if n > 1 else max(k, 1), q.blocked.address() if along else None, t.blocked.address() if across else None)
    return q, t


def matmul(a: Blocked, b: Stack, order: Plan, dtype=torch.bfloat16):
    """Rows r of each expert e of a (capacity, k) times b_e^T: (capacity, n) of
    `dtype`, zeros behind the last expert's rows.  An expert's rows without a choice are
    multiplied like its others: zeros from `quantize_rows`' zeros, where the expert's
    weights are finite.  Sums as `linear.matmul` sums `dtype`: a 16-bit result drops, from
    each eight products, what lies below 2^-13 of the largest of them."""
    e, n, k = b.shape
    pa, pb, device = a.address(), b.blocked.address(), a.codes.device
    if a.shape != (order.capacity, k) or e != order.n_experts:
        raise ValueError(f"a is {a.shape} and b {b.shape}, the plan has {order.capacity} rows of {order.n_experts} experts")
    if b.blocked.codes.device != device or order.device != device:
        raise ValueError(f"a is on {device}, b on {b.blocked.codes.device}, the plan on {order.device}")
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    out = torch.empty((order.capacity, n), dtype=dtype, device=device)
    _call("okls_experts_matmul", device, order.address(), pa, pb, n, out.data_ptr(), DTYPES[dtype], max(n, 1))
    return out


def weight_grad(a: Blocked, b: Blocked, order: Plan, dtype=torch.float32):
    """(n_experts, n, k) of `dtype`: for each expert a[:, rows] b[:, rows]^T over its
    rows, for the transposed forms a (n, capacity) and b (k, capacity); zeros for an
    expert without rows.  Its rows without a choice are summed too: `quantize_rows` makes
    them zeros.  The plan's align must be 128."""
    pa, pb, device = a.address(), b.address(), a.codes.device
    (n, ra), (k, rb) = a.shape, b.shape
    if ra != order.capacity or rb != order.capacity:
        raise ValueError(f"a is {a.shape} and b {b.shape}, the plan has {order.capacity} rows")
    if b.codes.device != device or order.device != device:
        raise ValueError(f"a is on {device}, b on {b.codes.device}, the plan on {order.device}")
    if order.align != 128:
        raise ValueError(f"the weights' gradient needs a plan with align=128, got {order.align}")
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    out = torch.empty((order.n_experts, n, k), dtype=dtype, device=device)
    _call("okls_experts_weight_grad", device, order.address(), pa, pb, out.data_ptr(), DTYPES[dtype], max(k, 1))
    return out


# --------------------------------------------------------------------------
# Autograd
# --------------------------------------------------------------------------
def _keep(ctx, order):
    """Keeps the plan for the backward pass.  Not by save_for_backward, which refuses inference tensors: a plan has no gradient."""
    ctx.order, ctx.versions = order, order._versions()


def _kept(ctx):
    """The forward pass's plan, which must be as it was: its gradients follow the same rows."""
    if ctx.order._versions() != ctx.versions:
        raise RuntimeError("the plan was modified in place after the forward pass, whose gradients need it as it was")
    return ctx.order


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order):
        _keep(ctx, order)
        return _gather(x, order)

    @staticmethod
    @once_differentiable     # the kernels below have no gradients of their own
    def backward(ctx, dout):
        _no_tangents(dout)
        return _combine(_rows(dout), None, _kept(ctx)), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, order):
        _keep(ctx, order)
        weights = None if weights is None else _weights(weights, order)
        out = _combine(y, weights, order)
        ctx.save_for_backward(*([] if weights is None else [y, weights]))
        return out

    @staticmethod
    @once_differentiable     # the kernels below have no gradients of their own
    def backward(ctx, dout):
        _no_tangents(dout)
        order, dout = _kept(ctx), _rows(dout)
        if not ctx.saved_tensors:
            return _gather(dout, order), None, None
        y, weights = ctx.saved_tensors
        need_y, need_w = ctx.needs_input_grad[:2]
        cols = y.shape[1]
        dy = torch.empty((order.capacity, cols), dtype=y.dtype, device=y.device)
        dweights = torch.empty_like(weights)
        if cols == 0:
            return dy if need_y else None, dweights.zero_() if need_w else None, None
        _call("okls_experts_combine_backward", y.device, order.address(), dout.data_ptr(), _matrix("dout", dout), y.data_ptr(),
              _matrix("y", y), DTYPES[y.dtype], cols, weights.data_ptr(), DTYPES[weights.dtype], dy.data_ptr(), cols, dweights.data_ptr())
        return dy if need_y else None, dweights if need_w else None, None


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, order, grad_dtype, gathered):
        need_x, need_w = ctx.needs_input_grad[:2]
        q, t = _quantize_rows(x, order, torch.float8_e4m3fn, gathered, True, need_w)
        w, wt = _quantize_stack(weight, torch.float8_e4m3fn, True, need_x)
        ctx.save_for_backward(*([t.codes, t.scales] if need_w else []), *([wt.blocked.codes, wt.blocked.scales] if need_x else []))
        _keep(ctx, order)
        ctx.grad_dtype, ctx.gathered, ctx.dtypes, ctx.shape = grad_dtype, gathered, (x.dtype, weight.dtype), weight.shape
        return matmul(q, w, order, dtype=x.dtype)

    @staticmethod
    @once_differentiable     # the kernels below have no gradients of their own
    def backward(ctx, dy):
        _no_tangents(dy)
        need_x, need_w = ctx.needs_input_grad[:2]
        order, (e, n, k), saved = _kept(ctx), ctx.shape, ctx.saved_tensors
        dq, dt = _quantize_rows(_rows(dy), order, ctx.grad_dtype, False, need_x, need_w)
        dx = dweight = None
        if need_w:
            dweight = weight_grad(dt, Blocked(saved[0], saved[1], (k, order.capacity)), order, dtype=ctx.dtypes[1])
        if need_x:
            dx = matmul(dq, Stack(saved[-2], saved[-1], (e, k, n)), order, dtype=ctx.dtypes[0])
            if ctx.gathered:
                dx = _combine(dx, None, order)
        return dx, dweight, None, None, None


def gather(x, order: Plan):
    """Tokens' rows x (tokens, k) in the sorted order: (order.capacity, k), zeros in rows without a choice."""
    _no_tangents(x)
    if x.requires_grad and torch.is_grad_enabled():
        return _Gather.apply(x, order)
    return _gather(x, order)


def combine(y, weights, order: Plan):
    """Each token's sum over its choices of weights (tokens, each) times their rows of
    y (order.capacity, k), in fp32, rounded once: (tokens, k) in y's dtype.  Dropped choices add
    nothing, and what y holds in rows without a choice is not read.  weights=None: ones."""
    _no_tangents(y, weights)
    if torch.is_grad_enabled() and (y.requires_grad or (weights is not None and weights.requires_grad)):
        return _Combine.apply(y, weights, order)
    return _combine(y, None if weights is None else _weights(weights, order), order)


def linear(x, weight, order: Plan, grad_dtype=torch.float8_e4m3fn):
    """Sorted rows x (order.capacity, k) through their experts' matrices, weight
    (n_experts, n, k): (order.capacity, n) in x's dtype, zeros in rows without a choice
    of an expert whose weights are finite.  Products and gradients as
    `linear.scaled_linear`'s; weight's gradient needs a plan with align=128 and is zeros
    for an expert without tokens."""
    return _apply(x, weight, order, grad_dtype, False)


def token_linear(x, weight, order: Plan, grad_dtype=torch.float8_e4m3fn):
    """`linear` of gather(x): the tokens x (tokens, k) are brought to 8 bits straight
    into the sorted order, and x's gradient is the sum over its choices, each rounded to
    x's dtype before the fp32 sum, as `gather`'s gradient would be."""
    return _apply(x, weight, order, grad_dtype, True)


def _apply(x, weight, order, grad_dtype, gathered):
    _no_tangents(x, weight)
    if weight.dim() != 3 or x.dim() != 2 or weight.shape[0] != order.n_experts or weight.shape[2] != x.shape[1]:
        raise ValueError(f"x is {tuple(x.shape)} and weight {tuple(weight.shape)}, the plan has {order.n_experts} experts")
    # all of it before the first launch, and what only the backward pass uses too
    _sorted("x", x, order, order.tokens if gathered else order.capacity)
    if weight.dtype not in DTYPES or weight.device != order.device:
        raise ValueError(f"weight must be float32, bfloat16 or float16 on {order.device}, got {weight.dtype} on {weight.device}")
    if grad_dtype not in _dense.FORMATS:
        raise ValueError(f"grad_dtype must be float8_e4m3fn or float8_e5m2, got {grad_dtype}")
    # summed over: the rows' columns, and in gradients the result's columns and the sorted rows
    grad, (_, n, k) = torch.is_grad_enabled(), weight.shape
    if max(k, n if grad and x.requires_grad else 0, order.capacity if grad and weight.requires_grad else 0) > MAX_SUMMED:
        raise ValueError(f"products sum over at most {MAX_SUMMED}, got k = {k}, n = {n} and {order.capacity} sorted rows")
    if order.align != 128 and torch.is_grad_enabled() and weight.requires_grad:
        raise ValueError(f"the weights' gradient needs a plan with align=128, got {order.align}")
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad):
        return _Linear.apply(x, weight, order, grad_dtype, gathered)
    # no transposed forms, which only gradients read
    q, _ = _quantize_rows(x, order, torch.float8_e4m3fn, gathered, True, False)
    return matmul(q, quantize_stack(weight), order, dtype=x.dtype)
