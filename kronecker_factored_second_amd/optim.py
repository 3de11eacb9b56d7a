"""The optimizer step for parameters that `okls.OKLS` does not take (embeddings,
norm weights, biases, routers): AdamW over many tensors at once, with moments in
32 or in 8 bits, and the norm of all gradients that it clips them by.

Binding of the entry points declared in include/okls_optim.h, with the same rules
as `okls`: argument checks and marshalling only, every step runs in the HIP
library on the current stream, and there is no fallback.

    opt = AdamW([embedding, *norms], lr=3e-4, weight_decay=0.1, moments="8bit")
    loss.backward()
    opt.step(norm=grad_norm([p.grad for p in everything]), max_norm=1.0)
    opt.zero_grad()
"""
from __future__ import annotations

import array
import ctypes
import itertools
import operator
from typing import NamedTuple, Optional

import torch

from . import linear, okls

EXPORTED = ("okls_grad_norm_workspace_size", "okls_grad_norm", "okls_adamw")
BITS = {"fp32": 32, "8bit": 8}


class GradientStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class TensorStruct(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("n", ctypes.c_int64), ("g_dtype", ctypes.c_int32)]


class ConfigStruct(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("max_norm", ctypes.c_double), ("moment_bits", ctypes.c_int32)]


class Moments(NamedTuple):
    """One tensor's moments, contiguous and of its number of elements n.
    32 bits: m and v in float32, scales None.  8 bits: m and the root of v in
    float8_e4m3fn, scales (2, ceil(n / 128)) float8_e8m0fnu, m's and the root's."""
    m: torch.Tensor
    v: torch.Tensor
    scales: Optional[torch.Tensor] = None


_lib = None


def load():
    """The library with this module's entry points declared; raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    lib = okls.load()
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.okls_grad_norm_workspace_size.argtypes = [i32, vp]
    lib.okls_grad_norm_workspace_size.restype = sz
    lib.okls_grad_norm.argtypes = [i32, vp, vp, vp, sz, vp]
    lib.okls_grad_norm.restype = ctypes.c_int
    lib.okls_adamw.argtypes = [ctypes.POINTER(ConfigStruct), i64, i32, vp, vp, vp]
    lib.okls_adamw.restype = ctypes.c_int
    _lib = lib
    return lib


def _on(device, name, *args):
    """One library call on the current stream of `device`."""
    fn, index = getattr(_lib or load(), name), device.index
    if index == torch.cuda.current_device():
        st = fn(*args, linear._raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, linear._raw_stream(index))
    if st != okls.OKLS_OK:
        raise okls.OKLSError(name, st)


def grad_norm(grads) -> torch.Tensor:
    """The 2-norm of all gradients together, a float32 scalar on their device:
    float32, bfloat16 or float16 tensors of any shapes, squared and summed in fp64.
    It records no gradient."""
    grads = [g if g.is_contiguous() else g.contiguous() for g in grads]
    if not grads:
        raise ValueError("no gradients")
    device, index, dtypes = grads[0].device, grads[0].get_device(), linear.DTYPES
    codes = [dtypes.get(g.dtype) for g in grads]
    if None in codes or index < 0 or set(map(_device, grads)) != {index}:
        for i, g in enumerate(grads):
            if codes[i] is None:
                raise ValueError(f"gradient {i} must be float32, bfloat16 or float16, got {g.dtype}")
            if g.get_device() != index or index < 0:
                raise ValueError(f"gradient {i} is on {g.device}, the first on {device}: all must be on one GPU")
    table = array.array("Q", itertools.chain.from_iterable(zip(map(_address, grads), map(_numel, grads), codes)))      # of GradientStruct
    at = table.buffer_info()[0]
    need = (_lib or load()).okls_grad_norm_workspace_size(len(grads), at)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    norm = torch.empty((), dtype=torch.float32, device=device)
    _on(device, "okls_grad_norm", len(grads), at, norm.data_ptr(), ws.data_ptr() if need else None, need)
    return norm


_numel, _address, _device, _contiguous = torch.Tensor.numel, torch.Tensor.data_ptr, torch.Tensor.get_device, torch.Tensor.is_contiguous
_dtype = operator.attrgetter("dtype")


def _scales_fit(s, n, index, eight):
    if not eight or s is None:
        return not eight and s is None
    return s.dtype is torch.float8_e8m0fnu and s.shape == (2, -(-n // 128)) and s.get_device() == index and s.is_contiguous()


def _refuse(params, grads, moments, index, device, held, eight):
    """Raises for the first tensor that is not as `adamw` says."""
    for i, (p, g, (m, v, scales)) in enumerate(zip(params, grads, moments)):
        n = p.numel()
        if p.dtype is not torch.float32 or p.get_device() != index or not p.is_contiguous():
            raise ValueError(f"parameter {i} must be a contiguous float32 tensor on {device}, got {p.dtype} on {p.device}")
        if g is None or g.dtype not in linear.DTYPES:
            raise ValueError(f"gradient {i} must be float32, bfloat16 or float16, got {'none' if g is None else g.dtype}")
        if not g.is_same_size(p) or g.get_device() != index:
            raise ValueError(f"gradient {i} is {tuple(g.shape)} on {g.device}, parameter {tuple(p.shape)} on {device}")
        if any(x.dtype is not held or x.numel() != n or x.get_device() != index or not x.is_contiguous() for x in (m, v)):
            raise ValueError(f"moments {i} must be contiguous {held} tensors of {n} elements on {device}, got "
                             f"{tuple(m.shape)} {m.dtype} on {m.device} and {tuple(v.shape)} {v.dtype} on {v.device}")
        if not _scales_fit(scales, n, index, eight):
            raise ValueError(f"scales {i} must be {f'contiguous float8_e8m0fnu {(2, -(-n // 128))} on {device}' if eight else 'None'}, "
                             f"got {None if scales is None else (scales.dtype, tuple(scales.shape), scales.device)}")
    raise ValueError("parameters, gradients and moments do not fit")


def adamw(params, grads, moments, t, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, norm=None, max_norm=None):
    """Step t (from 1 on) of AdamW on every float32 tensor of `params` and its `Moments`, in place:

        g <- g min(1, max_norm / (norm + 1e-6))      with norm, a float32 scalar on the device (`grad_norm`'s)
        m <- beta1 m + (1 - beta1) g
        v <- beta2 v + (1 - beta2) g^2
        p <- (1 - lr weight_decay) p - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)

    Where norm is no finite number nothing is written; without norm max_norm is not read.  8-bit moments are rounded
    up or down in proportion, by thresholds that t, the tensor's place in the list and
    the element's number give; the update takes them before they are rounded.  Roots of v
    below 3.5e-5 of the largest of their 128 always round up, and do not fall while that
    one stays.  With steady gradients a held root scatters by 15 %, and updates differ
    by 17 % in norm from those of fp32 moments.
    Tensors may have any shape and be views; all must be contiguous, on one GPU
    and apart from each other.  Captured into a graph, a replay reuses t and lr."""
    params, grads, moments = list(params), list(grads), list(moments)
    if not params:
        raise ValueError("no parameters")
    if len(grads) != len(params) or len(moments) != len(params):
        raise ValueError(f"{len(grads)} gradients and {len(moments)} moments for {len(params)} parameters")
    device, index, dtypes, float32 = params[0].device, params[0].get_device(), linear.DTYPES, torch.float32
    if index < 0:
        raise ValueError(f"parameter 0 must be on a GPU, got {device}")
    ms, vs, scales = zip(*moments)
    eight = scales[0] is not None
    held = torch.float8_e4m3fn if eight else float32
    counts = list(map(_numel, params))
    # all at once where everything is as it should be; one by one to say what is not
    grads = [g if g is None or g.is_contiguous() else g.contiguous() for g in grads]
    codes = [None if g is None else dtypes.get(g.dtype) for g in grads]
    if (None in codes or set(map(_dtype, params)) != {float32} or set(map(_dtype, ms + vs)) != {held}
            or {*map(_device, params), *map(_device, grads), *map(_device, ms), *map(_device, vs)} != {index}
            or not all(map(_contiguous, params)) or not all(map(_contiguous, ms)) or not all(map(_contiguous, vs))
            or not all(map(torch.Tensor.is_same_size, grads, params)) or list(map(_numel, ms)) != counts or list(map(_numel, vs)) != counts
            or not all(_scales_fit(s, n, index, eight) for s, n in zip(scales, counts))):
        _refuse(params, grads, moments, index, device, held, eight)
    places, m_places, v_places = list(map(_address, params)), list(map(_address, ms)), list(map(_address, vs))
    every = places + m_places + v_places
    if len(set(every)) != len(every) and len({a for a, n in zip(every, counts * 3) if n}) != 3 * sum(n > 0 for n in counts):
        raise ValueError("a parameter or one of its moments is in the lists twice")
    rows = zip(places, map(_address, grads), m_places, v_places, map(_address, scales) if eight else itertools.repeat(0), counts, codes)
    table = array.array("Q", itertools.chain.from_iterable(rows))        # of TensorStruct
    if norm is not None:
        if norm.dtype != float32 or norm.numel() != 1 or norm.device != device:
            raise ValueError(f"norm must be one float32 on {device}, got {tuple(norm.shape)} {norm.dtype} on {norm.device}")
        if max_norm is None:
            raise ValueError("norm needs max_norm")
    config = ConfigStruct(lr, beta1, beta2, eps, weight_decay, max_norm if norm is not None else 0.0, 8 if eight else 32)
    _on(device, "okls_adamw", config, operator.index(t), len(params), table.buffer_info()[0], None if norm is None else norm.data_ptr())
    # a graph that kept one has to know, as of torch's own writes
    linear._written([p for p in params if not p.is_inference()])


def new_moments(p, moments="fp32") -> Moments:
    """Zero moments of the tensor p, "fp32" or "8bit"."""
    if moments not in BITS:
        raise ValueError(f"moments must be 'fp32' or '8bit', got {moments!r}")
    if moments == "fp32":
        return Moments(torch.zeros_like(p, dtype=torch.float32), torch.zeros_like(p, dtype=torch.float32))
    m, v = (torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn) for _ in range(2))
    return Moments(m, v, torch.full((2, -(-p.numel() // 128)), 127, dtype=torch.uint8, device=p.device).view(torch.float8_e8m0fnu))


class AdamW:
    """AdamW over a list of float32 tensors of any shapes, with the interface of
    `okls.OKLS`: .step(), .zero_grad(), .state_dict(), .load_state_dict().  Gradients are
    read from p.grad (float32, bfloat16 or float16) unless `grads` is passed to
    step().  moments="8bit" holds both moments in 2 bytes a parameter instead of 8, as `adamw` says.
    A step that a norm without a finite value holds back counts in .t all the same: the
    host does not wait to learn of it."""

    def __init__(self, params, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, moments="fp32"):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        for p in self.params:
            if p.dtype != torch.float32 or not p.is_contiguous():
                raise ValueError("parameters must be contiguous fp32 tensors")
        self.lr, self.beta1, self.beta2 = float(lr), float(beta1), float(beta2)
        self.eps, self.weight_decay, self.moments = float(eps), float(weight_decay), moments
        self.state = [new_moments(p.detach(), moments) for p in self.params]
        self.t = 0

    def step(self, grads=None, lr=None, norm=None, max_norm=None):
        lr = self.lr if lr is None else float(lr)
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        # the counter and the learning rate change only once the library has accepted the step
        adamw(self.params, grads, self.state, self.t + 1, lr=lr, beta1=self.beta1, beta2=self.beta2, eps=self.eps,
              weight_decay=self.weight_decay, norm=norm, max_norm=max_norm)
        self.t += 1
        self.lr = lr

    def zero_grad(self):
        for p in self.params:
            p.grad = None

    def state_dict(self):
        return {"t": self.t, "lr": self.lr, "moments": self.moments,
                "state": [Moments(*[None if x is None else x.clone() for x in s])._asdict() for s in self.state]}

    def load_state_dict(self, sd):
        # every tensor is checked before anything is copied, so a mismatched checkpoint leaves this optimizer untouched
        if sd["moments"] != self.moments:
            raise ValueError(f"state holds {sd['moments']} moments, this optimizer {self.moments}")
        if len(sd["state"]) != len(self.state):
            raise ValueError(f"state holds {len(sd['state'])} parameters, this optimizer has {len(self.state)}")
        for i, (dst, src) in enumerate(zip(self.state, sd["state"])):
            for k, d in dst._asdict().items():
                s = src[k]
                if (s is None) != (d is None) or (d is not None and (s.shape != d.shape or s.dtype != d.dtype)):
                    raise ValueError(f"parameter {i} {k}: {None if s is None else (tuple(s.shape), s.dtype)}, "
                                     f"expected {None if d is None else (tuple(d.shape), d.dtype)}")
        self.t, self.lr = int(sd["t"]), float(sd["lr"])
        for dst, src in zip(self.state, sd["state"]):
            for k, d in dst._asdict().items():
                if d is not None:
                    # by bytes: copies of 8-bit floats are not everywhere
                    d.view(torch.uint8).copy_(src[k].view(torch.uint8)) if d.element_size() == 1 else d.copy_(src[k])
