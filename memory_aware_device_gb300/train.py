"""Python binding of the training-step operators in libnest (include/nest_train.h).

The parts of a training step that decide two inputs of the placement solver:

    r = route(logits, k=2)              # gates, chosen experts, counts, balance loss
    g = route_backward(logits, r, grad_weights, grad_loss)
    opt = AdamW(weights, grads, state_bits=8)
    opt.step(lr, grad_scale=opt.grad_norm(max_norm=1.0)[1])

`gate` is `route` as a differentiable function of the logits.  `capacity_milli` turns expert
counts into the capacity factor of an all-to-all, `AdamW.opt_factor` is the optimizer bytes per
bf16 weight byte of the solver's instances.

Argument marshalling and checks only: every result is computed by the library's CUDA kernels on
the caller's stream, and there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
from typing import NamedTuple, Sequence

import numpy as np

from . import nest
from .nest import NestError

F32, BF16, F16 = 0, 1, 2
BLOCK = 256   # NEST_OPT_BLOCK

# Every function declared in include/nest_train.h.
EXPORTS = ("nest_route_workspace_size", "nest_route", "nest_route_backward", "nest_table_query",
           "nest_table_pack", "nest_grad_norm_workspace_size", "nest_grad_norm", "nest_adamw",
           "nest_adamw_values")


class RouteDesc(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("experts", C.c_int32), ("k", C.c_int32), ("row_stride", C.c_int64),
                ("col_stride", C.c_int64), ("dtype", C.c_int32), ("normalize", C.c_int32)]


class TableInfo(C.Structure):
    _fields_ = [("table_bytes", C.c_int64), ("blocks", C.c_int64), ("items", C.c_int64), ("tensors", C.c_int32),
                ("workers", C.c_int32)]


class AdamWArgs(C.Structure):
    _fields_ = [("weight_type", C.c_int32), ("grad_type", C.c_int32), ("state_bits", C.c_int32),
                ("seed", C.c_uint32), ("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("master", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("m_exp", C.c_void_p), ("v_exp", C.c_void_p), ("state", C.c_void_p), ("grad_scale", C.c_void_p)]


TENSOR_DT = np.dtype([("weight", "<u8"), ("grad", "<u8"), ("numel", "<i8"), ("weight_decay", "<f4"),
                      ("lr_scale", "<f4")])
STATE_DT = np.dtype([("beta1_t", "<f8"), ("beta2_t", "<f8"), ("step", "<i8"), ("ticket", "<u4"),
                     ("reserved", "<u4")])

_lib = None


def lib():
    """libnest.so with the operators' signatures; raises if it has not been built."""
    global _lib
    if _lib is None:
        L = nest.lib()
        P, V = C.POINTER, C.c_void_p
        L.nest_route_workspace_size.argtypes = [P(RouteDesc)]
        L.nest_route_workspace_size.restype = C.c_size_t
        L.nest_route.argtypes = [P(RouteDesc), V, V, V, V, V, V, V, V, V, C.c_size_t, V]
        L.nest_route_backward.argtypes = [P(RouteDesc), V, V, V, V, V, V, V, V, V, C.c_int64, V]
        L.nest_table_query.argtypes = [V, C.c_int32, P(TableInfo)]
        L.nest_table_pack.argtypes = [V, C.c_int32, P(TableInfo), V]
        L.nest_grad_norm_workspace_size.argtypes = [P(TableInfo)]
        L.nest_grad_norm_workspace_size.restype = C.c_size_t
        L.nest_grad_norm.argtypes = [P(TableInfo), V, C.c_int32, C.c_float, V, V, C.c_size_t, V]
        L.nest_adamw.argtypes = [P(TableInfo), V, P(AdamWArgs), V]
        L.nest_adamw_values.argtypes = [P(TableInfo), V, V, V, V, V, V, V]
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc:
        raise NestError(rc, what)


_torch = _codes = _raw_stream = _written = None


def _load_torch():
    """torch, imported at the first call, with what every call looks up.  `_written` tells autograd
    that tensors were written in place, so that a backward pass which saved them raises."""
    global _torch, _codes, _raw_stream, _written
    import torch
    _codes = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _written = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version
    _torch = torch
    return torch


def _type(t, what: str) -> int:
    if _torch is None:
        _load_torch()
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} is {t.dtype}: float32, bfloat16 and float16 are supported")
    return code


def _want(t, what: str, dtype, shape, device):
    """t as a contiguous tensor of this type, shape and device, or an error."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device} with strides {t.stride()}")
    return t


class _Guard:
    """A device made current, and a stream (new tensors belong to it), which is recorded as a user
    of `used`; `leave` undoes it."""

    def __init__(self, device, stream, used):
        torch = _torch
        self.guards = []
        if device.index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(device))
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))
            if stream != torch.cuda.current_stream(device):
                for t in used:
                    if t is not None:
                        t.record_stream(stream)
        for g in self.guards:
            g.__enter__()

    def leave(self):
        for g in reversed(self.guards):
            g.__exit__(None, None, None)


def _enter(device, stream, used=()):
    """Before a call on this device and stream (None = the device's current one): what has to be
    left after it, or None where both are current."""
    torch = _torch or _load_torch()
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}: the operators run on CUDA devices only")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is of {stream.device}, the tensors are on {device}")
    elif device.index == torch.cuda.current_device():
        return None
    return _Guard(device, stream, used)


# ---------------------------------------------------------------------------------
# Routing
# ---------------------------------------------------------------------------------

class Routing(NamedTuple):
    """What `route` computes (CUDA tensors)."""
    ids: object         # int32 [T, k] chosen experts, largest logit first, -1 = none
    weights: object     # float32 [T, k]
    counts: object      # int32 [E] how often each expert was chosen
    tokens: object      # int32 [1] rows that count
    mean_prob: object   # float32 [E]
    loss: object        # float32 [] balance loss, 1 for an even router

    @staticmethod
    def empty(tokens: int, experts: int, k: int, device="cuda") -> "Routing":
        """Uninitialised result buffers, and the workspace of calls into them, for `route(..., out=)`."""
        import torch
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        i, f = dict(dtype=torch.int32, device=device), dict(dtype=torch.float32, device=device)
        out = _Buffers(torch.empty((tokens, k), **i), torch.empty((tokens, k), **f), torch.empty(experts, **i),
                       torch.empty(1, **i), torch.empty(experts, **f), torch.empty((), **f))
        out.call = _RouteCall(tokens, experts, k, device)
        return out


class _Buffers(Routing):
    """Buffers of `Routing.empty`, with the workspace of calls that write them."""
    call = None


def _route_workspace(ref) -> int:
    size = lib().nest_route_workspace_size(ref)
    if not size:   # the call says which limit is broken
        _check(lib().nest_route(ref, None, None, None, None, None, None, None, None, None, 0, None), "nest_route")
    return size


@functools.lru_cache(maxsize=1024)
def _described(*fields):
    """A description of these numbers, by reference (what is passed on, not what it is of)."""
    return C.byref(RouteDesc(*fields))


class _RouteCall:
    """The workspace of calls of these sizes, and its address: a deep copy gets its own, and nothing is
    pickled (calls into unpickled buffers make one)."""

    def __init__(self, tokens, experts, k, device):
        import torch
        self.key = (tokens, experts, k, device)
        size = _route_workspace(_described(tokens, experts, k, 0, 0, F32, 0))
        self.workspace = torch.zeros(size, dtype=torch.uint8, device=device)   # every call leaves its head zero
        self.tail = (self.workspace.data_ptr(), size)
        self.streams = set()   # which come behind the clearing, and which the workspace's memory waits for
        if device.type == "cuda":
            self.made = torch.cuda.current_stream(device)
            self.streams.add(self.made.cuda_stream)

    def join(self):
        """Before the first call on another stream than the one that clears the workspace.  (A capture
        cannot wait for what is outside it; its replays come later.)"""
        here = _torch.cuda.current_stream(self.key[3])
        self.workspace.record_stream(here)
        if not _torch.cuda.is_current_stream_capturing():
            here.wait_stream(self.made)
            self.streams.add(here.cuda_stream)

    def __deepcopy__(self, memo):
        return _RouteCall(*self.key)

    def __reduce__(self):
        return type(None), ()


def _mask_ptr(mask, logits):
    if mask is None:
        return None
    if mask.dtype not in (_torch.bool, _torch.uint8):
        raise TypeError(f"mask is {mask.dtype}: bool and uint8 are supported")
    return _want(mask, "mask", mask.dtype, logits.shape[:1], logits.device).data_ptr()


def route(logits, k: int, mask=None, normalize: bool = True, out: Routing | None = None, stream=None) -> Routing:
    """nest_route: softmax gates of the k best experts per token, counts and balance loss.

    logits [T, E] (any strides; float32, bfloat16 or float16); mask [T] (bool or uint8, True = the
    token counts); normalize: gates of a token sum to 1.  out: buffers to write instead of new ones
    (quickest those of `Routing.empty`); calls that overlap on the GPU need buffers of their own."""
    dtype = _type(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [tokens, experts], not of shape {tuple(logits.shape)}")
    T, E = logits.shape
    dev = logits.device
    call = getattr(out, "call", None)
    if call is None or call.key != (T, E, k, dev):
        call = None
        _route_workspace(_described(T, E, k, 0, 0, dtype, 0))
    guard = _enter(dev, stream, () if stream is None else (logits, mask, *(out or ())))
    given = out is not None
    try:
        if out is None:
            out = Routing.empty(T, E, k, dev)
            call = out.call
        elif call is None:
            torch = _torch
            _want(out.ids, "out.ids", torch.int32, (T, k), dev)
            _want(out.weights, "out.weights", torch.float32, (T, k), dev)
            _want(out.counts, "out.counts", torch.int32, (E,), dev)
            _want(out.tokens, "out.tokens", torch.int32, (1,), dev)
            _want(out.mean_prob, "out.mean_prob", torch.float32, (E,), dev)
            _want(out.loss, "out.loss", torch.float32, (), dev)
            call = _RouteCall(T, E, k, dev)
        ids, weights, counts, tokens, mean_prob, loss = out
        raw = _raw_stream(dev.index)
        if raw not in call.streams:
            call.join()
        rc = _lib.nest_route(_described(T, E, k, *logits.stride(), dtype, 1 if normalize else 0), logits.data_ptr(),
                             None if mask is None else _mask_ptr(mask, logits), ids.data_ptr(), weights.data_ptr(),
                             counts.data_ptr(), tokens.data_ptr(), mean_prob.data_ptr(), loss.data_ptr(), *call.tail,
                             raw)
    finally:
        if guard is not None:
            guard.leave()
    _check(rc, "nest_route")
    if given:
        _written(out)
    return out


def route_backward(logits, routing: Routing, grad_weights=None, grad_loss=None, mask=None, normalize: bool = True,
                   out=None, stream=None):
    """nest_route_backward: gradient with respect to the logits, in their type, from the gradients
    of the weights (float32 [T, k]) and of the loss (float32 scalar tensor); None counts as zero.
    routing, mask and normalize as in the forward call."""
    dtype = _type(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [tokens, experts], not of shape {tuple(logits.shape)}")
    torch, dev = _torch, logits.device
    T, E = logits.shape
    ids, weights, counts, tokens = routing[:4]
    k = ids.shape[-1]
    i32, f32, one = torch.int32, torch.float32, (T, k)
    if T and not (   # an empty batch reads none of them
            ids.dtype is i32 and ids.shape == one and ids.is_contiguous() and ids.device == dev and
            weights.dtype is f32 and weights.shape == one and weights.is_contiguous() and weights.device == dev and
            counts.dtype is i32 and counts.shape == (E,) and counts.is_contiguous() and counts.device == dev and
            tokens.dtype is i32 and tokens.shape == (1,) and tokens.device == dev):
        _want(ids, "routing.ids", i32, one, dev)
        _want(weights, "routing.weights", f32, one, dev)
        _want(counts, "routing.counts", i32, (E,), dev)
        _want(tokens, "routing.tokens", i32, (1,), dev)
    if grad_weights is not None:
        _want(grad_weights, "grad_weights", f32, one, dev)
    if grad_loss is not None:
        _want(grad_loss, "grad_loss", torch.float32, grad_loss.shape, dev)
        if grad_loss.numel() != 1:
            raise ValueError(f"grad_loss must be one number, not of shape {tuple(grad_loss.shape)}")
    guard = _enter(dev, stream, () if stream is None else
                   (logits, mask, ids, weights, counts, tokens, grad_weights, grad_loss, out))
    given = out is not None
    try:
        if not given:
            out = torch.empty((T, E), dtype=logits.dtype, device=dev)
            step = E
        else:
            step, col = out.stride() if out.dim() == 2 else (0, 0)
            if out.dtype is not logits.dtype or out.shape != logits.shape or out.device != dev or \
                    (E > 1 and col != 1) or (T > 1 and step < E):
                raise ValueError(f"out must be a {logits.dtype} tensor of shape {(T, E)} on {dev} with rows of its own")
        rc = lib().nest_route_backward(
            _described(T, E, k, *logits.stride(), dtype, 1 if normalize else 0), logits.data_ptr(),
            None if mask is None else _mask_ptr(mask, logits), ids.data_ptr(), weights.data_ptr(),
            counts.data_ptr(), tokens.data_ptr(), None if grad_weights is None else grad_weights.data_ptr(),
            None if grad_loss is None else grad_loss.data_ptr(), out.data_ptr(), max(step, E), _raw_stream(dev.index))
    finally:
        if guard is not None:
            guard.leave()
    _check(rc, "nest_route_backward")
    if given:
        _written((out,))
    return out


def _gate_function():
    import torch

    class Gate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, k, mask, normalize):
            r = route(logits, k, mask=mask, normalize=normalize)
            ctx.save_for_backward(logits, mask, *r)
            ctx.normalize = normalize
            ctx.mark_non_differentiable(r.ids, r.counts, r.tokens, r.mean_prob)
            return tuple(r)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, _ids, grad_weights, _counts, _tokens, _mean, grad_loss):
            logits, mask, *r = ctx.saved_tensors
            return (route_backward(logits, Routing(*r), grad_weights.contiguous(), grad_loss.contiguous(), mask=mask,
                                   normalize=ctx.normalize), None, None, None)

    return Gate


_gate = None


def gate(logits, k: int, mask=None, normalize: bool = True) -> Routing:
    """`route` with gradients: the result's weights and loss are differentiable in the logits (the
    counts are constants of the gradient; mean_prob carries none).  Once: a derivative of that
    gradient raises."""
    global _gate
    if _gate is None:
        _gate = _gate_function()
    return Routing(*_gate.apply(logits, k, mask, normalize))


def capacity_milli(counts, tokens: int, k: int) -> int:
    """Capacity factor in thousandths, rounded up, that a layer's all-to-all needs for these expert
    counts: the fullest expert's share over the even share, at least 1000 (even).  counts: integers
    on the host."""
    c = np.asarray(counts, dtype=np.int64)
    if not tokens or not k or not c.size:
        return 1000
    return max(1000, -(-int(c.max()) * c.size * 1000 // (int(tokens) * k)))


# ---------------------------------------------------------------------------------
# Lists of tensors
# ---------------------------------------------------------------------------------

class _Table:
    """The packed table of a list of tensors, on their device."""

    def __init__(self, grads, weights=None, weight_decay=0.0, lr_scale=1.0):
        import torch
        if not grads:
            raise ValueError("an empty list of tensors")
        n, self.device = len(grads), grads[0].device
        if self.device.type != "cuda":
            raise ValueError(f"tensors are on {self.device}: the operators run on CUDA devices only")
        rec = self.rec = np.zeros(n, TENSOR_DT)
        rec["numel"] = [t.numel() for t in grads]
        rec["grad"] = self._addresses("grads", grads, grads[0].dtype)
        if weights is not None:
            rec["weight"] = self._addresses("weights", weights, weights[0].dtype if len(weights) else None)
        rec["weight_decay"], rec["lr_scale"] = weight_decay, lr_scale
        # aliases: the storage whose addresses the table holds, also when a tensor is given another
        self.keep = [t.detach() for t in (*grads, *(weights or ()))]
        if weights is not None:
            at = np.argsort(rec["weight"], kind="stable")
            at = at[rec["numel"][at] > 0]
            start = rec["weight"][at].astype(np.int64)
            if (start[:-1] + rec["numel"][at][:-1] * weights[0].element_size() > start[1:]).any():
                raise ValueError("weights overlap")
        self.grad_type = _type(grads[0], "grads")
        self.info = TableInfo()
        _check(lib().nest_table_query(rec.ctypes.data, n, C.byref(self.info)), "nest_table_query")
        ws = lib().nest_grad_norm_workspace_size(C.byref(self.info))
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=self.device)
        self.table = self._packed().to(self.device)   # waits for the stream, the clearing with it
        self.out = torch.empty(2, dtype=torch.float32, device=self.device)
        self.head = (C.byref(self.info), self.table.data_ptr())
        self.tail = (self.out.data_ptr(), self.workspace.data_ptr(), ws)
        self.own = [self.table, self.workspace, self.out]   # made here, as an optimizer's buffers
        self.streams = {torch.cuda.current_stream(self.device).cuda_stream}   # which their memory waits for

    def join(self, raw):
        """Before the first call on a stream."""
        here = _torch.cuda.current_stream(self.device)
        for t in self.own:
            t.record_stream(here)
        self.streams.add(raw)

    def _addresses(self, what, ts, dtype):
        """The tensors' addresses, or an error where they are not the list's."""
        if len(ts) != len(self.rec):
            raise ValueError(f"{len(ts)} {what} for {len(self.rec)} tensors")
        for i, (t, n) in enumerate(zip(ts, self.rec["numel"].tolist())):
            if t.dtype != dtype or t.device != self.device or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{what}[{i}] must be a contiguous {dtype} tensor of {n} elements on {self.device}")
        return [t.data_ptr() for t in ts]

    def _packed(self):
        import torch
        packed = np.zeros(self.info.table_bytes, np.uint8)
        _check(lib().nest_table_pack(self.rec.ctypes.data, len(self.rec), C.byref(self.info), packed.ctypes.data),
               "nest_table_pack")
        return torch.from_numpy(packed)

    def bind_grads(self, grads):
        import torch
        self.rec["grad"] = self._addresses("grads", grads, self.keep[0].dtype)
        torch.cuda.synchronize(self.device)     # calls under way read the table and the gradients before
        self.table.copy_(self._packed())        # in its place: captured calls read it too
        self.keep[:len(grads)] = [t.detach() for t in grads]

    def norm(self, max_norm, stream):
        guard = _enter(self.device, stream, () if stream is None else self.held())
        try:
            raw = _raw_stream(self.device.index)
            if raw not in self.streams:
                self.join(raw)
            rc = _lib.nest_grad_norm(*self.head, self.grad_type, max_norm, *self.tail, raw)
        finally:
            if guard is not None:
                guard.leave()
        _check(rc, "nest_grad_norm")
        return self.out

    def held(self):
        """The tensors that were given to the list."""
        return self.keep


class GradNorm:
    """nest_grad_norm over a list of contiguous CUDA tensors of one type, bound by reference: the
    storage that they have now is kept and read by every `run`."""

    def __init__(self, grads: Sequence):
        self._table = _Table(grads)

    def run(self, max_norm: float = math.inf, stream=None):
        """float32 [2]: the global norm, and min(1, max_norm / (norm + 1e-6)), NaN when the norm is
        not finite.  The same buffer every call; calls that overlap on the GPU race on it."""
        return self._table.norm(max_norm, stream)

    def bind_grads(self, grads: Sequence):
        """Read these tensors from now on: as many, of the same type and sizes (synchronises)."""
        self._table.bind_grads(grads)


class AdamW:
    """nest_adamw over a list of tensors, bound by reference.

    weights, grads: lists of contiguous CUDA tensors, each list of one type (float32, bfloat16 or
    float16); the step reads the gradients and updates the weights in place, in the storage that they
    have now, which is kept.  The object owns the
    float32 master weights (weights of 16 bits only), the moments m and v (state_bits 32: float32;
    8: uint8 codes with the scales m_exp and v_exp) and the device's step count: copy into them to
    set them.  Buffers hold the tensors in order, each from a multiple of 256 elements on (`starts`).  weight_decay and
    lr_scale: one number, or one per tensor."""

    def __init__(self, weights: Sequence, grads: Sequence, state_bits: int = 32, betas=(0.9, 0.999),
                 eps: float = 1e-8, weight_decay=0.01, lr_scale=1.0, seed: int = 0):
        import torch
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits is {state_bits}: 8 and 32 are supported")
        self._table = tb = _Table(grads, weights, weight_decay, lr_scale)
        self.weights, self.grads, self.state_bits, self.betas = list(weights), list(grads), state_bits, tuple(betas)
        dev, n = tb.device, tb.info.blocks * BLOCK
        sizes = [-(-t.numel() // BLOCK) * BLOCK for t in weights]
        self.starts = [0] + np.cumsum(sizes, dtype=np.int64)[:-1].tolist()
        kind = dict(dtype=torch.float32 if state_bits == 32 else torch.uint8, device=dev)
        self.m, self.v = torch.zeros(n, **kind), torch.zeros(n, **kind)
        self.m_exp = self.v_exp = self.master = None
        if state_bits == 8:
            self.m_exp, self.v_exp = (torch.full((n // BLOCK,), -100, dtype=torch.int8, device=dev) for _ in "mv")
        weight_type = _type(weights[0], "weights")
        if weight_type != F32:
            self.master = torch.zeros(n, dtype=torch.float32, device=dev)
            for t, a in zip(weights, self.starts):
                self.master[a:a + t.numel()] = t.detach().reshape(-1)
        # one tensor for each version counter: views share their base's
        self._counters = list({id(b): b for b in (t if t._base is None else t._base for t in weights)}.values())
        self._state = torch.zeros(STATE_DT.itemsize, dtype=torch.uint8, device=dev)
        own = (self._state, self.master, self.m, self.v, self.m_exp, self.v_exp)
        tb.own += [t.detach() for t in own if t is not None]   # what the calls use, whatever the names hold later
        self._used = None   # stream of the last step

        def ptr(t):
            return t.data_ptr() if t is not None else None
        self._args = AdamWArgs(weight_type, tb.grad_type, state_bits, seed & 0xFFFFFFFF, 0.0, betas[0], betas[1], eps,
                               ptr(self.master), ptr(self.m), ptr(self.v), ptr(self.m_exp), ptr(self.v_exp),
                               self._state.data_ptr(), None)
        self._ref = C.byref(self._args)
        self._codes = tuple(ptr(t) for t in (self.m, self.v, self.m_exp, self.v_exp))
        self._length = n
        self.set_step(0)

    def _settle(self):
        """Lets the last step finish if it is on another stream than the current one, which reads and
        writes of the object's state come behind."""
        if self._used is not None and self._used != _raw_stream(self._table.device.index):
            _torch.cuda.synchronize(self._table.device)

    def set_step(self, step: int):
        """Set the number of steps taken (synchronises; 0 at the start).  Steps enqueued before, on
        whichever stream, come before it; replays of captured steps have to be waited for."""
        import torch
        if step < 0 or step != int(step):
            raise ValueError(f"the number of steps taken is {step}: it is a whole number of at least 0")
        self._settle()
        rec = np.zeros(1, STATE_DT)
        rec["beta1_t"], rec["beta2_t"], rec["step"] = self.betas[0] ** step, self.betas[1] ** step, step
        self._state.copy_(torch.from_numpy(rec.view(np.uint8)))

    @property
    def steps(self) -> int:
        """Steps taken (reads the device, behind the steps enqueued before as in `set_step`)."""
        self._settle()
        return int(self._state.cpu().numpy().view(STATE_DT)["step"][0])

    @property
    def opt_factor(self) -> int:
        """Optimizer-state bytes per bf16 weight byte, rounded down to the solver's whole number: 6
        for a float32 master and two float32 moments, 3 with 8-bit moments, whose scales are a
        further 1/256 of the bf16 weight bytes."""
        per = 2 * self.state_bits // 8 + (4 if self.master is not None else 0)
        return per // 2

    def bind_grads(self, grads: Sequence):
        """Read these gradients from now on - after they were allocated anew, as by a zero_grad that
        sets them to None: as many tensors, of the same type and sizes.  Moments and step count stay,
        and captured steps read the new ones too (synchronises)."""
        self._table.bind_grads(grads)
        self.grads = list(grads)

    def grad_norm(self, max_norm: float = math.inf, stream=None):
        """Norm and clip scale of the gradients, as `GradNorm.run`."""
        return self._table.norm(max_norm, stream)

    def step(self, lr: float, grad_scale=None, stream=None):
        """One step.  grad_scale: float32 CUDA scalar that multiplies the gradients (entry 1 of
        `grad_norm`); when it is not finite the call changes nothing."""
        a, tb = self._args, self._table
        if grad_scale is None:
            a.grad_scale = None
        else:
            if _codes.get(grad_scale.dtype) != F32 or grad_scale.numel() != 1 or grad_scale.device != tb.device:
                raise ValueError(f"grad_scale must be one float32 number on {tb.device}")
            a.grad_scale = grad_scale.data_ptr()
        a.lr = lr
        guard = _enter(tb.device, stream, () if stream is None else (grad_scale, *tb.held()))
        try:
            self._used = raw = _raw_stream(tb.device.index)
            if raw not in tb.streams:
                tb.join(raw)
            rc = _lib.nest_adamw(*tb.head, self._ref, raw)
        finally:
            if guard is not None:
                guard.leave()
        _check(rc, "nest_adamw")
        _written(self._counters)

    def state_values(self, stream=None):
        """(m, v): the moments, laid out like the object's buffers.  With 8-bit states new bfloat16
        tensors with the exact values of the codes, else the float32 buffers themselves."""
        if self.state_bits == 32:
            return self.m, self.v
        tb, kind = self._table, _torch.bfloat16
        guard = _enter(tb.device, stream)
        try:
            raw = _raw_stream(tb.device.index)
            if raw not in tb.streams:
                tb.join(raw)
            m = _torch.empty(self._length, dtype=kind, device=tb.device)
            v = _torch.empty(self._length, dtype=kind, device=tb.device)
            rc = _lib.nest_adamw_values(tb.head[0], *self._codes, m.data_ptr(), v.data_ptr(), raw)
        finally:
            if guard is not None:
                guard.leave()
        _check(rc, "nest_adamw_values")
        return m, v
