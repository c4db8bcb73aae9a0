"""Python binding of the output head's losses in libnest (include/nest_head.h).

The end of a training step's forward pass and the start of its backward pass: the product of the
hidden states with the output weights and a loss of its logits, which are never kept.

    r = cross_entropy(hidden, weight, labels)                  # loss, each token's loss
    dh, dw = cross_entropy_backward(hidden, weight, labels, r, grad_loss)
    r = distill(hidden, weight, ids, teacher, temperature=2.0)   # a teacher's largest logits
    dh, dw = distill_backward(hidden, weight, ids, teacher, r, grad_loss, temperature=2.0)

`label_loss` and `teacher_loss` are the same as differentiable functions of the hidden states and
the weights.

Argument marshalling and checks only, as in `train`: every result is computed by the library's CUDA
kernels on the caller's stream, and there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import functools
from typing import NamedTuple

from . import nest, train
from .train import BF16, F16, F32, _check, _enter, _want

I32, I64 = 0, 1
MAX_K = 256

# Every function declared in include/nest_head.h.
EXPORTS = ("nest_head_loss_workspace_size", "nest_head_backward_workspace_size", "nest_head_loss",
           "nest_head_loss_backward", "nest_head_waits_given_up")


class HeadDesc(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("tokens", "vocab", "hidden", "hidden_row", "hidden_col", "weight_row",
                                         "weight_col")] + \
               [(n, C.c_int32) for n in ("dtype", "index_type", "k", "teacher_type")] + \
               [("temperature", C.c_float), ("reserved", C.c_int32)]


_lib = None


def lib():
    """libnest.so with the losses' signatures; raises if it has not been built."""
    global _lib
    if _lib is None:
        L, P, V = nest.lib(), C.POINTER, C.c_void_p
        for f in (L.nest_head_loss_workspace_size, L.nest_head_backward_workspace_size):
            f.argtypes, f.restype = [P(HeadDesc), V], C.c_size_t
        L.nest_head_loss.argtypes = [P(HeadDesc)] + [V] * 10 + [C.c_size_t, V]
        L.nest_head_loss_backward.argtypes = [P(HeadDesc)] + [V] * 11 + [C.c_size_t, V]
        L.nest_head_waits_given_up.argtypes = [P(C.c_int64), V]
        _lib = L
    return _lib


class HeadLoss(NamedTuple):
    """What `cross_entropy` and `distill` compute (CUDA tensors)."""
    loss: object      # float32 [] mean over the tokens that count, 0 when there is none
    losses: object    # float32 [T], 0 for a token that does not count
    lse: object       # float32 [T] log of the sum of the exponentials of the (tempered) logits, 0 likewise
    tokens: object    # int32 [1] tokens that count


@functools.lru_cache(maxsize=1024)
def _described(*fields):
    """A description of these numbers, by reference."""
    return C.byref(HeadDesc(*fields, 0))


class _Inputs:
    """The checked inputs of a call: their description and their addresses."""
    __slots__ = ("device", "shape", "used", "ref", "pointers")

    def __init__(self, hidden, weight, index, teacher, mask, temperature):
        torch = train._torch or train._load_torch()
        if _lib is None:
            lib()
        kind = hidden.dtype
        dtype = train._codes.get(kind)
        if dtype not in (BF16, F16) or weight.dtype is not kind:
            raise TypeError(f"hidden is {kind} and weight {weight.dtype}: both bfloat16 or both float16 are supported")
        shape, across = self.shape = hidden.shape, weight.shape
        if len(shape) != 2 or len(across) != 2 or shape[1] != across[1]:
            raise ValueError(f"hidden must be [tokens, width] and weight [vocabulary, width], not of shapes "
                             f"{tuple(shape)} and {tuple(across)}")
        dev = self.device = hidden.device
        if weight.device != dev:
            raise ValueError(f"hidden is on {dev}, weight on {weight.device}")
        T, D = shape
        kind = index.dtype
        if kind is torch.int64:
            wide = I64
        elif kind is torch.int32:
            wide = I32
        else:
            raise TypeError(f"{'labels' if teacher is None else 'ids'} are {kind}: int64 and int32 are supported")
        k, listed = 0, F32
        if teacher is None:
            _want(index, "labels", kind, (T,), dev)
            second = third = None
        else:
            k = index.shape[-1] if index.dim() == 2 else 0
            if not 1 <= k <= MAX_K:
                raise ValueError(f"ids must be [tokens, k] with k from 1 to {MAX_K}, not of shape {tuple(index.shape)}")
            listed = train._type(teacher, "teacher")
            _want(index, "ids", kind, (T, k), dev)
            _want(teacher, "teacher", teacher.dtype, (T, k), dev)
            second, third = teacher.data_ptr(), None
            if mask is not None:
                if mask.dtype not in (torch.bool, torch.uint8):
                    raise TypeError(f"mask is {mask.dtype}: bool and uint8 are supported")
                third = _want(mask, "mask", mask.dtype, (T,), dev).data_ptr()
            temperature = float(temperature)   # as it is now: descriptions are kept by value
        self.used = (hidden, weight, index, teacher, mask)
        self.ref = _described(T, across[0], D, *hidden.stride(), *weight.stride(), dtype, wide, k, listed, temperature)
        self.pointers = (hidden.data_ptr(), weight.data_ptr(), index.data_ptr(), second, third)

    def workspace(self, size_of):
        """New memory, of the stream that the call is made on."""
        size = size_of(self.ref, self.pointers[1])
        if not size:   # the call says which limit is broken
            _check(_lib.nest_head_loss(self.ref, *self.pointers, *[None] * 5, 0, None), "nest_head_loss")
        return train._torch.empty(size, dtype=train._torch.uint8, device=self.device), size


def _span(t):
    """(first, behind the last) address of a tensor's numbers."""
    at = t.data_ptr()
    if t.is_contiguous():
        return at, at + t.nbytes
    return at, at + (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * t.element_size()


def _touches(low, high, t):
    """Whether a row of t, a matrix of any strides, has numbers in these addresses (its rows are the steps of its
    larger stride, and all between a row's first and last number counts as its own)."""
    (inner, across), (outer, down) = sorted(zip(t.stride(), t.shape))
    at, size = t.data_ptr(), t.element_size()
    length, step = ((across - 1) * inner + 1) * size, outer * size
    if not step:
        return low < at + length and at < high
    return max(0, (low - at - length) // step + 1) <= min(down - 1, (high - 1 - at) // step)


def _apart(results, names, inputs):
    """An error where a result shares memory with an input or with another result: the kernels read the
    inputs while they write the results."""
    spans = [(*_span(t), t) for t in inputs if t is not None]
    for t, name in zip(results, names):
        if t is None:
            continue
        low, high = _span(t)
        if low == high:
            continue
        for first, end, other in spans:
            if first < high and low < end and first != end and \
                    (other.is_contiguous() or other.dim() != 2 or _touches(low, high, other)):
                raise ValueError(f"{name} shares memory with an input or with another result")
        spans.append((low, high, t))


def _forward(x: _Inputs, out, stream) -> HeadLoss:
    torch, dev, T = train._torch, x.device, x.shape[0][0]
    guard = _enter(dev, stream, () if stream is None else (*x.used, *(out or ())))
    given = out is not None
    try:
        f32 = torch.float32
        if given:
            _want(out.loss, "out.loss", f32, (), dev)
            _want(out.losses, "out.losses", f32, (T,), dev)
            _want(out.lse, "out.lse", f32, (T,), dev)
            _want(out.tokens, "out.tokens", torch.int32, (1,), dev)
            _apart(out, ("out.loss", "out.losses", "out.lse", "out.tokens"), x.used)
        else:
            empty = torch.empty
            out = HeadLoss(empty((), dtype=f32, device=dev), empty(T, dtype=f32, device=dev),
                           empty(T, dtype=f32, device=dev), empty(1, dtype=torch.int32, device=dev))
        loss, losses, lse, tokens = out
        ws, size = x.workspace(_lib.nest_head_loss_workspace_size)
        rc = _lib.nest_head_loss(x.ref, *x.pointers, loss.data_ptr(), losses.data_ptr(), lse.data_ptr(), tokens.data_ptr(),
                                 ws.data_ptr(), size, train._raw_stream(dev.index))
    finally:
        if guard is not None:
            guard.leave()
    _check(rc, "nest_head_loss")
    if given:
        train._written(out)
    return out


def _backward(x: _Inputs, result, grad_loss, grad_losses, out, stream, needs=(True, True)):
    torch, dev, (T, D) = train._torch, x.device, x.shape[0]
    if not any(needs):
        raise ValueError("neither gradient is needed")
    lse = _want(result.lse, "result.lse", torch.float32, (T,), dev)
    if grad_loss is not None:
        _want(grad_loss, "grad_loss", torch.float32, grad_loss.shape, dev)
        if grad_loss.numel() != 1:
            raise ValueError(f"grad_loss must be one number, not of shape {tuple(grad_loss.shape)}")
    if grad_losses is not None:
        _want(grad_losses, "grad_losses", torch.float32, (T,), dev)
    kind = x.used[0].dtype
    guard = _enter(dev, stream, () if stream is None else (*x.used, lse, grad_loss, grad_losses, *(out or ())))
    given = out is not None
    try:
        for_hidden, for_weight = needs
        across, down = x.shape
        if given:
            first = _want(out[0], "out[0]", kind, across, dev) if for_hidden else None
            second = _want(out[1], "out[1]", kind, down, dev) if for_weight else None
            _apart((first, second), ("out[0]", "out[1]"), (*x.used, lse, grad_loss, grad_losses))
        else:
            first = torch.empty(across, dtype=kind, device=dev) if for_hidden else None
            second = torch.empty(down, dtype=kind, device=dev) if for_weight else None
        out = first, second
        ws, size = x.workspace(_lib.nest_head_backward_workspace_size)
        rc = _lib.nest_head_loss_backward(
            x.ref, *x.pointers, lse.data_ptr(), None if grad_loss is None else grad_loss.data_ptr(),
            None if grad_losses is None else grad_losses.data_ptr(), None if first is None else first.data_ptr(),
            None if second is None else second.data_ptr(), ws.data_ptr(), size, train._raw_stream(dev.index))
    finally:
        if guard is not None:
            guard.leave()
    _check(rc, "nest_head_loss_backward")
    if given:
        train._written(tuple(t for t in out if t is not None))
    return out


def cross_entropy(hidden, weight, labels, out: HeadLoss | None = None, stream=None) -> HeadLoss:
    """nest_head_loss with labels: the cross entropy of each token's label under the softmax of its
    logits hidden @ weight.T, and its mean.

    hidden [T, D] and weight [V, D] (any strides; both bfloat16 or both float16); labels [T] (int64 or
    int32): a token whose label is not in [0, V) does not count (-100, padding), whatever it holds.
    Weights whose rows are contiguous and 16-byte aligned are read in place, others are copied by
    every call.  out: buffers to write instead of new ones, which share no memory with the inputs or each
    other."""
    return _forward(_Inputs(hidden, weight, labels, None, None, 1.0), out, stream)


def cross_entropy_backward(hidden, weight, labels, result: HeadLoss, grad_loss=None, grad_losses=None, out=None,
                           stream=None, needs=(True, True)):
    """nest_head_loss_backward with labels: (grad_hidden [T, D], grad_weight [V, D]), in the inputs'
    type, from the gradients of the loss (float32 scalar tensor) and of the losses (float32 [T]);
    None counts as zero.  out: two contiguous tensors to write instead of new ones, which share no memory
    with the inputs or each other.  needs: which of the
    two gradients are computed (a frozen head's weights need none); None takes the other's place."""
    return _backward(_Inputs(hidden, weight, labels, None, None, 1.0), result, grad_loss, grad_losses, out, stream, needs)


def distill(hidden, weight, ids, teacher, temperature: float = 1.0, mask=None, out: HeadLoss | None = None,
            stream=None) -> HeadLoss:
    """nest_head_loss with a teacher: temperature^2 times the divergence of the teacher's softmax over
    its listed logits from the softmax of hidden @ weight.T, both at this temperature, per token
    and its mean.

    hidden, weight and out as for `cross_entropy`; ids [T, k] (int64 or int32, in any order, k up to
    256) and teacher [T, k] (float32, bfloat16 or float16): columns and the teacher's logits of them.
    A slot whose id is not in [0, V) or whose logit is minus infinity does not count; a token counts when
    one of its slots does and mask [T] (bool or uint8) is None or True.  temperature: a number from 2^-10 to
    2^10 (of a tensor its value at the call, which waits for the GPU where the tensor is there)."""
    return _forward(_Inputs(hidden, weight, ids, teacher, mask, temperature), out, stream)


def distill_backward(hidden, weight, ids, teacher, result: HeadLoss, grad_loss=None, grad_losses=None,
                     temperature: float = 1.0, mask=None, out=None, stream=None, needs=(True, True)):
    """nest_head_loss_backward with a teacher (which gets no gradient), as `cross_entropy_backward`;
    temperature and mask as in the forward call."""
    return _backward(_Inputs(hidden, weight, ids, teacher, mask, temperature), result, grad_loss, grad_losses, out,
                     stream, needs)


def waits_given_up(device="cuda", stream=None) -> int:
    """nest_head_waits_given_up: how many warps of these calls on the device gave up waiting (and left NaN) since the
    library was loaded, 0 unless the GPU failed or stood still.  Waits for the work of the stream; not under capture."""
    torch = train._torch or train._load_torch()
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    guard, count = _enter(device, stream), C.c_int64()
    try:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the count is read on the host: not under capture")
        _check(lib().nest_head_waits_given_up(C.byref(count), train._raw_stream(device.index)), "nest_head_waits_given_up")
    finally:
        if guard is not None:
            guard.leave()
    return count.value


def _functions():
    import torch

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, hidden, weight, index, teacher, mask, temperature):
            r = _forward(_Inputs(hidden, weight, index, teacher, mask, temperature), None, None)
            ctx.save_for_backward(hidden, weight, index, teacher, mask, r.lse)   # the losses may be changed in place
            ctx.temperature = temperature
            ctx.set_materialize_grads(False)   # of the two losses mostly one has a gradient
            ctx.mark_non_differentiable(r.lse, r.tokens)
            return tuple(r)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, grad_loss, grad_losses, _lse, _tokens):
            hidden, weight, index, teacher, mask, lse = ctx.saved_tensors
            x = _Inputs(hidden, weight, index, teacher, mask, ctx.temperature)
            return (*_backward(x, HeadLoss(None, None, lse, None), None if grad_loss is None else grad_loss.contiguous(),
                               None if grad_losses is None else grad_losses.contiguous(), None, None,
                               ctx.needs_input_grad[:2]), None, None, None, None)

    return Loss


_function = None


def _differentiable(*args) -> HeadLoss:
    global _function
    if _function is None:
        _function = _functions()
    torch = train._torch or train._load_torch()
    if torch.is_grad_enabled() and any(t.requires_grad for t in args[:2]) and args[0].is_cuda and \
            torch.cuda.is_current_stream_capturing():
        raise RuntimeError("a captured backward pass ends the process where an eager graph of the same leaves lives: "
                           "capture cross_entropy or distill and its backward function instead")
    return HeadLoss(*_function.apply(*args))


def label_loss(hidden, weight, labels) -> HeadLoss:
    """`cross_entropy` with gradients: the result's loss and losses are differentiable in the hidden
    states and the weights (lse carries none).  Once: a derivative of that gradient raises.  Not under
    capture: the functions above can be captured in a CUDA graph."""
    return _differentiable(hidden, weight, labels, None, None, 1.0)


def teacher_loss(hidden, weight, ids, teacher, temperature: float = 1.0, mask=None) -> HeadLoss:
    """`distill` with gradients, as `label_loss`; the teacher's logits and the temperature get none, and the
    backward pass is at the temperature of this call."""
    return _differentiable(hidden, weight, ids, teacher, mask, float(temperature))
