"""The gated feed-forward block in front of the head:

    y = (act(x W_gate^T) * (x W_up^T)) W_down^T

``gated_ffn`` is differentiable (in reverse mode); ``ffn_forward`` and
``ffn_backward`` are the single passes, outside autograd.  Everything runs in
the CUDA library on the current stream."""

from __future__ import annotations

import ctypes
from functools import lru_cache

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from .binding import DT_BF16, DT_FP32, RKLError, _check, _on_device, _raw_stream, lib

ACT_SILU = 0
ACT_GELU = 1
ACT_GELU_TANH = 2
ACT_RELU = 3

_CODES = {torch.bfloat16: DT_BF16, torch.float32: DT_FP32}


def _sizes(x, W_gate, W_up, W_down):
    """(dtype code, T, H, F, O) of a block, checked."""
    dtype, index = x.dtype, x.get_device()
    if not (W_gate.dtype == W_up.dtype == W_down.dtype == dtype and x.is_cuda and
            W_gate.get_device() == W_up.get_device() == W_down.get_device() == index):
        for name, t in (("x", x), ("W_gate", W_gate), ("W_up", W_up), ("W_down", W_down)):
            if not t.is_cuda or t.get_device() != index:
                raise RKLError(2, "%s must be a CUDA tensor on the device of x" % name)
            if t.dtype != dtype:
                raise RKLError(3, "%s is %s, x is %s" % (name, t.dtype, dtype))
    code = _CODES.get(dtype)
    if code is None:
        raise RKLError(3, "unsupported dtype %s" % (dtype,))
    shape = W_gate.shape
    if x.dim() != 2 or len(shape) != 2 or W_up.shape != shape or W_down.dim() != 2:
        raise RKLError(2, "x [T, H], W_gate and W_up [F, H], W_down [O, F] expected")
    (T, H), (F, H2), (O, F2) = x.shape, shape, W_down.shape
    if H != H2 or F != F2:
        raise RKLError(2, "sizes do not fit: x %s, W_gate %s, W_down %s" % (tuple(x.shape), tuple(shape),
                                                                            tuple(W_down.shape)))
    return code, T, H, F, O


def _ready(t):
    """t, or a copy that is contiguous from a 16-byte boundary."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


@lru_cache(maxsize=1024)
def _workspace_size(code, T, H, F, O, backward):
    nbytes = ctypes.c_size_t(0)
    _check(lib().rkl_ffn_workspace_size(code, T, H, F, O, backward, ctypes.byref(nbytes)))
    return nbytes.value


@lru_cache(maxsize=1024)
def _saved_size(T, F):
    n = ctypes.c_int64(0)
    _check(lib().rkl_ffn_saved_size(T, F, ctypes.byref(n)))
    return n.value


def ffn_forward(x, W_gate, W_up, W_down, activation=ACT_SILU, save=False):
    """(y [T, O], saved): saved (fp32, g and u in the library's own order, for
    ``ffn_backward``) is None unless ``save``."""
    code, T, H, F, O = _sizes(x, W_gate, W_up, W_down)
    # (bound to names: a copy has to live until the call returns)
    x, W_gate, W_up, W_down = _ready(x), _ready(W_gate), _ready(W_up), _ready(W_down)
    device = x.device
    with _on_device(device.index):
        y = torch.empty((T, O), dtype=x.dtype, device=device)
        saved = torch.empty(_saved_size(T, F), dtype=torch.float32, device=device) if save else None
        nbytes = _workspace_size(code, T, H, F, O, 0)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _check(lib().rkl_ffn_forward(x.data_ptr(), W_gate.data_ptr(), W_up.data_ptr(), W_down.data_ptr(), code, activation,
                                     T, H, F, O, y.data_ptr(), saved.data_ptr() if save else None, ws.data_ptr(), nbytes,
                                     _raw_stream(device.index)))
    return y, saved


def ffn_backward(x, W_gate, W_up, W_down, dy, saved, activation=ACT_SILU, needs=(True, True, True, True)):
    """(dx, dW_gate, dW_up, dW_down) in the dtype of x; None where ``needs``
    says so."""
    code, T, H, F, O = _sizes(x, W_gate, W_up, W_down)
    device = x.device
    if dy.shape != (T, O) or dy.device != device or dy.dtype != x.dtype:
        raise RKLError(2, "dy must be a [%d, %d] tensor of x's dtype and device" % (T, O))
    if saved.shape != (_saved_size(T, F),) or saved.dtype != torch.float32 or saved.device != device \
            or not saved.is_contiguous():
        raise RKLError(2, "saved must be what ffn_forward gave for the same sizes")
    x, W_gate, W_up, W_down, dy = _ready(x), _ready(W_gate), _ready(W_up), _ready(W_down), _ready(dy)
    with _on_device(device.index):
        out = [torch.empty_like(t) if need else None for t, need in zip((x, W_gate, W_up, W_down), needs)]
        nbytes = _workspace_size(code, T, H, F, O, 1)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _check(lib().rkl_ffn_backward(x.data_ptr(), W_gate.data_ptr(), W_up.data_ptr(), W_down.data_ptr(), code, activation,
                                      T, H, F, O, dy.data_ptr(), saved.data_ptr(),
                                      *[None if t is None else t.data_ptr() for t in out], ws.data_ptr(), nbytes,
                                      _raw_stream(device.index)))
    return tuple(out)


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W_gate, W_up, W_down, activation):
        y, saved = ffn_forward(x, W_gate, W_up, W_down, activation, save=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, W_gate, W_up, W_down, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        if forward_ad._current_level >= 0 and forward_ad.unpack_dual(dy).tangent is not None:
            raise NotImplementedError("gated_ffn has no jvp: no forward mode through its backward pass")
        x, W_gate, W_up, W_down, saved = ctx.saved_tensors
        return ffn_backward(x, W_gate, W_up, W_down, dy, saved, ctx.activation, ctx.needs_input_grad[:4]) + (None,)


def gated_ffn(x, W_gate, W_up, W_down, activation=ACT_SILU):
    """y = (act(x W_gate^T) * (x W_up^T)) W_down^T for x [..., H], W_gate and
    W_up [F, H], W_down [O, F]; differentiable in all four, in reverse mode (a
    tangent of forward mode is refused).  Keeps g and u (fp32) for the backward
    pass only where a gradient is wanted.

    To capture a backward pass in a CUDA graph, let no autograd graph of the
    same leaves from another stream be alive (PyTorch would tie the capture to
    that stream and break it), or capture ``ffn_forward`` and ``ffn_backward``."""
    if activation not in (ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU):
        raise RKLError(3, "unknown activation %r" % (activation,))
    if x.dim() < 1:
        raise RKLError(2, "x [..., H] expected")
    rows = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    # (inside a forward-mode level autograd looks for tangents and refuses them)
    if forward_ad._current_level >= 0 or \
            torch.is_grad_enabled() and any(t.requires_grad for t in (x, W_gate, W_up, W_down)):
        y = _GatedFFN.apply(rows, W_gate, W_up, W_down, activation)
    else:
        y = ffn_forward(rows, W_gate, W_up, W_down, activation)[0]
    return y if x.dim() == 2 else y.view(*x.shape[:-1], W_down.shape[0])
