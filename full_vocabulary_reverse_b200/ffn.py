"""The gated feed-forward block in front of the head:

    y = (act(x W_gate^T) * (x W_up^T)) W_down^T

``gated_ffn`` is differentiable; ``ffn_forward`` and ``ffn_backward`` are the
single passes.  Everything runs in the CUDA library on the current stream."""

from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from .binding import RKLError, _check, _dtype_code, _ptr, _stream, lib

ACT_SILU = 0
ACT_GELU = 1
ACT_GELU_TANH = 2
ACT_RELU = 3


def _sizes(x, W_gate, W_up, W_down):
    """(T, H, F, O) of a block, checked."""
    for name, t in (("x", x), ("W_gate", W_gate), ("W_up", W_up), ("W_down", W_down)):
        if not t.is_cuda or t.device != x.device or t.layout != torch.strided:
            raise RKLError(2, "%s must be a dense CUDA tensor beside x" % name)
        if t.dtype != x.dtype:
            raise RKLError(3, "%s is %s, x is %s" % (name, t.dtype, x.dtype))
    _dtype_code(x)
    if x.dim() != 2 or W_gate.dim() != 2 or W_up.shape != W_gate.shape or W_down.dim() != 2:
        raise RKLError(2, "x [T, H], W_gate and W_up [F, H], W_down [O, F] expected")
    (T, H), (F, H2), (O, F2) = x.shape, W_gate.shape, W_down.shape
    if H != H2 or F != F2:
        raise RKLError(2, "sizes do not fit: x %s, W_gate %s, W_down %s" % (tuple(x.shape), tuple(W_gate.shape),
                                                                            tuple(W_down.shape)))
    return T, H, F, O


def _workspace(x, T, H, F, O, backward):
    nbytes = ctypes.c_size_t(0)
    _check(lib().rkl_ffn_workspace_size(_dtype_code(x), T, H, F, O, backward, ctypes.byref(nbytes)))
    return torch.empty(nbytes.value, dtype=torch.uint8, device=x.device)


def _saved_size(T, F):
    n = ctypes.c_int64(0)
    _check(lib().rkl_ffn_saved_size(T, F, ctypes.byref(n)))
    return n.value


def ffn_forward(x, W_gate, W_up, W_down, activation=ACT_SILU, save=False):
    """(y [T, O], saved): saved (fp32, g and u in the library's own order, for
    ``ffn_backward``) is None unless ``save``."""
    T, H, F, O = _sizes(x, W_gate, W_up, W_down)
    x, W_gate, W_up, W_down = (t.contiguous() for t in (x, W_gate, W_up, W_down))
    with torch.cuda.device(x.device):
        y = torch.empty((T, O), dtype=x.dtype, device=x.device)
        saved = torch.empty(_saved_size(T, F), dtype=torch.float32, device=x.device) if save else None
        ws = _workspace(x, T, H, F, O, 0)
        _check(lib().rkl_ffn_forward(_ptr(x), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _dtype_code(x), activation,
                                     T, H, F, O, _ptr(y), _ptr(saved), _ptr(ws), ws.numel(), _stream(x.device)))
    return y, saved


def ffn_backward(x, W_gate, W_up, W_down, dy, saved, activation=ACT_SILU, needs=(True, True, True, True)):
    """(dx, dW_gate, dW_up, dW_down) in the dtype of x; None where ``needs``
    says so."""
    T, H, F, O = _sizes(x, W_gate, W_up, W_down)
    if dy.shape != (T, O) or dy.device != x.device or dy.dtype != x.dtype:
        raise RKLError(2, "dy must be a [%d, %d] tensor of x's dtype and device" % (T, O))
    if saved.shape != (_saved_size(T, F),) or saved.dtype != torch.float32 or saved.device != x.device or not saved.is_contiguous():
        raise RKLError(2, "saved must be what ffn_forward gave for the same sizes")
    x, W_gate, W_up, W_down, dy = (t.contiguous() for t in (x, W_gate, W_up, W_down, dy))
    with torch.cuda.device(x.device):
        out = [torch.empty_like(t) if need else None for t, need in zip((x, W_gate, W_up, W_down), needs)]
        ws = _workspace(x, T, H, F, O, 1)
        _check(lib().rkl_ffn_backward(_ptr(x), _ptr(W_gate), _ptr(W_up), _ptr(W_down), _dtype_code(x), activation,
                                      T, H, F, O, _ptr(dy), _ptr(saved), *[_ptr(t) for t in out], _ptr(ws), ws.numel(),
                                      _stream(x.device)))
    return tuple(out)


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W_gate, W_up, W_down, activation):
        y, saved = ffn_forward(x, W_gate, W_up, W_down, activation, save=True)
        ctx.save_for_backward(x, W_gate, W_up, W_down, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, W_gate, W_up, W_down, saved = ctx.saved_tensors
        return ffn_backward(x, W_gate, W_up, W_down, dy, saved, ctx.activation, ctx.needs_input_grad[:4]) + (None,)


def gated_ffn(x, W_gate, W_up, W_down, activation=ACT_SILU):
    """y = (act(x W_gate^T) * (x W_up^T)) W_down^T for x [..., H], W_gate and
    W_up [F, H], W_down [O, F]; differentiable in all four.  Keeps g and u (fp32)
    for the backward pass only where a gradient is wanted.

    To capture a backward pass in a CUDA graph, let no autograd graph of the
    same leaves from another stream be alive (PyTorch would tie the capture to
    that stream and break it), or capture ``ffn_forward`` and ``ffn_backward``."""
    if activation not in (ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU):
        raise RKLError(3, "unknown activation %r" % (activation,))
    if x.dim() < 1:
        raise RKLError(2, "x [..., H] expected")
    rows = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    if torch.is_grad_enabled() and any(t.requires_grad for t in (x, W_gate, W_up, W_down)):
        y = _GatedFFN.apply(rows, W_gate, W_up, W_down, activation)
    else:
        y = ffn_forward(rows, W_gate, W_up, W_down, activation)[0]
    return y if x.dim() == 2 else y.view(*x.shape[:-1], W_down.shape[0])
