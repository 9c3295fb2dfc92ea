"""The optimizer step behind the loss: ``grad_norm`` over many gradients and
``AdamW`` over many tensors, with moments in 32 bits or in 8.

    opt = AdamW([W_gate, W_up, W_down, W_s], lr=1e-4, weight_decay=[0.1] * 4, state_bits=8)
    loss.backward()
    norm = opt.step(max_norm=1.0)
    for w in opt.params:
        w.grad = None  # backward passes add to .grad; a step leaves it

A step is one launch (two more with ``max_norm``), with nothing copied to the
device and no host synchronisation: it can be captured in a CUDA graph, whose
replays count the steps themselves.
"""

from __future__ import annotations

import ctypes
from array import array
from functools import lru_cache
from operator import attrgetter

import torch

from .binding import DT_BF16, DT_FP32, RKLError, _check, _on_device, _raw_stream, lib

_CODES = {torch.bfloat16: DT_BF16, torch.float32: DT_FP32}
STATE_BLOCK = 256  # elements under one scale of an 8-bit state; each tensor's place in the state is a multiple


def _code(t, what):
    c = _CODES.get(t.dtype)
    if c is None:
        raise RKLError(3, "%s has dtype %s: bfloat16 or float32" % (what, t.dtype))
    return c


def _address(a):
    """Of the entries of an `array` (which the caller keeps)."""
    return a.buffer_info()[0]


@lru_cache(maxsize=64)
def _norm_workspace_size(n):
    nbytes = ctypes.c_size_t(0)
    _check(lib().rkl_grad_norm_workspace_size(n, ctypes.byref(nbytes)))
    return nbytes.value


_shape = attrgetter("shape")


def _plain(tensors, shapes, index):
    """Whether all are dense and contiguous tensors of these shapes (None: any)
    on device `index`; False where one has to be looked at by itself."""
    try:
        return (all(map(torch.Tensor.is_contiguous, tensors)) and
                set(map(torch.Tensor.get_device, tensors)) == {index} and
                (shapes is None or list(map(_shape, tensors)) == shapes))
    except (RuntimeError, TypeError):  # no layout with strides; a None
        return False


def _norm_into(n, ptrs, numel, codes, device):
    """The launches of grad_norm over n contiguous gradients on the current
    device, given as arrays of addresses (0: absent), element counts and dtype
    codes."""
    nbytes = _norm_workspace_size(n)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    norm = torch.empty(1, dtype=torch.float32, device=device)
    _check(lib().rkl_grad_norm(n, _address(ptrs), _address(numel), _address(codes), norm.data_ptr(), ws.data_ptr(), nbytes,
                               _raw_stream(device.index)))
    return norm


@lru_cache(maxsize=64)
def _codes_of(dtypes):
    return array("i", [_CODES[d] for d in dtypes])


def _dtype_codes(tensors, what):
    """Their dtype codes as an array (of a ``None``: fp32's)."""
    try:
        return _codes_of(tuple([torch.float32 if t is None else t.dtype for t in tensors]))
    except KeyError:
        for i, t in enumerate(tensors):
            if t is not None:
                _code(t, "%s %d" % (what, i))
        raise


def grad_norm(grads):
    """The 2-norm of all gradients together, a 1-element fp32 tensor on their
    device (no host synchronisation), outside autograd.  ``None`` entries are
    passed over."""
    grads = [g for g in grads if g is not None]
    if not grads:
        raise RKLError(2, "grad_norm needs a gradient")
    device = grads[0].device
    index = grads[0].get_device()
    if index < 0:
        raise RKLError(2, "gradients must be CUDA tensors")
    with _on_device(index):
        if not _plain(grads, None, index):
            for g in grads:
                if g.get_device() != index or g.layout != torch.strided:
                    raise RKLError(2, "gradients must be dense tensors on one device")
            grads = [g.contiguous() for g in grads]
        codes = _dtype_codes(grads, "gradient")
        return _norm_into(len(grads), array("Q", [g.data_ptr() for g in grads]), array("q", [g.numel() for g in grads]), codes,
                          device)


class AdamW:
    """AdamW with decoupled weight decay over a fixed list of tensors.

    ``params``: contiguous bf16 or fp32 CUDA tensors on one device, updated in
    place.  ``weight_decay``: one number, or one for each tensor.  ``lr``: a
    number, or a 1-element fp32 tensor on the device, which a captured step
    reads anew at each replay.  ``state_bits``: 32 (fp32 moments) or 8 (e4m3
    codes with an fp32 scale for 256 elements).  ``master_weights``: keep fp32
    copies of the parameters and update those; the parameters are their
    rounded values (without it a bf16 parameter loses updates below half its
    last place).  ``seed``: of the 8-bit form's stochastic rounding.  To follow a
    schedule, give ``step`` its ``lr`` (or change the number in the tensor); there
    are no parameter groups, and gradients are cleared by the caller.

    The state: ``exp_avg``, ``exp_avg_sq`` (flat; tensor i at
    ``[offsets[i], offsets[i] + numel)``), for 8 bits ``exp_avg_scale`` and
    ``exp_avg_sq_scale``, ``master`` and ``steps`` (1 int32 on the device).
    A step keeps running on the caller's current stream; steps of one object
    must be ordered by the caller.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32,
                 master_weights=False, seed=0):
        self.params = list(params)
        n = len(self.params)
        if n == 0:
            raise RKLError(2, "AdamW needs a parameter")
        device = self.params[0].device
        if not self.params[0].is_cuda:
            raise RKLError(2, "parameters must be CUDA tensors")
        for i, p in enumerate(self.params):
            if not p.is_cuda or p.device != device or p.layout != torch.strided or not p.is_contiguous():
                raise RKLError(2, "parameter %d: parameters must be contiguous CUDA tensors on one device" % i)
            _code(p, "parameter %d" % i)
        spans = sorted((p.data_ptr(), p.data_ptr() + p.numel() * p.element_size()) for p in self.params if p.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise RKLError(2, "two parameters share memory (is a tied weight listed twice?)")
        if state_bits not in (32, 8):
            raise RKLError(3, "state_bits = %r is neither 32 nor 8" % (state_bits,))
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(w) for w in weight_decay]
        if len(decay) != n:
            raise RKLError(2, "%d weight decays for %d parameters" % (len(decay), n))
        if len(betas) != 2 or not all(0 <= b < 1 for b in betas):
            raise RKLError(2, "betas %r outside [0, 1)" % (betas,))
        if not eps >= 0:
            raise RKLError(2, "eps = %r is negative" % (eps,))
        self.lr, self.betas, self.eps = self._checked_lr(lr, device), tuple(betas), eps
        self.weight_decay, self.state_bits, self.seed, self.device = decay, state_bits, int(seed) & 0xFFFFFFFF, device

        self._numel = array("q", [p.numel() for p in self.params])
        offsets, total = array("q", [0] * n), ctypes.c_int64(0)
        _check(lib().rkl_adamw_state_size(n, _address(self._numel), _address(offsets), ctypes.byref(total)))
        self.offsets, total = list(offsets), total.value
        dt = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        self.exp_avg = torch.zeros(total, dtype=torch.uint8 if state_bits == 8 else dt, device=device).view(dt)
        self.exp_avg_sq = torch.zeros_like(self.exp_avg)
        blocks = total // STATE_BLOCK
        self.exp_avg_scale = torch.zeros(blocks, device=device) if state_bits == 8 else None
        self.exp_avg_sq_scale = torch.zeros(blocks, device=device) if state_bits == 8 else None
        self.master = None
        if master_weights:
            self.master = torch.zeros(total, device=device)
            for p, at in zip(self.params, self.offsets):
                self.master[at:at + p.numel()] = p.detach().reshape(-1)
        self._control = torch.zeros(2, dtype=torch.int32, device=device)
        self.steps = self._control[:1]

        self._shapes = [p.shape for p in self.params]
        self._ptrs = array("Q", [p.data_ptr() for p in self.params])
        self._dtypes = _dtype_codes(self.params, "parameter")
        self._decay = array("f", decay)
        # an update moves a tensor's version, so that a backward pass through an older value is refused
        self._tracked = [p for p in self.params if not p.is_inference()]

    @staticmethod
    def _checked_lr(lr, device):
        if isinstance(lr, torch.Tensor):
            if lr.dtype != torch.float32 or lr.numel() != 1 or lr.device != device:
                raise RKLError(2, "a learning rate on the device must be a 1-element float32 tensor beside the parameters")
        elif not lr >= 0:
            raise RKLError(2, "lr = %r is negative" % (lr,))
        return lr

    def step(self, grads=None, lr=None, max_norm=None, norm=None):
        """One step.  ``grads``: a gradient for each parameter (default: their
        ``.grad``); ``None`` leaves a tensor and its moments as they are.
        ``max_norm`` scales the gradients down to this global norm, which is
        ``norm`` (a 1-element fp32 tensor, of ``grad_norm``) or found here.
        With either, a step whose norm is infinite or NaN changes nothing and
        does not count.  Returns the norm (None without either)."""
        n, device = len(self.params), self.device
        if array("Q", [p.data_ptr() for p in self.params]) != self._ptrs:
            raise RKLError(2, "a parameter moved in memory since AdamW was made")
        grads = [p.grad for p in self.params] if grads is None else list(grads)
        if len(grads) != n:
            raise RKLError(2, "%d gradients for %d parameters" % (len(grads), n))
        lr = self.lr if lr is None else self._checked_lr(lr, device)
        if max_norm is not None and not max_norm > 0:
            raise RKLError(2, "max_norm = %r is not positive" % (max_norm,))
        if norm is not None and (norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != device):
            raise RKLError(2, "norm must be a 1-element float32 tensor beside the parameters")
        index = device.index
        with _on_device(index):
            if _plain(grads, self._shapes, index):
                ptrs = array("Q", [g.data_ptr() for g in grads])
            else:
                grads = self._each_checked(grads, index)
                ptrs = array("Q", [0 if g is None else g.data_ptr() for g in grads])
            codes = _dtype_codes(grads, "gradient")
            if max_norm is not None and norm is None:
                norm = _norm_into(n, ptrs, self._numel, codes, device)
            lr_dev = lr if isinstance(lr, torch.Tensor) else None
            small = self.state_bits == 8
            _check(lib().rkl_adamw_step(
                n, _address(self._ptrs), _address(ptrs), _address(self._numel), _address(self._dtypes), _address(codes),
                _address(self._decay), self.state_bits, self.exp_avg.data_ptr(), self.exp_avg_sq.data_ptr(),
                self.exp_avg_scale.data_ptr() if small else None, self.exp_avg_sq_scale.data_ptr() if small else None,
                None if self.master is None else self.master.data_ptr(), self._control.data_ptr(),
                0.0 if lr_dev is not None else float(lr), None if lr_dev is None else lr_dev.data_ptr(),
                self.betas[0], self.betas[1], self.eps, self.seed, None if norm is None else norm.data_ptr(),
                float("inf") if max_norm is None else float(max_norm), _raw_stream(index)))
        if self._tracked:
            torch.autograd.graph.increment_version(self._tracked)
        return norm

    def _each_checked(self, grads, index):
        """The gradients one by one: contiguous, or the reason why not."""
        out = []
        for i, (g, shape) in enumerate(zip(grads, self._shapes)):
            if g is not None:
                if g.shape != shape or g.get_device() != index or g.layout != torch.strided:
                    raise RKLError(2, "gradient %d must be a dense tensor of its parameter's shape and device" % i)
                g = g.contiguous()
            out.append(g)
        return out

    def moments(self, i):
        """(exp_avg, exp_avg_sq) of parameter i as fp32 tensors of its shape."""
        at, n = self.offsets[i], self.params[i].numel()
        out = []
        for x, scale in ((self.exp_avg, self.exp_avg_scale), (self.exp_avg_sq, self.exp_avg_sq_scale)):
            first, last = at // STATE_BLOCK, -(-(at + n) // STATE_BLOCK)
            v = x[first * STATE_BLOCK:last * STATE_BLOCK].float()
            if scale is not None:
                v = (v.view(-1, STATE_BLOCK) * scale[first:last, None]).view(-1)
            out.append(v[:n].clone().view(self._shapes[i]))
        return tuple(out)

    def state_dict(self):
        """The state's tensors by name (the live ones, not copies)."""
        names = ["exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master", "steps"]
        return {k: getattr(self, k) for k in names if getattr(self, k) is not None}

    def load_state_dict(self, state):
        """Copies a ``state_dict`` of the same tensors and options in."""
        mine = self.state_dict()
        if set(state) != set(mine):
            raise RKLError(2, "state has %s, expected %s" % (sorted(state), sorted(mine)))
        for k, t in mine.items():
            if state[k].shape != t.shape or state[k].dtype != t.dtype:
                raise RKLError(2, "%s is %s %s, expected %s %s" % (k, tuple(state[k].shape), state[k].dtype,
                                                                  tuple(t.shape), t.dtype))
        for k, t in mine.items():
            t.copy_(state[k])
