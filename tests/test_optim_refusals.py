"""Refusals of the optimizer step's and the gradient norm's entry points,
before anything reaches a device (no GPU)."""

import ctypes

import pytest
import torch

from full_vocabulary_reverse_b200 import AdamW, RKLError, binding, grad_norm
from full_vocabulary_reverse_b200.build import build

GOOD = 0x10000


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def _adamw(L, **kw):
    a = dict(n=2, params=[GOOD, GOOD + 4], grads=[GOOD, GOOD + 4], numel=[3, 5], pd=[1, 1], gd=[1, 1], wd=[0.0, 0.0],
             bits=32, m=GOOD, v=GOOD, ms=0, vs=0, master=0, control=GOOD, lr=0.1, lr_dev=0, b1=0.9, b2=0.999, eps=1e-8,
             norm=0, max_norm=1.0)
    a.update(kw)
    vp = lambda x: ctypes.c_void_p(x) if x else None  # noqa: E731
    arr = lambda t, x: None if x is None else (t * len(x))(*x)  # noqa: E731
    return L.rkl_adamw_step(a["n"], arr(ctypes.c_void_p, a["params"]), arr(ctypes.c_void_p, a["grads"]),
                            arr(ctypes.c_int64, a["numel"]), arr(ctypes.c_int32, a["pd"]), arr(ctypes.c_int32, a["gd"]),
                            arr(ctypes.c_float, a["wd"]), a["bits"], vp(a["m"]), vp(a["v"]), vp(a["ms"]), vp(a["vs"]),
                            vp(a["master"]), vp(a["control"]), a["lr"], vp(a["lr_dev"]), a["b1"], a["b2"], a["eps"], 0,
                            vp(a["norm"]), a["max_norm"], None)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), 2), (dict(numel=None), 1), (dict(numel=[3, -1]), 2), (dict(numel=[3, 1 << 40]), 2),
    (dict(params=None), 1), (dict(grads=None), 1), (dict(pd=None), 1), (dict(gd=None), 1), (dict(wd=None), 1),
    (dict(params=[None, GOOD]), 1), (dict(pd=[1, 7]), 3), (dict(gd=[2, 1]), 3), (dict(bits=16), 3),
    (dict(params=[GOOD + 2, GOOD]), 4), (dict(grads=[GOOD + 2, GOOD]), 4), (dict(gd=[0, 0], grads=[GOOD + 1, GOOD]), 4),
    (dict(m=0), 1), (dict(v=0), 1), (dict(m=GOOD + 16), 4), (dict(master=GOOD + 16), 4), (dict(bits=8), 1),
    (dict(bits=8, ms=GOOD), 1), (dict(control=0), 1), (dict(control=GOOD + 4), 4), (dict(lr=-0.1), 2),
    (dict(lr=float("nan")), 2), (dict(lr_dev=GOOD + 2), 4), (dict(b1=1.0), 2), (dict(b2=-0.1), 2), (dict(eps=-1.0), 2),
    (dict(norm=GOOD, max_norm=0.0), 2), (dict(norm=GOOD, max_norm=float("nan")), 2), (dict(norm=GOOD + 1), 4),
])
def test_adamw_argument_errors(L, change, status):
    assert _adamw(L, **change) == status, L.rkl_last_error()
    assert L.rkl_last_error()


def test_grad_norm_argument_errors(L):
    one = (ctypes.c_int64 * 1)(5)
    ptr = (ctypes.c_void_p * 1)(GOOD)
    code = (ctypes.c_int32 * 1)(1)
    g = ctypes.c_void_p(GOOD)
    need = ctypes.c_size_t(0)
    assert L.rkl_grad_norm_workspace_size(1, None) == 1
    assert L.rkl_grad_norm_workspace_size(-1, ctypes.byref(need)) == 2
    assert L.rkl_grad_norm_workspace_size(1, ctypes.byref(need)) == 0 and need.value > 0
    few = need.value
    assert L.rkl_grad_norm_workspace_size(1000, ctypes.byref(need)) == 0 and need.value > few
    ok = dict(n=1, grads=ptr, numel=one, dt=code, norm=g, ws=g, nbytes=few)

    def call(**kw):
        a = dict(ok, **kw)
        return L.rkl_grad_norm(a["n"], a["grads"], a["numel"], a["dt"], a["norm"], a["ws"], a["nbytes"], None)
    assert call(n=-1) == 2
    assert call(numel=None) == 1
    assert call(grads=None) == 1
    assert call(dt=None) == 1
    assert call(norm=None) == 1
    assert call(norm=ctypes.c_void_p(GOOD + 2)) == 4
    assert call(grads=(ctypes.c_void_p * 1)(GOOD + 2)) == 4
    assert call(dt=(ctypes.c_int32 * 1)(9)) == 3
    assert call(ws=None) == 5
    assert call(nbytes=few - 1) == 5
    assert call(ws=ctypes.c_void_p(GOOD + 8)) == 4


def test_state_size(L):
    numel = (ctypes.c_int64 * 4)(1, 0, 256, 257)
    at, total = (ctypes.c_int64 * 4)(), ctypes.c_int64(0)
    assert L.rkl_adamw_state_size(4, numel, at, ctypes.byref(total)) == 0
    assert list(at) == [0, 256, 256, 512] and total.value == 1024
    assert L.rkl_adamw_state_size(4, numel, None, None) == 1
    assert L.rkl_adamw_state_size(-2, numel, None, ctypes.byref(total)) == 2
    assert L.rkl_adamw_state_size(0, None, None, ctypes.byref(total)) == 0 and total.value == 0


def test_python_refusals_without_a_device():
    with pytest.raises(RKLError, match="a parameter"):
        AdamW([])
    with pytest.raises(RKLError, match="CUDA"):
        AdamW([torch.zeros(3)])
    with pytest.raises(RKLError, match="a gradient"):
        grad_norm([None])
    with pytest.raises(RKLError, match="CUDA"):
        grad_norm([torch.zeros(3)])
