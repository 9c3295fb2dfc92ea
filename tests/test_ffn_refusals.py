"""Refusals of the gated feed-forward block's entry points, before anything
reaches a device (no GPU)."""

import ctypes

import pytest
import torch

from full_vocabulary_reverse_b200 import RKLError, binding, gated_ffn
from full_vocabulary_reverse_b200.build import build

GOOD = 0x10000
BASE = dict(x=GOOD, wg=GOOD, wu=GOOD, wd=GOOD, dtype=0, act=0, T=4, H=16, F=32, O=8, y=GOOD, dy=GOOD, saved=GOOD, dx=GOOD,
            dwg=GOOD, dwu=GOOD, dwd=GOOD, ws=GOOD, nbytes=1 << 30)


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def vp(x):
    return ctypes.c_void_p(x) if x else None


def forward(L, **kw):
    a = dict(BASE, **kw)
    return L.rkl_ffn_forward(vp(a["x"]), vp(a["wg"]), vp(a["wu"]), vp(a["wd"]), a["dtype"], a["act"], a["T"], a["H"], a["F"],
                             a["O"], vp(a["y"]), vp(a["saved"]), vp(a["ws"]), a["nbytes"], None)


def backward(L, **kw):
    a = dict(BASE, **kw)
    return L.rkl_ffn_backward(vp(a["x"]), vp(a["wg"]), vp(a["wu"]), vp(a["wd"]), a["dtype"], a["act"], a["T"], a["H"], a["F"],
                              a["O"], vp(a["dy"]), vp(a["saved"]), vp(a["dx"]), vp(a["dwg"]), vp(a["dwu"]), vp(a["dwd"]),
                              vp(a["ws"]), a["nbytes"], None)


BOTH = [(dict(dtype=5), 3), (dict(act=4), 3), (dict(act=-1), 3), (dict(T=-1), 2), (dict(H=0), 2), (dict(F=0), 2),
        (dict(O=0), 2), (dict(T=1 << 31), 2), (dict(F=1 << 21), 2), (dict(x=0), 1), (dict(wg=0), 1), (dict(wu=0), 1),
        (dict(wd=0), 1), (dict(x=GOOD + 1), 4), (dict(x=GOOD + 8), 4), (dict(wd=GOOD + 2), 4), (dict(wd=GOOD + 1, H=15), 4),
        (dict(wg=GOOD + 2, dtype=1), 4), (dict(ws=0), 5), (dict(nbytes=64), 5),
        (dict(ws=GOOD + 4), 4), (dict(saved=GOOD + 4), 4)]


@pytest.mark.parametrize("change,status", BOTH + [(dict(y=0), 1), (dict(y=GOOD + 1), 4)])
def test_forward_argument_errors(L, change, status):
    assert forward(L, **change) == status
    assert L.rkl_last_error()


@pytest.mark.parametrize("change,status", BOTH + [(dict(dy=0), 1), (dict(dy=GOOD + 1), 4), (dict(saved=0), 1),
                                                  (dict(dx=GOOD + 1), 4), (dict(dwd=GOOD + 1), 4)])
def test_backward_argument_errors(L, change, status):
    assert backward(L, **change) == status
    assert L.rkl_last_error()


def test_no_rows_needs_no_rows(L):
    assert forward(L, T=0, x=0, y=0, saved=0, ws=0, nbytes=0) == 0
    assert backward(L, T=0, x=0, dy=0, saved=0, dx=0, dwg=0, dwu=0, dwd=0, ws=0, nbytes=0) == 0


def test_workspace_size(L):
    need = ctypes.c_size_t(0)
    assert L.rkl_ffn_workspace_size(0, 4, 16, 32, 8, 0, None) == 1
    assert L.rkl_ffn_workspace_size(9, 4, 16, 32, 8, 0, ctypes.byref(need)) == 3
    assert L.rkl_ffn_workspace_size(0, 4, 16, 32, 8, 0, ctypes.byref(need)) == 0
    one = need.value
    assert one >= 4 * 32 * 2
    assert L.rkl_ffn_workspace_size(0, 4, 16, 32, 8, 1, ctypes.byref(need)) == 0 and need.value >= 3 * 4 * 32 * 2
    assert backward(L, nbytes=need.value - 1) == 5
    # the workspace that is asked for is enough, one byte less is not
    assert forward(L, nbytes=one - 1) == 5


def test_saved_size(L):
    n = ctypes.c_int64(0)
    assert L.rkl_ffn_saved_size(1, 1, None) == 1
    assert L.rkl_ffn_saved_size(-1, 1, ctypes.byref(n)) == 2
    assert L.rkl_ffn_saved_size(33, 65, ctypes.byref(n)) == 0 and n.value == 2 * 64 * 96
    assert L.rkl_ffn_saved_size(0, 65, ctypes.byref(n)) == 0 and n.value == 0


def test_python_refusals_without_a_device():
    t = torch.zeros(4, 4)
    with pytest.raises(RKLError, match="CUDA"):
        gated_ffn(t, t, t, t)
    with pytest.raises(RKLError, match="activation"):
        gated_ffn(t, t, t, t, "silu")
