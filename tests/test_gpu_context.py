"""A context that a caller of the C ABI has made current stays current, and its
memory is what the call works on; a thread with none gets the device's own."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = r'''
import ctypes, sys, threading
sys.path.insert(0, sys.argv[1])
import numpy as np
import torch
from cuda.bindings import driver as cu
from full_vocabulary_reverse_b200 import binding as rb, ffn_forward

def ok(r):
    assert r[0] == cu.CUresult.CUDA_SUCCESS, r
    return r[1] if len(r) == 2 else r[1:]

L = rb.lib()
x = torch.ones(8, 64, dtype=torch.bfloat16, device="cuda")
own = int(ok(cu.cuCtxGetCurrent()))
device = ok(cu.cuCtxGetDevice())
try:
    other = ok(cu.cuCtxCreate(0, device))
except TypeError:  # (newer bindings take creation parameters)
    other = ok(cu.cuCtxCreate(None, 0, device))
here = lambda: int(ok(cu.cuCtxGetCurrent()))
assert here() == int(other) != own

# a call without rows sets the device up and launches nothing
p = ctypes.c_void_p(0x10000)
assert L.rkl_forward_logits_pair(p, p, 0, 1, 4, 64, p, 0, None, 1, None, None, p, p, 1 << 20, None) == 0, L.rkl_last_error()
print("current stays", here() == int(other))
assert here() == int(other)

# one that computes, on that context's memory
g = np.arange(1, 1001, dtype=np.float32)
buf = ok(cu.cuMemAlloc(g.nbytes + 256))
ok(cu.cuMemcpyHtoD(buf, g.ctypes.data, g.nbytes))
need = ctypes.c_size_t(0)
assert L.rkl_grad_norm_workspace_size(1, ctypes.byref(need)) == 0
ws = ok(cu.cuMemAlloc(need.value))
norm = int(buf) + g.nbytes
assert L.rkl_grad_norm(1, (ctypes.c_void_p * 1)(int(buf)), (ctypes.c_int64 * 1)(g.size), (ctypes.c_int32 * 1)(1),
                       ctypes.c_void_p(norm), ctypes.c_void_p(int(ws)), need.value, None) == 0, L.rkl_last_error()
ok(cu.cuCtxSynchronize())
out = np.zeros(1, dtype=np.float32)
ok(cu.cuMemcpyDtoH(out.ctypes.data, norm, 4))
want = float(np.sqrt((g.astype(np.float64) ** 2).sum()))
assert abs(float(out[0]) - want) <= 4 * 2.0 ** -24 * want and here() == int(other)
for q in (ws, buf):
    ok(cu.cuMemFree(q))
ok(cu.cuCtxDestroy(other))
assert here() == own

# a thread that has made no call yet, through the raw entry point
w, wd = torch.ones(16, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(8, 16, dtype=torch.bfloat16, device="cuda")
y = ffn_forward(x, w, w, wd)[0]
z = torch.zeros_like(y)
assert L.rkl_ffn_workspace_size(0, 8, 64, 16, 8, 0, ctypes.byref(need)) == 0
ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
args = [ctypes.c_void_p(t.data_ptr()) for t in (x, w, w, wd)] + [0, 0, 8, 64, 16, 8, ctypes.c_void_p(z.data_ptr()), None,
        ctypes.c_void_p(ws.data_ptr()), need.value, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)]
got = []
t = threading.Thread(target=lambda: got.append(L.rkl_ffn_forward(*args)))
t.start()
t.join()
torch.cuda.synchronize()
assert got == [0] and torch.equal(y, z) and rb.device_error() == 0
print("checked")
'''


def test_the_callers_context_stays_current():
    out = subprocess.run([sys.executable, "-c", CODE, ROOT], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "checked" in out.stdout, out.stdout + out.stderr
