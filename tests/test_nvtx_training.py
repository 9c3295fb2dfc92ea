"""The training operators' entry points open and close NVTX ranges of their own
names, on refused arguments too (see test_nvtx.py; no GPU)."""

import os
import subprocess
import sys

from tests.test_nvtx import ROOT, recorder  # noqa: F401

ENTRY_POINTS = ["rkl_ffn_forward", "rkl_ffn_backward", "rkl_adamw_step", "rkl_grad_norm"]

CALLER = r'''
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from full_vocabulary_reverse_b200 import binding as rb
L = rb.lib()
for name in sys.argv[2:]:
    fn = getattr(L, name)
    assert fn(*[None if t is ctypes.c_void_p else 0 for t in fn.argtypes]) != 0, name  # NULL pointers
'''


def test_every_training_entry_point_opens_and_closes_a_named_range(recorder, tmp_path):  # noqa: F811
    from full_vocabulary_reverse_b200.build import build
    build()
    log = tmp_path / "ranges.log"
    env = dict(os.environ, NVTX_INJECTION64_PATH=recorder, RKL_NVTX_LOG=str(log))
    subprocess.run([sys.executable, "-c", CALLER, ROOT] + ENTRY_POINTS, env=env, check=True, timeout=300)
    lines = log.read_text().split("\n")[:-1]
    assert [ln for ln in lines if ln.split()[1:] and ln.split()[1] in ENTRY_POINTS or ln == "pop"] == \
        [x for name in ENTRY_POINTS for x in ("push " + name, "pop")]
