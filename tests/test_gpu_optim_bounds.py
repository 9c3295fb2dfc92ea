"""The 8-bit step's look-ahead in the bounds-checking build: with more blocks
than the grid takes at once, and a last block that is only partly there, no
address is formed behind a gradient's or a parameter's end."""

import os
import subprocess
import sys

import pytest

from full_vocabulary_reverse_b200.build import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# 24 blocks of 8 warps an SM, a state block of 256 each: 148 x 24 x 8 x 256 elements are one round of the grid.
CODE = r'''
import sys
sys.path.insert(0, %r)
import torch
from full_vocabulary_reverse_b200 import AdamW, binding as rb
assert b"debug bounds checks" in rb.lib().rkl_version()
sms = torch.cuda.get_device_properties(0).multi_processor_count
rounds = sms * 24 * 8 * 256
for n in (rounds + 1, rounds + 131, 2 * rounds + 256 + 9):
    for dtype in (torch.float32, torch.bfloat16):
        for master in (False, True):
            p, g = torch.ones(n, dtype=dtype, device="cuda"), torch.full((n,), 0.5, dtype=dtype, device="cuda")
            AdamW([p], lr=0.25, weight_decay=0.0, state_bits=8, master_weights=master).step([g])
            # the first step of a steady gradient moves by lr
            assert rb.device_error() == 0 and float((p.float() - 0.75).abs().max()) <= 2.0 ** -9
print("checked")
'''


def test_look_ahead_stays_inside_the_tensors():
    build(debug=True)
    out = subprocess.run([sys.executable, "-c", CODE % ROOT], env=dict(os.environ, RKL_LIBRARY="debug"), cwd=ROOT,
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "checked" in out.stdout, out.stdout + out.stderr
