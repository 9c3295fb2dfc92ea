"""The training operators through the bounds-checking build: same results, no
check fires."""

import os
import subprocess
import sys

import pytest

from full_vocabulary_reverse_b200.build import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = r'''
import sys
sys.path.insert(0, %r)
import torch
from full_vocabulary_reverse_b200 import AdamW, ffn_backward, ffn_forward, binding as rb
from tests import ffn_reference as R
assert b"debug bounds checks" in rb.lib().rkl_version()
gen = torch.Generator().manual_seed(0)
r = lambda shape, s: (torch.randn(shape, generator=gen) * s).bfloat16().cuda()
for T, H, F, O in ((3, 64, 72, 40), (100, 136, 264, 520), (300, 136, 264, 520), (513, 1160, 344, 72)):
    ins, dy = [r((T, H), 1.0), r((F, H), H ** -0.5), r((F, H), H ** -0.5), r((O, F), F ** -0.5)], r((T, O), 0.1)
    y, saved = ffn_forward(*ins, save=True)
    grads = ffn_backward(*ins, dy, saved)
    R.check([y, *grads], R.block(*ins, 0, dy), torch.bfloat16)
    for bits in (32, 8):
        params = [t.clone() for t in ins[1:]]
        AdamW(params, state_bits=bits).step(list(grads[1:]), max_norm=1.0)
        assert not torch.equal(params[0], ins[1])
    assert rb.device_error() == 0
print("checked")
'''


def test_training_operators_in_the_debug_build():
    build(debug=True)
    out = subprocess.run([sys.executable, "-c", CODE % ROOT], env=dict(os.environ, RKL_LIBRARY="debug"), cwd=ROOT,
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "checked" in out.stdout, out.stdout + out.stderr
