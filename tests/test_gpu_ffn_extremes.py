"""The gated feed-forward block beyond the ordinary call: infinite rows at odd
widths."""

import pytest
import torch

from full_vocabulary_reverse_b200 import ACT_RELU, ffn_backward, ffn_forward
from full_vocabulary_reverse_b200 import binding as rb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,F,O", [(5, 16, 32, 24), (5, 16, 33, 24), (5, 15, 33, 23), (100, 16, 1001, 24), (300, 16, 33, 24),
                                     (300, 17, 129, 40)])
def test_infinite_rows_at_odd_widths(T, H, F, O):
    """With positive numbers everywhere no product of an infinite row is 0 x infinity: its results are infinite, not
    NaN, whatever the widths, and the other rows are finite."""
    gen = torch.Generator().manual_seed(T)
    x, wg, wu, wd, dy = ((torch.rand(s, generator=gen) + 0.5).bfloat16().cuda()
                         for s in ((T, H), (F, H), (F, H), (O, F), (T, O)))
    for bad in ("x", "dy"):
        rows, up = x.clone(), dy.clone()
        (rows if bad == "x" else up)[T // 2] = float("inf")
        y, saved = ffn_forward(rows, wg, wu, wd, ACT_RELU, save=True)
        dx, dwg, dwu, dwd = ffn_backward(rows, wg, wu, wd, up, saved, ACT_RELU)
        assert rb.device_error() == 0
        others = torch.arange(T, device="cuda") != T // 2
        if bad == "x":
            assert y[T // 2].isinf().all()
        assert y[others].isfinite().all()
        assert dx[T // 2].isinf().all() and dx[others].isfinite().all()
        if T > 64:  # (in two terms, which few rows may take, a weight's gradient may be infinity - infinity)
            assert all(w.isinf().all() for w in (dwg, dwu, dwd))
