"""The gated feed-forward block beyond the ordinary call: infinite rows at odd
widths, and how many bf16 terms its operands have."""

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


@pytest.mark.parametrize("T,F,N", [(5, 2048, 1024), (9, 1000, 256), (64, 128, 1032)])
def test_a_width_beside_the_result_does_not_change_its_digits(T, F, N):
    """y [T, N] does not know how wide x is, nor dx [T, N] how wide dy: a's, dg's and du's terms go by the results."""
    gen = torch.Generator().manual_seed(F)
    r = lambda *s: torch.randn(s, generator=gen).bfloat16().cuda()  # noqa: E731
    wide = lambda t: torch.cat([t, torch.zeros(t.shape[0], 248 - t.shape[1], dtype=t.dtype, device="cuda")], 1)  # noqa: E731
    x, wg, wu, wd = r(T, 8), r(F, 8), r(F, 8), r(N, F)
    y = ffn_forward(x, wg, wu, wd)[0]
    # zeros beside x and the weights add nothing to g and u
    assert torch.equal(y, ffn_forward(wide(x), wide(wg), wide(wu), wd)[0])
    x, wg, wu, wd, dy = r(T, N), r(F, N), r(F, N), r(8, F), r(T, 8)
    saved = ffn_forward(x, wg, wu, wd, save=True)[1]
    dx = ffn_backward(x, wg, wu, wd, dy, saved)[0]
    tall = wide(wd.t().contiguous()).t().contiguous()
    assert torch.equal(dx, ffn_backward(x, wg, wu, tall, wide(dy), saved)[0])
