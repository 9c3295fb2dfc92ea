"""The gated feed-forward block beyond the ordinary call: infinite rows at odd
widths, how many bf16 terms its operands have, forward mode (which it has not),
gates far out, offsets past 32 bits, two streams at once."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

from full_vocabulary_reverse_b200 import (ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_SILU, ffn_backward, ffn_forward,
                                          gated_ffn)
from full_vocabulary_reverse_b200 import binding as rb
from tests import ffn_reference as R

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


def block(T=4, H=16, F=32, O=8):
    gen = torch.Generator().manual_seed(0)
    return [torch.randn(s, generator=gen).bfloat16().cuda() for s in ((T, H), (F, H), (F, H), (O, F))]


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(which, grad):
    ins = block()
    with fwd.dual_level(), torch.set_grad_enabled(grad):
        ins[which] = fwd.make_dual(ins[which], torch.ones_like(ins[which]))
        with pytest.raises(NotImplementedError, match="jvp"):
            gated_ffn(*ins)


def test_forward_mode_over_the_backward_pass_is_refused():
    ins = [t.requires_grad_(True) for t in block()]
    y = gated_ffn(*ins)
    with fwd.dual_level():
        dy = fwd.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(NotImplementedError, match="jvp"):
            torch.autograd.grad(y, ins, dy)


def test_a_level_without_tangents_changes_nothing():
    ins = block()
    y = gated_ffn(*ins)
    with fwd.dual_level():
        assert torch.equal(gated_ffn(*ins), y)
        ins[0].requires_grad_(True)
        z = gated_ffn(*ins)
        assert torch.equal(z, y)
        a, = torch.autograd.grad(z, [ins[0]], torch.ones_like(z))
    b, = torch.autograd.grad(gated_ffn(*ins), [ins[0]], torch.ones_like(y))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", [ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU])
@pytest.mark.parametrize("T", [1, 300])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_gates_whose_square_leaves_fp32(sign, T, kind, dtype):
    """g = +-2^67 and u = 1, powers of two throughout: act' is 1 or 0, and nothing is NaN."""
    full = lambda shape, v: torch.full(shape, v, dtype=dtype, device="cuda")  # noqa: E731
    x, wg, wu, wd = full((T, 8), 2.0 ** 31), full((8, 8), sign * 2.0 ** 33), full((8, 8), 2.0 ** -34), full((8, 8), 1.0)
    dy = full((T, 8), 2.0 ** -3)
    y, saved = ffn_forward(x, wg, wu, wd, kind, save=True)
    dx, dwg, dwu, dwd = ffn_backward(x, wg, wu, wd, dy, saved, kind)
    on = 1.0 if sign > 0 else 0.0
    # a = g u = 2^67; da = 8 x 2^-3 = 1, dg = 1, du = 2^67; dx = 8 (2^33 + 2^67 2^-34), the weights over T rows
    for got, want in ((y, 2.0 ** 70), (dx, 2.0 ** 37), (dwg, T * 2.0 ** 31), (dwu, T * 2.0 ** 98), (dwd, T * 2.0 ** 64)):
        assert torch.equal(got, torch.full_like(got, on * want)), (got.flatten()[0], want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,F,O", [(270003, 8, 8192, 8), (270003, 9, 8193, 7)])
def test_offsets_past_32_bits(T, H, F, O, dtype):
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of free memory")
    gen = torch.Generator("cuda").manual_seed(1)
    r = lambda rows, cols, s: (torch.randn((rows, cols), generator=gen, device="cuda") * s).to(dtype)  # noqa: E731
    x, wg, wu, wd, dy = r(T, H, 1), r(F, H, H ** -0.5), r(F, H, H ** -0.5), r(O, F, F ** -0.5), r(T, O, 0.1)
    n = 700
    dy[:-n] = 0  # the other rows add exact zeros to the weights' gradients
    y, saved = ffn_forward(x, wg, wu, wd, save=True)
    grads = ffn_backward(x, wg, wu, wd, dy, saved)
    assert rb.device_error() == 0 and saved.numel() > 1 << 32
    R.check([y[-n:], grads[0][-n:], *grads[1:]], R.block(x[-n:], wg, wu, wd, R.SILU, dy[-n:]), dtype)
    R.check([y[:n]], R.block(x[:n], wg, wu, wd, R.SILU), dtype)
    assert not grads[0][:-n].any()


def test_two_streams_at_once():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: (torch.randn(s, generator=gen) * s[-1] ** -0.5).bfloat16().cuda()  # noqa: E731
    blocks = [[r(T, 512), r(1024, 512), r(1024, 512), r(512, 1024)] for T in (3, 700)]
    want = [ffn_forward(*b)[0] for b in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for b, s, g in zip(blocks, streams, got):
            with torch.cuda.stream(s):
                g.append(ffn_forward(*b)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for w, g in zip(want, got) for y in g) and rb.device_error() == 0


def test_one_row_without_a_batch_and_no_batch():
    x, wg, wu, wd = block()
    y = gated_ffn(x[0], wg, wu, wd)
    assert y.shape == (8,) and torch.equal(y, gated_ffn(x[:1], wg, wu, wd)[0])
    assert gated_ffn(x.new_empty(0, 5, 16), wg, wu, wd).shape == (0, 5, 8)
