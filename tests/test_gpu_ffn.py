"""The gated feed-forward block against the formulas in 64 bits (bounds in
ffn_reference.py)."""

import ctypes

import pytest
import torch

from full_vocabulary_reverse_b200 import (ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_SILU, RKLError, ffn_backward, ffn_forward,
                                          gated_ffn)
from full_vocabulary_reverse_b200 import binding as rb
from tests import ffn_reference as R

pytestmark = pytest.mark.gpu
ACTS = [ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU]


def inputs(T, H, F, O, dtype, seed=0, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda shape, s: (torch.randn(shape, generator=gen) * s).to(dtype).cuda()  # noqa: E731
    return [r((T, H), scale), r((F, H), H ** -0.5), r((F, H), H ** -0.5), r((O, F), F ** -0.5)], r((T, O), 0.1)


def both(T, H, F, O, dtype, kind, seed=0, scale=1.0):
    ins, dy = inputs(T, H, F, O, dtype, seed, scale)
    y, saved = ffn_forward(*ins, kind, save=True)
    grads = ffn_backward(*ins, dy, saved, kind)
    torch.cuda.synchronize()
    assert rb.device_error() == 0
    R.check([y, *grads], R.block(*ins, kind, dy), dtype)
    assert torch.equal(y, ffn_forward(*ins, kind)[0])
    return ins, dy, y, grads


SIZES = [(1, 8, 8, 8), (1, 1, 1, 1), (1, 512, 1032, 264), (2, 64, 72, 40), (3, 65, 33, 17), (5, 1032, 200, 520),
         (8, 256, 2048, 256), (9, 264, 136, 8), (31, 200, 77, 64), (64, 128, 128, 128), (127, 96, 264, 72),
         (128, 256, 256, 256), (129, 136, 520, 328), (255, 64, 1000, 64), (257, 320, 264, 1032), (300, 515, 131, 67),
         (513, 72, 88, 2056), (700, 1160, 344, 120), (1500, 349, 699, 351)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,F,O", SIZES)
def test_sizes(T, H, F, O, dtype):
    both(T, H, F, O, dtype, ACT_SILU, seed=T + H)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("T", [1, 37, 261])
def test_activations(T, kind, dtype):
    both(T, 128, 200, 136, dtype, kind, seed=kind, scale=3.0)


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("T,H,F,O", [(1, 64, 64, 64), (1, 1032, 2056, 520), (2, 856, 112, 256), (2, 857, 113, 255), (5, 64, 72, 2056),
                                     (9, 136, 1000, 72), (31, 64, 128, 72), (33, 200, 77, 65), (63, 264, 64, 136), (64, 72, 64, 264)])
def test_few_elements_round_the_result_alone(T, H, F, O, kind):
    # a, dg and du in two terms: the rest of the first (half a step, 2^-8) is rounded by 2^-8 of itself
    ins, dy = inputs(T, H, F, O, torch.bfloat16, T + F)
    y, saved = ffn_forward(*ins, kind, save=True)
    grads = ffn_backward(*ins, dy, saved, kind)
    assert rb.device_error() == 0
    for k, (t, (value, bound)) in enumerate(zip([y, *grads], R.block(*ins, kind, dy, operand=2.0 ** -16))):
        off = (t.double() - value).abs()
        assert torch.all(off <= bound), (k, float((off / bound.clamp(min=1e-300)).max()))


def test_few_elements_that_overflow():
    # an a beyond the type's range is infinite in its first term, with no rest beside it
    x = torch.full((3, 8), 2.0 ** 60, dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0
    w = torch.ones(16, 8, dtype=torch.bfloat16, device="cuda") * 8.0
    y = ffn_forward(x, w, w, torch.ones(8, 16, dtype=torch.bfloat16, device="cuda"))[0]
    assert torch.isinf(y[0]).all() and torch.isinf(y[2]).all()
    assert torch.equal(y[1].float(), torch.full((8,), 65536.0, device="cuda"))  # 16 x 64 x 64


@pytest.mark.parametrize("T", [1, 4, 16, 200])
def test_long_and_wide(T):
    both(T, 4096, 5632, 2048, torch.bfloat16, ACT_SILU, seed=T)


def test_training_size():
    both(8192, 2048, 6144, 2048, torch.bfloat16, ACT_GELU_TANH, seed=3)


def test_wide_output_and_narrow_hidden():
    both(1031, 24, 6152, 16, torch.bfloat16, ACT_SILU)
    both(40, 6152, 8, 4104, torch.bfloat16, ACT_SILU)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_autograd_shapes_strides_and_partial_gradients(dtype):
    ins, _ = inputs(30, 64, 48, 40, dtype, 5)
    x = ins[0].view(2, 15, 64)
    dy = torch.randn(2, 15, 40, device="cuda").to(dtype)
    ref = R.block(*ins, ACT_SILU, dy.reshape(30, 40))
    leaves = [x.clone().requires_grad_(True)] + [w.clone().requires_grad_(True) for w in ins[1:]]
    y = gated_ffn(*leaves)
    assert y.shape == (2, 15, 40)
    grads = torch.autograd.grad(y, leaves, dy)
    R.check([y.detach().view(30, 40), grads[0].view(30, 64), *grads[1:]], ref, dtype)
    # weights and rows stored the other way round, and a sliced one
    wide = torch.zeros(48, 70, dtype=dtype, device="cuda")
    wide[:, 3:67] = ins[1]
    turned = [ins[0].t().contiguous().t(), wide[:, 3:67], ins[2].t().contiguous().t(), ins[3].t().contiguous().t()]
    assert not any(t.is_contiguous() for t in turned)
    z = gated_ffn(*turned)
    assert torch.equal(z, y.detach().view(30, 40))
    # one gradient alone is the same as among all
    for k in range(4):
        part = [t.detach().requires_grad_(i == k) for i, t in enumerate(leaves)]
        got, = torch.autograd.grad(gated_ffn(*part), [part[k]], dy)
        assert torch.equal(got, grads[k])
    with torch.no_grad():
        assert not gated_ffn(*leaves).requires_grad
    # an expanded upstream gradient
    y = gated_ffn(*leaves)
    g1 = torch.autograd.grad(y.sum(), leaves)
    g2 = torch.autograd.grad(gated_ffn(*leaves), leaves, torch.ones_like(y))
    assert all(torch.equal(a, b) for a, b in zip(g1, g2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_addresses_off_16_bytes(dtype):
    ins, dy = inputs(40, 64, 128, 64, dtype, 6)
    shifted = []
    for t in ins + [dy]:
        buf = torch.empty(t.numel() + 1, dtype=dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        shifted.append(buf[1:].view(t.shape))
    y, saved = ffn_forward(*shifted[:4], save=True)
    R.check([y, *ffn_backward(*shifted[:4], shifted[4], saved)], R.block(*ins, ACT_SILU, dy), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_rows(dtype):
    ins, _ = inputs(0, 64, 48, 40, dtype)
    leaves = [t.requires_grad_(True) for t in ins]
    y = gated_ffn(*leaves)
    assert y.shape == (0, 40)
    grads = torch.autograd.grad(y, leaves, torch.zeros(0, 40, dtype=dtype, device="cuda"))
    assert grads[0].shape == (0, 64) and all(not g.any() and g.shape == t.shape for g, t in zip(grads[1:], leaves[1:]))


@pytest.mark.parametrize("T,H,F,O", [(5, 64, 72, 40), (100, 64, 72, 40), (300, 520, 264, 136), (300, 515, 131, 67)])
def test_memory_behind_the_results_is_left_alone(T, H, F, O):
    """Every output sits in a larger buffer; nothing but its own elements changes, and a NaN row of x or dy stays in
    its row of y and dx."""
    ins, dy = inputs(T, H, F, O, torch.bfloat16, 9)
    sizes = [(T, O), (T, H), (F, H), (F, H), (O, F)]
    bufs = [torch.full((a * b + 4096,), 5.0, dtype=torch.bfloat16, device="cuda") for a, b in sizes]
    L = rb.lib()
    need = [ctypes.c_size_t(0), ctypes.c_size_t(0)]
    for way in (0, 1):  # one workspace for both directions
        assert L.rkl_ffn_workspace_size(0, T, H, F, O, way, ctypes.byref(need[way])) == 0
    nbytes = max(need, key=lambda b: b.value)
    ws = torch.full((nbytes.value + 4096,), 7, dtype=torch.uint8, device="cuda")
    count = ctypes.c_int64(0)
    assert L.rkl_ffn_saved_size(T, F, ctypes.byref(count)) == 0
    saved = torch.full((count.value + 1024,), 5.0, device="cuda")
    p = [rb._ptr(t) for t in ins]
    s = rb._stream("cuda")

    def run():
        rb._check(L.rkl_ffn_forward(*p, 0, 0, T, H, F, O, rb._ptr(bufs[0]), rb._ptr(saved), rb._ptr(ws), nbytes, s))
        rb._check(L.rkl_ffn_backward(*p, 0, 0, T, H, F, O, rb._ptr(dy), rb._ptr(saved), *[rb._ptr(b) for b in bufs[1:]],
                                     rb._ptr(ws), nbytes, s))
        torch.cuda.synchronize()
        for (a, b), buf in zip(sizes, bufs):
            assert (buf[a * b:] == 5.0).all()
        assert (ws[nbytes.value:] == 7).all() and (saved[count.value:] == 5.0).all()
    run()
    out = [buf[:a * b].view(a, b) for (a, b), buf in zip(sizes, bufs)]
    R.check(out, R.block(*ins, ACT_SILU, dy), torch.bfloat16)
    y, dx = out[0].clone(), out[1].clone()
    ins[0][T // 2] = float("nan")
    run()
    rows = torch.arange(T, device="cuda") != T // 2
    assert out[0][T // 2].isnan().all() and out[1][T // 2].isnan().all()
    assert torch.equal(out[0][rows], y[rows]) and torch.equal(out[1][rows], dx[rows])


@pytest.mark.parametrize("T,H", [(1, 128), (20, 128), (500, 128), (20, 125), (500, 125)])
def test_captured_pass_and_other_stream(T, H):
    ins, dy = inputs(T, H, 264, 72, torch.bfloat16, 4)
    leaves = [t.requires_grad_(True) for t in ins]

    def step():
        y = gated_ffn(*leaves)
        return [y.detach()] + list(torch.autograd.grad(y, leaves, dy))  # (no graph of the leaves outlives the pass)
    ref = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(ref, step()))
    torch.cuda.current_stream().wait_stream(side)
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.cuda.graph(second, pool=graph.pool()):
        again = step()
    with torch.no_grad():
        kept = leaves[0].clone()
        leaves[0].mul_(0.5)
    graph.replay()
    assert not torch.equal(out[0], ref[0])
    with torch.no_grad():
        leaves[0].copy_(kept)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    second.replay()
    assert all(torch.equal(a, b) for a, b in zip(ref, again))
    # the single passes can be captured whatever graphs of the leaves live
    alive = gated_ffn(*leaves)
    third = torch.cuda.CUDAGraph()
    with torch.cuda.graph(third), torch.no_grad():
        y, saved = ffn_forward(*leaves, save=True)
        out = [y, *ffn_backward(*leaves, dy, saved)]
    third.replay()
    assert all(torch.equal(a, b) for a, b in zip(ref, out)) and alive.requires_grad


def test_rows_do_not_depend_on_the_batch_beside_them():
    """Rows of one large call equal the same rows of another batch with the same row count."""
    ins, _ = inputs(600, 136, 264, 72, torch.bfloat16, 2)
    y = ffn_forward(*ins)[0]
    other = ins[0].clone()
    other[100:] = torch.randn_like(other[100:])
    assert torch.equal(y[:100], ffn_forward(other, *ins[1:])[0][:100])


def test_gradients_against_differences():
    """fp32, directional derivatives of L = sum(y dy): central differences of step e are off by e^2 / 6 of the third
    derivative along the direction (below 10 |L|-sized here, v of norm 1 entries) and 4 u L / e; with e = 2^-6 both
    stay below 2^-8 of the sizes involved."""
    ins, dy = inputs(6, 24, 40, 16, torch.float32, 8)
    y, saved = ffn_forward(*ins, ACT_GELU, save=True)
    grads = ffn_backward(*ins, dy, saved, ACT_GELU)
    gen = torch.Generator().manual_seed(1)
    for k in range(4):
        v = torch.randn(ins[k].shape, generator=gen).cuda() * ins[k].std()
        e = 2.0 ** -6
        L = []
        for sign in (1, -1):
            moved = [t + sign * e * v if i == k else t for i, t in enumerate(ins)]
            L.append(float((ffn_forward(*moved, ACT_GELU)[0].double() * dy.double()).sum()))
        want = (L[0] - L[1]) / (2 * e)
        got = float((grads[k].double() * v.double()).sum())
        size = float(grads[k].double().norm() * v.double().norm())
        assert abs(got - want) <= 2.0 ** -8 * size, (k, got, want)


def test_refusals_with_tensors_on_the_device():
    ins, dy = inputs(4, 8, 16, 8, torch.bfloat16)
    x, wg, wu, wd = ins
    with pytest.raises(RKLError, match="W_up"):
        gated_ffn(x, wg, wu[:8], wd)
    with pytest.raises(RKLError, match="do not fit"):
        gated_ffn(x, wg, wu, wd.t())
    with pytest.raises(RKLError, match="W_gate is torch.float32"):
        gated_ffn(x, wg.float(), wu, wd)
    with pytest.raises(RKLError, match="dtype"):
        gated_ffn(x.half(), wg.half(), wu.half(), wd.half())
    with pytest.raises(RKLError, match="activation"):
        gated_ffn(x, wg, wu, wd, 7)
    with pytest.raises(RKLError, match="CUDA"):
        gated_ffn(x, wg.cpu(), wu, wd)
    _, saved = ffn_forward(*ins, save=True)
    with pytest.raises(RKLError, match="dy"):
        ffn_backward(*ins, dy[:3], saved)
    with pytest.raises(RKLError, match="saved"):
        ffn_backward(*ins, dy, saved[:-1])
