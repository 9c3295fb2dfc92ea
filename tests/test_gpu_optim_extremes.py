"""AdamW at the ends of its range: second moments below and above fp32's,
scales, no eps.  Codes and scales against the 64-bit formulas of
optim_reference.py."""

import math

import pytest
import torch

from full_vocabulary_reverse_b200 import AdamW
from full_vocabulary_reverse_b200 import binding as rb
from tests import optim_reference as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LR, BETAS, EPS = 3e-3, (0.9, 0.999), 1e-8


def state(opt):
    """(m, v) of the 8-bit state's one tensor, code x scale in float64 on the CPU."""
    n = opt.params[0].numel()
    return tuple((x.double().view(-1, 256) * s.double()[:, None]).view(-1)[:n].cpu()
                 for x, s in ((opt.exp_avg, opt.exp_avg_scale), (opt.exp_avg_sq, opt.exp_avg_sq_scale)))


def after(opt, g, t, betas=BETAS, clip=1.0):
    """(m, v) that a step makes of the state, in float64."""
    m, v = state(opt)
    _, m, v = R.adamw(torch.zeros_like(m), m, v, g.double().cpu(), t, LR, betas, EPS, 0.0, clip)
    return m, v


def same(codes, ref):
    # (2^-40 of a step: the order of the reference's own 64-bit operations)
    value, _, edge, _, _ = ref
    return not ((codes.double().cpu() != value) & (edge > 2.0 ** -40)).any()


def mixed(n, small, seed):
    """Gradients near 1e-3, of `small` size and 0, side by side in every block."""
    gen = torch.Generator().manual_seed(seed)
    g = torch.randn(n, generator=gen) * 1e-3
    g[1::3] = torch.randn(g[1::3].shape, generator=gen).abs() * small + small
    g[2::5] = 0.0
    return g.cuda()


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("small,max_norm", [(1e-22, None), (1e-26, None), (1e-16, 4e-8), (1e-30, 1e-4)])
def test_second_moments_below_fp32_are_not_zero(small, max_norm, grad):
    """A gradient whose square fp32 cannot hold still makes a second moment above 0, whose code is never 0."""
    n = 4096 + 77
    g = mixed(n, small, 3).to(grad)
    opt = AdamW([torch.zeros(n, device="cuda")], lr=LR, betas=BETAS, eps=EPS, weight_decay=0.0, state_bits=8, seed=6)
    for t in (1, 2):
        zero = (state(opt)[1] == 0) & (g.cpu() == 0)
        norm = opt.step([g], max_norm=max_norm) if t == 1 else opt.step([g])
        if t == 1:
            fresh = AdamW([torch.zeros(n, device="cuda")], state_bits=8)
            m, v = after(fresh, g, t, clip=1.0 if norm is None else min(1.0, max_norm / float(norm)))
        else:
            m, v = after(kept, g, t)
        assert same(opt.exp_avg, R.codes(m)), t
        assert same(opt.exp_avg_sq, R.codes(v, R.random20(torch.arange(n), t, 6))), t
        code = opt.exp_avg_sq[:n].view(torch.uint8).cpu()
        assert (code[zero] == 0).all() and (code[~zero] > 0).all()
        kept = AdamW([torch.zeros(n, device="cuda")], state_bits=8)
        kept.load_state_dict(opt.state_dict())
    assert rb.device_error() == 0 and opt.params[0].isfinite().all()


def test_second_moment_that_beta2_takes_below_fp32_is_not_zero():
    """The old moment times a beta2 below fp32's normal numbers, beside new gradients and zeros."""
    n, betas = 1024, (0.9, 1e-42)
    g = mixed(n, 1e-3, 4)
    opt = AdamW([torch.zeros(n, device="cuda")], lr=LR, betas=betas, weight_decay=0.0, state_bits=8, seed=1)
    opt.step([g])
    turned = torch.where(g == 0, torch.full_like(g, 1e-3), torch.zeros_like(g))
    m, v = after(opt, turned, 2, betas)
    opt.step([turned])
    assert (v > 0).all() and (opt.exp_avg_sq.view(torch.uint8) > 0).all()
    assert same(opt.exp_avg_sq, R.codes(v, R.random20(torch.arange(n), 2, 1)))


@pytest.mark.parametrize("size", [1e21, 2e23, 3e38])
def test_second_moment_above_fp32_leaves_its_neighbours_alone(size):
    """One gradient whose square fp32 cannot hold: the block's scale is the formula's, the largest number at most, and
    the values beside it stay finite, zeros stay zeros."""
    n, top = 512, torch.finfo(torch.float32).max
    g = mixed(n, 1e-4, 9)
    g[7] = size
    g[300] = 0.25
    opt = AdamW([torch.zeros(n, device="cuda")], lr=LR, betas=BETAS, eps=EPS, weight_decay=0.0, state_bits=8, seed=2)
    for t in (1, 2, 3):
        _, v = after(opt, g, t)
        opt.step([g])
        scale = opt.exp_avg_sq_scale.double().cpu()
        assert scale.isfinite().all() and opt.params[0].isfinite().all()
        largest = float(v[:256].max())
        assert abs(float(scale[0]) - min(largest / 448, top)) <= 2.0 ** -24 * float(scale[0])
        if largest / 448 <= top:  # codes of the first block: the formula's
            assert same(opt.exp_avg_sq[:256], R.codes(v[:256], R.random20(torch.arange(256), t, 2)))
        code = opt.exp_avg_sq.view(torch.uint8).cpu()
        assert code[7] == 126 and (code[(g == 0).cpu()] == 0).all() and (code[(g != 0).cpu()] > 0).all()
    # the other block is as it would be without its neighbour
    twin = AdamW([torch.zeros(n, device="cuda")], lr=LR, betas=BETAS, eps=EPS, weight_decay=0.0, state_bits=8, seed=2)
    h = g.clone()
    h[7] = 0.0
    for _ in range(3):
        twin.step([h])
    assert torch.equal(twin.params[0][256:], opt.params[0][256:])
    assert torch.equal(twin.exp_avg_sq.view(torch.uint8)[256:], opt.exp_avg_sq.view(torch.uint8)[256:])


def test_scales_are_the_rounded_quotient():
    """Where fp32 holds a block's largest exactly (betas of 0: the gradient and its square), its scale is that number
    over 448, rounded once."""
    n = 256 * 4000
    g = torch.randn(n, generator=torch.Generator().manual_seed(8)).bfloat16()
    opt = AdamW([torch.zeros(n, device="cuda")], lr=LR, betas=(0.0, 0.0), weight_decay=0.0, state_bits=8)
    opt.step([g.cuda()])
    most = g.double().abs().view(-1, 256).amax(1)
    assert torch.equal(opt.exp_avg_scale.cpu(), (most / 448).float())
    assert torch.equal(opt.exp_avg_sq_scale.cpu(), (most * most / 448).float())


@pytest.mark.parametrize("bits", [32, 8])
def test_no_eps_leaves_the_elements_between_tensors_zero(bits):
    counts = [257, 3, 256]
    gen = torch.Generator().manual_seed(1)
    ps = [torch.randn(n, generator=gen).cuda() for n in counts]
    gs = [torch.randn(n, generator=gen).cuda() for n in counts]
    opt = AdamW(ps, lr=LR, betas=BETAS, eps=0.0, weight_decay=0.1, state_bits=bits, master_weights=True)
    old = [p.double().cpu() for p in ps]
    opt.step(gs)
    for p, g, p0, at in zip(ps, gs, old, opt.offsets):
        z = torch.zeros_like(p0)
        ref, _, _ = R.adamw(p0, z, z, g.double().cpu(), 1, LR, BETAS, 0.0, 0.1)
        assert torch.all((p.double().cpu() - ref).abs() <= 4 * U * ref.abs() + 2.0 ** -19 * LR)
        pad = slice(at + p.numel(), at + -(-p.numel() // 256) * 256)
        for x in (opt.master, opt.exp_avg.float(), opt.exp_avg_sq.float()):
            assert not x[pad].any()


@pytest.mark.parametrize("size", [1e-17, 1e-19, 3e-21])
def test_no_eps_and_second_moments_below_the_normal_numbers(size):
    """32-bit states without eps: a first step moves by lr whatever the gradient's size.  v = (1 - b2) g^2 is off by the
    half steps of two operations, 2^-149 in all, beside the 12 u of a normal v; its root by half of that, relative."""
    n = 300
    gen = torch.Generator().manual_seed(7)
    g = ((torch.rand(n, generator=gen) + 1) * size * (torch.randint(0, 2, (n,), generator=gen) * 2 - 1)).cuda()
    opt = AdamW([torch.zeros(n, device="cuda")], lr=LR, betas=BETAS, eps=0.0, weight_decay=0.0)
    opt.step([g])
    z = torch.zeros(n, dtype=torch.float64)
    ref, _, v = R.adamw(z, z, z, g.double().cpu(), 1, LR, BETAS, 0.0, 0.0)
    part = 2.0 ** -149 / v
    assert (part < 0.5).all()
    assert torch.all((opt.params[0].double().cpu() - ref).abs() <= LR * (2.0 ** -19 + part))


def test_no_eps_and_faint_gradients_in_8_bits():
    """Beside larger gradients, where their second moment has no digits: no update goes beyond lr."""
    n = 2048
    gen = torch.Generator().manual_seed(5)
    size = 10.0 ** (torch.randint(-24, -2, (n,), generator=gen))
    g = ((torch.rand(n, generator=gen) + 1) * size * (torch.randint(0, 2, (n,), generator=gen) * 2 - 1)).cuda()
    opt = AdamW([torch.zeros(n, device="cuda")], lr=LR, betas=BETAS, eps=0.0, weight_decay=0.0, state_bits=8)
    opt.step([g])
    p = opt.params[0]
    assert (p.abs() <= LR * (1 + 2.0 ** -18)).all() and (p * g <= 0).all()
    large = g.abs() >= 1e-14
    assert torch.all((p.abs() - LR)[large].abs() <= LR * 2.0 ** -11)  # eps beside 1e-14: 2^-58 / 1e-14 < 2^-11
