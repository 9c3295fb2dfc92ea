"""AdamW and grad_norm against a plain implementation in 64 bits.

Tolerances count roundings of fp32 (half a step, u = 2^-24) in the kernel:
  m   c grad, (1-b1) x, the fused multiply-add, and b1, 1-b1 and c rounded to
      fp32 (c: the norm's and the quotient's roundings too): 8 u of the terms'
      magnitudes.
  v   one square more of c grad: 12 u of v (all terms are positive).
  p   keep = 1 - lr wd, the fused multiply-add, lr's and wd's roundings: 4 u of
      |p|; the update: m (8 u of its terms' magnitudes), sqrt of v (6 u + 2^-22),
      the quotient (2^-22), the bias corrections by expm1f of t log b (argument
      rounded, 2 u, and expm1f's 2^-22 each): below 2^-19 of the magnitude that
      m's terms give the update.
A parameter in bf16 adds half a step of bf16, 2^-9 of a value below a power of
two's double: 2^-8 relative covers every place in the binade."""

import math

import pytest
import torch

from full_vocabulary_reverse_b200 import AdamW, RKLError, grad_norm
from full_vocabulary_reverse_b200 import binding as rb
from tests import optim_reference as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LR, BETAS, EPS = 3e-3, (0.9, 0.999), 1e-8
COUNTS = [1, 255, 256, 257, 0, 8, 2048 + 3, 70001]


def unaligned(t):
    """The same values one element behind an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


def make(counts, param, grad, seed, shift=False):
    gen = torch.Generator().manual_seed(seed)
    ps = [(torch.randn(n, generator=gen) * 0.05).to(param).cuda() for n in counts]
    gs = [[(torch.randn(n, generator=gen) * 10 ** (k - 3.0)).to(grad).cuda() for n in counts] for k in range(3)]
    if shift:
        ps, gs = [unaligned(p) for p in ps], [[unaligned(g) for g in s] for s in gs]
    return ps, gs


def state64(opt, i):
    """(p, m, v) of tensor i as the step will see them, in float64 on the CPU."""
    n, at = opt.params[i].numel(), opt.offsets[i]
    m, v = opt.moments(i)
    p = opt.master[at:at + n] if opt.master is not None else opt.params[i].reshape(-1)
    if opt.state_bits == 8:  # code x scale without the rounding of their product
        blocks = slice(at // 256, -(-(at + n) // 256))
        m, v = ((x[blocks.start * 256:blocks.stop * 256].double().view(-1, 256) * s[blocks].double()[:, None]
                 ).view(-1)[:n] for x, s in ((opt.exp_avg, opt.exp_avg_scale), (opt.exp_avg_sq, opt.exp_avg_sq_scale)))
    return p.double().cpu(), m.double().cpu().view(-1), v.double().cpu().view(-1)


def check_step(opt, grads, before, t, clip=1.0, decay=None):
    for i, (p, g) in enumerate(zip(opt.params, grads)):
        n, at = p.numel(), opt.offsets[i]
        if n == 0:
            continue
        wd = opt.weight_decay[i] if decay is None else decay
        p0, m0, v0 = before[i]
        g64 = g.double().cpu().reshape(-1)
        rp, rm, rv = R.adamw(p0, m0, v0, g64, t, LR, BETAS, EPS, wd, clip)
        terms = BETAS[0] * m0.abs() + (1 - BETAS[0]) * (g64 * clip).abs()
        upd = LR / (1 - BETAS[0] ** t) * terms / (rv.sqrt() / math.sqrt(1 - BETAS[1] ** t) + EPS)
        tol = 4 * U * rp.abs() + 2.0 ** -19 * upd
        if opt.master is not None:
            got = opt.master[at:at + n].double().cpu()
            assert torch.all((got - rp).abs() <= tol), i
            assert torch.equal(p.reshape(-1), opt.master[at:at + n].to(p.dtype)), i
        else:
            low = rp.abs() * 2.0 ** -8 if p.dtype == torch.bfloat16 else 0.0
            assert torch.all((p.double().cpu().reshape(-1) - rp).abs() <= tol + low), i
        if opt.state_bits == 32:
            m, v = opt.moments(i)
            assert torch.all((m.double().cpu().view(-1) - rm).abs() <= 8 * U * terms), i
            assert torch.all((v.double().cpu().view(-1) - rv).abs() <= 12 * U * rv), i
            pad = slice(at + n, at + -(-n // 256) * 256)
            assert not opt.exp_avg[pad].any() and not opt.exp_avg_sq[pad].any()
            continue
        where = torch.arange(at, at + n)
        blocks = slice(at // 256, -(-(at + n) // 256))
        for x, scale, ref, rnd in ((opt.exp_avg, opt.exp_avg_scale, rm, None),
                                   (opt.exp_avg_sq, opt.exp_avg_sq_scale, rv, R.random20(where, t, opt.seed))):
            value, s, edge, r, gap = R.codes(ref, rnd)
            got = x[blocks.start * 256:blocks.stop * 256].double().cpu()
            # off: what the value is off by (above); the block's largest is off as much, its scale rounds once more
            off = torch.nn.functional.pad(8 * U * terms if rnd is None else 12 * U * rv, (0, -n % 256))
            most = off.view(-1, 256).amax(1)
            assert torch.all((scale[blocks].double().cpu() - s).abs() <= most / 448 + U * s), i
            # Another code only where the value lies on the border.  r = value / scale is off by the value's and the
            # scale's errors and 4 roundings; below 2^-6 the sum with the random number rounds too (8 u).
            per = s.repeat_interleave(256).clamp(min=1e-300)
            slack = (off / per + r * (most.repeat_interleave(256) / (448 * per) + 4 * U)) / gap + 8 * U
            wrong = (got != value) & (edge > slack)
            assert not wrong.any(), (i, int(wrong.sum()))


@pytest.mark.parametrize("shift", [False, True])
@pytest.mark.parametrize("param,grad,master", [(torch.float32, torch.float32, False), (torch.bfloat16, torch.bfloat16, False),
                                               (torch.bfloat16, torch.float32, True), (torch.float32, torch.bfloat16, True)])
@pytest.mark.parametrize("bits", [32, 8])
def test_three_steps(bits, param, grad, master, shift):
    ps, gs = make(COUNTS, param, grad, 7 + bits, shift)
    opt = AdamW(ps, lr=LR, betas=BETAS, eps=EPS, weight_decay=[0.1 * (i % 3) for i in range(len(ps))], state_bits=bits,
                master_weights=master, seed=5)
    for t, grads in enumerate(gs, 1):
        before = [state64(opt, i) for i in range(len(ps))]
        assert opt.step(grads) is None
        torch.cuda.synchronize()
        assert int(opt.steps) == t and rb.device_error() == 0
        check_step(opt, grads, before, t)


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_and_far_step_count(bits):
    ps, gs = make([1031, 5], torch.float32, torch.float32, 3)
    opt = AdamW(ps, lr=LR, betas=BETAS, eps=EPS, weight_decay=0.1, state_bits=bits)
    opt.step(gs[0])
    opt.steps.fill_(100000)
    before = [state64(opt, i) for i in range(2)]
    norm = opt.step(gs[2], max_norm=0.5)
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in gs[2]))
    assert abs(float(norm) - ref) <= 4 * U * ref and ref > 0.5
    check_step(opt, gs[2], before, 100001, clip=0.5 / ref)
    # a norm below the limit scales nothing
    twin = AdamW([p.clone() for p in ps], lr=LR, betas=BETAS, eps=EPS, weight_decay=0.1, state_bits=bits)
    twin.load_state_dict(opt.state_dict())
    opt.step(gs[0], max_norm=1e4)
    twin.step(gs[0])
    assert all(torch.equal(a, b) for a, b in zip(opt.params, twin.params))
    assert torch.equal(opt.exp_avg.view(torch.uint8), twin.exp_avg.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_changes_nothing(bits, bad):
    ps, gs = make([300, 257], torch.bfloat16, torch.float32, 4)
    opt = AdamW(ps, state_bits=bits, master_weights=True)
    opt.step(gs[0])
    kept = {k: t.clone() for k, t in opt.state_dict().items()}
    params = [p.clone() for p in ps]
    gs[1][1][200] = bad
    norm = opt.step(gs[1], max_norm=1.0)
    assert not math.isfinite(float(norm))
    assert all(torch.equal(a, b) for a, b in zip(params, ps))
    assert all(torch.equal(t.view(torch.uint8), kept[k].view(torch.uint8)) for k, t in opt.state_dict().items())
    assert opt.step(gs[2], norm=grad_norm(gs[2])) is not None  # found outside, no limit
    assert int(opt.steps) == 2


@pytest.mark.parametrize("bits", [32, 8])
def test_absent_gradients_and_zero_gradients(bits):
    ps, gs = make([300, 257, 3], torch.float32, torch.float32, 8)
    opt = AdamW(ps, lr=LR, betas=BETAS, eps=EPS, weight_decay=0.0, state_bits=bits)
    kept = ps[1].clone()
    before = [state64(opt, i) for i in range(3)]
    zero = torch.zeros_like(gs[0][2])
    was = ps[2].clone()
    opt.step([gs[0][0], None, zero])
    assert torch.equal(ps[1], kept) and torch.equal(ps[2], was) and int(opt.steps) == 1
    assert all(not x.any() for i in (1, 2) for x in opt.moments(i))
    n = ps[0].numel()
    rp, _, _ = R.adamw(before[0][0], before[0][1], before[0][2], gs[0][0].double().cpu(), 1, LR, BETAS, EPS, 0.0)
    assert torch.all((ps[0].double().cpu() - rp).abs() <= 4 * U * rp.abs() + 2.0 ** -19 * LR) and n == 300
    opt.step([None, None, None], max_norm=1.0)  # nothing to do still counts
    assert int(opt.steps) == 2


def test_parameters_own_gradients_and_version():
    w = torch.nn.Parameter(torch.randn(40, 33, device="cuda"))
    b = torch.nn.Parameter(torch.zeros(33, device="cuda"))
    x = torch.randn(5, 40, device="cuda")
    opt = AdamW([w, b], lr=1e-2)
    loss = ((x @ w + b) ** 2).mean()
    loss.backward()
    old = w.detach().clone()
    opt.step()
    assert not torch.equal(old, w)
    x.requires_grad_(True)  # its gradient reads w as it was
    loss = ((x @ w + b) ** 2).sum()
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(loss, [x])


def test_many_tensors_take_several_launches():
    n = 905  # three tables
    counts = [(7 * i) % 600 for i in range(n)]
    ps, gs = make(counts, torch.float32, torch.float32, 9)
    opt = AdamW(ps, lr=LR, betas=BETAS, eps=EPS, weight_decay=0.1, state_bits=8, seed=3)
    before = [state64(opt, i) for i in range(n)]
    norm = opt.step(gs[2], max_norm=1.0)
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in gs[2]))
    assert abs(float(norm) - ref) <= 4 * U * ref
    assert int(opt.steps) == 1
    check_step(opt, gs[2], before, 1, clip=1.0 / ref)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_replays_and_counts(bits):
    ps, gs = make([5000, 257], torch.bfloat16, torch.bfloat16, 11)
    twin = [p.clone() for p in ps]
    lr = torch.tensor([1e-2], device="cuda")
    a = AdamW(ps, lr=lr, state_bits=bits, master_weights=True, seed=2)
    b = AdamW(twin, lr=1e-2, state_bits=bits, master_weights=True, seed=2)
    grads = [g.clone() for g in gs[0]]
    a.step(grads, max_norm=1.0)
    b.step(gs[0], max_norm=1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        norm = a.step(grads, max_norm=1.0)
    for k, rate in ((1, 1e-2), (2, 5e-3), (0, 0.0)):
        for x, g in zip(grads, gs[k]):
            x.copy_(g)
        lr.fill_(rate)
        graph.replay()
        ref = b.step(gs[k], lr=rate, max_norm=1.0)
        assert torch.equal(norm, ref)
        assert all(torch.equal(x, y) for x, y in zip(ps, twin))
        assert all(torch.equal(x.view(torch.uint8), b.state_dict()[n].view(torch.uint8)) for n, x in a.state_dict().items())
    assert int(a.steps) == 4


def test_memory_around_the_tensors_is_left_alone():
    buf = torch.full((4096,), 7.0, device="cuda", dtype=torch.bfloat16)
    ps = [buf[3:300], buf[1000:1001], buf[2048:2048 + 256]]
    opt = AdamW(ps, lr=0.5, state_bits=8)  # 7 - 0.5: well over bf16's half step of 2^-6 there
    opt.step([torch.ones_like(p) for p in ps])
    untouched = torch.ones(4096, dtype=torch.bool, device="cuda")
    for lo, hi in ((3, 300), (1000, 1001), (2048, 2304)):
        untouched[lo:hi] = False
        assert not (buf[lo:hi] == 7.0).any()
    assert (buf[untouched] == 7.0).all()


def test_other_stream_and_strided_gradient():
    w = torch.randn(64, 48, device="cuda")
    g = torch.randn(48, 64, device="cuda")
    twin = w.clone()
    AdamW([twin]).step([g.t().contiguous()], max_norm=1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        AdamW([w]).step([g.t()], max_norm=1.0)
    side.synchronize()
    assert torch.equal(w, twin)


def test_stochastic_rounding_follows_a_slow_moment():
    """v far below its target moves by less than half a code each step; the
    stochastic form follows all the same.  4096 equal elements: after 200 steps
    of g^2 = 2 v0 the mean of v is v0 (2 - 0.999^200) within 6 standard errors,
    a step's rounding being off by less than one code step (1/8) of v."""
    n = 4096
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), math.sqrt(2e-6), device="cuda")
    g[::256] = math.sqrt(64e-6)  # keeps every block's scale well above
    opt = AdamW([p], lr=0.0, weight_decay=0.0, state_bits=8, seed=1)
    start = torch.full((n,), 1e-6, device="cuda")
    start[::256] = 64e-6
    value, scale = R.codes(start.double().cpu())[:2]
    opt.exp_avg_sq.copy_(value.float().cuda())
    opt.exp_avg_sq_scale.copy_(scale.float().cuda())
    _, v0 = opt.moments(0)
    for _ in range(200):
        opt.step([g])
    _, v = opt.moments(0)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[::256] = False
    want = 2e-6 + (float(v0[keep].double().mean()) - 2e-6) * 0.999 ** 200
    mean = float(v[keep].double().mean())
    bound = 6 * math.sqrt(200) * 2e-6 / 8 / math.sqrt(int(keep.sum()))
    assert abs(mean - want) <= bound, (mean, want, bound)


def test_codes_are_the_formulas_everywhere():
    """Every one of a million codes, over steps of steady, growing, vanishing and cancelling gradients, is the one that
    64-bit arithmetic gives: fp32's error never picks the neighbour."""

    def same(codes, ref):
        # Values of bf16 gradients can lie on a border exactly (the first step's m is 0.1 g: a ratio of two bf16
        # numbers); there the order of the reference's own operations decides.  A value is off by a few 2^-53 of
        # itself, at most 16 code steps: below 2^-40 of a step.
        value, _, edge, _, _ = ref
        return not ((codes.double().cpu() != value) & (edge > 2.0 ** -40)).any()
    n = 1 << 20
    gen = torch.Generator().manual_seed(6)
    base = torch.randn(n, generator=gen) * torch.exp(2 * torch.randn(n, generator=gen))
    p = torch.zeros(n, device="cuda")
    opt = AdamW([p], lr=1e-3, betas=BETAS, weight_decay=0.0, state_bits=8, seed=77)
    where = torch.arange(n)
    for t, factor in enumerate([1.0, 1.0, 1.0, -7.0, 1e-3, 30.0, 1.0, 1e4, -3e-2, 1.0], 1):
        g = (base * factor * 1e-3).bfloat16().cuda()
        _, m0, v0 = state64(opt, 0)
        norm = opt.step([g], max_norm=1.0)
        g64 = g.double().cpu() * min(1.0, 1.0 / float(norm))
        _, m, v = R.adamw(torch.zeros_like(m0), m0, v0, g64, t, 1e-3, BETAS, EPS, 0.0)
        assert same(opt.exp_avg, R.codes(m)), t
        assert same(opt.exp_avg_sq, R.codes(v, R.random20(where, t, 77))), t


def test_large_and_tiny_moments_in_8_bits():
    """Gradients up to the end of fp32's range and below its squares' range: codes by the formula, blocks too small for
    a scale held as zeros."""
    sizes = [1e-18, 1e-10, 1.0, 1e4, 1e9, 1e18]
    n = 256 * len(sizes)
    gen = torch.Generator().manual_seed(2)
    g = (torch.randn(len(sizes), 256, generator=gen) * torch.tensor(sizes)[:, None]).view(-1).cuda()
    opt = AdamW([torch.zeros(n, device="cuda")], lr=1e-3, betas=BETAS, weight_decay=0.0, state_bits=8, seed=3)
    for t in (1, 2):
        _, m0, v0 = state64(opt, 0)
        opt.step([g])
        _, m, v = R.adamw(torch.zeros_like(m0), m0, v0, g.double().cpu(), t, 1e-3, BETAS, EPS, 0.0)
        assert torch.equal(opt.exp_avg.double().cpu(), R.codes(m)[0])
        assert torch.equal(opt.exp_avg_sq.double().cpu(), R.codes(v, R.random20(torch.arange(n), t, 3))[0])
    assert not opt.exp_avg_sq[:256].view(torch.uint8).any() and opt.exp_avg[:256].view(torch.uint8).any()
    assert opt.params[0].isfinite().all()


def test_places_past_32_bits():
    n = (1 << 31) + 300
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free memory")
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    q = torch.full((515,), 0.5, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = (torch.randn(700, generator=torch.Generator().manual_seed(1)) * 0.1).bfloat16().cuda()
    g[-700:] = tail
    gq = tail[:515].clone()
    opt = AdamW([p, q], lr=LR, betas=BETAS, eps=EPS, weight_decay=0.0, state_bits=8, seed=9)
    norm = opt.step([g, gq], max_norm=1e3)
    ref = math.sqrt(float(tail.double().square().sum() + gq.double().square().sum()))
    assert abs(float(norm) - ref) <= 4 * U * ref
    assert (p[:1000] == 1).all() and (p[-1000:-700] == 1).all()
    for w, grad, first, at in ((p[-300:], tail[-300:], 1.0, 1 << 31), (q, gq, 0.5, opt.offsets[1])):
        m = w.numel()
        z = torch.zeros(m, dtype=torch.float64)
        rp, rm, rv = R.adamw(z + first, z, z, grad.double().cpu(), 1, LR, BETAS, EPS, 0.0)
        assert torch.all((w.double().cpu() - rp).abs() <= 2.0 ** -8 * rp.abs() + 2.0 ** -19 * LR)
        rnd = R.random20(torch.arange(at, at + m), 1, 9)
        value, _, edge, r, gap = R.codes(rv, rnd)
        got = opt.exp_avg_sq[at:at + value.numel()].double().cpu()
        assert not ((got != value) & (edge > 28 * U * r / gap + 8 * U)).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 1e-30, 1e25])
def test_norm(dtype, scale):
    gen = torch.Generator().manual_seed(5)
    gs = [(torch.randn(n, generator=gen) * scale).to(dtype).cuda() for n in [1, 1023, 1024, 1025, 0, 100003, 8]]
    gs[3] = unaligned(gs[3])
    gs.insert(2, None)
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in gs if g is not None))
    got = grad_norm(gs)
    # 8 squares summed in fp32: at most 8 roundings of positive terms, half of that in the root, one for the result
    assert got.shape == (1,) and abs(float(got) - ref) <= 5 * U * ref
    assert torch.equal(got, grad_norm(gs))


def test_norm_extremes():
    big = torch.full((10,), 3e38, device="cuda")
    assert float(grad_norm([big])) == math.inf
    assert float(grad_norm([torch.zeros(5, device="cuda")])) == 0.0
    assert float(grad_norm([torch.zeros(0, device="cuda")])) == 0.0
    mixed = torch.tensor([1e-30, 2e18, 1e-45], device="cuda")
    assert abs(float(grad_norm([mixed])) - 2e18) <= 2e18 * 2 * U
    for bad in (math.inf, -math.inf, math.nan):
        x = torch.ones(3000, device="cuda")
        x[2999] = bad
        assert not math.isfinite(float(grad_norm([x, x])))


def test_refusals_with_tensors_on_the_device():
    w = torch.randn(16, 16, device="cuda")
    with pytest.raises(RKLError, match="share memory"):
        AdamW([w, w])
    with pytest.raises(RKLError, match="share memory"):
        AdamW([w, w[3:5]])
    with pytest.raises(RKLError, match="contiguous"):
        AdamW([w.t()[:, :3]])
    with pytest.raises(RKLError, match="dtype"):
        AdamW([w.half()])
    opt = AdamW([w])
    with pytest.raises(RKLError, match="1 parameters"):
        opt.step([w, w])
    with pytest.raises(RKLError, match="shape"):
        opt.step([torch.ones(16, device="cuda")])
    with pytest.raises(RKLError, match="dtype"):
        opt.step([w.double()])
    with pytest.raises(RKLError, match="max_norm"):
        opt.step([w.clone()], max_norm=0.0)
    with pytest.raises(RKLError, match="lr"):
        opt.step([w.clone()], lr=-1.0)
    with pytest.raises(RKLError, match="moved"):
        w.data = w.data.clone()
        opt.step([w.clone()])
    assert int(opt.steps) == 0
