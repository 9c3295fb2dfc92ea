"""The operators of a training step together, as a user's loop runs them: the
gated block in front of the head, the reverse-KL loss on its output, both
backward passes, the clipped AdamW step over all four weights."""

import math

import pytest
import torch

from full_vocabulary_reverse_b200 import (REDUCE_TOKEN_MEAN, AdamW, ffn_backward, ffn_forward, gated_ffn, grad_norm,
                                          reverse_kl_hidden)
from full_vocabulary_reverse_b200 import binding as rb
from tests import ffn_reference, optim_reference

pytestmark = pytest.mark.gpu
B, SM1, H, F, V = 2, 150, 128, 264, 1000
LR, BETAS, EPS, DECAY = 1e-2, (0.9, 0.999), 1e-8, 0.1


def problem(seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda shape, s: (torch.randn(shape, generator=gen) * s).bfloat16().cuda()  # noqa: E731
    x, h_t = r((B * SM1, H), 1.0), r((B * SM1, H), 1.0)
    weights = [r((F, H), H ** -0.5), r((F, H), H ** -0.5), r((H, F), F ** -0.5), r((V, H), 3 * H ** -0.5)]
    W_t = r((V, H), 3 * H ** -0.5)
    mask = (torch.rand((B, SM1), generator=gen) < 0.6).to(torch.uint8).cuda()
    return x, h_t, weights, W_t, mask


def loss64(x, h_t, weights, W_t, mask):
    wg, wu, wd, ws = weights
    g = x @ wg.t()
    h = (ffn_reference.act(ffn_reference.SILU, g)[0] * (x @ wu.t())) @ wd.t()
    ps, pt = torch.log_softmax(h @ ws.t(), -1), torch.log_softmax(h_t @ W_t.t(), -1)
    per_row = (ps.exp() * (ps - pt)).sum(-1)
    keep = mask.reshape(-1).bool()
    return per_row[keep].mean()


def test_gradients_of_the_chain():
    """Against float64 autograd of the definition.  Operands rounded to bf16 on the way of a gradient: y (the head's
    input), the loss's dz, dH, then a, dg and du, and the result; the head's input moves the logits' gradient too.  Each
    is at most half a step, 2^-8 relative, of a value: eight of them, in 2-norms, below 8 x 2^-8."""
    x, h_t, weights, W_t, mask = problem()
    leaves = [w.requires_grad_(True) for w in weights]
    h = gated_ffn(x.requires_grad_(True), *leaves[:3])
    loss, _ = reverse_kl_hidden(h, h_t, leaves[3], W_t, mask, REDUCE_TOKEN_MEAN)
    got = torch.autograd.grad(loss, [x, *leaves])
    x64, w64 = x.detach().double().requires_grad_(True), [w.detach().double().requires_grad_(True) for w in weights]
    ref = loss64(x64, h_t.double(), w64, W_t.double(), mask)
    want = torch.autograd.grad(ref, [x64, *w64])
    # y's rounding moves a logit (standard deviation 3) by below 3 x 2^-8; the loss, some 7 a row, by less than that
    assert abs(float(loss.detach()) - float(ref.detach())) <= 3 * 2.0 ** -8
    for k, (a, b) in enumerate(zip(got, want)):
        assert float((a.double() - b).norm() / b.norm()) <= 8 * 2.0 ** -8, k
    masked = ~mask.reshape(-1).bool()
    assert not got[0][masked].any()  # rows outside the loss get exact zeros through the block as well


@pytest.mark.parametrize("bits", [32, 8])
def test_step_follows_its_own_gradients(bits):
    """The update is AdamW's of the gradients that the loop has in hand, clipped by their common norm."""
    x, h_t, weights, W_t, mask = problem(1)
    params = [torch.nn.Parameter(w) for w in weights]
    opt = AdamW(params, lr=LR, betas=BETAS, eps=EPS, weight_decay=[DECAY] * 4, state_bits=bits, master_weights=True)
    for t in (1, 2):
        loss, _ = reverse_kl_hidden(gated_ffn(x, *params[:3]), h_t, params[3], W_t, mask)
        loss.backward()
        before = []
        for i, p in enumerate(params):
            m, v = opt.moments(i)
            at = opt.offsets[i]
            before.append((opt.master[at:at + p.numel()].double().cpu(), m.double().cpu().view(-1), v.double().cpu().view(-1)))
        grads = [p.grad.clone() for p in params]
        total = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        limit = total / 3
        norm = opt.step(max_norm=limit)
        assert abs(float(norm) - total) <= 2.0 ** -21 * total
        assert torch.equal(norm, grad_norm(grads))
        for i, p in enumerate(params):
            at = opt.offsets[i]
            p0, m0, v0 = before[i]
            g = grads[i].double().cpu().reshape(-1)
            rp, _, _ = optim_reference.adamw(p0, m0, v0, g, t, LR, BETAS, EPS, DECAY, clip=limit / total)
            # p: 4 half steps of fp32; the update, at most lr |m| / sqrt(v) sized, 2^-19 of the terms in m
            terms = BETAS[0] * m0.abs() + (1 - BETAS[0]) * g.abs() * limit / total
            v = BETAS[1] * v0 + (1 - BETAS[1]) * (g * limit / total) ** 2
            upd = LR / (1 - BETAS[0] ** t) * terms / (v.sqrt() / math.sqrt(1 - BETAS[1] ** t) + EPS)
            # (a moment's code x scale is rounded once more in fp32 than here: 2^-23 of the update)
            off = (opt.master[at:at + p.numel()].double().cpu() - rp).abs()
            assert torch.all(off <= 4 * 2.0 ** -24 * rp.abs() + 2.0 ** -18 * upd), i
            assert torch.equal(p.detach().reshape(-1), opt.master[at:at + p.numel()].bfloat16())
            p.grad = None
    assert int(opt.steps) == 2 and rb.device_error() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_training_step(bits):
    """One graph holds the whole step; its replays on changing inputs equal the same calls made eagerly."""
    def build(seed=2):
        x, h_t, weights, W_t, mask = problem(seed)
        return x, h_t, weights, W_t, mask, AdamW(weights, lr=1e-3, state_bits=bits, master_weights=True, seed=4)

    def step(s):
        x, h_t, (wg, wu, wd, ws), W_t, mask, opt = s
        h, saved = ffn_forward(x, wg, wu, wd, save=True)
        row_idx, n = rb.compact_rows(mask, on_device=True)
        _, loss, kept = rb.forward_hidden(h, h_t, ws, W_t, B, SM1, row_idx, n, REDUCE_TOKEN_MEAN)
        one = torch.ones(1, device="cuda")
        dh, dws = rb.backward(rb.PAYLOAD_HIDDEN, h, h_t, ws, W_t, B, SM1, row_idx, n, REDUCE_TOKEN_MEAN, kept, grad_loss=one)
        _, dwg, dwu, dwd = ffn_backward(x, wg, wu, wd, dh.bfloat16(), saved, needs=(False, True, True, True))
        norm = opt.step([dwg, dwu, dwd, dws], max_norm=0.1)
        return loss, norm

    a, b = build(), build()
    for s in (a, b):
        step(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        loss, norm = step(a)
    torch.cuda.current_stream().wait_stream(side)
    for k in range(3):
        fresh = problem(10 + k)
        for s in (a, b):
            s[0].copy_(fresh[0])
            s[1].copy_(fresh[1])
            s[4].copy_(fresh[4] if k < 2 else torch.zeros_like(fresh[4]))  # the last batch has no row in the loss
        graph.replay()
        ref_loss, ref_norm = step(b)
        assert torch.equal(loss, ref_loss) and torch.equal(norm, ref_norm)
        assert all(torch.equal(p, q) for p, q in zip(a[2], b[2]))
    assert int(a[5].steps) == 4 and float(norm) == 0.0
    assert rb.device_error() == 0
