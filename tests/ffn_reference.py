"""The gated feed-forward block in 64 bits, from its formulas, with bounds of
what a computation with fp32 sums and operands rounded to the inputs' type may
be off by (test infrastructure: shares no code with the package).

Bounds, with u = 2^-24 and b half a step of the inputs' type (0 for fp32: its
values are not rounded further):
  a sum of n products in fp32, in any order, each addition off by at most one
      step (tensor cores cut instead of rounding):  2 (n + 2) u sum |x_k w_k|
  act:  |act'| <= 1.13 and |act''| <= 1.2 for all four away from relu's corner;
      act itself 2^-19 relative, act' 2^-19 (1 + |g|) (the hardware's exponential
      and reciprocal, 2^-21 each, and e^-g's argument)
  each operand or result rounded to the type:  b relative
"""

import math

import torch

U = 2.0 ** -24
SILU, GELU, GELU_TANH, RELU = range(4)
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def act(kind, g):
    """(act, act') in float64."""
    if kind == SILU:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == GELU:
        c = torch.special.ndtr(g)
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if kind == GELU_TANH:
        k = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(k * (g + 0.044715 * g ** 3))
        return g * s, s + g * s * (1 - s) * k * (1 + 3 * 0.044715 * g * g)
    return torch.clamp(g, min=0), (g > 0).double()


def dot(x, w, ex, ew):
    """Bound of x @ w for |x| off by ex and |w| off by ew, all given as magnitudes."""
    e = 2 * (x.shape[1] + 2) * U * (x @ w)
    if ex is not None:
        e = e + ex @ (w if ew is None else w + ew)
    if ew is not None:
        e = e + x @ ew
    return e


def block(x, wg, wu, wd, kind, dy=None, operand=None):
    """[(value, bound)] of y, and with dy of dx, dWg, dWu, dWd.  operand: what a, dg and du may be rounded by, relative
    (None: half a step of the type)."""
    b = HALF_STEP[x.dtype]
    o = b if operand is None else operand
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = dot(x.abs(), wg.abs().t(), None, None), dot(x.abs(), wu.abs().t(), None, None)
    h, s = act(kind, g)
    a = h * u
    ea = 1.13 * eg * (u.abs() + eu) + h.abs() * eu + (2.0 ** -19 + o) * a.abs()
    y = a @ wd.t()
    out = [(y, dot(a.abs(), wd.abs().t(), ea, None) + b * y.abs())]
    if dy is None:
        return out
    dy = dy.double()
    da = dy @ wd
    eda = dot(dy.abs(), wd.abs(), None, None)
    du, dg = da * h, da * u * s
    edu = h.abs() * eda + (da.abs() + eda) * 1.13 * eg + (2.0 ** -19 + o) * du.abs()
    es = 1.2 * eg + 2.0 ** -19 * (1 + g.abs())
    if kind == RELU:
        es = (g.abs() <= eg).double()
    edg = (u * s).abs() * eda + ((da.abs() + eda) * (s.abs() * eu + (u.abs() + eu) * es)) + (2.0 ** -22 + o) * dg.abs()
    # an output is off by its operands' bounds, its own sum's and its rounding
    dx = dg @ wg + du @ wu
    out.append((dx, dot(dg.abs(), wg.abs(), edg, None) + dot(du.abs(), wu.abs(), edu, None)
                + 2 * wg.shape[0] * U * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()) + b * dx.abs()))
    for d, ed in ((dg, edg), (du, edu)):
        w = d.t() @ x
        out.append((w, dot(d.abs().t(), x.abs(), ed.t(), None) + b * w.abs()))
    w = dy.t() @ a
    out.append((w, dot(dy.abs().t(), a.abs(), None, ea) + b * w.abs()))
    return out


def check(got, ref, dtype):
    """Elements within their bounds; and, for sums of many independent roundings, the whole within 3 half steps of
    its 2-norm (operands, saved values and the result, each at most half a step)."""
    for k, (t, (value, bound)) in enumerate(zip(got, ref)):
        t = t.double().to(value.device)
        assert t.shape == value.shape, k
        off = (t - value).abs()
        assert torch.all(off <= bound), (k, float((off / bound.clamp(min=1e-300)).max()))
        if dtype == torch.bfloat16 and value.numel() > 64 and value.norm() > 0:
            assert float(off.norm() / value.norm()) <= 3 * HALF_STEP[dtype], k
