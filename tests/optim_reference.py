"""The optimizer step and the gradient norm in 64 bits, from their formulas
(test infrastructure: shares no code with the package)."""

import math

import torch

BLOCK = 256
M32 = 0xFFFFFFFF


def e4m3_table():
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def mix32(h):
    """MurmurHash3's final mix on a tensor of 32-bit numbers held in int64."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & M32
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & M32
    return h ^ (h >> 16)


def random20(at, t, seed):
    """The 20 bits of the state's elements `at` at step t."""
    key = int(mix32(torch.tensor((t * 0x9E3779B1 + seed) & M32)))
    hi = mix32((key + (at >> 32)) & M32)
    return mix32((at & M32) ^ hi) >> 12


def adamw(p, m, v, g, t, lr, betas, eps, decay, clip=1.0):
    """One step on float64 tensors; returns (p, m, v)."""
    b1, b2 = betas
    g = g * clip
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - lr * decay) - lr / (1 - b1 ** t) * m / (v.sqrt() / math.sqrt(1 - b2 ** t) + eps)
    return p, m, v


def codes(x, rnd=None):
    """Of a float64 state, padded to blocks: (value of each code, scale of each
    block, distance of each element's choice from the border between its two
    codes, the magnitude before rounding in the code's units, the step between
    the two codes).  rnd None: to nearest; else stochastic."""
    table = e4m3_table()
    x = torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)
    most = x.abs().amax(1, keepdim=True)
    some = most > 2.0 ** -100
    r = torch.where(some, x.abs() / torch.where(some, most, torch.ones_like(most)) * 448, torch.zeros_like(x))
    lo = (torch.searchsorted(table, r.reshape(-1), right=True) - 1).clamp(max=125).view_as(r)
    part = (r - table[lo]) / (table[lo + 1] - table[lo])
    if rnd is None:
        edge = part - 0.5
        up = (edge > 0) | ((edge == 0) & (lo % 2 == 1))
    else:
        edge = part + torch.nn.functional.pad(rnd, (0, x.numel() - rnd.numel())).view_as(x).double() / 2 ** 20 - 1
        forced = (lo == 0) & (r > 0)
        up = (edge >= 0) | forced
        edge = torch.where(forced, torch.ones_like(edge), edge)
    value = table[lo + up.long()] * torch.sign(x)
    scale = torch.where(some, most / 448, torch.zeros_like(most)).view(-1)
    return value.view(-1), scale, edge.abs().view(-1), r.view(-1), (table[lo + 1] - table[lo]).view(-1)
