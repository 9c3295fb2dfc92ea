"""Cases of the training-step operators: the gated feed-forward block, the
AdamW step over many tensors (32-bit and 8-bit states) and the global gradient
norm.

``own`` False computes every operator in its plain form (elementary torch
operations, 32 bits or more, rounded once at the end); ``own`` True makes the
calls a user of the package makes.  ``exact`` gives the same results in 64
bits, straight from the operators' definitions.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}
_ACTS = ("silu", "gelu", "gelu_tanh", "relu")
_BLOCK = 256  # elements that share one scale of an 8-bit state, and the alignment of a tensor's place in the state
_LR, _B1, _B2, _EPS, _WD, _MAX_NORM, _SEED = 1e-3, 0.9, 0.999, 1e-8, 0.1, 1.0, 17
_FIRST = 100  # optimizer steps behind the state that a case starts from


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through the block: serving's smallest call, latency and the reading of the weights
        dict(name="ffn_token", op="ffn", train=False, dtype="bf16", act="silu", T=1, H=2048, F=6144, O=2048),
        # a small decoding batch through a wider block, an odd number of rows
        dict(name="ffn_batch_23", op="ffn", train=False, dtype="bf16", act="gelu_tanh", T=23, H=4096, F=11008, O=4096),
        # a prompt of odd length
        dict(name="ffn_prompt", op="ffn", train=False, dtype="bf16", act="silu", T=2047, H=4096, F=11008, O=4096),
        # training: all B (S-1) = 4 x 2048 rows of the default workload, forward and backward
        dict(name="ffn_train", op="ffn", train=True, dtype="bf16", act="silu", T=8192, H=2048, F=6144, O=2048),
        # training on a ragged batch: row count, widths and output width off every tile border
        dict(name="ffn_train_ragged", op="ffn", train=True, dtype="bf16", act="gelu", T=1171, H=1160, F=2712, O=840),
        # training in 32 bits (the small parity configuration's type), sizes off every border
        dict(name="ffn_train_fp32", op="ffn", train=True, dtype="fp32", act="silu", T=509, H=515, F=1031, O=515),
        # the LM head of the default workload and one block's weights, bf16 with 32-bit master copies, fp32
        # gradients as the loss's backward gives them, clipped by the global norm
        dict(name="adamw_head", op="adamw", bits=32, param="bf16", grad="fp32", master=True, clip=True,
             shapes="151936x2048 6144x2048 6144x2048 2048x6144 2048"),
        # the norm weights and biases of a small model: many little fp32 tensors, launch latency
        dict(name="adamw_little", op="adamw", bits=32, param="fp32", grad="fp32", master=False, clip=False,
             shapes=" ".join(["2048 515 77 1"] * 12)),
        # the head again with 8-bit states
        dict(name="adamw8_head", op="adamw", bits=8, param="bf16", grad="bf16", master=False, clip=True,
             shapes="151936x2048 6144x2048 6144x2048 2048x6144 2048"),
        # an adapter's tensors with 8-bit states, sizes off the border of a scale's block
        dict(name="adamw8_odd", op="adamw", bits=8, param="fp32", grad="fp32", master=False, clip=False,
             shapes="1031x515 1031x515 515x1031 515 4097 255 1 2048x64 64x2049"),
        # the norm alone, as a training log wants it each step: a head's and a block's gradients
        dict(name="norm_head", op="norm", grad="bf16", shapes="151936x2048 6144x2048 6144x2048 2048x6144 2048"),
        # the norm over many tensors of odd sizes
        dict(name="norm_little", op="norm", grad="fp32", shapes=" ".join(["2048x33 515 77 1"] * 12)),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "adamw", "adamw", "norm"])
    if op == "ffn":
        if rng.random() < 0.2:  # 32 bits: any sizes
            return dict(op="ffn", train=rng.random() < 0.7, dtype="fp32", act=rng.choice(_ACTS), T=_log_int(rng, 1, 700),
                        H=_log_int(rng, 30, 900), F=_log_int(rng, 30, 1500), O=_log_int(rng, 30, 900))
        train = rng.random() < 0.6
        unit = 8 if rng.random() < 0.9 else 1  # widths of 16-byte rows, now and then others
        most = 4096 if unit == 8 else 700
        wide = lambda lo, hi: max(unit, _log_int(rng, lo, hi) // unit * unit)  # noqa: E731
        return dict(op="ffn", train=train, dtype="bf16", act=rng.choice(_ACTS), T=_log_int(rng, 1, 6000),
                    H=wide(64, most // 2), F=wide(64, most), O=wide(64, most // 2))
    shapes = []
    total = _log_int(rng, 2_000, 200_000_000)
    for _ in range(rng.randint(1, 48)):
        n = max(1, min(total, _log_int(rng, 1, 2 * total)))
        cols = max(1, min(n, rng.choice([1, 64, 255, 1031, 2048, 4097])))
        shapes.append("%dx%d" % (max(1, n // cols), cols) if cols > 1 else "%d" % n)
        total -= n
        if total <= 0:
            break
    shapes = " ".join(shapes)
    if op == "norm":
        return dict(op="norm", grad=rng.choice(["bf16", "fp32"]), shapes=shapes)
    param = rng.choice(["bf16", "fp32"])
    return dict(op="adamw", bits=rng.choice([8, 32]), param=param, grad=rng.choice([param, "fp32"]),
                master=param == "bf16" and rng.random() < 0.5, clip=rng.random() < 0.5, shapes=shapes)


def _shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["shapes"].split()]


def _places(shapes):
    """(element counts, first element of each tensor in the state, elements of the state)."""
    counts = [math.prod(s) for s in shapes]
    firsts, at = [], 0
    for n in counts:
        firsts.append(at)
        at += -(-n // _BLOCK) * _BLOCK
    return counts, firsts, at


def work(case):
    if case["op"] == "ffn":
        T, H, F, O, es = case["T"], case["H"], case["F"], case["O"], _BYTES[case["dtype"]]
        weights, rows = F * (2 * H + O), T * (H + O)
        if not case["train"]:
            return {"bytes": es * (weights + rows), "flops": 2 * T * weights}
        return {"bytes": es * (2 * weights + 2 * rows), "flops": 6 * T * weights}
    n = sum(math.prod(s) for s in _shapes(case))
    g = _BYTES[case["grad"]]
    if case["op"] == "norm":
        return {"bytes": n * g, "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 + 16 / _BLOCK
    param = 2 + 8 if case["master"] else 2 * _BYTES[case["param"]]
    return {"bytes": int(n * (param + g + state)), "flops": 16 * n}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(shape, scale, dtype):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    if case["op"] == "ffn":
        T, H, F, O, dt = case["T"], case["H"], case["F"], case["O"], _DT[case["dtype"]]
        s = {"case": case, "x": normal((T, H), 1.0, dt), "w_gate": normal((F, H), H ** -0.5, dt),
             "w_up": normal((F, H), H ** -0.5, dt), "w_down": normal((O, F), F ** -0.5, dt)}
        if case["train"]:
            s["dy"] = normal((T, O), 0.01, dt)
            if own:
                for k in ("x", "w_gate", "w_up", "w_down"):
                    s[k].requires_grad_(True)
        return s

    shapes = _shapes(case)
    if case["op"] == "norm":
        return {"case": case, "grads": [normal(s, 0.01, _DT[case["grad"]]) for s in shapes]}

    params = [normal(s, 0.02, _DT[case["param"]]) for s in shapes]
    grads = [normal(s, 1e-3, _DT[case["grad"]]) for s in shapes]
    counts, firsts, total = _places(shapes)
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for n, at in zip(counts, firsts):
        live[at: at + n] = True
    s = {"case": case, "params": params, "grads": grads, "live": live,
         "decay": [_WD if len(sh) > 1 else 0.0 for sh in shapes],  # matrices decay, vectors do not
         "steps": torch.full((1,), _FIRST, dtype=torch.int32, device="cuda")}
    # the state of a run under way: moments of the size that such gradients leave
    if case["bits"] == 32:
        s["m"] = torch.randn(total, generator=gen, device="cuda") * 3e-4 * live
        s["v"] = (torch.rand(total, generator=gen, device="cuda") + 0.1) * 1e-7 * live
    else:
        blocks = total // _BLOCK
        code = torch.randn(total, generator=gen, device="cuda") * 120 * live
        s["m"] = code.clamp_(-448, 448).to(torch.float8_e4m3fn)
        code = (torch.rand(total, generator=gen, device="cuda") * 440 + 4) * live
        s["v"] = code.to(torch.float8_e4m3fn)
        s["m_scale"] = (torch.rand(blocks, generator=gen, device="cuda") + 0.5) * (1e-3 / 448)
        s["v_scale"] = (torch.rand(blocks, generator=gen, device="cuda") + 0.5) * (2e-7 / 448)
    if case["master"]:
        s["master"] = torch.zeros(total, device="cuda")
        for p, n, at in zip(params, counts, firsts):
            s["master"][at: at + n] = p.reshape(-1)
    if own:
        from full_vocabulary_reverse_b200 import AdamW
        opt = AdamW(params, lr=_LR, betas=(_B1, _B2), eps=_EPS, weight_decay=s["decay"], state_bits=case["bits"],
                    master_weights=case["master"], seed=_SEED)
        opt.exp_avg.copy_(s.pop("m"))
        opt.exp_avg_sq.copy_(s.pop("v"))
        opt.steps.copy_(s.pop("steps"))
        if case["bits"] == 8:
            opt.exp_avg_scale.copy_(s.pop("m_scale"))
            opt.exp_avg_sq_scale.copy_(s.pop("v_scale"))
        s["opt"] = opt
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if case["op"] == "ffn":
        return _run_ffn(state, case)
    if case["op"] == "norm":
        if own:
            from full_vocabulary_reverse_b200 import grad_norm
            return grad_norm(state["grads"])
        return _plain_norm(state["grads"])
    if own:
        opt = state["opt"]
        norm = opt.step(state["grads"], max_norm=_MAX_NORM if case["clip"] else None)
        out = {"params": state["params"], "m": opt.exp_avg, "v": opt.exp_avg_sq, "steps": opt.steps}
        if case["bits"] == 8:
            out.update(m_scale=opt.exp_avg_scale, v_scale=opt.exp_avg_sq_scale)
        if case["master"]:
            out["master"] = opt.master
        if case["clip"]:
            out["norm"] = norm
        return out
    return _plain_adamw(state, case)


def _run_ffn(state, case):
    x, wg, wu, wd = state["x"], state["w_gate"], state["w_up"], state["w_down"]
    if own:
        import full_vocabulary_reverse_b200 as fvr
        act = {"silu": fvr.ACT_SILU, "gelu": fvr.ACT_GELU, "gelu_tanh": fvr.ACT_GELU_TANH, "relu": fvr.ACT_RELU}
        y = fvr.gated_ffn(x, wg, wu, wd, act[case["act"]])
        if not case["train"]:
            return y
        return [y.detach()] + list(torch.autograd.grad(y, [x, wg, wu, wd], state["dy"]))
    dt = x.dtype
    x, wg, wu, wd = x.float(), wg.float(), wu.float(), wd.float()
    g, u = x @ wg.t(), x @ wu.t()
    act, slope = _activation(case["act"], g)
    a = act * u
    y = (a @ wd.t()).to(dt)
    if not case["train"]:
        return y
    dy = state["dy"].float()
    da = dy @ wd
    dg, du = da * u * slope, da * act
    return [y] + [t.to(dt) for t in (dg @ wg + du @ wu, dg.t() @ x, du.t() @ x, dy.t() @ a)]


def _activation(kind, g):
    """(the activation of g, its derivative)."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if kind == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if kind == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _plain_norm(grads):
    parts = torch.stack([g.reshape(-1).double().square().sum() for g in grads])
    return parts.sum().sqrt().float().reshape(1)


def _padded(tensors, dtype):
    """The tensors one behind another, each up to the border of a block."""
    pad = torch.nn.functional.pad
    return torch.cat([pad(t.reshape(-1).to(dtype), (0, -t.numel() % _BLOCK)) for t in tensors])


def _spread(values, counts, dtype):
    """values[i] for each element of tensor i and of its padding."""
    reps = torch.tensor([-(-n // _BLOCK) * _BLOCK for n in counts], device="cuda")
    return torch.repeat_interleave(torch.tensor(values, dtype=dtype, device="cuda"), reps, output_size=sum(
        -(-n // _BLOCK) * _BLOCK for n in counts))


def _plain_adamw(state, case):
    # 8-bit states: in 64 bits, since a value next to the border of two codes takes the one or the other
    dt = torch.float32 if case["bits"] == 32 else torch.float64
    params, live = state["params"], state["live"]
    counts, firsts, total = _places([tuple(p.shape) for p in params])
    state["steps"] += 1
    t = state["steps"].double()
    g = _padded(state["grads"], dt)
    norm = None
    if case["clip"]:
        norm = _plain_norm(state["grads"])
        g = g * (_MAX_NORM / norm.double()).clamp(max=1.0).to(dt)
    p = state["master"].to(dt) if case["master"] else _padded(params, dt)
    if case["bits"] == 32:
        m, v = state["m"], state["v"]
    else:
        m = state["m"].to(dt) * state["m_scale"].to(dt).repeat_interleave(_BLOCK)
        v = state["v"].to(dt) * state["v_scale"].to(dt).repeat_interleave(_BLOCK)
    m = _B1 * m + (1 - _B1) * g
    v = _B2 * v + (1 - _B2) * g * g
    root = torch.sqrt(v) / torch.sqrt(1 - _B2 ** t).to(dt) + _EPS
    p = p * (1 - _LR * _spread(state["decay"], counts, dt)) - (_LR / (1 - _B1 ** t)).to(dt) * m / root
    if case["bits"] == 32:
        state["m"], state["v"] = m, v
    else:
        state["m"], state["m_scale"] = _to_codes(m, None)
        state["v"], state["v_scale"] = _to_codes(v, _random_bits(total, int(_SEED), state["steps"]))
    new = [p[at: at + n].reshape(w.shape).to(w.dtype) for w, n, at in zip(params, counts, firsts)]
    torch._foreach_copy_(params, new)
    out = {"params": params, "m": state["m"], "v": state["v"], "steps": state["steps"]}
    if case["bits"] == 8:
        out.update(m_scale=state["m_scale"], v_scale=state["v_scale"])
    if case["master"]:
        state["master"] = torch.where(live, p, torch.zeros_like(p)).float()
        out["master"] = state["master"]
    if case["clip"]:
        out["norm"] = norm
    return out


def _mix(h):
    """The final mix of MurmurHash3 on 32-bit numbers held in 64 bits."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random_bits(total, seed, steps):
    """20 bits for each element of the state, from the seed, the step and the element's place."""
    at = torch.arange(total, dtype=torch.int64, device="cuda")
    key = _mix((steps.long() * 0x9E3779B1 + seed) & 0xFFFFFFFF)
    return _mix((at & 0xFFFFFFFF) ^ _mix((key + (at >> 32)) & 0xFFFFFFFF)) >> 12


def _to_codes(x, bits):
    """Blocks of 256 values as e4m3 times the block's scale = largest magnitude / 448.

    To the nearest code (ties to even) where bits is None; else up with the probability that the rest has, by 20
    random bits, and never from a value above zero to zero."""
    x = x.reshape(-1, _BLOCK)
    most = x.abs().amax(dim=1, keepdim=True)
    some = most > 2.0 ** -100
    r = torch.where(some, x * (448.0 / most), torch.zeros_like(x))
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6))) - 3)
    if bits is None:
        code = torch.round(r / step) * step
    else:
        code = torch.floor(r / step + bits.reshape(-1, _BLOCK).to(x.dtype) * 2.0 ** -20) * step
        code = torch.where(r > 0, code.clamp(min=2.0 ** -9), code)
    code = code.clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn)
    scale = torch.where(some, most / 448.0, torch.zeros_like(most)).float()
    return code.reshape(-1), scale.reshape(-1)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    if own:
        raise RuntimeError("the exact values use none of the package's code")
    s = prepare(case, seed)
    if case["op"] == "ffn":
        return _exact_ffn(s, case)
    if case["op"] == "norm":
        return torch.linalg.vector_norm(torch.cat([g.double().flatten() for g in s["grads"]])).reshape(1)
    return _exact_adamw(s, case)


def _exact_ffn(s, case):
    # differentiates the definition itself
    x, wg, wu, wd = (s[k].double().requires_grad_(case["train"]) for k in ("x", "w_gate", "w_up", "w_down"))
    z = torch.einsum("th,fh->tf", x, wg)
    kind = case["act"]
    if kind == "silu":
        a = z * torch.sigmoid(z)
    elif kind == "relu":
        a = torch.maximum(z, torch.zeros_like(z))
    elif kind == "gelu":
        a = z * torch.special.ndtr(z)
    else:
        a = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    y = torch.einsum("tf,of->to", a * torch.einsum("th,fh->tf", x, wu), wd)
    if not case["train"]:
        return y
    return [y.detach()] + list(torch.autograd.grad(y, [x, wg, wu, wd], s["dy"].double()))


def _exact_adamw(s, case):
    t = _FIRST + 1
    counts, firsts, total = _places(_shapes(case))
    sq = sum(float(g.double().pow(2).sum()) for g in s["grads"])
    clip = min(1.0, _MAX_NORM / math.sqrt(sq)) if case["clip"] and sq > 0 else 1.0
    out = {"params": [], "steps": torch.tensor([t], dtype=torch.int32)}
    m = torch.zeros(total, dtype=torch.float64, device="cuda")
    v, master = torch.zeros_like(m), torch.zeros_like(m)
    for w, g, decay, n, at in zip(s["params"], s["grads"], s["decay"], counts, firsts):
        here = slice(at, at + n)
        m0, v0 = s["m"][here].double(), s["v"][here].double()
        if case["bits"] == 8:
            block = torch.arange(at, at + n, device="cuda") // _BLOCK
            m0, v0 = m0 * s["m_scale"].double()[block], v0 * s["v_scale"].double()[block]
        g = g.double().flatten() * clip
        m[here] = m0 + (g - m0) * (1 - _B1)
        v[here] = v0 + (g.pow(2) - v0) * (1 - _B2)
        p = (s["master"][here] if case["master"] else w.flatten()).double()
        p = p - _LR * decay * p - _LR * (m[here] / (1 - _B1 ** t)) / ((v[here] / (1 - _B2 ** t)).sqrt() + _EPS)
        out["params"].append(p.reshape(w.shape))
        master[here] = p
    if case["master"]:
        out["master"] = master
    if case["clip"]:
        out["norm"] = torch.tensor([math.sqrt(sq)], dtype=torch.float64)
    if case["bits"] == 32:
        out["m"], out["v"] = m, v
        return out
    out["m"], out["m_scale"] = _exact_codes(m, None)
    out["v"], out["v_scale"] = _exact_codes(v, t)
    return out


def _exact_codes(x, t):
    """Every value between its two neighbours in the table of e4m3's numbers."""
    table = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    most = x.view(-1, _BLOCK).abs().amax(1)
    r = (x.abs() / most.clamp(min=2.0 ** -100).repeat_interleave(_BLOCK) * 448).clamp(max=448)
    lo = (torch.searchsorted(table, r, right=True) - 1).clamp(max=125)
    part = (r - table[lo]) / (table[lo + 1] - table[lo])
    if t is None:
        up = (part > 0.5) | ((part == 0.5) & (lo % 2 == 1))
    else:
        word = lambda h, a, b: (h ^ (h >> a)) * b % 2 ** 32  # noqa: E731
        fmix = lambda h: word(word(h, 16, 0x85EBCA6B), 13, 0xC2B2AE35) ^ (word(word(h, 16, 0x85EBCA6B), 13, 0xC2B2AE35) >> 16)  # noqa: E731
        key = fmix((t * 0x9E3779B1 + _SEED) % 2 ** 32)
        at = torch.arange(x.numel(), device="cuda")
        rnd = fmix(at % 2 ** 32 ^ fmix((key + at // 2 ** 32) % 2 ** 32)) // 4096
        up = (part + rnd / 2.0 ** 20 >= 1) | ((lo == 0) & (r > 0))
    code = table[lo + up.long()] * torch.sign(x)
    return code, torch.where(most > 2.0 ** -100, most / 448, torch.zeros_like(most))
