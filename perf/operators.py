"""The training and serving operators as measured cases: the fused linear layer, its gradient and the AdamW step.

``linear``  OUT = act(X W + b) + R, on request with Z = X W + b kept
``grad``    D = G * act'(Z); dX = D W^T, dW = X^T D, db = the column sums of D
``adamw``   one AdamW step over a list of tensors, states in 32 bits or in 8

X is (m, n), W (n, k); ``w_t`` stores W's transpose row by row (W is then the transposed view).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 256  # elements that share a scale where the AdamW states are held in 8 bits
ADAM = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01}
STEPS = 1000  # steps taken before the measured one


# ---------------------------------------------------------------------------- cases
def _linear(name, dtype, m, n, k, act, bias=True, residual=False, pre=False, w_t=False):
    return {"name": name, "op": "linear", "dtype": dtype, "m": m, "n": n, "k": k, "act": act, "bias": bias,
            "residual": residual, "pre": pre, "w_t": w_t}


def _grad(name, dtype, m, n, k, act, w_t=False):
    return {"name": name, "op": "grad", "dtype": dtype, "m": m, "n": n, "k": k, "act": act, "w_t": w_t}


def _adamw(name, tensors, numel, param, grad, bits, copy="none"):
    return {"name": name, "op": "adamw", "tensors": tensors, "numel": numel, "param": param, "grad": grad, "bits": bits,
            "copy": copy}


def listed():
    return [
        # serving one row: the weights are read once, latency counts
        _linear("token_bf16", "bf16", 1, 4096, 4096, "silu", residual=True),
        # serving a small batch, weights stored output by output
        _linear("batch_f16", "f16", 24, 8192, 8192, "gelu_tanh", w_t=True),
        # a prompt's rows, of no round number, with a residual
        _linear("prompt_bf16", "bf16", 777, 4096, 2056, "silu", residual=True),
        # the forward pass of training a wide layer, with Z kept for the gradient
        _linear("train_bf16", "bf16", 8192, 4096, 16384, "gelu", pre=True),
        # the first layer on the library's tall data matrix (32 features)
        _linear("tall_f32", "f32", 1_000_000, 32, 32, "relu", pre=True),
        # a square layer on full-precision data
        _linear("wide_f32", "f32", 2048, 2048, 8192, "sigmoid"),
        # the gradient of a wide layer in training
        _grad("grad_bf16", "bf16", 8192, 4096, 16384, "gelu"),
        # the gradient of the first layer on the tall data matrix
        _grad("grad_tall_f32", "f32", 1_000_000, 32, 32, "relu"),
        # a small ragged gradient: odd row pitches, weights stored output by output
        _grad("grad_ragged_f16", "f16", 301, 1001, 503, "silu", w_t=True),
        # the step of a small network: latency counts
        _adamw("adamw_small", 20, 200_000, "f32", "f32", 32),
        # full-precision weights with 16-bit gradients and a 16-bit working copy
        _adamw("adamw_master", 120, 100_000_000, "f32", "bf16", 32, copy="bf16"),
        # 16-bit weights with states in 8 bits, for a network that has to fit
        _adamw("adamw_8bit", 300, 250_000_000, "bf16", "bf16", 8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: shapes spread over their logarithm, three quarters of the widths multiples of 8."""
    op = rng.choice(["linear", "linear", "grad", "adamw"])
    if op == "adamw":
        numel = _log(rng, 1_000, 250_000_000)
        return {"op": "adamw", "tensors": min(_log(rng, 1, 400), numel), "numel": numel,
                "param": rng.choice(["f32", "bf16", "f16"]), "grad": rng.choice(["f32", "bf16"]),
                "bits": rng.choice([8, 32]), "copy": rng.choice(["none", "none", "bf16"])}
    dtype = rng.choice(["f32", "bf16", "f16"])
    while True:
        if rng.random() < 0.2:  # tall data with few features
            m, n, k = _log(rng, 50_000, 1_000_000), _log(rng, 8, 64), _log(rng, 8, 64)
        else:
            m, n, k = _log(rng, 1, 16384), _log(rng, 16, 16384), _log(rng, 16, 16384)
        if rng.random() < 0.75:
            n, k = (n + 7) // 8 * 8, (k + 7) // 8 * 8
        if m * n * k <= 8192 * 4096 * 16384 // (8 if dtype == "f32" else 1):
            break
    case = {"op": op, "dtype": dtype, "m": m, "n": n, "k": k, "act": rng.choice(list(ACTS)), "w_t": rng.random() < 0.5}
    if op == "linear":
        case |= {"bias": rng.random() < 0.7, "residual": rng.random() < 0.4, "pre": rng.random() < 0.4}
    return case


def _sizes(case):
    """The tensors' sizes: like a network's, many small and a few that hold most, and of no round number."""
    t, total = case["tensors"], case["numel"]
    weights = [(1.0 if i % 3 == 0 else 0.3 if i % 3 == 1 else 0.002) * (1 + 0.1 * (i % 7)) for i in range(t)]
    unit = (total - t) / sum(weights)
    sizes = [1 + int(w * unit) for w in weights]
    sizes[0] += total - sum(sizes)
    return sizes


def _offsets(sizes):
    at, got = 0, []
    for s in sizes:
        got.append(at)
        at += (s + BLOCK - 1) // BLOCK * BLOCK
    return got, at


# ---------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    if case["op"] != "adamw":
        dt, m, n, k = TYPES[case["dtype"]], case["m"], case["n"], case["k"]
        s = {"X": normal(m, n, dtype=dt)}
        w = (k, n) if case["w_t"] else (n, k)
        s["W"] = normal(*w, scale=1 / math.sqrt(n), dtype=dt)
        if case["w_t"]:
            s["W"] = s["W"].t()
        if case["op"] == "grad":
            s["G"], s["Z"] = normal(m, k, dtype=dt), normal(m, k, dtype=dt)
        else:
            s["b"] = normal(k, scale=0.1, dtype=dt) if case["bias"] else None
            s["R"] = normal(m, k, dtype=dt) if case["residual"] else None
        return s

    # a network in mid-training: weights, gradients and moments of different sizes from block to block; the padding up
    # to whole blocks is zero
    sizes = _sizes(case)
    at, total = _offsets(sizes)
    blocks = total // BLOCK
    real = torch.zeros(total + 1, dtype=torch.int8, device="cuda")
    ends = torch.tensor([[a, a + n] for a, n in zip(at, sizes)], device="cuda")
    real.index_add_(0, ends[:, 0], torch.ones(len(sizes), dtype=torch.int8, device="cuda"))
    real.index_add_(0, ends[:, 1], torch.full((len(sizes),), -1, dtype=torch.int8, device="cuda"))
    real = real.cumsum(0, dtype=torch.int8)[:total].bool()
    size = torch.exp(normal(blocks, 1)) * 1e-3
    g = (normal(blocks, BLOCK) * size).view(-1).mul_(real).to(TYPES[case["grad"]])
    p = normal(total, scale=0.02).mul_(real).to(TYPES[case["param"]])
    s = {"p": p, "g": g, "sizes": sizes, "at": at, "steps": STEPS}
    if case["bits"] == 32:
        s["m"] = (normal(blocks, BLOCK) * size * 0.3).view(-1).mul_(real)
        s["v"] = (normal(blocks, BLOCK) * size).square_().add_(size.square() * 0.1).view(-1).mul_(real)
    else:
        s["m"] = torch.randint(-127, 128, (total,), generator=gen, device="cuda", dtype=torch.int8).mul_(real)
        s["v"] = torch.randint(1, 256, (total,), generator=gen, device="cuda", dtype=torch.uint8).mul_(real)
        s["ms"], s["vs"] = (size * (0.6 / 127**2)).view(-1), (size * (2.0 / 255**2)).view(-1)
    s["copy"] = torch.zeros_like(p, dtype=TYPES[case["copy"]]) if case["copy"] != "none" else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own and case["op"] == "adamw":
        import dense_linear_algebra_gb300 as fx

        def views(t):
            return [t[a:a + n] for a, n in zip(s["at"], s["sizes"])]

        s["grads"] = views(s["g"])
        opt = fx.AdamW(views(s["p"]), state_bits=case["bits"], copies=None if s["copy"] is None else views(s["copy"]),
                       lr=ADAM["lr"], betas=(ADAM["beta1"], ADAM["beta2"]), eps=ADAM["eps"],
                       weight_decay=ADAM["weight_decay"])
        state = {"exp_avg": s["m"], "exp_avg_sq": s["v"], "steps": STEPS}
        if case["bits"] == 8:
            state |= {"exp_avg_scale": s["ms"], "exp_avg_sq_scale": s["vs"]}
        opt.load_state_dict(state)
        s["opt"] = opt
        for key in ("m", "v", "ms", "vs"):
            s.pop(key, None)
    return s


# ---------------------------------------------------------------------------- the plain forms
C0, C1 = math.sqrt(2 / math.pi), 0.044715

ACTS = {
    "none": lambda z: z,
    "relu": lambda z: torch.where(z < 0, torch.zeros_like(z), z),
    "gelu": lambda z: 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5))),
    "gelu_tanh": lambda z: 0.5 * z * (1 + torch.tanh(C0 * (z + C1 * z * z * z))),
    "silu": lambda z: z / (1 + torch.exp(-z)),
    "sigmoid": lambda z: 1 / (1 + torch.exp(-z)),
}


def _slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), torch.ones_like(z))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(C0 * (z + C1 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C0 * (1 + 3 * C1 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s)) if act == "silu" else s * (1 - s)


def _plain_linear(s, case):
    dt = s["X"].dtype
    z = s["X"].float() @ s["W"].float()
    if s["b"] is not None:
        z = z + s["b"].float()
    out = ACTS[case["act"]](z)
    if s["R"] is not None:
        out = out + s["R"].float()
    return (out.to(dt), z.to(dt)) if case["pre"] else (out.to(dt),)


def _plain_grad(s, case):
    dt = s["X"].dtype
    d = s["G"].float() * _slope(case["act"], s["Z"].float())
    return (d @ s["W"].float().t()).to(dt), (s["X"].float().t() @ d).to(dt), d.sum(0).to(dt)


def _plain_adamw(s, case):
    h = ADAM
    s["steps"] += 1
    t = s["steps"]
    g = s["g"].float()
    if case["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        c = s["m"].view(-1, BLOCK).float()
        m = (c * c.abs() * s["ms"][:, None]).view(-1)
        c = s["v"].view(-1, BLOCK).float()
        r = c * c * s["vs"][:, None]
        v = (r * r).view(-1)
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1 - h["beta2"])
    r = torch.sqrt(v)
    step = m / (r * (1 / math.sqrt(1 - h["beta2"] ** t)) + h["eps"])
    p = s["p"].float() * (1 - h["lr"] * h["weight_decay"]) - step * (h["lr"] / (1 - h["beta1"] ** t))
    s["p"].copy_(p)
    out = {"p": s["p"]}
    if s["copy"] is not None:
        s["copy"].copy_(p)
        out["copy"] = s["copy"]
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return out | {"m": s["m"], "v": s["v"]}
    x, r = m.view(-1, BLOCK), r.view(-1, BLOCK)
    top = x.abs().amax(1)
    fine = ~(top < 1e-30)
    inv = torch.where(fine, 127.0**2 / top, torch.zeros_like(top))
    s["ms"] = torch.where(fine, top / 127.0**2, torch.zeros_like(top))
    c = torch.round(torch.sqrt(x.abs() * inv[:, None])).clamp(max=127).nan_to_num(0.0) * torch.sign(x).nan_to_num(0.0)
    s["m"].copy_(c.view(-1))
    top = r.amax(1)
    fine = ~(top < 1e-30)
    inv = torch.where(fine, 255.0**2 / top, torch.zeros_like(top))
    s["vs"] = torch.where(fine, top / 255.0**2, torch.zeros_like(top))
    d = torch.round(torch.sqrt(r * inv[:, None])).clamp(max=255).nan_to_num(0.0)
    d = torch.maximum(d, (r > 0).float())
    s["v"].copy_(d.view(-1))
    # the states as the values they stand for
    r = d * d * s["vs"][:, None]
    return out | {"m": (c * c.abs() * s["ms"][:, None]).view(-1), "v": (r * r).view(-1)}


# ---------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if not own:
        return {"linear": _plain_linear, "grad": _plain_grad, "adamw": _plain_adamw}[case["op"]](s, case)
    import dense_linear_algebra_gb300 as fx

    if case["op"] == "linear":
        out = fx.linear(s["X"], s["W"], s["b"], act=case["act"], residual=s["R"], pre=case["pre"])
        return out if case["pre"] else (out,)
    if case["op"] == "grad":
        return fx.linear_grad(s["G"], s["X"], s["W"], pre=s["Z"], act=case["act"])
    opt = s["opt"]
    opt.step(s["grads"])
    out = {"p": s["p"]}
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    m, v = opt.moments()
    return out | {"m": m, "v": v}


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] != "adamw":
        m, n, k, e = case["m"], case["n"], case["k"], size[case["dtype"]]
        if case["op"] == "grad":
            return {"bytes": e * (2 * m * k + 2 * m * n + 2 * n * k + k), "flops": 4 * m * n * k}
        wide = 1 + case["residual"] + case["pre"]
        return {"bytes": e * (m * n + n * k + case["bias"] * k + wide * m * k), "flops": 2 * m * n * k}
    n = case["numel"]
    b = 2 * size[case["param"]] + size[case["grad"]] + (0 if case["copy"] == "none" else 2)
    # 32 bits: both moments read and written; 8 bits: their codes too, and the values that they stand for written out
    b += 16 if case["bits"] == 32 else 2 * (2 + 8 / BLOCK) + 8
    return {"bytes": b * n, "flops": 15 * n}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f = torch.float64
    if case["op"] != "adamw":
        X, W = s["X"].to(f), s["W"].to(f)
        if case["op"] == "grad":
            z = s["Z"].to(f).requires_grad_(True)
            a = _exact_act(case["act"], z)
            if a is not z:
                (d,) = torch.autograd.grad(a, z, s["G"].to(f))
            else:
                d = s["G"].to(f)
            return torch.mm(d, W.t()), torch.mm(X.t(), d), torch.einsum("ik->k", d)
        z = torch.mm(X, W) if s["b"] is None else torch.addmm(s["b"].to(f), X, W)
        out = _exact_act(case["act"], z)
        if s["R"] is not None:
            out = s["R"].to(f) + out
        return (out, z) if case["pre"] else (out,)
    t, b1, b2 = STEPS + 1, ADAM["beta1"], ADAM["beta2"]
    g, p = s["g"].to(f), s["p"].to(f)
    if case["bits"] == 32:
        m, v = s["m"].to(f), s["v"].to(f)
    else:
        m = _held(s["m"], s["ms"].to(f))
        v = _held(s["v"], s["vs"].to(f)).square()
    m.lerp_(g, 1 - b1)
    v.lerp_(g.square_(), 1 - b2)
    del g
    root = v.sqrt()
    hat = root / math.sqrt(1 - b2**t)
    p = p - ADAM["lr"] * (m / (1 - b1**t) / hat.add_(ADAM["eps"]) + ADAM["weight_decay"] * p)
    out = {"p": p}
    if s["copy"] is not None:
        out["copy"] = p
    if case["bits"] == 32:
        return out | {"m": m, "v": v}
    return out | {"m": _requantised(m, 127), "v": _requantised(root, 255).square_()}


def _exact_act(act, z):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return torch.sigmoid(z) if act == "sigmoid" else z


def _held(codes, scale):
    c = codes.view(scale.numel(), -1).to(torch.float64)
    return (c.sign() * c.pow(2) * scale.unsqueeze(1)).flatten()


def _requantised(x, levels):
    x = x.view(-1, BLOCK)
    top = x.abs().max(dim=1, keepdim=True).values
    unit = (x.abs() / top.clamp(min=1e-300)).sqrt_()
    c = torch.round(unit * levels)
    if levels == 255:
        c = torch.where((x > 0) & (c < 1), torch.ones_like(c), c)
    return (x.sign() * (c / levels).square_() * top).flatten()
