"""What training a classifier takes besides its layers, as measured cases: layer norm, the embedding lookup, and softmax
cross entropy on a linear layer's outputs, each with its gradient.

``norm``        OUT = (X - mean) * rstd * w + b over each row, mean and rstd kept
``norm_grad``   dX (plus the gradient that arrives on the residual path), dw, db
``embed``       OUT_i = scale * E[ids_i]; a row of zeros for an id outside the table
``embed_grad``  dE_v = scale * the sum of G's rows with id v, zeros where there is none
``loss``        z = X W + b; loss_i = lse_i - z_i,label, lse_i = log sum_j exp z_ij, without the logits being kept
``loss_grad``   D_ij = g_i (exp(z_ij - lse_i) - [j = label_i]); dX = D W^T, dW = X^T D, db = the column sums of D

X is (m, n), W (n, k); ``w_t`` stores W's transpose row by row (W is then the transposed view). A label outside 0 .. k - 1
leaves its row out.
"""
import functools
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
SPREAD = 3.0  # standard deviation of the logits


# ---------------------------------------------------------------------------- cases
def _norm(name, dtype, m, n, affine=True):
    return {"name": name, "op": "norm", "dtype": dtype, "m": m, "n": n, "affine": affine}


def _norm_grad(name, dtype, m, n, residual=False):
    return {"name": name, "op": "norm_grad", "dtype": dtype, "m": m, "n": n, "residual": residual}


def _embed(name, dtype, m, n, k, scale=1.0):
    return {"name": name, "op": "embed", "dtype": dtype, "m": m, "n": n, "k": k, "scale": scale}


def _embed_grad(name, dtype, m, n, k, scale=1.0):
    return {"name": name, "op": "embed_grad", "dtype": dtype, "m": m, "n": n, "k": k, "scale": scale}


def _loss(name, dtype, m, n, k, bias=False, w_t=True):
    return {"name": name, "op": "loss", "dtype": dtype, "m": m, "n": n, "k": k, "bias": bias, "w_t": w_t}


def _loss_grad(name, dtype, m, n, k, bias=False, w_t=True, weighted=False, input_grad=True):
    return {"name": name, "op": "loss_grad", "dtype": dtype, "m": m, "n": n, "k": k, "bias": bias, "w_t": w_t,
            "weighted": weighted, "input_grad": input_grad}


def listed():
    return [
        # serving one row: latency counts
        _norm("norm_token_bf16", "bf16", 1, 4096),
        # the forward pass of training, statistics kept for the gradient
        _norm("norm_train_bf16", "bf16", 16384, 4096),
        # its gradient, with the residual path's added
        _norm_grad("norm_grad_bf16", "bf16", 16384, 4096, residual=True),
        # the gradient over the library's tall data matrix (32 features)
        _norm_grad("norm_grad_tall_f32", "f32", 1_000_000, 32),
        # a prompt's rows, of no round number: latency counts
        _embed("embed_prompt_f16", "f16", 777, 2056, 32000, scale=math.sqrt(2056)),
        # a training batch over a large table
        _embed("embed_train_bf16", "bf16", 65536, 4096, 131072, scale=64.0),
        # its gradient: frequent ids have thousands of rows, most of the table none
        _embed_grad("embed_grad_bf16", "bf16", 65536, 2048, 131072, scale=64.0),
        # a small ragged gradient: odd row pitch
        _embed_grad("embed_grad_ragged_f32", "f32", 5001, 301, 20011),
        # scoring one row against a vocabulary: the weights are read once
        _loss("loss_row_bf16", "bf16", 1, 4096, 32000, bias=True),
        # the loss of a training batch over a large vocabulary
        _loss("loss_train_bf16", "bf16", 8192, 2048, 65536),
        # its gradient, each row with its own weight
        _loss_grad("loss_grad_bf16", "bf16", 8192, 2048, 65536, weighted=True),
        # softmax regression on the tall data matrix: ten classes, no gradient for the data
        _loss_grad("loss_grad_tall_f32", "f32", 1_000_000, 32, 10, bias=True, w_t=False, input_grad=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over their logarithm, three quarters of the widths multiples of 8."""
    op = rng.choice(["norm", "norm_grad", "embed", "embed_grad", "loss", "loss", "loss_grad", "loss_grad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    even = rng.random() < 0.75

    def width(lo, hi):
        n = _log(rng, lo, hi)
        return (n + 7) // 8 * 8 if even else n

    if op in ("norm", "norm_grad"):
        top = 16384 * 4096 // (2 if dtype == "f32" else 1)
        while True:
            m, n = _log(rng, 1, 1_000_000), width(8, 16384)
            if m * n <= top:
                break
        case = {"op": op, "dtype": dtype, "m": m, "n": n}
        return case | ({"affine": rng.random() < 0.8} if op == "norm" else {"residual": rng.random() < 0.5})
    if op in ("embed", "embed_grad"):
        while True:
            m, n, k = _log(rng, 1, 262_144), width(8, 8192), _log(rng, 16, 262_144)
            if (m + k) * n * SIZE[dtype] <= 65536 * 4096 * 2:
                break
        return {"op": op, "dtype": dtype, "m": m, "n": n, "k": k, "scale": rng.choice([1.0, math.sqrt(n)])}
    while True:
        if rng.random() < 0.25:  # tall data with few features and classes
            m, n, k = _log(rng, 50_000, 1_000_000), width(8, 64), _log(rng, 2, 64)
        else:
            m, n, k = _log(rng, 1, 16384), width(16, 8192), _log(rng, 16, 131072)
        if m * n * k <= 8192 * 2048 * 65536 // (8 if dtype == "f32" else 1) and n * k <= 2**29:
            break
    case = {"op": op, "dtype": dtype, "m": m, "n": n, "k": k, "bias": rng.random() < 0.5, "w_t": rng.random() < 0.7}
    if op == "loss_grad":
        case |= {"weighted": rng.random() < 0.5, "input_grad": rng.random() < 0.8}
    return case


# ---------------------------------------------------------------------------- inputs
def _ids(m, k, gen):
    """Ids as texts have them: the frequency of id v falls as 1 / (v + 1); one in 32 stands for padding (-1)."""
    u = torch.rand(m, generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(k + 1)).long().sub_(1).clamp_(0, k - 1)
    pad = torch.rand(m, generator=gen, device="cuda") < 1 / 32
    return torch.where(pad, torch.full_like(ids, -1), ids)


@functools.lru_cache(maxsize=None)
def _distinct(m, k):
    """The expected number of different ids among m."""
    total, norm = 0.0, math.log(k + 1)
    for v in range(k):
        total += -math.expm1(m * math.log1p(-(31 / 32) * math.log1p(1 / (v + 1)) / norm))
    return total


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    op, dt, m, n = case["op"], TYPES[case["dtype"]], case["m"], case["n"]
    if op in ("norm", "norm_grad"):
        # rows of different sizes around different means, as a residual stream's
        rows = torch.exp(normal(m, 1, scale=0.5))
        s = {"X": (normal(m, n) * rows + normal(m, 1, scale=0.3)).to(dt)}
        s["w"] = (1 + normal(n, scale=0.1)).to(dt) if case.get("affine", True) else None
        s["b"] = normal(n, scale=0.1, dtype=dt) if case.get("affine", True) else None
        if op == "norm_grad":
            x = s["X"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
            s["G"] = normal(m, n, dtype=dt)
            s["R"] = normal(m, n, dtype=dt) if case["residual"] else None
        return s
    k = case["k"]
    if op in ("embed", "embed_grad"):
        s = {"ids": _ids(m, k, gen)}
        if op == "embed":
            s["E"] = normal(k, n, scale=0.02, dtype=dt)
        else:
            s["G"] = normal(m, n, scale=1e-2, dtype=dt)
        return s
    s = {"X": normal(m, n, dtype=dt), "labels": _ids(m, k, gen)}
    s["W"] = normal(*((k, n) if case["w_t"] else (n, k)), scale=SPREAD / math.sqrt(n), dtype=dt)
    if case["w_t"]:
        s["W"] = s["W"].t()
    s["b"] = normal(k, scale=0.5, dtype=dt) if case["bias"] else None
    if op == "loss_grad":
        z = s["X"].float() @ s["W"].float()
        s["lse"] = torch.logsumexp(z if s["b"] is None else z.add_(s["b"].float()), 1)
        del z
        s["g"] = 1.0 / m
        if case["weighted"]:
            s["g"] = torch.rand(m, generator=gen, device="cuda").add_(0.5).div_(m)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------- the plain forms
def _plain_norm(s, case):
    x = s["X"].float()
    mean = x.mean(1)
    x = x - mean[:, None]
    rstd = torch.rsqrt((x * x).mean(1) + EPS)
    x = x * rstd[:, None]
    if s["w"] is not None:
        x = x * s["w"].float() + s["b"].float()
    return x.to(s["X"].dtype), mean, rstd


def _plain_norm_grad(s, case):
    dt = s["X"].dtype
    g = s["G"].float()
    x = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dw, db = (g * x).sum(0), g.sum(0)
    h = g * s["w"].float()
    dx = (h - h.mean(1, keepdim=True) - x * (h * x).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["R"] is not None:
        dx = dx + s["R"].float()
    return dx.to(dt), dw.to(dt), db.to(dt)


def _plain_embed(s, case):
    ids, E = s["ids"], s["E"]
    inside = (ids >= 0) & (ids < E.shape[0])
    rows = E[torch.where(inside, ids, torch.zeros_like(ids))].float() * case["scale"]
    return (torch.where(inside[:, None], rows, torch.zeros_like(rows)).to(E.dtype),)


def _plain_embed_grad(s, case):
    ids, G, k = s["ids"], s["G"], case["k"]
    # the rows of no id go to one more row, which is left out
    at = torch.where((ids >= 0) & (ids < k), ids, torch.full_like(ids, k))
    dE = torch.zeros(k + 1, G.shape[1], device="cuda", dtype=torch.float32).index_add_(0, at, G.float())
    return ((dE[:k] * case["scale"]).to(G.dtype),)


def _logits(s):
    z = s["X"].float() @ s["W"].float()
    return z if s["b"] is None else z + s["b"].float()


def _plain_loss(s, case):
    labels, k = s["labels"], case["k"]
    z = _logits(s)
    top = z.max(1).values
    lse = torch.log(torch.exp(z - top[:, None]).sum(1)) + top
    inside = (labels >= 0) & (labels < k)
    at = z.gather(1, torch.where(inside, labels, torch.zeros_like(labels))[:, None])[:, 0]
    return torch.where(inside, lse - at, torch.zeros_like(lse)), lse


def _plain_loss_grad(s, case):
    dt, labels, k = s["X"].dtype, s["labels"], case["k"]
    inside = (labels >= 0) & (labels < k)
    g = torch.where(inside, torch.zeros_like(s["lse"]) + s["g"], torch.zeros_like(s["lse"]))
    d = torch.exp(_logits(s) - s["lse"][:, None]) * g[:, None]
    rows = torch.arange(case["m"], device="cuda")
    d[rows, torch.where(inside, labels, torch.zeros_like(labels))] -= g
    dx = (d @ s["W"].float().t()).to(dt) if case["input_grad"] else None
    dw = (s["X"].float().t() @ d).to(dt)
    db = d.sum(0).to(dt) if case["bias"] else None
    return [t for t in (dx, dw, db) if t is not None]


# ---------------------------------------------------------------------------- one pass
PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "embed": _plain_embed, "embed_grad": _plain_embed_grad,
         "loss": _plain_loss, "loss_grad": _plain_loss_grad}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s, case)
    import dense_linear_algebra_gb300 as fx

    if op == "norm":
        return fx.layer_norm(s["X"], s["w"], s["b"], eps=EPS, stats=True)
    if op == "norm_grad":
        return fx.layer_norm_grad(s["G"], s["X"], s["w"], s["mean"], s["rstd"], residual=s["R"])
    if op == "embed":
        return (fx.embedding(s["ids"], s["E"], scale=case["scale"]),)
    if op == "embed_grad":
        return (fx.embedding_grad(s["G"], s["ids"], case["k"], scale=case["scale"]),)
    if op == "loss":
        return fx.cross_entropy(s["X"], s["W"], s["labels"], s["b"])
    got = fx.cross_entropy_grad(s["X"], s["W"], s["labels"], s["lse"], s["b"], g=s["g"],
                                need=(case["input_grad"], True, case["bias"]))
    return [t for t in got if t is not None]


def work(case):
    op, m, n, e = case["op"], case["m"], case["n"], SIZE[case["dtype"]]
    if op == "norm":
        return {"bytes": e * (2 * m * n + (2 * n if case["affine"] else 0)) + 8 * m, "flops": 8 * m * n}
    if op == "norm_grad":
        return {"bytes": e * ((3 + case["residual"]) * m * n + 3 * n) + 8 * m, "flops": 14 * m * n}
    k = case["k"]
    if op == "embed":
        return {"bytes": int(e * n * (m + _distinct(m, k))) + 8 * m, "flops": m * n}
    if op == "embed_grad":
        return {"bytes": e * n * (m * 31 // 32 + k) + 8 * m, "flops": m * n}
    b = k if case["bias"] else 0
    if op == "loss":
        return {"bytes": e * (m * n + n * k + b) + 16 * m, "flops": 2 * m * n * k + 4 * m * k}
    products = 2 + case["input_grad"]
    return {"bytes": e * (m * n * (1 + case["input_grad"]) + 2 * n * k + 2 * b) + (16 if case["weighted"] else 12) * m,
            "flops": 2 * products * m * n * k + 4 * m * k}


# ---------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f = torch.float64
    op = case["op"]
    if op in ("norm", "norm_grad"):
        x = s["X"].to(f)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        w, b = (None if s[c] is None else s[c].to(f) for c in ("w", "b"))
        if op == "norm":
            out = torch.nn.functional.layer_norm(x, (case["n"],), w, b, EPS)
            return out, mean, (var + EPS).pow(-0.5)
        G = s["G"].to(f)
        # with the statistics as they are given, rounded to 32 bits
        u = torch.addcmul(-s["mean"].to(f)[:, None] * s["rstd"].to(f)[:, None], x, s["rstd"].to(f)[:, None])
        dw, db = torch.einsum("ij,ij->j", G, u), torch.einsum("ij->j", G)
        h = G * w
        c = torch.einsum("ij,ij->i", h, u) / case["n"]
        dx = torch.addcmul(h - torch.einsum("ij->i", h)[:, None] / case["n"], u, c[:, None], value=-1)
        dx *= s["rstd"].to(f)[:, None]
        return dx if s["R"] is None else dx + s["R"].to(f), dw, db
    if op == "embed":
        E = torch.cat([s["E"].to(f) * case["scale"], torch.zeros(1, case["n"], device="cuda", dtype=f)])
        return (E.index_select(0, s["ids"] % (case["k"] + 1)),)
    if op == "embed_grad":
        keep = s["ids"] >= 0
        dE = torch.zeros(case["k"], case["n"], device="cuda", dtype=f)
        return (dE.index_put_((s["ids"][keep],), s["G"][keep].to(f) * case["scale"], accumulate=True),)
    X, W, labels = s["X"].to(f), s["W"].to(f), s["labels"]
    z = torch.mm(X, W) if s["b"] is None else torch.addmm(s["b"].to(f), X, W)
    if op == "loss":
        loss = torch.nn.functional.cross_entropy(z, labels, reduction="none", ignore_index=-1)
        return loss, torch.logsumexp(z, 1)
    d = z.sub_(s["lse"].to(f)[:, None]).exp_()
    d.scatter_add_(1, labels.clamp(min=0)[:, None], torch.full((case["m"], 1), -1.0, device="cuda", dtype=f))
    g = s["g"].to(f) if case["weighted"] else torch.full((case["m"],), s["g"], device="cuda", dtype=f)
    d *= (g * (labels >= 0))[:, None]
    out = [torch.mm(d, W.t())] if case["input_grad"] else []
    out.append(torch.mm(X.t(), d))
    return out + ([torch.einsum("ik->k", d)] if case["bias"] else [])
