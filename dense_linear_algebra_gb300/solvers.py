"""Whole ML algorithms whose inner loop is the fused pattern.

"On optimizing machine learning workloads via kernel fusion" (abstract) closes by
applying the fused kernel inside an entire ML algorithm. The two here are the
textbook consumers of ``alpha * X^T (v * (X p)) + beta * z``:

* ``ridge_cg``: least squares with an L2 penalty, ``min ||X w - b||^2 + lam ||w||^2``,
  solved by conjugate gradients on ``(X^T X + lam I) w = X^T b``. Every operator
  application ``X^T (X p) + lam p`` is ONE fused call (v = 1, z = p, beta = lam).
* ``ridge_cg_multi``: the same for k targets at once (block CG); every iteration applies
  the operator to all k search directions in ONE multi-vector call, one pass over X.
* ``logistic_newton_cg``: L2-regularised logistic regression by Newton's method;
  each Newton step solves ``(X^T D X + lam I) d = -g`` by conjugate gradients, where
  every Hessian-vector product ``X^T (D * (X p)) + lam p`` is ONE fused call with
  v = D = mu (1 - mu).

``mlp_adamw`` trains a network of more than one layer on the rows of X with the layer operators
(``layers.linear``, ``layers.linear_grad``, ``layers.AdamW``).

For the linear models X may be dense (a 2-D CUDA tensor) or CSR (a tuple ``(row_ptr, col_idx, vals, n)``).
The few operations outside the pattern (``X^T b`` once, and per Newton step the
margins ``X w`` and the gradient ``X^T (mu - b)``) are plain matrix-vector products
done by torch (for CSR X on torch CSR copies built once per solve); vector updates on
n-vectors are torch operations as well.
"""
from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import _lib


def _is_csr(X) -> bool:
    return isinstance(X, tuple)


def _shape(X):
    if _is_csr(X):
        row_ptr, _, vals, n = X
        return row_ptr.shape[0] - 1, n, vals.dtype, vals.device
    return X.shape[0], X.shape[1], X.dtype, X.device


def fused(X, p, v, alpha: float, beta: float, z, out=None):
    """alpha * X^T (v * (X p)) + beta * z, dense or CSR."""
    if _is_csr(X):
        row_ptr, col_idx, vals, n = X
        return _lib.csr(row_ptr, col_idx, vals, p, n, v, alpha, beta, z, out=out)
    return _lib.dense(X, p, v, alpha, beta, z, out=out)


def _torch_csr(X):
    row_ptr, col_idx, vals, n = X
    return torch.sparse_csr_tensor(row_ptr, col_idx.to(torch.int64), vals, size=(row_ptr.shape[0] - 1, n))


class TorchOps:
    """X w and X^T r outside the pattern (torch). For CSR X the torch CSR tensor and its
    transposed copy are built once, when the operator is made, not per product."""

    def __init__(self, X):
        if _is_csr(X):
            self.A = _torch_csr(X)
            self.AT = self.A.t().to_sparse_csr()
        else:
            self.A, self.AT = X, X.t()

    def matvec(self, w):
        return torch.mv(self.A, w)

    def rmatvec(self, r):
        return torch.mv(self.AT, r)


def matvec(X, w):
    """X w (outside the pattern; torch)."""
    return TorchOps(X).matvec(w) if _is_csr(X) else torch.mv(X, w)


def rmatvec(X, r):
    """X^T r (outside the pattern; torch)."""
    return TorchOps(X).rmatvec(r) if _is_csr(X) else torch.mv(X.t(), r)


@dataclass
class CGInfo:
    iterations: int = 0
    residual: float = 0.0
    converged: bool = False
    history: list = field(default_factory=list)


def cg(apply, rhs, tol: float = 1e-6, max_iter: int = 100, x0=None, check_every: int = 1):
    """Conjugate gradients for the symmetric positive definite operator `apply` (one fused call each).

    The residual is read back to the host (a synchronisation) every `check_every`
    iterations and at the last one; between checks the iterations queue on the
    stream back to back.
    """
    x = torch.zeros_like(rhs) if x0 is None else x0.clone()
    r = rhs - apply(x) if x0 is not None else rhs.clone()
    p = r.clone()
    rs = torch.dot(r, r)
    bnorm = float(torch.linalg.vector_norm(rhs))
    info = CGInfo()
    if bnorm == 0.0:
        info.converged = True
        return x, info
    for k in range(max_iter):
        q = apply(p)
        pq = torch.dot(p, q)
        # once the residual is exactly zero, stop moving (no 0/0 on the device)
        a = torch.where(pq > 0, rs / torch.where(pq > 0, pq, torch.ones_like(pq)), torch.zeros_like(pq))
        x.add_(a * p)
        r.sub_(a * q)
        rs_new = torch.dot(r, r)
        info.iterations = k + 1
        if (k + 1) % check_every == 0 or k + 1 == max_iter:
            res = float(torch.sqrt(rs_new)) / bnorm
            info.residual = res
            info.history.append(res)
            if res <= tol:
                info.converged = True
                break
        p.mul_(torch.where(rs > 0, rs_new / torch.where(rs > 0, rs, torch.ones_like(rs)), torch.zeros_like(rs))).add_(r)
        rs = rs_new
    return x, info


def ridge_cg(X, b, lam: float, tol: float = 1e-6, max_iter: int = 200):
    """Ridge regression by CG: each iteration applies X^T (X p) + lam p in one fused call."""
    m, n, dt, dev = _shape(X)
    rhs = rmatvec(X, b)
    return cg(lambda p: fused(X, p, None, 1.0, lam, p), rhs, tol=tol, max_iter=max_iter)


def fused_multi(X, P, V, alpha: float, beta: float, Z, out=None):
    """alpha * X^T (V * (X P)) + beta * Z for k right-hand sides (dense X): one pass over X."""
    return _lib.dense_multi(X, P, V, alpha, beta, Z, out=out)


def cg_block(apply, rhs, tol: float = 1e-6, max_iter: int = 100, check_every: int = 1):
    """k independent conjugate-gradient solves in lockstep, one per column of `rhs` (n, k).

    `apply` maps an (n, k) block to the operator applied to each column, so one call
    serves all k solves. Each column has its own step sizes; a column whose residual
    reaches zero stops moving. Converged when every column's relative residual is <= tol.
    """
    x = torch.zeros_like(rhs)
    r = rhs.clone()
    p = r.clone()
    rs = (r * r).sum(dim=0)
    bnorm = torch.linalg.vector_norm(rhs, dim=0)
    info = CGInfo()
    safe_b = torch.where(bnorm > 0, bnorm, torch.ones_like(bnorm))
    if float(bnorm.max()) == 0.0:
        info.converged = True
        return x, info
    for k in range(max_iter):
        q = apply(p)
        pq = (p * q).sum(dim=0)
        a = torch.where(pq > 0, rs / torch.where(pq > 0, pq, torch.ones_like(pq)), torch.zeros_like(pq))
        x.add_(a * p)
        r.sub_(a * q)
        rs_new = (r * r).sum(dim=0)
        info.iterations = k + 1
        if (k + 1) % check_every == 0 or k + 1 == max_iter:
            res = float((torch.sqrt(rs_new) / safe_b).max())
            info.residual = res
            info.history.append(res)
            if res <= tol:
                info.converged = True
                break
        b = torch.where(rs > 0, rs_new / torch.where(rs > 0, rs, torch.ones_like(rs)), torch.zeros_like(rs))
        p.mul_(b).add_(r)
        rs = rs_new
    return x, info


def ridge_cg_multi(X, B, lam: float, tol: float = 1e-6, max_iter: int = 200):
    """Ridge regression for k targets at once (B is (m, k)): block CG in which every
    iteration applies X^T (X P) + lam P to all k directions in one multi-vector call."""
    rhs = torch.mm(X.t(), B).contiguous()
    return cg_block(lambda P: fused_multi(X, P.contiguous(), None, 1.0, lam, P.contiguous()), rhs, tol=tol,
                    max_iter=max_iter)


@dataclass
class NewtonInfo:
    newton_steps: int = 0
    cg_iterations: int = 0
    grad_norm: float = 0.0
    converged: bool = False


def logistic_newton_cg(X, labels, lam: float, newton_steps: int = 20, tol: float = 1e-6, cg_tol: float = 1e-4,
                       cg_max: int = 100):
    """L2 logistic regression (labels in {0, 1}) by Newton-CG.

    Minimises sum_i log(1 + exp(x_i . w)) - b_i (x_i . w) + lam / 2 ||w||^2. Each Hessian-vector
    product X^T (D * (X p)) + lam p, D = mu (1 - mu), is one fused call with v = D.
    """
    m, n, dt, dev = _shape(X)
    ops = TorchOps(X)  # the margins' and the gradient's products; CSR copies built once per solve
    w = torch.zeros(n, dtype=dt, device=dev)
    info = NewtonInfo()
    g0 = None
    for step in range(newton_steps):
        mu = torch.sigmoid(ops.matvec(w))
        g = ops.rmatvec(mu - labels) + lam * w
        gn = float(torch.linalg.vector_norm(g))
        if g0 is None:
            g0 = max(gn, 1e-300)
        info.grad_norm = gn
        if gn <= tol * g0:
            info.converged = True
            break
        D = (mu * (1.0 - mu)).contiguous()
        d, ci = cg(lambda p: fused(X, p, D, 1.0, lam, p), -g, tol=cg_tol, max_iter=cg_max)
        w.add_(d)
        info.newton_steps = step + 1
        info.cg_iterations += ci.iterations
    return w, info


@dataclass
class MLPInfo:
    steps: int = 0
    losses: list = field(default_factory=list)


class MLP:
    """A residual network on the rows of X: h = act(X W0 + b0), then h = h + act(h Wi + bi) for each hidden layer, and
    the result h Wn + bn. Every layer is one fused call, forward and backward (``layers.linear``, ``layers.linear_grad``).

    ``weights`` and ``biases`` are float32; ``dtype`` (bfloat16, float16 or float32) is what the layers compute in: the
    working copies of 16-bit types are refreshed by the optimiser.
    """

    def __init__(self, features: int, hidden: int, outputs: int, layers: int = 1, act: str = "gelu",
                 dtype=torch.float32, device="cuda", seed: int = 0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        sizes = [features] + [hidden] * (layers + 1) + [outputs]
        self.act, self.dtype = act, dtype
        self.weights = [torch.randn(a, b, generator=gen, device=device) / a ** 0.5 for a, b in zip(sizes, sizes[1:])]
        self.biases = [torch.zeros(b, device=device) for b in sizes[1:]]
        self.copies = None
        if dtype != torch.float32:
            self.copies = [p.to(dtype) for p in self.parameters()]

    def parameters(self):
        return self.weights + self.biases

    def _working(self):
        if self.copies is None:
            return self.weights, self.biases
        return self.copies[:len(self.weights)], self.copies[len(self.weights):]

    def forward(self, X, keep: bool = False):
        """The result for the rows of X; with ``keep`` also what ``backward`` needs."""
        from . import layers

        W, b = self._working()
        last, saved, h = len(W) - 1, [], X
        for i in range(last + 1):
            residual = h if 0 < i < last else None
            act = self.act if i < last else None
            if keep and act:
                out, pre = layers.linear(h, W[i], b[i], act=act, residual=residual, pre=True)
            else:
                out, pre = layers.linear(h, W[i], b[i], act=act, residual=residual), None
            saved.append((h, pre))
            h = out
        return (h, saved) if keep else h

    def backward(self, G, saved):
        """The gradients of ``parameters()`` from the gradient at the result."""
        from . import layers

        W, _ = self._working()
        last = len(W) - 1
        dW, db = [None] * (last + 1), [None] * (last + 1)
        for i in range(last, -1, -1):
            h, pre = saved[i]
            dh, dW[i], db[i] = layers.linear_grad(G, h, W[i], pre=pre, act=self.act if i < last else None,
                                                  need=(i > 0, True, True))
            # the residual passes the gradient on as it is
            G = dh.add_(G) if 0 < i < last else dh
        return dW + db


def _mean_square_gradients(net, err, saved):
    """The gradients of mean(err^2) in the network's parameters."""
    rate = 2.0 / err.numel()
    if net.dtype != torch.float16:
        return net.backward((err * rate).to(net.dtype), saved)
    # float16 has nothing below 6e-8, where the gradient of a mean over millions of entries lies: it goes through the layers
    # relative to the largest error, held down so that a sum over the rows stays below 4,096 times an entry of the layer's
    # input, and gets its size in float32
    top, part = err.abs().amax().clamp_min(1e-30), min(1.0, 4096 / err.shape[0])
    grads = net.backward((err * (part / top)).to(net.dtype), saved)
    return [g.float().mul_(top * (rate / part)) for g in grads]


def mlp_adamw(X, B, hidden: int, layers: int = 1, act: str = "gelu", steps: int = 100, batch: int = 0, lr: float = 1e-3,
              weight_decay: float = 0.0, state_bits: int = 32, dtype=torch.float32, seed: int = 0):
    """Least squares by a residual network (``MLP``) trained with AdamW: min mean((net(X) - B)^2).

    X (m, n) and B (m, outputs) are float32 or ``dtype``; each step takes ``batch`` rows in turn (0: all of them), the
    last step of a pass over X what is left of its rows. Returns the network and the losses of the steps (left on the
    GPU until read).
    """
    from .layers import AdamW

    X, B = X.to(dtype), B.to(dtype)
    net = MLP(X.shape[1], hidden, B.shape[1], layers, act, dtype, X.device, seed)
    opt = AdamW(net.parameters(), lr=lr, weight_decay=weight_decay, state_bits=state_bits, copies=net.copies)
    info, m = MLPInfo(), X.shape[0]
    batch = m if batch <= 0 else min(batch, m)
    at = 0
    for _ in range(steps):
        out, saved = net.forward(X[at:at + batch], keep=True)
        err = out.float() - B[at:at + batch].float()
        info.losses.append(err.square().mean())
        opt.step(_mean_square_gradients(net, err, saved))
        info.steps += 1
        at = at + batch if at + batch < m else 0
    return net, info


class Classifier:
    """A residual network with layer norms and a softmax over classes, on rows of features or of ids.

    With ``tokens`` = 0 the rows of X (m, features) go in as they are. Else they are ids (m, slots), each looked up in a
    (tokens, width) table: a row is its slots' rows side by side (features = slots * width; an id outside the table is
    padding and gives zeros). Then h = act(x W0 + b0), h = h + act(norm(h) Wi + bi) for each hidden layer, and the
    classes' logits norm(h) P^T + c, which only ``logits`` writes out: the loss and its gradient do without
    (``training.cross_entropy``). ``params`` are float32; ``dtype`` is what the layers compute in, as for ``MLP``.
    """

    def __init__(self, features: int, hidden: int, classes: int, layers: int = 1, tokens: int = 0, width: int = 0, act: str = "gelu",
                 dtype=torch.float32, device="cuda", seed: int = 0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def normal(a, b, scale):
            return torch.randn(a, b, generator=gen, device=device) * scale

        self.act, self.dtype, self.layers, self.tokens, self.width = act, dtype, layers, tokens, width
        self.params = {}
        if tokens:
            self.params["table"] = normal(tokens, width, width**-0.5)
        for i in range(layers + 1):
            n = hidden if i else features
            self.params[f"W{i}"], self.params[f"b{i}"] = normal(n, hidden, n**-0.5), torch.zeros(hidden, device=device)
            # the norm before layer i + 1, the last one before the classes
            self.params[f"g{i}"], self.params[f"s{i}"] = torch.ones(hidden, device=device), torch.zeros(hidden, device=device)
        self.params["P"], self.params["c"] = normal(classes, hidden, hidden**-0.5), torch.zeros(classes, device=device)
        self.copies = None if dtype == torch.float32 else {name: p.to(dtype) for name, p in self.params.items()}

    def parameters(self):
        return list(self.params.values())

    def working(self):
        """The parameters that the layers compute with."""
        return self.params if self.copies is None else self.copies

    def forward(self, X, keep: bool = False):
        """norm(h) of the rows of X before the classes; with ``keep`` also what ``backward`` needs."""
        from . import layers, training

        p, saved = self.working(), []
        if self.tokens:
            rows = training.embedding(X.reshape(-1), p["table"], scale=self.width**0.5)
            x = rows.view(X.shape[0], X.shape[1] * self.width)
        else:
            x = X
        v, h = x, None
        for i in range(self.layers + 1):
            entry, pre = h, None
            out = layers.linear(v, p[f"W{i}"], p[f"b{i}"], act=self.act, residual=h, pre=keep)
            h, pre = out if keep else (out, None)
            saved.append((entry, v, pre))
            v, mean, rstd = training.layer_norm(h, p[f"g{i}"], p[f"s{i}"], stats=True)
            saved[-1] += (h, mean, rstd)
        return (v, saved) if keep else v

    def logits(self, X):
        """The logits of the rows of X."""
        from . import layers

        p = self.working()
        return layers.linear(self.forward(X), p["P"].t(), p["c"])

    def loss(self, X, labels):
        """The rows' losses and what ``backward`` needs. A label outside the classes leaves its row out."""
        from . import training

        p = self.working()
        v, saved = self.forward(X, keep=True)
        loss, lse = training.cross_entropy(v, p["P"].t(), labels, p["c"])
        return loss, (X, labels, v, lse, saved)

    def backward(self, g, kept):
        """The gradients of ``parameters()`` from the gradient ``g`` at the losses (a number, or a float32 tensor of the rows)."""
        from . import layers, training

        p, grads = self.working(), {}
        X, labels, v, lse, saved = kept
        dv, dP, grads["c"] = training.cross_entropy_grad(v, p["P"].t(), labels, lse, p["c"], g=g)
        grads["P"], dh = dP.t(), None
        for i in range(self.layers, -1, -1):
            _, v, pre, h, mean, rstd = saved[i]
            # what reaches h through the norm, and past it
            dh, grads[f"g{i}"], grads[f"s{i}"] = training.layer_norm_grad(dv, h, p[f"g{i}"], mean, rstd, residual=dh)
            dv, grads[f"W{i}"], grads[f"b{i}"] = layers.linear_grad(dh, v, p[f"W{i}"], pre=pre, act=self.act,
                                                                    need=(i > 0 or self.tokens > 0, True, True))
        if self.tokens:
            grads["table"] = training.embedding_grad(dv.view(-1, self.width), X.reshape(-1), self.tokens, scale=self.width**0.5)
        return [grads[name] for name in self.params]


def _mean_loss_gradients(net, labels, kept):
    """The gradients of the mean loss of the rows that have a label, in the network's parameters."""
    classes = net.params["P"].shape[0]
    rate = 1.0 / ((labels >= 0) & (labels < classes)).sum().clamp_min(1).float()
    if net.dtype != torch.float16:
        return net.backward(rate.expand(labels.shape[0]).contiguous(), kept)
    # float16 has nothing below 6e-8, where the gradient of a mean over millions of rows lies: it goes through the layers at a
    # size that a sum over the rows leaves below 4,096 times an entry of the layer's input, and gets its own in float32
    part = min(1.0, 4096 / max(labels.shape[0], 1))
    return [g.float().mul_(rate / part) for g in net.backward(part, kept)]


def classify_adamw(X, labels, classes: int, hidden: int, layers: int = 1, tokens: int = 0, width: int = 0, act: str = "gelu",
                   steps: int = 100, batch: int = 0, lr: float = 1e-3, weight_decay: float = 0.0, state_bits: int = 32,
                   dtype=torch.float32, seed: int = 0):
    """Classification by a residual network (``Classifier``) trained with AdamW: min mean cross entropy of softmax(net(X)).

    X is (m, n) features, or with ``tokens`` > 0 (m, slots) ids, int32 or int64, into a table of ``tokens`` rows of ``width``.
    ``labels`` (m,) are int32 or int64; rows with a label outside 0 .. classes - 1 are left out. Each step takes ``batch``
    rows in turn (0: all of them), the last step of a pass over X what is left of its rows. Returns the network and the
    steps' mean losses (left on the GPU until read).
    """
    from .layers import AdamW

    m, features = X.shape
    if tokens:
        features *= width
    else:
        X = X.to(dtype)
    net = Classifier(features, hidden, classes, layers, tokens, width, act, dtype, X.device, seed)
    opt = AdamW(net.parameters(), lr=lr, weight_decay=weight_decay, state_bits=state_bits,
                copies=None if net.copies is None else list(net.copies.values()))
    info = MLPInfo()
    batch = m if batch <= 0 else min(batch, m)
    at = 0
    for _ in range(steps):
        y = labels[at:at + batch]
        loss, kept = net.loss(X[at:at + batch], y)
        inside = ((y >= 0) & (y < classes)).sum().clamp_min(1)
        info.losses.append(loss.sum() / inside)
        opt.step(_mean_loss_gradients(net, y, kept))
        info.steps += 1
        at = at + batch if at + batch < m else 0
    return net, info
