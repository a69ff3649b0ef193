"""Plain 64-bit forms of the block operators, on the CPU, and the bounds their
GPU results are held to.

The bounds, with u = 2^-24 (half a step of FP32, relative); close() adds half
a step of the output's type:

  dropout   one FP32 product: u |ref|.

  norms     a sum of squares: a lane adds at most 32 terms in one chain, the
            wave and the workgroup at most 23 more; the product with 1 / dim
            and eps two: relative error at most 58 u, half of that in the
            root, v_rsq_f32 2 u: R = 32 u.
  h         x + scale * term: the term is off by R and 5 roundings.
  out       h's error e: the root moves by sum |h| e / sum h^2; 3 roundings.

  gradient  stated at residual_grad(): every sum along a row has at most 58
            roundings, a sum over rows `rows` of them (a worker's rows), the
            join is in 64 bits.

  balance   stated at balance().
"""
from __future__ import annotations

import math

import numpy as np
import torch

from vocab_helpers import U, f32

DOUBLE = torch.float64
ROW = 58 * U   # a sum along a row, relative to its terms' magnitudes
R = 32 * U     # the reciprocal root of a mean square

_M0, _M1, _W0, _W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key):
    """Philox 4x32 with ten rounds, word by word: counter 4 and key 2 numbers
    or numpy arrays of numbers below 2^32."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = np.uint64(_M0) * c[0], np.uint64(_M1) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + _W0) & 0xFFFFFFFF, (k[1] + _W1) & 0xFFFFFFFF]
    return c


def threshold(p):
    return math.floor(65536 * p + 0.5)


def keep_mask(n, dim, p, seed, offset, first_row=0):
    """Truth values [n, dim]: which elements are kept."""
    groups = -(-dim // 8)
    col, row = np.meshgrid(np.arange(groups), np.arange(n) + first_row)
    words = philox((col, row, np.full_like(col, offset & 0xFFFFFFFF), np.full_like(col, offset >> 32)),
                   (seed & 0xFFFFFFFF, seed >> 32))
    numbers = np.empty((n, groups, 8), np.int64)
    for i, w in enumerate(words):
        numbers[:, :, 2 * i] = (w & np.uint64(0xFFFF)).astype(np.int64)
        numbers[:, :, 2 * i + 1] = (w >> np.uint64(16)).astype(np.int64)
    return torch.from_numpy(numbers.reshape(n, groups * 8)[:, :dim] >= threshold(p))


def keep_factor(p):
    t = threshold(p)
    return f32(65536 / (65536 - t)) if t < 65536 else 0.0


def dropout(x, p, seed, offset, first_row=0):
    """(reference, bound) of radamw_dropout."""
    keep = keep_mask(x.shape[0], x.shape[1], p, seed, offset, first_row)
    ref = torch.where(keep, x.double() * keep_factor(p), 0.0)
    return ref, U * ref.abs()


class Residual:
    """One residual call's inputs in 64 bits (absent ones None)."""

    def __init__(self, x, branch, gate=None, per=None, post=None, pre=None, eps=1e-6, offset=0.0, scale=1.0, p=0.0,
                 seed=0, counter=0, first_row=0):
        self.x = x.double()
        self.n, self.dim = x.shape
        self.y = None if branch is None else branch.double()
        self.groups = torch.arange(self.n) // (per or max(1, self.n))
        self.gate_rows = 0 if gate is None else gate.shape[0]
        self.g = torch.ones(()).double() if gate is None else gate.double()[self.groups]
        self.post = None if post is None else post.double() + f32(offset)
        self.pre = None if pre is None else pre.double() + f32(offset)
        self.eps, self.scale = f32(eps), f32(scale)
        self.factor = keep_factor(p)
        self.keep = keep_mask(self.n, self.dim, p, seed, counter, first_row)

    def _rstd(self, v):
        return (v.square().mean(1, keepdim=True) + self.eps).rsqrt()

    def forward(self):
        """{name: (reference, bound)} of h, out and both rows of rstd."""
        got = {}
        h, e = self.x, torch.zeros_like(self.x)
        if self.y is not None:
            term = self.y * self.factor * self.g * self.scale
            if self.post is not None:
                rb = self._rstd(self.y)
                got["rstd_branch"] = (rb[:, 0], R * rb[:, 0])
                term = term * rb * self.post
            term = torch.where(self.keep, term, 0.0)
            h = self.x + term
            e = 1.01 * term.abs() * (R + 5 * U) + U * h.abs()
            got["h"] = (h, e)
        if self.pre is not None:
            rh = self._rstd(h)
            rho = R + (h.abs() * e).sum(1, keepdim=True) / (h.square().sum(1, keepdim=True) + self.dim * self.eps)
            got["rstd_h"] = (rh[:, 0], 1.01 * (rho * rh)[:, 0])
            out = h * rh * self.pre
            got["out"] = (out, 1.01 * ((self.pre * rh).abs() * e + out.abs() * (rho + 3 * U)))
        return got

    def backward(self, grad_h, grad_out, rstd):
        """{name: (reference, bound)} of the gradients, with the rstd given
        (2 n values)."""
        n, dim = self.n, self.dim
        rows = -(-n // 256) + 2  # a worker's rows, and two roundings
        got = {}
        d = torch.zeros(n, dim, dtype=DOUBLE) if grad_h is None else grad_h.double()
        size = d.abs()
        e = torch.zeros_like(d)
        if self.pre is not None:
            r = rstd.double()[n:, None]
            hat = self.x * r
            c = grad_out.double() * hat
            got["pre"] = (c.sum(0), c.abs().sum(0) * (2 + rows) * U)
            q = grad_out.double() * self.pre
            mean = (q * hat).mean(1, keepdim=True)
            e_mean = (q * hat).abs().mean(1, keepdim=True) * (ROW + 4 * U)
            d = d + r * (q - hat * mean)
            size = size + r * (q.abs() + (hat * mean).abs())
            e = r * hat.abs() * e_mean + 6 * U * size
        got["x"] = (d, e)
        if self.y is None:
            return got
        fs = self.factor * self.scale
        b = torch.where(self.keep, d * fs, 0.0)
        e = torch.where(self.keep, e * abs(fs), 0.0) + 2 * U * b.abs()
        rb = rstd.double()[:n, None] if self.post is not None else torch.ones(n, 1, dtype=DOUBLE)
        hat = self.y * rb
        post = torch.ones(dim, dtype=DOUBLE) if self.post is None else self.post
        u = torch.where(self.keep, hat * post, 0.0)
        dg = torch.where(self.keep, b * u, 0.0)
        e_dg = 1.01 * (e * u.abs() + 4 * U * dg.abs())
        if self.gate_rows:
            sums = torch.zeros(3, self.gate_rows, dim, dtype=DOUBLE)
            for s, v in zip(sums, (dg, e_dg, dg.abs())):
                s.index_add_(0, self.groups, v)
            alone = self.gate_rows == n
            got["gate"] = (sums[0], sums[1] + (0 if alone else rows * U) * sums[2])
        c = torch.where(self.keep, b * self.g, 0.0)
        e = torch.where(self.keep, e * self.g.abs(), 0.0) + U * c.abs()
        hat = torch.where(self.keep, hat, 0.0) if self.post is None else hat
        if self.post is not None:
            got["post"] = ((c * hat).sum(0), 1.01 * (e * hat.abs()).sum(0) + (c * hat).abs().sum(0) * (2 + rows) * U)
        du = c * post
        e = e * post.abs() + 2 * U * du.abs()
        if self.post is not None:
            mean = (du * hat).mean(1, keepdim=True)
            e_mean = (e * hat.abs()).mean(1, keepdim=True) + (du * hat).abs().mean(1, keepdim=True) * (ROW + 4 * U)
            dy = rb * (du - hat * mean)
            e = 1.01 * rb * (e + hat.abs() * e_mean) + 6 * U * rb * (du.abs() + (hat * mean).abs())
            du = dy
        got["branch"] = (du, e)
        return got


def balance(logits, ids, mask=None, bounds=None, weights=None, coef=0.01, z=0.0, score="softmax", scale=1.0):
    """{name: (reference, bound)} of a balance call; counts and tokens exactly.

    An exponential: the difference (or the logit itself), the product with
    log2 e and that constant are rounded, v_exp_f32 is within 1 ulp: 3 u |d| +
    2 u relative, and one below 2^-126 may be flushed.  A sigmoid adds 3
    roundings.  A row's sum: at most 64 + 6 additions; its reciprocal and the
    product 3 more.  Sums over rows: a piece's rows, at most n / 256 + 12.
    """
    x = logits.double()
    n, experts = x.shape
    k = ids.shape[1]
    live = torch.ones(n, dtype=torch.bool) if mask is None else mask.bool().clone()
    bounds = [0, n] if bounds is None else bounds
    groups = len(bounds) - 1
    group = torch.full((n,), -1)
    for g in range(groups):
        group[bounds[g]:bounds[g + 1]] = g
    live &= group >= 0
    w = torch.ones(groups, dtype=DOUBLE) if weights is None else weights.double()
    x = torch.where(live[:, None], x, 0.0)
    if score == "softmax":
        top = x.amax(1, keepdim=True)
        m = torch.where(top == -math.inf, 0.0, top)
        s = (x - m).exp()
        rel = torch.where(s > 0, 3 * U * (x - m).abs() + 2 * U, 0.0)
        rest = torch.ones_like(s)
        lse = m[:, 0] + s.sum(1).log()
    else:
        s = x.sigmoid()
        rel = torch.where(s > 0, 3 * U * x.abs() + 5 * U, 0.0)
        rest = (-x).sigmoid()
        lse = torch.zeros(n, dtype=DOUBLE)
    norm = s.sum(1, keepdim=True)
    p = torch.where(norm == 0, 0.0, s / norm)
    lse = torch.where(norm[:, 0] == 0, 0.0, lse)
    sum_rel = (p * rel).sum(1, keepdim=True) + 70 * U
    p_err = 1.01 * p * (rel + sum_rel + 3 * U) + 2.0 ** -120
    lse_err = sum_rel[:, 0] + 4 * U * (torch.where(x == -math.inf, 0.0, x).abs().amax(1) + math.log(experts) + 1)
    p, p_err = torch.where(live[:, None], p, 0.0), torch.where(live[:, None], p_err, 0.0)
    lse, lse_err = torch.where(live, lse, 0.0), torch.where(live, lse_err, 0.0)
    counts = torch.zeros(groups, experts, dtype=torch.int64)
    tokens = torch.zeros(groups, dtype=torch.int64)
    mean, mean_err = torch.zeros(2, groups, experts, dtype=DOUBLE)
    loss, loss_err = torch.zeros(2, groups, dtype=DOUBLE)
    grad, grad_err = torch.zeros(2, n, experts, dtype=DOUBLE)
    chain = (n // 256 + 12) * U
    for g in range(groups):
        rows = torch.nonzero(live & (group == g))[:, 0]
        t = max(1, len(rows))
        tokens[g] = len(rows)
        chosen = ids[rows].reshape(-1).long()
        chosen = chosen[(chosen >= 0) & (chosen < experts)]
        counts[g] = torch.bincount(chosen, minlength=experts)
        mean[g] = p[rows].sum(0) / t
        mean_err[g] = p_err[rows].sum(0) / t + chain * mean[g]
        f = coef * experts / (k * t) * counts[g].double()
        loss[g] = (f * mean[g]).sum() + z * lse[rows].square().sum() / t
        loss_err[g] = (f * (mean_err[g] + U * mean[g])).sum() + \
            z * (2 * lse[rows].abs() * lse_err[rows] + lse_err[rows] ** 2 + chain * lse[rows].square()).sum() / t
        up = f32(scale) * w[g] / t
        cost = f * up
        zc = 2 * z * up
        inner = (cost * p[rows]).sum(1, keepdim=True)
        inner_err = (cost.abs() * p_err[rows]).sum(1, keepdim=True) + 73 * U * inner.abs()
        away = cost - inner + zc * lse[rows, None]
        away_err = inner_err + 4 * U * (cost.abs() + inner.abs() + (zc * lse[rows, None]).abs()) + \
            abs(zc) * lse_err[rows, None]
        factor = p[rows] * (rest[rows] if score == "sigmoid" else 1.0)
        # of a sigmoid, 1 - s has the error of s
        factor_err = p_err[rows] * (rest[rows] if score == "sigmoid" else 1.0) * (2.0 if score == "sigmoid" else 1.0)
        grad[rows] = factor * away
        grad_err[rows] = 1.01 * (factor_err * away.abs() + factor * away_err) + 3 * U * (factor * away).abs()
    total = (w * loss).sum()
    total_err = (w.abs() * (loss_err + U * loss.abs())).sum()
    return {"counts": counts, "tokens": tokens, "mean_prob": (mean, mean_err), "loss": (loss, loss_err),
            "total": (total, total_err), "grad": (grad, grad_err)}
