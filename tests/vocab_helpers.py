"""Plain 64-bit forms of the vocabulary operators, on the CPU, and the bounds
their GPU results are held to.

The bounds, with u = 2^-24 (half a step of FP32, relative) and h = half a
step of the output type (torch.finfo(t).eps / 2):

  lookup    one FP32 product and one rounding: torch forms the same bits.

  gradient  k terms are summed in FP32 in some order and multiplied by the
            scale (fused with the old value): at most k + 2 roundings, each
            of at most u times the sum of the terms' magnitudes T (the old
            value's among them), then the output's rounding:
            (k + 2) u T + h |ref|, and half the smallest subnormal.

  logp      e_j = exp(x_j - m): the difference, the product with log2 e and
            that constant are each rounded (3 u |x_j - m| relative), v_exp_f32
            is within 1 ulp (2 u); a lane adds at most `chain` of them in
            FP32, the rest is in 64 bits.  So the sum is off by at most
            E = sum p_j (3 u |x_j - m| + 2 u) + chain u relative, logp by E
            and its own rounding u |logp|.
  loss      what E does to it by its derivative, to first order with a factor
            1.01 for the rest (E < 1e-4), and its rounding.
  gradient  g_j = c (1[j = a] - p_j): p_j is off by p_j (3 u |x_j - m| + 2 u
            + E), plus the roundings of c / s, of the product and of the
            label's factor (4 u |g_j|); c by what E does to it; then h |g_j|
            and half the smallest subnormal.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def half_tiny(dtype) -> float:
    """Half the smallest subnormal (what a result next to zero rounds by)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def f32(x: float) -> float:
    return float(torch.tensor(x, dtype=torch.float64).float())


def embedding_grad(grad_out, ids, rows, scale, padding_id, old):
    """(reference, bound without the output's rounding) of the lookup's
    gradient, both [rows, dim] in 64 bits."""
    g = grad_out.double()
    ids = ids.reshape(-1).long()
    keep = (ids >= 0) & (ids < rows)
    if padding_id is not None:
        keep &= ids != padding_id
    g, ids = g[keep], ids[keep]
    dim = g.shape[1]
    s = f32(scale)
    ref = torch.zeros(rows, dim, dtype=torch.float64).index_add_(0, ids, g) * s
    mag = torch.zeros(rows, dim, dtype=torch.float64).index_add_(0, ids, g.abs()) * abs(s)
    count = torch.zeros(rows, dtype=torch.float64).index_add_(0, ids, torch.ones(len(ids), dtype=torch.float64))
    if old is not None:
        ref += old.double()
        mag += old.double().abs()
    return ref, (count[:, None] + 2) * U * mag


def close(got, ref, slack, what):
    """|got - ref| <= slack + the rounding of got's type; NaN where ref is."""
    got64 = got.detach().cpu().double()
    ref = ref.detach().cpu().double()
    assert got64.shape == ref.shape, (what, got64.shape, ref.shape)
    assert torch.equal(got64.isnan(), ref.isnan()), f"{what}: NaN in other places"
    inf = ref.isinf()
    assert torch.equal(got64[inf], ref[inf]), f"{what}: infinities differ"
    fine = ref.isfinite()
    slack = slack.cpu() if torch.is_tensor(slack) else torch.full_like(ref, slack)
    tol = slack + half_step(got.dtype) * (ref.abs() + slack) + half_tiny(got.dtype)
    err = (got64 - ref).abs()
    bad = fine & ~(err <= tol)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got64[tuple(i)].item()} against {ref[tuple(i)].item()}, "
                             f"allowed {tol[tuple(i)].item():.3g}")


class Rows:
    """A loss's rows in 64 bits: logp, probabilities, the error E of logp."""

    def __init__(self, logits, labels, taken):
        x = logits.detach().cpu().double()
        self.taken = taken
        n, vocab = x.shape
        self.label = torch.where(taken, labels.cpu().long(), 0)
        x = torch.where(taken[:, None], x, 0.0)
        top = x.amax(1, keepdim=True)
        self.y = x - top
        e = self.y.exp()
        self.p = e / e.sum(1, keepdim=True)
        self.logp = (x.gather(1, self.label[:, None]) - top)[:, 0] - e.sum(1).log()
        # a lane's longest chain of FP32 additions into one of its four sums
        lanes = 256
        chain = math.ceil(math.ceil(vocab / lanes) / 4) + 8
        away = torch.where(self.p > 0, self.y.abs(), 0.0)
        self.e_rel = 3 * U * away + 2 * U
        self.err = (self.p * self.e_rel).sum(1) + chain * U

    def grad(self, coef, coef_err, scale):
        """(reference, bound) of scale * coef * (1[label] - p)."""
        one = torch.zeros_like(self.p).scatter_(1, self.label[:, None], 1.0)
        c = (coef * scale)[:, None]
        ref = c * (one - self.p)
        # 2^-126: an exponential below FP32's normal range may be flushed
        p_err = self.p * (self.e_rel + self.err[:, None]) + 2.0 ** -126
        # the label's factor 1 - p comes from logp itself
        slack = 1.01 * (c.abs() * p_err + (coef_err * abs(scale))[:, None] * (one - self.p).abs()) + 4 * U * ref.abs()
        # a row that takes no part, or without a coefficient, is exactly zero
        dead = (~self.taken | (coef == 0))[:, None]
        return torch.where(dead, 0.0, ref), torch.where(dead, 0.0, slack)


def policy(rows, old, ref, adv, weights, lo, hi, kl):
    """loss, coef and their bounds from the rows' logp, in 64 bits."""
    lp, err = rows.logp, rows.err
    old = lp if old is None else old.cpu().double()
    err_r = torch.zeros_like(err) if old is lp else err
    a = adv.cpu().double()
    w = torch.ones_like(lp) if weights is None else weights.cpu().double()
    r = (lp - old).exp()
    loss = -torch.minimum(r * a, r.clamp(1 - lo, 1 + hi) * a)
    active = torch.where(a >= 0, r <= 1 + hi, r >= 1 - lo)
    d = torch.where(active | r.isnan(), -a * r, 0.0)  # a NaN ratio is not clipped away
    loss_err = 1.01 * (a * r).abs() * err_r
    d_err = torch.where(active, loss_err, 0.0)
    if kl:
        away = ref.cpu().double() - lp
        loss = loss + kl * (away.exp() - away - 1)
        d = d + kl * (1 - away.exp())
        loss_err = loss_err + 1.01 * kl * (away.exp() + 1) * err
        d_err = d_err + 1.01 * kl * away.exp() * err
    zero = torch.zeros_like(loss)
    t = rows.taken
    return (torch.where(t, loss, zero), torch.where(t, loss_err, zero), torch.where(t, d * w, zero),
            torch.where(t, d_err * w.abs(), zero))


def preference(rows, bounds, ref, weights, beta, smoothing):
    """(loss, its bound, sums, their bound, coef per row, its bound) from
    the rows' logp; ``bounds`` are the offsets, as a list."""
    s = len(bounds) - 1
    pairs = s // 2
    lp = torch.where(rows.taken, rows.logp, 0.0)
    er = torch.where(rows.taken, rows.err, 0.0)
    sums = torch.stack([lp[bounds[i]:bounds[i + 1]].sum() for i in range(s)])
    errs = torch.stack([er[bounds[i]:bounds[i + 1]].sum() for i in range(s)])
    # what a record keeps of logp beside its FP32 value is an FP32 value too: 2^-48
    m = sums - ref.cpu().double()
    h = beta * (m[:pairs] - m[pairs:])
    h_err = beta * (errs[:pairs] + errs[pairs:])
    ls = torch.nn.functional.logsigmoid
    loss = -(1 - smoothing) * ls(h) - smoothing * ls(-h)
    w = torch.ones(pairs, dtype=torch.float64) if weights is None else weights.cpu().double()
    d = beta * w * (smoothing * h.sigmoid() - (1 - smoothing) * (-h).sigmoid())
    d_err = 1.01 * beta * w.abs() * 0.25 * h_err + U * d.abs()
    coef = torch.zeros_like(lp)
    coef_err = torch.zeros_like(lp)
    for i in range(s):
        coef[bounds[i]:bounds[i + 1]] = d[i % pairs] * (1 if i < pairs else -1)
        coef_err[bounds[i]:bounds[i + 1]] = d_err[i % pairs]
    coef = torch.where(rows.taken, coef, 0.0)
    return loss, 1.01 * h_err, sums, errs, coef, torch.where(rows.taken, coef_err, 0.0)
