"""The operators at the vocabulary's two ends of a training step, as cases to
time and compare: the scaled embedding lookup, its gradient, the clipped
policy loss with a KL term and the preference loss over pairs of sequences.

A case is a dict of plain values.  ``op`` names the operator:

  lookup      out[t] = scale * table[ids[t]]
  grad        table_grad[v] (+)= scale * sum of grad_out[t] over ids[t] == v
  policy      clipped policy loss of N token rows, with the logits' gradient
  preference  preference loss of pairs of packed sequences, likewise

``run`` computes it in plain torch (32 bits, 64 where sums are long) or, with
``own`` set, by the library's entry points; ``exact`` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_ID = {"i32": torch.int32, "i64": torch.int64}
_ID_SIZE = {"i32": 4, "i64": 8}
_CLIP_LOW, _CLIP_HIGH = 0.2, 0.28
_PAD = 0  # the padding token of the gradient cases


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a decoding batch's tokens, from the 16-bit model copy: latency
        dict(name="lookup decode", op="lookup", tokens=64, vocab=32000, dim=4096, table="bf16", out="bf16", ids="i64",
             scale=1.0),
        # a training micro-batch read from the FP32 masters of the 1.1B decoder, scaled by sqrt(dim)
        dict(name="lookup train", op="lookup", tokens=8191, vocab=32000, dim=2048, table="f32", out="bf16", ids="i64",
             scale=45.254833995939045),
        # a long packed batch over a large vocabulary
        dict(name="lookup long", op="lookup", tokens=65536, vocab=131072, dim=8192, table="bf16", out="bf16",
             ids="i32", scale=1.0),
        # one short sequence's gradient, loss-scaled, added into the FP16 gradient bucket of the 1.1B decoder
        dict(name="grad few accumulate", op="grad", tokens=511, vocab=32000, dim=2048, grad="f16", into="f16",
             ids="i64", scale=1.0, pad=False, accumulate=True),
        # a micro-batch of the 6.7B decoder, BF16 activations' gradient into FP32, padded sequences
        dict(name="grad dense", op="grad", tokens=8192, vocab=32000, dim=4096, grad="bf16", into="f32", ids="i64",
             scale=1.0, pad=True, accumulate=False),
        # a long packed batch over a large vocabulary
        dict(name="grad long", op="grad", tokens=131072, vocab=131072, dim=4096, grad="bf16", into="bf16", ids="i32",
             scale=1.0, pad=False, accumulate=False),
        # the end of one short answer: few rows, FP32 logits
        dict(name="policy few", op="policy", rows=16, vocab=32000, dtype="f32", ids="i64", taken=1.0, kl=True,
             gradient=True),
        # answers behind prompts that take no part, a vocabulary that leaves rows unaligned
        dict(name="policy ragged", op="policy", rows=4097, vocab=50001, dtype="f16", ids="i64", taken=0.6, kl=True,
             gradient=True),
        # a large batch over a large vocabulary
        dict(name="policy large", op="policy", rows=8192, vocab=131072, dtype="bf16", ids="i64", taken=0.85, kl=True,
             gradient=True),
        # two pairs, loss and margins alone, as an evaluation computes them
        dict(name="preference few", op="preference", pairs=2, longest=48, vocab=32000, dtype="bf16", ids="i64",
             taken=0.7, gradient=False),
        # pairs of sequences of uneven lengths, FP32 logits, an odd vocabulary
        dict(name="preference ragged", op="preference", pairs=8, longest=513, vocab=32001, dtype="f32", ids="i64",
             taken=0.7, gradient=True),
        # long pairs over a large vocabulary
        dict(name="preference long", op="preference", pairs=8, longest=1024, vocab=131072, dtype="bf16", ids="i32",
             taken=0.7, gradient=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, its logarithm spread evenly; odd as often as even."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["lookup", "grad", "policy", "preference"])
        ids = rng.choice(["i32", "i64"])
        any_type = lambda: rng.choice(["f32", "f16", "bf16"])  # noqa: E731
        if op == "lookup":
            c = dict(op=op, tokens=_log(rng, 1, 65536), vocab=_log(rng, 1000, 131072), dim=_log(rng, 64, 8192),
                     table=any_type(), out=any_type(), ids=ids, scale=rng.choice([1.0, round(rng.uniform(0.5, 90), 3)]))
        elif op == "grad":
            c = dict(op=op, tokens=_log(rng, 1, 131072), vocab=_log(rng, 1000, 131072), dim=_log(rng, 64, 8192),
                     grad=any_type(), into=any_type(), ids=ids, scale=rng.choice([1.0, round(rng.uniform(0.5, 8), 3)]),
                     pad=rng.random() < 0.5, accumulate=rng.random() < 0.5)
        elif op == "policy":
            c = dict(op=op, rows=_log(rng, 1, 8192), vocab=_log(rng, 1000, 160000), dtype=any_type(), ids=ids,
                     taken=rng.choice([1.0, round(rng.uniform(0.3, 1), 2)]), kl=rng.random() < 0.7,
                     gradient=rng.random() < 0.7)
        else:
            c = dict(op=op, pairs=_log(rng, 1, 16), longest=_log(rng, 1, 1024), vocab=_log(rng, 1000, 160000),
                     dtype=any_type(), ids=ids, taken=rng.choice([1.0, round(rng.uniform(0.3, 1), 2)]),
                     gradient=rng.random() < 0.7)
        if work(c)["bytes"] <= most and _values(c) <= 8192 * 131072:
            return c


def _values(c):
    """Values of the largest array of a case."""
    if c["op"] == "lookup":
        return max(c["tokens"], c["vocab"]) * c["dim"]
    if c["op"] == "grad":
        return max(c["tokens"], c["vocab"]) * c["dim"]
    return _rows(c) * c["vocab"]


def _lengths(c):
    """Lengths of a preference case's 2 * pairs sequences: the first has the longest, the others are spread over
    1 .. longest, and with several pairs one of them is empty."""
    n = 2 * c["pairs"]
    out = [c["longest"]] + [1 + (i * 7919 + 104729) % c["longest"] for i in range(1, n)]
    if n > 4:
        out[3] = 0
    return out


def _rows(c):
    return c["rows"] if c["op"] == "policy" else sum(_lengths(c))


def _taken(c):
    """Truth values [rows]: which rows take part.  Of every sequence (512 rows of a policy case) the leading ones are
    the prompt, which does not."""
    if c["op"] == "policy":
        n = c["rows"]
        lengths = [512] * (n // 512) + ([n % 512] if n % 512 else [])
    else:
        lengths = _lengths(c)
    lengths = np.array(lengths, np.int64)
    at = np.arange(lengths.sum()) - np.repeat(np.cumsum(lengths) - lengths, lengths)
    return at >= np.repeat(np.rint(lengths * (1 - c["taken"])), lengths)


def _loss_scale(c):
    """The factor that FP16 gradients are stored with, and the optimizer step divides out."""
    return 1024.0 if c["dtype"] == "f16" else 1.0


def _shares(vocab):
    """Share of each token id in a text: the Zipf-Mandelbrot law 1 / (rank + 2.7), ids in order of rank."""
    p = 1.0 / (np.arange(vocab) + 2.7)
    return p / p.sum()


def _padded(c):
    """Padding tokens of a gradient case: the last eighth of the batch."""
    return c["tokens"] // 8 if c["pad"] else 0


def _distinct(c, tokens):
    """How many distinct ids that many tokens hold, on average."""
    return float(np.sum(-np.expm1(tokens * np.log1p(-_shares(c["vocab"])))))


def work(case):
    c = case
    if c["op"] == "lookup":
        rows = _distinct(c, c["tokens"])
        return {"bytes": rows * c["dim"] * _SIZE[c["table"]] + c["tokens"] * (c["dim"] * _SIZE[c["out"]] + _ID_SIZE[c["ids"]]),
                "flops": c["tokens"] * c["dim"]}
    if c["op"] == "grad":
        tokens = c["tokens"] - _padded(c)
        moved = 2 * _distinct(c, tokens) if c["accumulate"] else c["vocab"]
        return {"bytes": tokens * c["dim"] * _SIZE[c["grad"]] + c["tokens"] * _ID_SIZE[c["ids"]]
                + moved * c["dim"] * _SIZE[c["into"]], "flops": tokens * c["dim"]}
    n, s = _rows(c), _SIZE[c["dtype"]]
    taken = int(_taken(c).sum())
    return {"bytes": taken * c["vocab"] * s + (n * c["vocab"] * s if c["gradient"] else 0) + n * (_ID_SIZE[c["ids"]] + 24),
            "flops": taken * c["vocab"] * (8 if c["gradient"] else 4)}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    return torch.Generator("cuda").manual_seed(int(seed))


def _normal(shape, std, dtype, g):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _text(c, n, g):
    """n token ids of a text."""
    cdf = torch.from_numpy(np.cumsum(_shares(c["vocab"]))).cuda()
    u = torch.rand(n, dtype=torch.float64, device="cuda", generator=g)
    return torch.searchsorted(cdf, u).clamp_(max=c["vocab"] - 1).to(_ID[c["ids"]])


def _logits(c, n, g):
    """Logits of n rows with their labels: the label's logit is raised, as a trained model's is.  Rows that take no
    part have the label -100."""
    x = _normal((n, c["vocab"]), 2.0, _DT[c["dtype"]], g)
    labels = torch.randint(0, c["vocab"], (n,), device="cuda", generator=g)
    lift = 4.0 + 6.0 * torch.rand((n, 1), device="cuda", generator=g)
    x.scatter_add_(1, labels[:, None], lift.to(x.dtype))
    # log-probabilities of the labels
    logp = x.float().log_softmax(1).gather(1, labels[:, None])[:, 0]
    taken = torch.from_numpy(_taken(c)).cuda()
    labels = torch.where(taken, labels, torch.full_like(labels, -100))
    return x, labels.to(_ID[c["ids"]]), taken, logp


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "lookup":
        s["table"] = _normal((c["vocab"], c["dim"]), 0.02, _DT[c["table"]], g)
        s["ids"] = _text(c, c["tokens"], g)
        s["out"] = torch.empty((c["tokens"], c["dim"]), dtype=_DT[c["out"]], device="cuda")
        return s
    if c["op"] == "grad":
        # gradients as the optimizer's decoder lists have them: 1e-4, scaled by 1024 where FP16 holds them
        std = 1e-4 * (1024 if "f16" in (c["grad"], c["into"]) else 1)
        s["grad_out"] = _normal((c["tokens"], c["dim"]), std, _DT[c["grad"]], g)
        s["ids"] = _text(c, c["tokens"], g)
        if c["pad"]:
            s["ids"][c["tokens"] - _padded(c):] = _PAD
        s["table_grad"] = (_normal((c["vocab"], c["dim"]), std, _DT[c["into"]], g) if c["accumulate"] else
                           torch.empty((c["vocab"], c["dim"]), dtype=_DT[c["into"]], device="cuda"))
        return s
    n = _rows(c)
    s["logits"], s["labels"], taken, logp = _logits(c, n, g)
    if c["op"] == "policy":
        # the policy has moved a little since the tokens were sampled, and the reference is further away
        s["old_logp"] = logp + 0.15 * _normal((n,), 1.0, torch.float32, g)
        s["ref_logp"] = logp + 0.3 * _normal((n,), 1.0, torch.float32, g) if c["kl"] else None
        # a ratio within a thousandth of a clipping bound is moved off it: 32 bits do not tell its side
        for edge in (1 - _CLIP_LOW, 1 + _CLIP_HIGH):
            near = ((logp - s["old_logp"]) - math.log(edge)).abs() < 1e-3
            s["old_logp"] += 4e-3 * near
        s["advantages"] = _normal((n,), 1.0, torch.float32, g)
        # the mean over the rows that take part
        s["weights"] = torch.full((n,), 1.0 / max(1, int(taken.sum())), device="cuda")
    else:
        lengths = torch.tensor(_lengths(c), device="cuda")
        s["offsets"] = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)]).to(_ID[c["ids"]])
        seq = torch.repeat_interleave(torch.arange(len(_lengths(c)), device="cuda"), lengths)
        total = torch.zeros(len(_lengths(c)), dtype=torch.float64, device="cuda")
        total.index_add_(0, seq, torch.where(taken, logp, 0).double())
        s["seq"] = seq
        s["ref_logp"] = (total + 8.0 * _normal((len(_lengths(c)),), 1.0, torch.float64, g)).float()
        s["weights"] = torch.full((c["pairs"],), 1.0 / c["pairs"], device="cuda")
        s["seq_logp"] = torch.empty(2 * c["pairs"], device="cuda")
    s["total"] = torch.empty((), device="cuda")
    s["loss"] = torch.empty(n if c["op"] == "policy" else c["pairs"], device="cuda")
    s["logp"] = torch.empty(n, device="cuda")
    s["row_stats"] = torch.empty((n, 4), device="cuda")
    s["grad"] = torch.empty_like(s["logits"]) if c["gradient"] else None
    return s


# --------------------------------------------------------------------- run --

_BETA, _SMOOTHING, _KL = 0.1, 0.05, 0.04


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import optimizer_step_dl_amd as ra
    c = s["case"]
    if c["op"] == "lookup":
        ra.radamw_embedding_lookup(s["table"], s["ids"], s["out"], scale=c["scale"])
        return s["out"]
    if c["op"] == "grad":
        need = ra.radamw_embedding_grad_workspace_bytes(c["tokens"], c["vocab"], c["dim"])
        workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        ra.radamw_embedding_grad(s["grad_out"], s["ids"], s["table_grad"], workspace, scale=c["scale"],
                                 padding_id=_PAD if c["pad"] else None, accumulate=c["accumulate"])
        return s["table_grad"]
    if c["op"] == "policy":
        opts = ra.policy_options(clip_low=_CLIP_LOW, clip_high=_CLIP_HIGH, kl_coef=_KL if c["kl"] else 0.0)
        ra.radamw_policy_loss(s["logits"], s["labels"], s["old_logp"], s["advantages"], opts, s["total"], s["loss"],
                              s["logp"], ref_logp=s["ref_logp"], weights=s["weights"], grad=s["grad"],
                              grad_scale=_loss_scale(c))
        return _answer(s)
    opts = ra.preference_options(beta=_BETA, label_smoothing=_SMOOTHING)
    ra.radamw_preference_loss(s["logits"], s["labels"], s["offsets"], s["ref_logp"], opts, s["total"], s["loss"],
                              s["seq_logp"], s["logp"], s["row_stats"], weights=s["weights"], grad=s["grad"],
                              grad_scale=_loss_scale(c))
    return _answer(s)


def _answer(s):
    out = {"total": s["total"], "loss": s["loss"], "logp": s["logp"]}
    if s["case"]["op"] == "preference":
        out["seq_logp"] = s["seq_logp"]
    if s["grad"] is not None:
        out["grad"] = s["grad"]
    return out


def _run_plain(s):
    c = s["case"]
    if c["op"] == "lookup":
        return (s["table"][s["ids"]].float() * c["scale"]).to(_DT[c["out"]])
    if c["op"] == "grad":
        into = s["table_grad"]
        acc = into.float() if c["accumulate"] else torch.zeros(into.shape, device="cuda")
        src = s["grad_out"].float() * c["scale"]
        if c["pad"]:
            src *= (s["ids"] != _PAD)[:, None]
        acc = acc.clone() if acc is into else acc
        into.copy_(acc.index_add_(0, s["ids"], src))
        return into
    taken = s["labels"] >= 0
    label = torch.where(taken, s["labels"], 0).long()[:, None]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    e = (x - top).exp_()
    norm = e.sum(1, dtype=torch.float64)
    logp = (x.gather(1, label) - top)[:, 0].double() - norm.log()
    logp = torch.where(taken, logp, 0)
    del x
    if c["op"] == "policy":
        ratio = (logp - s["old_logp"]).exp()
        a = s["advantages"].double()
        loss = -torch.minimum(ratio * a, ratio.clamp(1 - _CLIP_LOW, 1 + _CLIP_HIGH) * a)
        active = torch.where(a >= 0, ratio <= 1 + _CLIP_HIGH, ratio >= 1 - _CLIP_LOW)
        d = torch.where(active, -a * ratio, 0)
        if c["kl"]:
            away = s["ref_logp"] - logp
            loss = loss + _KL * (away.exp() - away - 1)
            d = d + _KL * (1 - away.exp())
        loss = torch.where(taken, loss, 0)
        coef = torch.where(taken, d * s["weights"], 0)
        total = (loss * s["weights"]).sum()
        out = {"total": total.float(), "loss": loss.float(), "logp": logp.float()}
    else:
        p = c["pairs"]
        sums = torch.zeros(2 * p, dtype=torch.float64, device="cuda").index_add_(0, s["seq"], logp)
        margin = sums - s["ref_logp"]
        h = _BETA * (margin[:p] - margin[p:])
        # -log sigmoid(h) = log(1 + exp(-h)) = max(-h, 0) + log(1 + exp(-|h|))
        tail = (1 + (-h.abs()).exp()).log()
        loss = (1 - _SMOOTHING) * ((-h).clamp(min=0) + tail) + _SMOOTHING * (h.clamp(min=0) + tail)
        sig = 1 / (1 + (-h).exp())
        d = _BETA * (_SMOOTHING * sig - (1 - _SMOOTHING) * (1 - sig)) * s["weights"]
        coef = torch.where(taken, torch.cat([d, -d])[s["seq"]], 0)
        out = {"total": (loss * s["weights"]).sum().float(), "loss": loss.float(), "logp": logp.float(),
               "seq_logp": sums.float()}
    if c["gradient"]:
        coef = coef * _loss_scale(c)
        grad = e.mul_((-coef / norm).float()[:, None])
        grad.scatter_add_(1, label, coef.float()[:, None])
        out["grad"] = grad.to(s["logits"].dtype)
    return out


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "lookup":
        return torch.index_select(s["table"], 0, s["ids"].long()).double().mul_(float(np.float32(c["scale"])))
    if c["op"] == "grad":
        ids = s["ids"].long()
        kept = ids != _PAD if c["pad"] else torch.ones_like(ids, dtype=torch.bool)
        out = s["table_grad"].double() if c["accumulate"] else \
            torch.zeros(s["table_grad"].shape, dtype=torch.float64, device="cuda")
        out.index_put_((ids[kept],), s["grad_out"][kept].double() * float(np.float32(c["scale"])), accumulate=True)
        return out
    n = _rows(c)
    keep = _taken(c)
    logp = torch.zeros(n, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // c["vocab"])
    for i in range(0, n, step):
        x = s["logits"][i:i + step].double()
        a = s["labels"][i:i + step].long()
        a = a.clamp(min=0)
        logp[i:i + step] = x[torch.arange(len(a), device="cuda"), a] - torch.logsumexp(x, 1)
    keep = torch.from_numpy(keep).cuda()
    logp = logp.masked_fill(~keep, 0.0)
    if c["op"] == "policy":
        lp = logp.clone().requires_grad_()
        ratio = torch.exp(lp - s["old_logp"].double())
        a = s["advantages"].double()
        loss = -torch.min(ratio * a, torch.clamp(ratio, 1 - _CLIP_LOW, 1 + _CLIP_HIGH) * a)
        if c["kl"]:
            log_ratio = s["ref_logp"].double() - lp
            loss = loss + _KL * (torch.expm1(log_ratio) - log_ratio)
        loss = loss.masked_fill(~keep, 0.0)
        total = torch.dot(loss, s["weights"].double())
        out = {"total": total.detach(), "loss": loss.detach(), "logp": logp}
        coef, = torch.autograd.grad(total, lp)
    else:
        p = c["pairs"]
        lp = logp.clone().requires_grad_()
        ends = np.concatenate([[0], np.cumsum(_lengths(c))])
        sums = torch.stack([lp[ends[i]:ends[i + 1]].sum() for i in range(2 * p)])
        gap = sums - s["ref_logp"].double()
        h = _BETA * (gap[:p] - gap[p:])
        loss = -(1 - _SMOOTHING) * torch.nn.functional.logsigmoid(h) - _SMOOTHING * torch.nn.functional.logsigmoid(-h)
        total = torch.dot(loss, s["weights"].double())
        out = {"total": total.detach(), "loss": loss.detach(), "logp": logp, "seq_logp": sums.detach()}
        coef, = torch.autograd.grad(total, lp)
    if c["gradient"]:
        coef = coef.masked_fill(~keep, 0.0) * _loss_scale(c)
        grad = torch.empty((n, c["vocab"]), dtype=torch.float64, device="cuda")
        for i in range(0, n, step):
            g = torch.softmax(s["logits"][i:i + step].double(), 1).mul_(-coef[i:i + step, None])
            a = s["labels"][i:i + step].long().clamp(min=0)
            g[torch.arange(len(a), device="cuda"), a] += coef[i:i + step]
            grad[i:i + step] = g
        out["grad"] = grad
    return out
