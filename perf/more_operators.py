"""The operators between the vocabulary's two ends of a training step, as cases
to time and compare: dropout from a counter-based generator, the residual
stream's norms with a block's gate, dropout and scale, their gradient, and the
balance loss of a router with its per-expert counts.

A case is a dict of plain values.  ``op`` names the operator:

  dropout   out = x / keep where the generator keeps an element, else 0
  residual  h = x + scale * gate * drop(norm(branch) * w_post),
            out = norm(h) * w_pre
  grad      the gradients of the stream, the branch, the gate and both weights
  balance   balance loss and z-loss of a router's logits over groups of
            tokens, with the counts and, in training, the logits' gradient

``run`` computes it in plain torch (32 bits, 64 where sums are long) or, with
``own`` set, by the library's entry points; ``exact`` computes it in 64 bits.

The generator is Philox 4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011): key = the seed, counter
= (column / 8, row, offset); the four words of a counter are eight 16-bit
numbers for the eight columns, and a column is dropped where its number is
below round(65536 p).
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_ID = {"i32": torch.int32, "i64": torch.int64}
_ID_SIZE = {"i32": 4, "i64": 8}
_EPS = 1e-6
_BALANCE, _Z = 0.01, 0.001
_MASK32 = 0xFFFFFFFF


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the embedding's dropout of one short sequence: latency
        dict(name="dropout few", op="dropout", rows=128, dim=2048, dtype="bf16", p=0.1),
        # FP32 activations of an odd width
        dict(name="dropout ragged", op="dropout", rows=4097, dim=1111, dtype="f32", p=0.25),
        # a long packed batch
        dict(name="dropout long", op="dropout", rows=32768, dim=8192, dtype="bf16", p=0.1),
        # a step of an evaluation batch: the 16-bit model copy's weights, no dropout, one gate for all rows
        dict(name="residual few", op="residual", rows=64, dim=2048, stream="bf16", branch="bf16", weight="bf16",
             gate="column", gate_type="bf16", per=64, post=True, pre=True, p=0.0, scale=1.0),
        # a micro-batch of the 6.7B decoder: FP32 stream, FP32 master weights, residual dropout
        dict(name="residual train", op="residual", rows=8192, dim=4096, stream="f32", branch="bf16", weight="f32",
             gate="column", gate_type="f32", per=8192, post=True, pre=True, p=0.1, scale=1.0),
        # a long batch of a wide model, a gate of its own for every sequence
        dict(name="residual long", op="residual", rows=32768, dim=8192, stream="bf16", branch="bf16", weight="bf16",
             gate="sequence", gate_type="bf16", per=2048, post=True, pre=True, p=0.0, scale=0.5),
        # one short sequence of the 1.1B decoder, FP16, a plain residual sum before the next norm
        dict(name="grad few", op="grad", rows=511, dim=2048, stream="f16", branch="f16", weight="f32", gate="none",
             gate_type="f32", per=511, post=False, pre=True, p=0.1, scale=1.0),
        # the micro-batch's backward pass
        dict(name="grad train", op="grad", rows=8192, dim=4096, stream="f32", branch="bf16", weight="f32",
             gate="column", gate_type="f32", per=8192, post=True, pre=True, p=0.1, scale=1.0),
        # the long batch's, with a gate for every element
        dict(name="grad long", op="grad", rows=32768, dim=8192, stream="bf16", branch="bf16", weight="bf16",
             gate="element", gate_type="bf16", per=1, post=True, pre=True, p=0.0, scale=0.5),
        # the router of a small mixture over one short batch, loss and counts alone
        dict(name="balance few", op="balance", rows=256, experts=8, top_k=2, dtype="bf16", ids="i64", groups=1,
             taken=1.0, score="softmax", z=True, gradient=False),
        # packed sequences of uneven lengths, each balanced by itself, padding between them, sigmoid scores
        dict(name="balance ragged", op="balance", rows=16383, experts=160, top_k=6, dtype="f32", ids="i32", groups=13,
             taken=0.8, score="sigmoid", z=False, gradient=True),
        # a large batch over many experts, FP32 logits as routers keep them
        dict(name="balance large", op="balance", rows=262144, experts=256, top_k=8, dtype="f32", ids="i64", groups=1,
             taken=1.0, score="softmax", z=True, gradient=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, its logarithm spread evenly; odd as often as even."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["dropout", "residual", "grad", "balance"])
        any_type = lambda: rng.choice(["f32", "f16", "bf16"])  # noqa: E731
        rows = _log(rng, 1, 65536)
        if op == "dropout":
            c = dict(op=op, rows=rows, dim=_log(rng, 64, 16384), dtype=any_type(), p=round(rng.uniform(0.01, 0.6), 3))
        elif op in ("residual", "grad"):
            branch = any_type()
            gate = rng.choice(["none", "column", "sequence", "element"])
            per = {"none": rows, "column": rows, "sequence": _log(rng, 1, rows), "element": 1}[gate]
            post, pre = rng.choice([(True, True), (True, False), (False, True), (False, False)])
            c = dict(op=op, rows=rows, dim=_log(rng, 64, 16384), stream=rng.choice(["f32", branch]), branch=branch,
                     weight=rng.choice(["f32", branch]), gate=gate, gate_type=rng.choice(["f32", branch]), per=per,
                     post=post, pre=pre, p=rng.choice([0.0, round(rng.uniform(0.01, 0.6), 3)]),
                     scale=rng.choice([1.0, round(rng.uniform(0.1, 2), 3)]))
        else:
            experts = _log(rng, 4, 1024)
            score = rng.choice(["softmax", "sigmoid"])
            rows = _log(rng, 1, 262144)
            c = dict(op=op, rows=rows, experts=experts, top_k=rng.randint(1, min(8, experts)), dtype=any_type(),
                     ids=rng.choice(["i32", "i64"]), groups=rng.choice([1, _log(rng, 1, min(64, rows))]),
                     taken=rng.choice([1.0, round(rng.uniform(0.3, 1), 2)]), score=score,
                     z=score == "softmax" and rng.random() < 0.6, gradient=rng.random() < 0.7)
        if work(c)["bytes"] <= most and c["rows"] * c.get("dim", 1) <= 1 << 28:
            return c


def _gate_rows(c):
    return 0 if c["gate"] == "none" else -(-c["rows"] // c["per"])


def _lengths(c):
    """Rows of a balance case's groups: uneven, together all rows; with several groups one of them is empty."""
    g, n = c["groups"], c["rows"]
    if g == 1:
        return [n]
    share = np.array([1 + (i * 7919 + 104729) % 97 for i in range(g)], np.float64)
    share[g // 2] = 0
    ends = np.rint(np.cumsum(share) / share.sum() * n).astype(np.int64)
    return np.diff(np.concatenate([[0], ends])).tolist()


def _taken(c):
    """Truth values [rows]: of every group (512 rows where there is one group) the trailing rows are padding."""
    n = c["rows"]
    lengths = _lengths(c) if c["groups"] > 1 else [512] * (n // 512) + ([n % 512] if n % 512 else [])
    lengths = np.array(lengths, np.int64)
    at = np.arange(n) - np.repeat(np.cumsum(lengths) - lengths, lengths)
    return at < np.rint(np.repeat(lengths, lengths) * c["taken"])


def _grad_scale(c):
    """The factor that FP16 gradients are stored with, and the optimizer step divides out."""
    if c["op"] == "balance":  # a mean over all tokens: small values
        return 65536.0 if c["dtype"] == "f16" else 1.0
    return 1024.0 if "f16" in (c["stream"], c["branch"]) else 1.0


def work(case):
    c = case
    n = c["rows"]
    if c["op"] == "dropout":
        return {"bytes": 2 * n * c["dim"] * _SIZE[c["dtype"]], "flops": n * c["dim"]}
    if c["op"] == "balance":
        s, taken = _SIZE[c["dtype"]], int(_taken(c).sum())
        moved = taken * (c["experts"] * s + c["top_k"] * _ID_SIZE[c["ids"]]) + n
        if c["gradient"]:
            moved += n * c["experts"] * s
        return {"bytes": moved + c["groups"] * c["experts"] * 8, "flops": taken * c["experts"] * (9 if c["gradient"] else 4)}
    d, s, b = c["dim"], _SIZE[c["stream"]], _SIZE[c["branch"]]
    gate = _gate_rows(c) * d * _SIZE[c["gate_type"]]
    weights = (c["post"] + c["pre"]) * d * _SIZE[c["weight"]]
    if c["op"] == "residual":
        return {"bytes": n * d * (2 * s + b + (b if c["pre"] else 0)) + gate + weights, "flops": n * d * 10}
    # the stream's gradient in and out, the branch and its gradient; with a norm after the sum its input and gradient
    return {"bytes": n * d * (2 * s + 2 * b + (s + b if c["pre"] else 0)) + 2 * gate + 2 * weights,
            "flops": n * d * 24}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    return torch.Generator("cuda").manual_seed(int(seed))


def _normal(shape, std, dtype, g, mean=0.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)


def _chunks(n, width):
    """Row ranges of about 2^25 values each."""
    step = max(1, (1 << 25) // width)
    return [(i, min(n, i + step)) for i in range(0, n, step)]


def _gate_of(s, a, b):
    """The gate's rows for the stream's rows a .. b - 1."""
    c = s["case"]
    if c["gate"] == "column":
        return s["gate"]
    return s["gate"][torch.arange(a, b, device="cuda") // c["per"]]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    n = c["rows"]
    # the generator's key is the run's seed, its offset names the step and the layer
    s = {"case": c, "seed": 0x9E3779B97F4A7C15 ^ int(seed), "offset": (int(seed) % 100003) * 64 + 5}
    if c["op"] == "dropout":
        s["x"] = _normal((n, c["dim"]), 1.0, _DT[c["dtype"]], g)
        s["out"] = torch.empty_like(s["x"])
        return s
    if c["op"] == "balance":
        return _prepare_balance(s, g)
    d, st, br = c["dim"], _DT[c["stream"]], _DT[c["branch"]]
    s["branch"] = _normal((n, d), 1.0, br, g)
    # the stream grows over the layers, and some of its columns are far larger than the others
    s["x"] = _normal((n, d), 3.0, st, g)
    s["x"][:, :: max(1, d // 5)] *= 8
    s["post"] = _normal((d,), 0.1, _DT[c["weight"]], g, 1.0) if c["post"] else None
    s["pre"] = _normal((d,), 0.1, _DT[c["weight"]], g, 1.0) if c["pre"] else None
    s["gate"] = _normal((_gate_rows(c), d), 0.3, _DT[c["gate_type"]], g, 0.5) if c["gate"] != "none" else None
    s["rstd"] = torch.empty((2, n), device="cuda")
    if c["op"] == "residual":
        s["h"] = torch.empty_like(s["x"])
        s["out"] = torch.empty_like(s["branch"]) if c["pre"] else None
        return s
    # what the forward pass left: its sum h, here x, and the reciprocal root mean squares of both norms
    s["h"] = s.pop("x")
    for a, b in _chunks(n, d):
        for i, t in enumerate((s["branch"], s["h"])):
            s["rstd"][i, a:b] = (t[a:b].double().square().mean(1) + _EPS).rsqrt().float()
    std = 1e-3 * _grad_scale(c)
    s["grad_h"] = _normal((n, d), std, st, g)
    s["grad_out"] = _normal((n, d), std, br, g) if c["pre"] else None
    s["grad_x"], s["grad_branch"] = torch.empty_like(s["h"]), torch.empty_like(s["branch"])
    for k in ("gate", "post", "pre"):
        s["grad_" + k] = None if s[k] is None else torch.empty_like(s[k])
    return s


def _prepare_balance(s, g):
    c = s["case"]
    n, e, k = c["rows"], c["experts"], c["top_k"]
    # some experts are favoured, as an unbalanced router's are
    favour = _normal((e,), 0.7, torch.float32, g)
    x = torch.empty((n, e), dtype=_DT[c["dtype"]], device="cuda")
    ids = torch.empty((n, k), dtype=_ID[c["ids"]], device="cuda")
    for a, b in _chunks(n, e):
        x[a:b] = (_normal((b - a, e), 1.0, torch.float32, g) + favour).to(x.dtype)
        ids[a:b] = x[a:b].float().topk(k, 1).indices.to(ids.dtype)
    s["logits"], s["ids"] = x, ids
    s["mask"] = None if c["taken"] == 1.0 else torch.from_numpy(_taken(c)).cuda()
    ends = np.concatenate([[0], np.cumsum(_lengths(c))])
    s["offsets"] = None if c["groups"] == 1 else torch.from_numpy(ends).cuda().to(ids.dtype)
    s["group"] = torch.repeat_interleave(torch.arange(c["groups"], device="cuda"),
                                         torch.tensor(_lengths(c), device="cuda"))
    s["ends"] = ends.tolist()
    s["weights"] = None if c["groups"] == 1 else torch.full((c["groups"],), 1.0 / c["groups"], device="cuda")
    s["total"] = torch.empty((), device="cuda")
    s["loss"] = torch.empty(c["groups"], device="cuda")
    s["counts"] = torch.empty((c["groups"], e), dtype=torch.int32, device="cuda")
    s["tokens"] = torch.empty(c["groups"], dtype=torch.int32, device="cuda")
    s["mean_prob"] = torch.empty((c["groups"], e), device="cuda")
    s["grad"] = torch.empty_like(x) if c["gradient"] else None
    return s


# --------------------------------------------------------------------- run --

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import optimizer_step_dl_amd as ra
    c = s["case"]
    if c["op"] == "dropout":
        ra.radamw_dropout(s["x"], s["out"], ra.dropout_options(c["p"], s["seed"], s["offset"]))
        return s["out"]
    if c["op"] == "balance":
        opts = ra.balance_options(balance_coef=_BALANCE, z_coef=_Z if c["z"] else 0.0, score=c["score"])
        need = ra.radamw_balance_workspace_bytes(c["rows"], c["experts"], c["groups"])
        workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        ra.radamw_balance_loss(s["logits"], s["ids"], opts, s["total"], s["loss"], s["counts"], s["tokens"],
                               s["mean_prob"], workspace, mask=s["mask"], offsets=s["offsets"], weights=s["weights"],
                               grad=s["grad"], grad_scale=_grad_scale(c))
        return _balance_answer(s)
    opts = ra.residual_options(eps=_EPS, residual_scale=c["scale"], p=c["p"], seed=s["seed"], offset=s["offset"])
    shared = dict(gate=s["gate"], rows_per_gate=c["per"], post_weight=s["post"], pre_weight=s["pre"])
    if c["op"] == "residual":
        ra.radamw_residual_norm(s["x"], s["branch"], opts, h=s["h"], out=s["out"], rstd=s["rstd"], **shared)
        return {"h": s["h"], "out": s["out"]} if c["pre"] else {"h": s["h"]}
    need = ra.radamw_residual_grad_workspace_bytes(c["rows"], c["dim"], c["per"])
    workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
    ra.radamw_residual_norm_grad(s["h"], s["branch"], opts, s["rstd"], workspace, grad_h=s["grad_h"],
                                 grad_out=s["grad_out"], grad_x=s["grad_x"], grad_branch=s["grad_branch"],
                                 grad_gate=s["grad_gate"], grad_post_weight=s["grad_post"],
                                 grad_pre_weight=s["grad_pre"], **shared)
    return _grad_answer(s)


def _grad_answer(s):
    out = {"x": s["grad_x"], "branch": s["grad_branch"]}
    out.update({k: s["grad_" + k] for k in ("gate", "post", "pre") if s["grad_" + k] is not None})
    return out


def _balance_answer(s):
    out = {k: s[k] for k in ("total", "loss", "counts", "tokens", "mean_prob")}
    if s["grad"] is not None:
        out["grad"] = s["grad"]
    return out


def _threshold(p):
    return int(math.floor(65536 * p + 0.5))


def _kept(s, a, b, d):
    """Truth values [b - a, d]: which elements of rows a .. b - 1 the generator keeps."""
    groups = -(-d // 8)
    c0 = torch.arange(groups, device="cuda").expand(b - a, groups)
    c1 = torch.arange(a, b, device="cuda")[:, None].expand(b - a, groups)
    c2 = torch.full_like(c0, s["offset"] & _MASK32)
    c3 = torch.full_like(c0, s["offset"] >> 32)
    k0, k1 = s["seed"] & _MASK32, s["seed"] >> 32
    for _ in range(10):
        # a product of two 32-bit numbers wraps in 64 signed bits, its bits stay right
        u, v = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((v >> 32) & _MASK32) ^ c1 ^ k0, v & _MASK32, ((u >> 32) & _MASK32) ^ c3 ^ k1, u & _MASK32)
        k0, k1 = (k0 + 0x9E3779B9) & _MASK32, (k1 + 0xBB67AE85) & _MASK32
    words = torch.stack([c0, c1, c2, c3], -1)
    halves = torch.stack([words & 0xFFFF, words >> 16], -1)
    return (halves.view(b - a, groups * 8) >= _threshold(s["case"]["p"]))[:, :d]


def _keep_factor(p):
    t = _threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def _run_plain(s):
    c = s["case"]
    n = c["rows"]
    if c["op"] == "balance":
        return _plain_balance(s)
    d = c["dim"]
    keep = _keep_factor(c["p"])
    if c["op"] == "dropout":
        for a, b in _chunks(n, d):
            s["out"][a:b] = torch.where(_kept(s, a, b, d), s["x"][a:b].float() * keep, 0).to(s["out"].dtype)
        return s["out"]
    if c["op"] == "residual":
        for a, b in _chunks(n, d):
            u = s["branch"][a:b].float()
            if c["post"]:
                u = u * (u.square().mean(1, keepdim=True) + _EPS).rsqrt() * s["post"].float()
            if c["p"]:
                u = torch.where(_kept(s, a, b, d), u * keep, 0)
            if c["gate"] != "none":
                u = u * _gate_of(s, a, b).float()
            h = s["x"][a:b].float() + c["scale"] * u
            s["h"][a:b] = h.to(s["h"].dtype)
            if c["pre"]:
                h = h * (h.square().mean(1, keepdim=True) + _EPS).rsqrt() * s["pre"].float()
                s["out"][a:b] = h.to(s["out"].dtype)
        return {"h": s["h"], "out": s["out"]} if c["pre"] else {"h": s["h"]}
    sums = {k: torch.zeros(s["grad_" + k].shape, dtype=torch.float64, device="cuda")
            for k in ("gate", "post", "pre") if s["grad_" + k] is not None and not (k == "gate" and c["gate"] == "element")}
    for a, b in _chunks(n, d):
        dh = s["grad_h"][a:b].float()
        if c["pre"]:
            r = s["rstd"][1, a:b, None]
            dn = s["grad_out"][a:b].float()
            hat = s["h"][a:b].float() * r
            sums["pre"] += (dn * hat).sum(0, dtype=torch.float64)
            dn = dn * s["pre"].float()
            dh = dh + r * (dn - hat * (dn * hat).mean(1, keepdim=True))
        s["grad_x"][a:b] = dh.to(s["grad_x"].dtype)
        du = dh * c["scale"]
        if c["p"]:
            kept = _kept(s, a, b, d)
            du = torch.where(kept, du * keep, 0)
        y = s["branch"][a:b].float()
        r = s["rstd"][0, a:b, None]
        hat = y * r
        u = hat * s["post"].float() if c["post"] else y
        if c["gate"] != "none":
            dg = du * u
            if c["gate"] == "element":
                s["grad_gate"][a:b] = dg.to(s["grad_gate"].dtype)
            elif c["gate"] == "column":
                sums["gate"] += dg.sum(0, dtype=torch.float64)
            else:
                sums["gate"].index_add_(0, torch.arange(a, b, device="cuda") // c["per"], dg.double())
            du = du * _gate_of(s, a, b).float()
        if c["post"]:
            sums["post"] += (du * hat).sum(0, dtype=torch.float64)
            du = du * s["post"].float()
            du = r * (du - hat * (du * hat).mean(1, keepdim=True))
        s["grad_branch"][a:b] = du.to(s["grad_branch"].dtype)
    for k, v in sums.items():
        s["grad_" + k].copy_(v)
    return _grad_answer(s)


def _plain_balance(s):
    c = s["case"]
    n, e, k, groups = c["rows"], c["experts"], c["top_k"], c["groups"]
    live = torch.ones(n, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    weights = torch.ones(groups, device="cuda") if s["weights"] is None else s["weights"]
    group = s["group"]

    def sums(v, dtype):
        """Sums over each group's rows, which lie together."""
        return torch.stack([v[a:b].sum(0, dtype=dtype) for a, b in zip(s["ends"], s["ends"][1:])])

    tokens = sums(live, torch.int64)
    hits = torch.zeros((n, e), dtype=torch.uint8, device="cuda")
    hits.scatter_add_(1, s["ids"].long(), live[:, None].expand(n, k).to(torch.uint8))
    counts = sums(hits, torch.int64)
    x = torch.where(live[:, None], s["logits"].float(), 0)
    if c["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        q = (x - top).exp()
        norm = q.sum(1, keepdim=True)
        p = q / norm
        lse = (top + norm.log())[:, 0]
    else:
        q = 1 / (1 + (-x).exp())
        norm = q.sum(1, keepdim=True)
        p = q / norm
    t = tokens.clamp(min=1).double()
    mean = sums(torch.where(live[:, None], p, 0), torch.float64) / t[:, None]
    share = _BALANCE * e / k * counts / t[:, None]
    loss = (share * mean).sum(1)
    if c["z"]:
        loss = loss + _Z * sums(torch.where(live, lse, 0).square(), torch.float64) / t
    out = {"total": (loss * weights).sum().float(), "loss": loss.float(), "counts": counts.int(),
           "tokens": tokens.int(), "mean_prob": mean.float()}
    if c["gradient"]:
        up = weights.double() * _grad_scale(c) / t
        cost = (share * up[:, None]).float()[group]
        inner = (cost * p).sum(1, keepdim=True)
        if c["score"] == "softmax":
            grad = p * (cost - inner)
            if c["z"]:
                grad = grad + 2 * _Z * up.float()[group][:, None] * lse[:, None] * p
        else:
            grad = p * (1 - q) * (cost - inner)
        out["grad"] = torch.where(live[:, None], grad, 0).to(s["logits"].dtype)
    return out


# ------------------------------------------------------------------- exact --

def _high_low(m, v):
    """The high and low 32 bits of m * v, both below 2^32, by products of 16 and 32 bits."""
    low, high = v * (m & 0xFFFF), v * (m >> 16)
    total = high + (low >> 16)
    return total >> 16, ((total & 0xFFFF) << 16) | (low & 0xFFFF)


def _dropped(s, a, b, d):
    """Truth values [b - a, d]: which elements the generator drops, number by number."""
    column = torch.arange(-(-d // 8), device="cuda")[None, :]
    row = torch.arange(a, b, device="cuda")[:, None]
    word = [column + 0 * row, row + 0 * column, torch.tensor(s["offset"] % 2 ** 32, device="cuda"),
            torch.tensor(s["offset"] // 2 ** 32, device="cuda")]
    for r in range(10):
        key = [(s["seed"] % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        h0, l0 = _high_low(0xD2511F53, word[0])
        h1, l1 = _high_low(0xCD9E8D57, word[2])
        word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
    out = torch.empty((b - a, column.numel() * 8), dtype=torch.bool, device="cuda")
    for j in range(8):
        number = word[j // 2] // 65536 if j % 2 else word[j // 2] % 65536
        out[:, j::8] = number < _threshold(s["case"]["p"])
    return out[:, :d]


def _norm64(v):
    return v / torch.sqrt(torch.mean(v * v, 1, keepdim=True) + _EPS)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    n = c["rows"]
    if c["op"] == "balance":
        return _exact_balance(s)
    d = c["dim"]
    left = 1 - _threshold(c["p"]) / 65536
    ends = _chunks(n, 2 * d)
    if c["op"] == "dropout":
        out = torch.empty((n, d), dtype=torch.float64, device="cuda")
        for a, b in ends:
            out[a:b] = s["x"][a:b].double().div_(left).masked_fill_(_dropped(s, a, b, d), 0)
        return out

    def term(a, b, y, gate, post):
        """What the block adds to rows a .. b - 1 of the stream."""
        u = _norm64(y) * post if c["post"] else y
        if c["p"]:
            u = (u / left).masked_fill(_dropped(s, a, b, d), 0)
        if c["gate"] == "column":
            u = u * gate
        elif c["gate"] != "none":
            u = u * gate.index_select(0, torch.div(torch.arange(a, b, device="cuda"), c["per"], rounding_mode="floor")
                                      - a // c["per"])
        return float(np.float32(c["scale"])) * u

    def gates(a, b):
        if c["gate"] == "none":
            return None
        return s["gate"].double() if c["gate"] == "column" else s["gate"][a // c["per"]:(b - 1) // c["per"] + 1].double()

    post = s["post"].double() if c["post"] else None
    pre = s["pre"].double() if c["pre"] else None
    if c["op"] == "residual":
        out = {"h": torch.empty((n, d), dtype=torch.float64, device="cuda")}
        if c["pre"]:
            out["out"] = torch.empty_like(out["h"])
        for a, b in ends:
            h = s["x"][a:b].double() + term(a, b, s["branch"][a:b].double(), gates(a, b), post)
            out["h"][a:b] = h
            if c["pre"]:
                out["out"][a:b] = _norm64(h) * pre
        return out
    out = {k: torch.zeros(s["grad_" + k].shape, dtype=torch.float64, device="cuda")
           for k in ("x", "branch", "gate", "post", "pre") if s["grad_" + k] is not None}
    for a, b in ends:
        up = s["grad_h"][a:b].double()
        if c["pre"]:
            h = s["h"][a:b].double().requires_grad_()
            w = pre.clone().requires_grad_()
            dh, dw = torch.autograd.grad(_norm64(h) * w, (h, w), s["grad_out"][a:b].double())
            up = up + dh
            out["pre"] += dw
        out["x"][a:b] = up
        leaves = {"branch": s["branch"][a:b].double(), "gate": gates(a, b), "post": None if post is None else post.clone()}
        leaves = {k: v.requires_grad_() for k, v in leaves.items() if v is not None}
        got = torch.autograd.grad(term(a, b, leaves["branch"], leaves.get("gate"), leaves.get("post")),
                                  list(leaves.values()), up)
        got = dict(zip(leaves, got))
        out["branch"][a:b] = got["branch"]
        if c["post"]:
            out["post"] += got["post"]
        if c["gate"] == "column":
            out["gate"] += got["gate"]
        elif c["gate"] != "none":
            out["gate"][a // c["per"]:(b - 1) // c["per"] + 1] += got["gate"]
    return out


def _exact_balance(s):
    c = s["case"]
    ends = np.concatenate([[0], np.cumsum(_lengths(c))])
    keep = torch.from_numpy(_taken(c)).cuda()
    out = {"total": torch.zeros((), dtype=torch.float64, device="cuda"), "loss": [], "counts": [], "tokens": [],
           "mean_prob": []}
    grad = torch.zeros((c["rows"], c["experts"]), dtype=torch.float64, device="cuda")
    for i in range(c["groups"]):
        rows = torch.nonzero(keep[ends[i]:ends[i + 1]])[:, 0] + int(ends[i])
        t = len(rows)
        z = s["logits"][rows].double().requires_grad_()
        counts = torch.bincount(s["ids"][rows].reshape(-1).long(), minlength=c["experts"])
        if c["score"] == "softmax":
            p = torch.softmax(z, 1)
        else:
            p = torch.sigmoid(z)
            p = p / p.sum(1, keepdim=True)
        mean = p.sum(0) / max(t, 1)
        loss = _BALANCE * torch.dot(counts.double() * (c["experts"] / (c["top_k"] * max(t, 1))), mean)
        if c["z"]:
            loss = loss + _Z * torch.logsumexp(z, 1).square().sum() / max(t, 1)
        w = 1.0 if s["weights"] is None else float(s["weights"][i])
        out["total"] += w * loss.detach()
        out["loss"].append(loss.detach())
        out["counts"].append(counts.int())
        out["tokens"].append(torch.tensor(t, dtype=torch.int32, device="cuda"))
        out["mean_prob"].append(mean.detach())
        if c["gradient"]:
            grad[rows] = w * _grad_scale(c) * torch.autograd.grad(loss, z)[0]
    for k in ("loss", "counts", "tokens", "mean_prob"):
        out[k] = torch.stack(out[k])
    if c["gradient"]:
        out["grad"] = grad
    return out
