"""GPU tests of the block operators' autograd forms, alone and together with
the vocabulary operators and FusedAdamW as a training loop uses them.

The autograd forms only hand tensors on, so their gradients are compared with
the binding's, bit for bit; whole steps with the same model in plain torch in
64 bits.  Those agree to 1e-4 of a gradient's largest value: the longest chain
of a model here is some ten operators of at most 130 FP32 roundings each, 2^-24
* 1300 = 8e-5 where nothing cancels beyond the largest value."""
import threading

import pytest
import torch

import optimizer_step_dl_amd as ra
from block_helpers import Residual, dropout as plain_dropout, keep_factor, keep_mask
from gpu_helpers import DEV, announce
from optimizer_step_dl_amd.functional import balance_loss, dropout, embedding, policy_loss, residual_norm
from optimizer_step_dl_amd.optim import FusedAdamW
from vocab_helpers import close

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def leaf(shape, dtype, seed, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen(seed)) * std + mean).to(dtype).to(DEV).requires_grad_()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_dropout_autograd(dtype):
    announce(f"functional dropout {dtype}")
    x = leaf((3, 5, 24), dtype, 1)
    g = torch.randn((3, 5, 24), generator=gen(2)).to(dtype)
    out = dropout(x, 0.4, seed=3, offset=4, first_row=5)
    out.backward(g.to(DEV))
    for got, t in ((out, x), (x.grad, g)):
        ref, slack = plain_dropout(t.detach().cpu().reshape(15, 24), 0.4, 3, 4, 5)
        close(got.reshape(15, 24), ref, slack, "dropout")
    # a slice of a wider tensor, and gradients that torch hands over expanded or transposed
    wide = leaf((6, 40), dtype, 3)
    y = dropout(wide[:, 3:27], 0.4, seed=3, offset=4)
    keep = keep_mask(6, 24, 0.4, 3, 4)
    y.sum().backward()
    assert torch.equal((wide.grad[:, 3:27] != 0).cpu(), keep) and not wide.grad[:, :3].any()
    x.grad = None
    dropout(x.transpose(0, 1), 0.4, seed=3).transpose(0, 1).mul(g.to(DEV)).sum().backward()
    assert torch.equal((x.grad.transpose(0, 1).reshape(15, 24) != 0).cpu(), keep_mask(15, 24, 0.4, 3, 0))


RESIDUAL = [dict(gate="one", post=True, pre=True, p=0.3), dict(gate="batch", post=True, pre=True, p=0.0),
            dict(gate="all", post=False, pre=True, p=0.3), dict(gate=None, post=True, pre=False, p=0.0),
            dict(gate="one", post=False, pre=False, p=0.5), dict(gate=None, post=False, pre=True, p=0.0)]


@pytest.mark.parametrize("stream,branch", [(F32, F32), (F32, BF16), (F16, F16)])
@pytest.mark.parametrize("kw", RESIDUAL, ids=str)
def test_residual_autograd(kw, stream, branch):
    announce(f"functional residual {kw} {stream} {branch}")
    b, s, d = 4, 6, 40
    n = b * s
    x, y = leaf((b, s, d), stream, 1), leaf((b, s, d), branch, 2)
    shape = {"one": (d,), "batch": (b, 1, d), "all": (b, s, d), None: None}[kw["gate"]]
    gate = None if shape is None else leaf(shape, branch, 3, 0.3, 1.0)
    post = leaf((d,), F32, 4, 0.1) if kw["post"] else None
    pre = leaf((d,), F32, 5, 0.1) if kw["pre"] else None
    dh, dout = leaf((b, s, d), stream, 6).detach(), leaf((b, s, d), branch, 7).detach()
    args = dict(eps=1e-5, residual_scale=0.5, weight_offset=1.0, p=kw["p"], seed=8, offset=9, first_row=10)
    res = residual_norm(x, y, gate=gate, post_weight=post, pre_weight=pre, **args)
    h, out = res if kw["pre"] else (res, None)
    assert h.shape == x.shape and h.dtype == stream and (out is None or out.dtype == branch)
    per = {"one": n, "batch": s, "all": 1, None: None}[kw["gate"]]
    # the binding by hand
    opts = ra.residual_options(**args)
    two = lambda t: None if t is None else t.detach().reshape(-1, d)  # noqa: E731
    one = lambda t: None if t is None else t.detach()  # noqa: E731
    shared = dict(gate=two(gate), rows_per_gate=per, post_weight=one(post), pre_weight=one(pre))
    h2 = torch.empty((n, d), dtype=stream, device=DEV)
    out2 = torch.empty((n, d), dtype=branch, device=DEV) if kw["pre"] else None
    rstd = torch.empty((2, n), device=DEV)
    ra.radamw_residual_norm(two(x), two(y), opts, h=h2, out=out2, rstd=rstd, **shared)
    assert torch.equal(h.view(n, d), h2) and (out is None or torch.equal(out.view(n, d), out2))
    ws = torch.empty(ra.radamw_residual_grad_workspace_bytes(n, d, per or 1), dtype=torch.uint8, device=DEV)

    def by_hand(dh, dout):
        like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
        g = dict(grad_x=like(h2), grad_branch=like(two(y)), grad_gate=like(two(gate)), grad_post_weight=like(one(post)),
                 grad_pre_weight=like(one(pre)) if dout is not None else None)
        kw2 = dict(shared, pre_weight=one(pre) if dout is not None else None)
        ra.radamw_residual_norm_grad(h2, two(y), opts, rstd, ws, grad_h=two(dh), grad_out=two(dout), **kw2, **g)
        return list(g.values())

    leaves = [x, y, gate, post, pre]
    both = ([(dh, dout), (dh, None), (None, dout)] if kw["pre"] else [(dh, None)])
    for gh, go in both:
        for t in leaves:
            if t is not None:
                t.grad = None
        roots = [(t, g) for t, g in ((h, gh), (out, go)) if g is not None]
        torch.autograd.backward([t for t, _ in roots], [g for _, g in roots], retain_graph=True)
        for t, want in zip(leaves, by_hand(gh, go)):
            assert (t is None or t.grad is None) == (want is None)
            if want is not None:
                assert torch.equal(t.grad.reshape(want.shape), want)


def test_residual_of_views_and_what_takes_no_gradient():
    """Columns of a wider tensor, a transposed gate, weights that are frozen;
    an output that nothing is asked of."""
    announce("functional residual views")
    n, d = 20, 32
    wide = leaf((n, 3 * d), F32, 1)
    x, y = wide[:, :d], wide[:, d:2 * d]
    gate = leaf((d, n), F32, 2)
    w = torch.ones(d, device=DEV)
    h, out = residual_norm(x, y, gate=gate.t(), post_weight=w, pre_weight=w)
    r = Residual(x.detach().cpu(), y.detach().cpu(), gate.detach().cpu().t(), 1, w.cpu(), w.cpu())
    leaves = [r.x.requires_grad_(), r.y.requires_grad_(), r.g.requires_grad_()]
    for power in (2, 3):
        wide.grad = gate.grad = None
        out.pow(power).sum().backward(retain_graph=True)
        f = r.forward()
        want = torch.autograd.grad(f["out"][0].pow(power).sum(), leaves, retain_graph=True)
        got = [wide.grad[:, :d].cpu(), wide.grad[:, d:2 * d].cpu(), gate.grad.t().cpu()]
        # The sum of squares of a norm is constant but for eps: its gradient D = r_h (q - hat_h mean(q hat_h)) with q =
        # 2 out is a difference of two equal terms.  So the bound of 1e-4 is of the terms, r_h |q|, times what the branch
        # makes of D: u for the gate, and for y gate r_b (1 + hat_b^2), as |hat_b mean(s hat_b)| <= max |s| hat_b^2.
        with torch.no_grad():
            q = float((power * f["out"][0].pow(power - 1).abs() * f["rstd_h"][0][:, None]).max())
            rb, hat = float(f["rstd_branch"][0].max()), float((r.y * f["rstd_branch"][0][:, None]).abs().max())
            sizes = [q, q * float(r.g.abs().max()) * rb * (1 + hat * hat), q * hat]
        for v, ref, size in zip(got, want, sizes):
            limit = size if power == 2 else float(ref.abs().max())
            assert float((v - ref).abs().max()) <= 1e-4 * limit
        assert not wide.grad[:, 2 * d:].any()
    (residual_norm(x, y, pre_weight=w)[0] * 0 + h.detach()).sum().backward()


def test_first_norm_and_evaluation():
    announce("functional first norm")
    x, w = leaf((2, 7, 48), F32, 1), leaf((48,), F32, 2, 0.1, 1.0)
    out = residual_norm(x, None, pre_weight=w, out_dtype=BF16)
    assert out.dtype == BF16 and out.shape == x.shape
    out.float().sum().backward()
    assert x.grad is not None and w.grad is not None
    y = leaf((2, 7, 48), BF16, 3)
    a, b = residual_norm(x, y, pre_weight=w, p=0.5, seed=1, training=False)
    c, d = residual_norm(x, y, pre_weight=w)
    assert torch.equal(a, c) and torch.equal(b, d)
    empty = residual_norm(x[:0], y[:0], pre_weight=w, post_weight=w)
    (empty[0].sum() + empty[1].sum()).backward()


@pytest.mark.parametrize("score,z", [("softmax", 0.01), ("sigmoid", 0.0)])
def test_balance_autograd(score, z):
    announce(f"functional balance {score}")
    x = leaf((6, 50, 24), F32, 1)
    ids = torch.randint(0, 24, (6, 50, 3), generator=gen(2)).to(DEV)
    mask = (torch.rand((6, 50), generator=gen(3)) < 0.7).to(DEV)
    off = torch.tensor([0, 100, 250, 300], device=DEV, dtype=torch.int32)  # of another type than the ids
    total, loss, counts, mean = balance_loss(x, ids, mask=mask, offsets=off, z_coef=z, score=score, balance_coef=0.1)
    assert not loss.requires_grad and not counts.requires_grad and not mean.requires_grad and counts.dtype == torch.int32
    (total * 12.0).backward()
    got = [torch.empty((), device=DEV), torch.empty(3, device=DEV), torch.empty((3, 24), dtype=torch.int32, device=DEV),
           torch.empty(3, dtype=torch.int32, device=DEV), torch.empty((3, 24), device=DEV)]
    grad = torch.empty((300, 24), device=DEV)
    ws = torch.empty(ra.radamw_balance_workspace_bytes(300, 24, 3), dtype=torch.uint8, device=DEV)
    w = torch.full((3,), 1 / 3, device=DEV)
    o = ra.balance_options(0.1, z, score)
    rows = x.detach().view(300, 24)
    ra.radamw_balance_loss(rows, ids.view(300, 3), o, *got, ws, mask=mask.view(-1), offsets=off.long(), weights=w)
    ra.radamw_balance_grad(rows, 3, o, got[2], got[3], grad, mask=mask.view(-1), offsets=off.long(), weights=w,
                           upstream=torch.tensor(12.0, device=DEV))
    assert torch.equal(total, got[0]) and torch.equal(loss, got[1]) and torch.equal(counts, got[2])
    assert torch.equal(mean, got[4]) and torch.equal(x.grad.view(300, 24), grad)


def test_second_derivatives_and_capture_are_refused():
    announce("functional refusals")
    x, w = leaf((4, 16), F32, 1), leaf((16,), F32, 2)
    for f in (lambda: dropout(x, 0.5, seed=1), lambda: residual_norm(x, x, pre_weight=w)[1],
              lambda: balance_loss(x, torch.zeros((4, 1), dtype=torch.int64, device=DEV))[0]):
        out = f()
        grad, = torch.autograd.grad(out.sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            grad.sum().backward()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
            for f in (lambda: dropout(x, 0.5, seed=1), lambda: residual_norm(x, x, pre_weight=w),
                      lambda: balance_loss(x, torch.zeros((4, 1), dtype=torch.int64, device=DEV))):
                with pytest.raises(ra.RadamwError):
                    f()
            y = x.detach() * 2  # a graph of torch's own work goes on
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, x.detach() * 2)


def test_streams_and_threads():
    """Calls on two streams at once share nothing; a backward pass on another
    thread runs on its forward pass's stream."""
    announce("functional streams")
    x = [leaf((700, 264), BF16, i) for i in (1, 2)]
    w = [leaf((264,), F32, i, 0.1, 1.0) for i in (3, 4)]

    def work(i):
        h, out = residual_norm(x[i], x[i] * 2, post_weight=w[i], pre_weight=w[i], p=0.2, seed=i)
        return h.float().sum() + out.float().square().sum()

    want = []
    for i in range(2):
        want.append(torch.autograd.grad(work(i), [x[i], w[i]]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        totals, got = [], [None, None]
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                totals.append(work(i))
        torch.cuda.synchronize()

        def back(i):
            with torch.cuda.stream(streams[i]):
                got[i] = torch.autograd.grad(totals[i], [x[i], w[i]])

        threads = [threading.Thread(target=back, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


class Model:
    """Two blocks around a stream, a router of four experts, tied to nothing:
    the parameters by name, and one step's total."""

    rows, dim, vocab, experts = 48, 64, 101, 4

    def __init__(self):
        d = self.dim
        g = gen(5)
        self.values = {"table": torch.randn((self.vocab, d), generator=g) * 0.5}
        for i in range(2):
            self.values[f"block{i}"] = torch.randn((d, d), generator=g) / d ** 0.5
            self.values[f"post{i}"] = 1 + 0.1 * torch.randn(d, generator=g)
            self.values[f"gate{i}"] = 0.5 + 0.1 * torch.randn(d, generator=g)
        for i in range(3):
            self.values[f"norm{i}"] = 1 + 0.1 * torch.randn(d, generator=g)
        self.values["router"] = torch.randn((d, self.experts), generator=g) / d ** 0.5
        self.values["head"] = torch.randn((d, self.vocab), generator=g) / d ** 0.5
        self.ids = torch.randint(0, self.vocab, (self.rows,), generator=g)
        self.labels = torch.randint(0, self.vocab, (self.rows,), generator=g)
        self.labels[:5] = -100
        self.mask = self.labels >= 0
        self.adv = torch.randn(self.rows, generator=g)

    def own(self, v, step):
        x = dropout(embedding(self.ids.to(DEV), v["table"]), 0.1, seed=7, offset=8 * step)
        y = residual_norm(x, None, pre_weight=v["norm0"])
        for i in range(2):
            x, y = residual_norm(x, (y @ v[f"block{i}"]).tanh(), post_weight=v[f"post{i}"], gate=v[f"gate{i}"],
                                 pre_weight=v[f"norm{i + 1}"], residual_scale=0.7, p=0.2, seed=7, offset=8 * step + i + 1)
        routed = y @ v["router"]
        chosen = routed.detach().topk(2, 1).indices
        balance, _, counts, _ = balance_loss(routed, chosen, mask=self.mask.to(DEV), z_coef=0.1, balance_coef=0.5)
        total, *_ = policy_loss(y @ v["head"], self.labels.to(DEV), self.adv.to(DEV))
        return total + balance, chosen, counts

    def plain(self, v, step, chosen):
        n, d = self.rows, self.dim

        def drop(t, p, offset):
            return torch.where(keep_mask(n, d, p, 7, offset), t * keep_factor(p), 0.0)

        def norm(t, w):
            return t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w

        x = drop(v["table"][self.ids], 0.1, 8 * step)
        y = norm(x, v["norm0"])
        for i in range(2):
            u = norm((y @ v[f"block{i}"]).tanh(), v[f"post{i}"])
            x = x + 0.7 * v[f"gate{i}"] * drop(u, 0.2, 8 * step + i + 1)
            y = norm(x, v[f"norm{i + 1}"])
        z = (y @ v["router"])[self.mask]
        t = len(z)
        counts = torch.bincount(chosen[self.mask].reshape(-1), minlength=self.experts)
        balance = 0.5 * self.experts / (2 * t) * (counts * z.softmax(1).mean(0)).sum() + 0.1 * z.logsumexp(1).square().mean()
        lp = (y @ v["head"]).log_softmax(1)[torch.arange(n), self.labels.clamp(min=0)]
        ratio = (lp - lp.detach()).exp()
        return -(ratio * self.adv.double())[self.mask].mean() + balance, counts


def test_gradients_of_a_model():
    """Lookup, dropout, norms with gates, a router's balance loss and the
    policy loss together, against the same model in 64 bits."""
    announce("functional model")
    m = Model()
    own = {k: v.to(DEV).requires_grad_() for k, v in m.values.items()}
    ref = {k: v.double().requires_grad_() for k, v in m.values.items()}
    total, chosen, counts = m.own(own, 3)
    want, want_counts = m.plain(ref, 3, chosen.cpu())
    assert torch.equal(counts[0].cpu().long(), want_counts)
    assert abs(float(total.detach()) - float(want.detach())) <= 1e-4 * abs(float(want.detach()))
    total.backward()
    want.backward()
    for k in own:
        err = float((own[k].grad.cpu() - ref[k].grad).abs().max())
        assert err <= 1e-4 * float(ref[k].grad.abs().max()), (k, err)


def test_training_steps():
    """Steps of FusedAdamW over one flattened bucket, with a loss scale and
    clipping: every parameter follows the gradients that are found without
    them, and a step runs like the one before it."""
    announce("functional training steps")
    m = Model()
    own = {k: v.to(DEV).requires_grad_() for k, v in m.values.items()}
    opt = FusedAdamW(list(own.values()), lr=1e-3, weight_decay=0.0, flatten=True)
    for step in range(3):
        grads = torch.autograd.grad(m.own(own, step)[0], list(own.values()))
        before = [v.detach().clone() for v in own.values()]
        opt.zero_grad()
        (m.own(own, step)[0] * 256.0).backward()
        got = [v.grad.clone() for v in own.values()]
        for g, s in zip(grads, got):  # a power of two scales every rounding
            assert float((s / 256.0 - g).abs().max()) <= 1e-5 * float(g.abs().max())
        opt.step(gradient_scale=256.0)
        assert all(bool(v.isfinite().all()) and not torch.equal(v, b) for v, b in zip(own.values(), before))
