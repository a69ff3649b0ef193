"""GPU tests of the autograd forms, alone and together with FusedAdamW as a
training loop uses them."""
import threading

import pytest
import torch

import optimizer_step_dl_amd as ra
from gpu_helpers import DEV, announce
from optimizer_step_dl_amd.functional import embedding, policy_loss, preference_loss
from optimizer_step_dl_amd.optim import FusedAdamW
from vocab_helpers import U, Rows, close, embedding_grad, policy

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_embedding_autograd(dtype):
    announce(f"functional embedding {dtype}")
    rows, dim = 50, 24
    table = torch.randn((rows, dim), generator=gen(1)).to(dtype)
    ids = torch.randint(0, rows, (3, 7), generator=gen(2))
    g = torch.randn((3, 7, dim), generator=gen(3)).to(dtype)
    t = table.to(DEV).requires_grad_()
    out = embedding(ids.to(DEV), t, scale=3.0, padding_id=4)
    assert out.shape == (3, 7, dim) and torch.equal(out.cpu(), (table.float() * 3.0)[ids].to(dtype))
    out.backward(g.to(DEV))
    ref, slack = embedding_grad(g.reshape(-1, dim), ids, rows, 3.0, 4, None)
    close(t.grad, ref, slack, "table gradient")
    # a gradient that torch hands over expanded or transposed
    t.grad = None
    embedding(ids.to(DEV), t, scale=3.0).sum().backward()
    ref, slack = embedding_grad(torch.ones(21, dim), ids, rows, 3.0, None, None)
    close(t.grad, ref, slack, "gradient of a sum")
    t.grad = None
    (embedding(ids.to(DEV), t).transpose(0, 2) * g.to(DEV).transpose(0, 2)).sum().backward()
    ref, slack = embedding_grad(g.reshape(-1, dim), ids, rows, 1.0, None, None)
    close(t.grad, ref, slack, "transposed gradient")


def test_embedding_grad_buffer_and_copy():
    """The buffer takes the rows that occur, twice when the table is used
    twice, and torch no gradient; the copy is what is read."""
    announce("functional embedding buffer")
    rows, dim = 30, 16
    master = torch.randn((rows, dim), generator=gen(1)).to(DEV).requires_grad_()
    copy = master.detach().to(BF16) * 2
    buffer = torch.ones((rows, dim), dtype=F16, device=DEV)
    a, b = (torch.randint(0, rows, (9,), generator=gen(s)) for s in (4, 5))
    x = embedding(a.to(DEV), master, model_copy=copy, grad_buffer=buffer)
    y = embedding(b.to(DEV), master, model_copy=copy, grad_buffer=buffer)
    assert x.dtype == BF16 and torch.equal(x, copy[a.to(DEV)])
    (x.float().sum() + 2 * y.float().sum()).backward()
    assert master.grad is None
    want = torch.ones(rows, dim)
    want.index_add_(0, a, torch.ones(9, dim)).index_add_(0, b, torch.full((9, dim), 2.0))
    assert torch.equal(buffer.float().cpu(), want)  # small whole numbers: exact


def test_embedding_of_a_computed_table():
    """A table that is itself a result (a tied, scaled or cast one)."""
    announce("functional computed table")
    leaf = torch.randn((9, 5), generator=gen(1)).to(DEV).requires_grad_()
    ids = torch.tensor([3, 3, 8], device=DEV)
    embedding(ids, leaf * 2).sum().backward()
    want = torch.zeros(9, 5)
    want[3], want[8] = 4, 2
    assert torch.equal(leaf.grad.cpu(), want)
    leaf.grad = None
    embedding(ids, leaf.to(BF16)).sum().backward()
    assert leaf.grad.dtype == F32 and torch.equal(leaf.grad.cpu(), want / 2)


def test_embedding_16_bit_gradient_of_a_master():
    announce("functional embedding grad_dtype")
    table = torch.zeros((8, 4), device=DEV, requires_grad=True)
    if not hasattr(table, "grad_dtype"):
        pytest.skip("this torch keeps no 16-bit gradient on an FP32 tensor")
    table.grad_dtype = BF16
    embedding(torch.tensor([1, 1, 7], device=DEV), table, out_dtype=BF16).sum().backward()
    assert table.grad.dtype == BF16
    assert table.grad[:, 0].tolist() == [0, 2, 0, 0, 0, 0, 0, 1]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_policy_autograd(dtype):
    announce(f"functional policy {dtype}")
    shape, vocab = (4, 11), 130
    x = (2 * torch.randn(shape + (vocab,), generator=gen(6))).to(dtype)
    labels = torch.randint(0, vocab, shape, generator=gen(7))
    labels[:, :3] = -100
    flat = labels.reshape(-1)
    taken = flat >= 0
    r = Rows(x.reshape(-1, vocab), flat, taken)
    adv = torch.randn(shape, generator=gen(8))
    old = (r.logp + 0.02).reshape(shape).float()
    ref = (r.logp - 0.3).reshape(shape).float()
    xd = x.to(DEV).requires_grad_()
    total, loss, logp = policy_loss(xd, labels.to(DEV), adv.to(DEV), old_logp=old.to(DEV), ref_logp=ref.to(DEV),
                                    kl_coef=0.2)
    assert loss.shape == shape and not loss.requires_grad and not logp.requires_grad
    (total * -32.0).backward()
    w = taken.float() / taken.sum()
    want, want_err, coef, coef_err = policy(r, old.reshape(-1), ref.reshape(-1), adv.reshape(-1), w, 0.2, 0.2, 0.2)
    ww = torch.where(taken, w.double(), 0.0)
    # the mean's weights are rounded: U more
    close(total, (want * ww).sum(), ((want_err + 2 * U * want.abs()) * ww).sum(), "total")
    g, slack = r.grad(coef, coef_err + 2 * U * coef.abs(), -32.0)
    close(xd.grad, g.reshape(x.shape), (slack + 2 * U * g.abs()).reshape(x.shape), "gradient")


def test_losses_of_views_and_none():
    """Logits that are a slice of a padded vocabulary; a total that nothing
    is asked of."""
    announce("functional views")
    wide = torch.randn((6, 40), generator=gen(9)).to(DEV)
    labels = torch.randint(0, 33, (6,), generator=gen(10)).to(DEV)
    adv = torch.ones(6, device=DEV)
    a = wide[:, :33].clone().requires_grad_()
    b = wide.clone().requires_grad_()
    policy_loss(a, labels, adv)[0].backward()
    policy_loss(b[:, :33], labels, adv)[0].backward()
    assert torch.equal(a.grad, b.grad[:, :33]) and bool((b.grad[:, 33:] == 0).all())
    c = wide.t().contiguous().t().requires_grad_()
    policy_loss(c[:, :33], labels, adv)[0].backward()
    assert torch.equal(a.grad, c.grad[:, :33])
    total, loss, _ = policy_loss(a, labels, adv)
    (total.detach() + loss.sum() + 0 * a.sum()).backward()  # no part of the loss asks for a gradient


def test_preference_autograd():
    announce("functional preference")
    n, vocab = 12, 50
    x = torch.randn((n, vocab), generator=gen(11), dtype=torch.float64)
    labels = torch.randint(0, vocab, (n,), generator=gen(12))
    labels[4] = -100
    offsets = [0, 3, 6, 10, 12]
    ref = torch.tensor([-11.0, -12.0, -14.0, -9.0])
    x32 = x.float()
    z = x32.double().requires_grad_()
    lp = z.log_softmax(1).gather(1, labels.clamp(min=0)[:, None])[:, 0] * (labels >= 0)
    m = torch.stack([lp[offsets[i]:offsets[i + 1]].sum() for i in range(4)]) - ref
    h = 0.3 * (m[:2] - m[2:])
    ls = torch.nn.functional.logsigmoid
    want = (-0.9 * ls(h) - 0.1 * ls(-h)).mean()
    want.backward()
    xd = x32.to(DEV).requires_grad_()
    total, loss, seq = preference_loss(xd, labels.to(DEV), torch.tensor(offsets, device=DEV, dtype=torch.int32),
                                       ref.to(DEV), beta=0.3, label_smoothing=0.1)
    total.backward()
    r = Rows(x32, labels, labels >= 0)
    err = 0.3 * torch.stack([torch.where(r.taken, r.err, 0.0)[offsets[i]:offsets[i + 1]].sum() for i in range(4)])
    close(total, want.detach(), err.sum(), "total")
    coef_err = 0.3 * 0.25 * err.sum() / 2 + U
    g, slack = r.grad(torch.where(r.taken, 0.3, 0.0).double(), coef_err.expand(n), 1.0)
    close(xd.grad, z.grad, slack + 4 * U * z.grad.abs(), "gradient")


def test_second_derivative_is_refused():
    announce("functional double backward")
    x = torch.randn((3, 9), device=DEV, requires_grad=True)
    total, *_ = policy_loss(x, torch.zeros(3, dtype=torch.int64, device=DEV), torch.ones(3, device=DEV))
    g, = torch.autograd.grad(total, x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_backward_on_the_forward_stream():
    """A forward pass on a side stream: its backward runs there too, also
    when called from another thread."""
    announce("functional streams")
    side = torch.cuda.Stream()
    table = torch.randn((500, 64), device=DEV).requires_grad_()
    ids = torch.randint(0, 500, (9000,), device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = embedding(ids, table)
        total, *_ = policy_loss(out, ids % 64, torch.ones(9000, device=DEV))
    t = threading.Thread(target=total.backward)
    t.start()
    t.join()
    torch.cuda.synchronize()
    got = table.grad.clone()
    table.grad = None
    del out, total  # the graph that lives on the side stream
    total, *_ = policy_loss(embedding(ids, table), ids % 64, torch.ones(9000, device=DEV))
    total.backward()
    assert torch.equal(got, table.grad)


def test_capture_is_refused():
    announce("functional capture")
    table = torch.randn((10, 8), device=DEV, requires_grad=True)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.capture_begin(capture_error_mode="relaxed")
        try:
            with pytest.raises(ra.RadamwError):
                embedding(ids, table)
            ids.add_(0)
        finally:
            graph.capture_end()
    torch.cuda.synchronize()


# ------------------------------------------------- together with the step --

@pytest.mark.parametrize("kind", ["policy", "preference"])
@pytest.mark.parametrize("grad_dtype", [F32, F16])
def test_training_steps(kind, grad_dtype):
    """Lookup from the flattened bucket's table, a linear layer, the loss,
    backward with a loss scale into the bucket, a fused step with clipping:
    every step's gradients are those of a 64-bit plain model at the
    parameters of that step, the report's norm is theirs, and an infinite
    advantage (or weight) skips the step."""
    announce(f"training {kind} {grad_dtype}")
    rows, dim, vocab, n, scale = 60, 32, 40, 48, 256.0
    table = torch.nn.Parameter(0.1 * torch.randn((rows, dim), generator=gen(1)).to(DEV))
    head = torch.nn.Parameter(0.3 * torch.randn((vocab, dim), generator=gen(2)).to(DEV))
    if grad_dtype != F32 and not hasattr(table, "grad_dtype"):
        pytest.skip("this torch keeps no 16-bit gradient on an FP32 parameter")
    opt = FusedAdamW([{"params": [table]}, {"params": [head], "weight_decay": 0.0}], lr=1e-2, fused_step=True,
                     max_grad_norm=1.0, hierarchical_stats=True, flatten=True, flatten_grad_dtype=grad_dtype)
    ids = torch.randint(0, rows, (n,), generator=gen(3))
    ids[-6:] = 0  # padding
    labels = torch.randint(0, vocab, (n,), generator=gen(4))
    labels[:5] = -100
    labels[-6:] = -100
    adv = torch.randn(n, generator=gen(5))
    old = torch.full((n,), -3.6)
    bounds = [0, 12, 20, 33, n]
    ref = torch.full((4,), -40.0)

    def plain(tab, w):
        emb = torch.where((ids == 0)[:, None], tab[ids].detach(), tab[ids]) * 4.0  # the padding row takes no gradient
        lp = (emb @ w.t()).log_softmax(1).gather(1, labels.clamp(min=0)[:, None])[:, 0]
        live = (labels >= 0).double()
        if kind == "policy":
            r = (lp - old.double()).exp()
            a = adv.double()
            loss = -torch.minimum(r * a, r.clamp(0.8, 1.2) * a)
            return (loss * live).sum() / live.sum()
        m = torch.stack([(lp * live)[bounds[i]:bounds[i + 1]].sum() for i in range(4)]) - ref.double()
        return -torch.nn.functional.logsigmoid(0.1 * (m[:2] - m[2:])).mean()

    for step in range(4):
        opt.zero_grad()
        broken = step == 2
        x = embedding(ids.to(DEV), table, scale=4.0, padding_id=0, grad_buffer=table.grad)
        logits = x @ head.t()
        if kind == "policy":
            a = adv.clone()
            if broken:
                a[9] = float("inf")
            total, *_ = policy_loss(logits, labels.to(DEV), a.to(DEV), old_logp=old.to(DEV))
        else:
            w = torch.tensor([0.5, float("inf") if broken else 0.5])
            total, *_ = preference_loss(logits, labels.to(DEV), torch.tensor(bounds, device=DEV), ref.to(DEV),
                                        weights=w.to(DEV))
        (total * scale).backward()
        tab, hd = table.detach().cpu().double().requires_grad_(), head.detach().cpu().double().requires_grad_()
        before = table.detach().clone()
        want = plain(tab, hd)
        want.backward()
        if not broken:
            for p, q in ((table, tab), (head, hd)):
                got, exact = p.grad.double().cpu() / scale, q.grad
                # sums of at most 48 x 40 products of FP32 values, logits of order 1: a relative error of
                # some hundred roundings of the largest gradient, and the storage's own rounding
                tol = 400 * U * exact.abs().max() + torch.finfo(grad_dtype).eps / 2 * exact.abs()
                tol = tol + torch.finfo(grad_dtype).smallest_normal * torch.finfo(grad_dtype).eps / scale
                good = bool(((got - exact).abs() <= tol).all())
                assert good, (step, (got - exact).abs().max(), exact.abs().max())
        opt.step(gradient_scale=scale)
        assert bool(opt.last_result.updated) == (not broken) and bool(opt.last_result.found_inf) == broken
        changed = not torch.equal(before, table.detach())
        assert changed == (not broken)
        if not broken:
            norm = torch.sqrt(tab.grad.square().sum() + hd.grad.square().sum())
            assert abs(opt.last_result.total_norm - float(norm)) <= 4 * torch.finfo(grad_dtype).eps * float(norm) + 1e-6
