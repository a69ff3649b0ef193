"""CPU tests of the vocabulary operators: the C entry points' refusals that
need no device, the binding's and the autograd forms' argument checks, the
workspace sizes, and the plain 64-bit forms of vocab_helpers.py against
torch's own autograd."""
import ctypes
import os

import pytest
import torch

import optimizer_step_dl_amd as ra
from optimizer_step_dl_amd import functional
from vocab_helpers import Rows, close, embedding_grad, policy, preference

INVALID, RANGE = -1, -5
DOUBLE = torch.float64


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ra.LIB_PATH):
        from optimizer_step_dl_amd import build
        build.build()
    return ra.load()


P = 0x10000  # a pointer that no refused call may look at


def lookup(lib, tdt=0, rows=8, dim=4, ts=4, idt=1, n=3, scale=1.0, odt=0, os_=4):
    return lib.radamw_embedding_lookup(P, tdt, rows, dim, ts, P, idt, n, scale, P, odt, os_, None)


def test_lookup_refusals(lib):
    for kw in (dict(tdt=3), dict(odt=-1), dict(idt=2), dict(dim=0), dict(ts=3), dict(os_=3), dict(n=-1), dict(rows=-1),
               dict(scale=float("inf")), dict(scale=1e39)):
        assert lookup(lib, **kw) == INVALID, kw
    for kw in (dict(dim=2 ** 24 + 1, ts=2 ** 24 + 1, os_=2 ** 24 + 1), dict(n=2 ** 31), dict(rows=2 ** 31),
               dict(ts=2 ** 47, rows=1000), dict(n=2 ** 24, dim=8192, ts=8192, os_=8192)):
        assert lookup(lib, **kw) == RANGE, kw
    assert lookup(lib, n=0) == 0


def grad(lib, gdt=0, gs=4, idt=1, n=3, rows=8, dim=4, scale=1.0, pad=-1, acc=0, tdt=0, ts=4, ws=1 << 40):
    return lib.radamw_embedding_grad(P, gdt, gs, P, idt, n, rows, dim, scale, pad, acc, P, tdt, ts, P, ws, None)


def test_grad_refusals(lib):
    for kw in (dict(gdt=3), dict(tdt=5), dict(idt=-1), dict(gs=3), dict(ts=3), dict(pad=-2), dict(acc=2), dict(dim=0),
               dict(scale=float("nan")), dict(n=-1)):
        assert grad(lib, **kw) == INVALID, kw
    need = ra.radamw_embedding_grad_workspace_bytes(3, 8, 4)
    for kw in (dict(pad=8), dict(ws=need - 1), dict(ws=0), dict(n=2 ** 31), dict(rows=2 ** 31, ts=4),
               dict(n=2 ** 31 - 100, dim=8192, gs=8192, ts=8192)):
        assert grad(lib, **kw) == RANGE, kw
    assert grad(lib, n=0, acc=1) == 0 and grad(lib, rows=0) == 0


def test_workspace_bytes(lib):
    last = 0
    for n in (0, 1, 7, 1000, 8192, 8193, 100_000, 10_000_000):
        b = ra.radamw_embedding_grad_workspace_bytes(n, 32000, 4096)
        assert b >= last and b % 256 == 0
        # ids and positions twice, counts, flags, and two partial rows per chunk of at least eight tokens
        assert b <= 16 * n + 1024 * (n + 8192) // 1024 * 4 + 32000 + 2 * 4096 * 4 * (n // 8 + 1) + 4096
        last = b
    for bad in ((-1, 8, 4), (3, 8, 0), (2 ** 31, 8, 4), (3, 2 ** 31, 4), (3, 8, 2 ** 25)):
        with pytest.raises(ra.RadamwError) as e:
            ra.radamw_embedding_grad_workspace_bytes(*bad)
        assert e.value.status in (INVALID, RANGE)


def policy_call(lib, opts, dt=0, n=3, vocab=8, st=8, idt=1, ref=P, scale=1.0, grad_=P, gs=8):
    o = None if opts is None else ctypes.byref(ra.policy_options(*opts))
    return lib.radamw_policy_loss(P, dt, n, vocab, st, P, idt, P, ref, P, P, o, scale, P, P, P, P, grad_, gs, None)


def preference_call(lib, opts, dt=0, n=3, vocab=8, st=8, idt=1, pairs=1, scale=1.0, grad_=P, gs=8):
    o = None if opts is None else ctypes.byref(ra.preference_options(*opts))
    return lib.radamw_preference_loss(P, dt, n, vocab, st, P, idt, P, pairs, P, P, o, scale, P, P, P, P, P, grad_, gs,
                                      None)


def test_loss_refusals(lib):
    good = (0.2, 0.2, 0.0)
    for bad in (None, (-0.1, 0.2, 0.0), (1.01, 0.2, 0.0), (0.2, -0.1, 0.0), (0.2, float("inf"), 0.0),
                (0.2, 0.2, -1.0), (float("nan"), 0.2, 0.0), (0.2, 0.2, float("nan"))):
        assert policy_call(lib, bad) == INVALID, bad
    assert policy_call(lib, (0.2, 0.2, 0.1), ref=None) == INVALID
    for bad in (None, (-0.1, 0.0), (float("inf"), 0.0), (0.1, -0.1), (0.1, 1.1), (0.1, float("nan"))):
        assert preference_call(lib, bad) == INVALID, bad
    for call, opts in ((policy_call, good), (preference_call, (0.1, 0.0))):
        for kw in (dict(dt=3), dict(idt=2), dict(n=-1), dict(vocab=0), dict(st=7), dict(gs=7),
                   dict(scale=float("nan")), dict(scale=-1e40)):
            assert call(lib, opts, **kw) == INVALID, kw
        for kw in (dict(n=2 ** 31), dict(vocab=2 ** 27 + 1, st=2 ** 27 + 1, gs=2 ** 27 + 1), dict(st=2 ** 47, n=1000)):
            assert call(lib, opts, **kw) == RANGE, kw
    assert preference_call(lib, (0.1, 0.0), pairs=0) == INVALID
    assert preference_call(lib, (0.1, 0.0), pairs=2 ** 24) == RANGE
    assert lib.radamw_logits_grad(P, 0, 3, 8, 8, P, 1, P, None, 1.0, None, 0, None) == INVALID
    assert lib.radamw_logits_grad(P, 0, 0, 8, 8, P, 1, P, None, 1.0, None, 0, None) == 0


def test_option_defaults(lib):
    p, q = ra.radamw_policy_options_default(), ra.radamw_preference_options_default()
    assert (p.clip_low, p.clip_high, p.kl_coef) == (0.2, 0.2, 0.0) and (q.beta, q.label_smoothing) == (0.1, 0.0)
    d, e = ra.policy_options(), ra.preference_options()
    assert (d.clip_low, d.clip_high, d.kl_coef, e.beta, e.label_smoothing) == (0.2, 0.2, 0.0, 0.1, 0.0)


def test_binding_refuses_host_tensors(lib):
    t, ids, out = torch.zeros(4, 4), torch.zeros(2, dtype=torch.int64), torch.zeros(2, 4)
    with pytest.raises(ValueError):
        ra.radamw_embedding_lookup(t, ids, out)
    with pytest.raises(ValueError):
        ra.radamw_embedding_grad(out, ids, t, torch.zeros(1000, dtype=torch.uint8))
    v = torch.zeros(2)
    with pytest.raises(ValueError):
        ra.radamw_policy_loss(out, ids, None, v, ra.policy_options(), v, v, v)
    with pytest.raises(ValueError):
        ra.radamw_logits_grad(out, ids, torch.zeros(2, 4), torch.zeros(2, 4))


def test_functional_argument_checks():
    t, ids = torch.zeros(5, 4, requires_grad=True), torch.zeros(2, 3, dtype=torch.int64)
    for bad in (dict(table=torch.zeros(5)), dict(model_copy=torch.zeros(5, 3)), dict(grad_buffer=torch.zeros(4, 4)),
                dict(grad_buffer=torch.zeros(5, 4, requires_grad=True)), dict(padding_id=5), dict(padding_id=-1)):
        kw = dict(table=t, **bad) if "table" not in bad else bad
        with pytest.raises(ValueError):
            functional.embedding(ids, **kw)
    x, labels = torch.zeros(2, 3, 7), torch.zeros(2, 3, dtype=torch.int64)
    adv = torch.zeros(6)
    for kw in (dict(labels=labels[:, :2]), dict(advantages=adv[:5]), dict(old_logp=adv[:5]), dict(ref_logp=adv[:4]),
               dict(weights=adv[:4])):
        with pytest.raises(ValueError):
            functional.policy_loss(**{**dict(logits=x, labels=labels, advantages=adv), **kw})
    off = torch.tensor([0, 2, 6])
    for kw in (dict(offsets=off[:2]), dict(offsets=torch.arange(4)), dict(offsets=off[None]), dict(ref_logp=adv[:3]),
               dict(weights=adv[:2])):
        with pytest.raises(ValueError):
            functional.preference_loss(**{**dict(logits=x, labels=labels, offsets=off, ref_logp=adv[:2]), **kw})


# ------------------------------------------------ the plain forms themselves --

def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_plain_embedding_gradient():
    rows, dim = 9, 5
    w = torch.randn(rows, dim, generator=gen(1), dtype=DOUBLE, requires_grad=True)
    ids = torch.randint(0, rows, (40,), generator=gen(2))
    g = torch.randn(40, dim, generator=gen(3))
    torch.nn.functional.embedding(ids, w, padding_idx=3).mul(0.5).backward(g.double())
    ref, slack = embedding_grad(g, ids, rows, 0.5, 3, None)
    assert torch.allclose(ref, w.grad, rtol=1e-14, atol=1e-14) and bool((slack >= 0).all())
    old = torch.ones(rows, dim)
    assert torch.allclose(embedding_grad(g, ids, rows, 0.5, 3, old)[0], w.grad + 1, rtol=1e-14)


def plain_inputs(n=14, vocab=23):
    x = (2 * torch.randn(n, vocab, generator=gen(4))).float()
    labels = torch.randint(0, vocab, (n,), generator=gen(5))
    labels[::4] = -100
    taken = labels >= 0
    z = x.double().requires_grad_()
    lp = z.log_softmax(1).gather(1, labels.clamp(min=0)[:, None])[:, 0]
    return x, labels, taken, z, torch.where(taken, lp, 0.0)


def test_plain_policy():
    x, labels, taken, z, lp = plain_inputs()
    n = len(labels)
    old = (lp.detach() + 0.4 * torch.randn(n, generator=gen(6))).float()
    ref = (lp.detach() + 0.4 * torch.randn(n, generator=gen(7))).float()
    adv, w = torch.randn(n, generator=gen(8)), torch.rand(n, generator=gen(9))
    r = (lp - old.double()).exp()
    a = adv.double()
    d = ref.double() - lp
    loss = -torch.minimum(r * a, r.clamp(0.8, 1.3) * a) + 0.25 * (d.exp() - d - 1)
    (torch.where(taken, loss, 0.0) * w.double()).sum().backward()
    rows = Rows(x, labels, taken)
    got, err, coef, coef_err = policy(rows, old, ref, adv, w, 0.2, 0.3, 0.25)
    assert torch.allclose(got[taken], loss[taken], rtol=1e-12, atol=1e-13) and bool((got[~taken] == 0).all())
    g, slack = rows.grad(coef, coef_err, 3.0)
    assert torch.allclose(g, 3 * z.grad, rtol=1e-11, atol=1e-13)
    assert bool((slack >= 0).all()) and float(slack.max()) < 1e-4 and float(err.max()) < 1e-4


def test_plain_preference():
    x, labels, taken, z, lp = plain_inputs()
    bounds = [1, 4, 4, 9, 13]
    ref, w = torch.tensor([-9.0, 0.5, -15.0, -12.0]), torch.tensor([0.5, 2.0])
    s = torch.stack([lp[bounds[i]:bounds[i + 1]].sum() for i in range(4)])
    h = 0.2 * ((s[:2] - ref[:2]) - (s[2:] - ref[2:]))
    loss = -0.9 * h.sigmoid().log() - 0.1 * (-h).sigmoid().log()
    (loss * w.double()).sum().backward()
    rows = Rows(x, labels, taken)
    got, err, sums, _, coef, coef_err = preference(rows, bounds, ref, w, 0.2, 0.1)
    assert torch.allclose(got, loss.detach(), rtol=1e-12) and torch.allclose(sums, s.detach(), rtol=1e-12)
    g, slack = rows.grad(coef, coef_err, 1.0)
    assert torch.allclose(g, z.grad, rtol=1e-11, atol=1e-13) and float(err.max()) < 1e-4


def test_close_finds_a_wrong_value():
    ref = torch.linspace(-2, 2, 50, dtype=DOUBLE)
    close(ref.float(), ref, 0.0, "rounded")
    close(ref.bfloat16(), ref, 0.0, "rounded")
    off = ref.float().clone()
    off[7] *= 1 + 2 ** -22
    with pytest.raises(AssertionError):
        close(off, ref, 0.0, "one value off")
    with pytest.raises(AssertionError):
        close(torch.where(torch.arange(50) == 3, float("nan"), ref).float(), ref, 1.0, "a NaN")
