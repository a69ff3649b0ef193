"""GPU tests of the losses where a row's exponents or its sum are hard to
hold: against the plain 64-bit forms, with and without the gradient (which
take different kernels)."""
import math

import pytest
import torch

import optimizer_step_dl_amd as ra
from gpu_helpers import announce
from test_gpu_losses import check_policy, check_preference, gen
from vocab_helpers import U, Rows, close

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.mark.parametrize("vocab", [1000, 4097, 8192, 50_001, 70_000])
def test_rows_on_both_sides_of_the_lowest_shift(vocab):
    """Rows around -2^24, where the shift by the maximum ends: the label's
    lane shifts, the others' values lie on or below the limit and are most
    of the row's sum where the maximum is near."""
    announce(f"lowest shift vocab={vocab}")
    low = -(2.0 ** 24)
    label = vocab // 2
    tops = [low + 1, low + 2, low + 20, low + 255, low + 256, low + 257, low + 400, low, low * 2]
    n = len(tops)
    x = torch.full((n, vocab), low)
    for i, t in enumerate(tops):
        x[i, label] = t
    x[7, label] = low
    x[8] = low * 2
    x[:, ::5] = torch.where(x[:, ::5] == low, low - 2, x[:, ::5])
    x[2, 3::7] = float("-inf")
    x[2, label] = tops[2]
    labels = torch.full((n,), label)
    labels[3] = 0  # a label that is not the maximum
    adv = torch.randn(n, generator=gen(1))
    o, _ = check_policy(x, labels, torch.ones(n, dtype=torch.bool), None, adv, ra.policy_options())
    plain = x[0].double().log_softmax(0)[label]
    assert abs(float(o["logp"][0]) - float(plain)) < 1e-5 * abs(float(plain))
    check_preference(x, labels, torch.ones(n, dtype=torch.bool), [0, 4, n], torch.tensor([-30.0, -20.0]),
                     ra.preference_options(0.1, 0.1))


@pytest.mark.parametrize("dtype,vocab", [(F32, 1000), (F32, 12_000), (F32, 50_001), (F32, 70_000), (torch.bfloat16, 131_072),
                                         (torch.float16, 3001)])
def test_exponents_carry_all_of_log2_e(dtype, vocab):
    """One logit stands g above the label and far above the rest, so that
    logp = -g to 1e-12 and an exponent's factor that is off by a relative d
    moves it by d g.  The policy loss -exp(logp - old) shows logp as it is
    before it is rounded.

    The bound: the exponents are exact to 2^-40 (the shift cancels), v_exp_f32
    is within 1 ulp (2 u), the loss is rounded once (u); 1 u for the rest.
    FP32's log2 e alone (d = 1.3e-8) gives 9 to 18 u here."""
    announce(f"exponents {dtype} vocab={vocab}")
    n = 24
    x = torch.zeros((n, vocab), dtype=dtype)
    g = torch.linspace(42, 84, n).to(dtype)
    labels = (torch.arange(n) * 37 + vocab // 3) % vocab
    rows = torch.arange(n)
    x[rows, (labels + vocab // 2) % vocab] = g
    if vocab > 10_000:  # leading columns that serve no shift
        x[::4, :9000] = float("-inf")
        labels[::4] = vocab - 3
        x[rows[::4], labels[::4]] = 0.0
        x[::4, -9] = g[::4]
    r = Rows(x, labels, torch.ones(n, dtype=torch.bool))
    old = r.logp.float()
    want = -(r.logp - old.double()).exp()
    d = "cuda"
    for grad in (False, True):
        total, loss, logp = torch.empty((), device=d), torch.empty(n, device=d), torch.empty(n, device=d)
        xd = x.to(d)
        ra.radamw_policy_loss(xd, labels.to(d), old.to(d), torch.ones(n, device=d), ra.policy_options(), total, loss,
                              logp, grad=xd if grad else None)
        close(loss, want, 3 * U * want.abs(), f"loss, grad={grad}")  # close adds the rounding itself
        close(logp, r.logp, 3 * U, f"logp, grad={grad}")


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [4096, 16_384])
def test_log_probabilities_are_off_to_no_side(dtype, vocab):
    """Errors of one sign add up over a sequence: the mean error of logp over
    N rows, from losses -exp(logp - old).

    The bound: a row's error is the rounding of the label's exponent (up to 8:
    2^-21 / 2 log 2 = 1.7e-7 at most, 1e-7 in the mean square), of a lane's
    chain (5e-8) and of the loss (3e-8): 1.2e-7 in the mean square, and four
    times that over sqrt N; v_exp_f32 is 3.4e-9 low in the mean."""
    announce(f"mean error {dtype} vocab={vocab}")
    n = 4096
    x = 2 * torch.randn((n, vocab), generator=gen(vocab))
    labels = torch.randint(0, vocab, (n,), generator=gen(3))
    x[torch.arange(n), labels] += 4 + 6 * torch.rand(n, generator=gen(4))
    xd = x.to(dtype).cuda()
    z = xd.double()
    logp = z.gather(1, labels.cuda()[:, None])[:, 0] - z.logsumexp(1)
    old = logp.float()
    bound = 4 * 1.2e-7 / math.sqrt(n) + 3.4e-9
    for grad in (False, True):
        total, loss, out = (torch.empty(s, device="cuda") for s in ((), n, n))
        ra.radamw_policy_loss(xd, labels.cuda(), old, torch.ones(n, device="cuda"), ra.policy_options(), total, loss,
                              out, grad=torch.empty_like(xd) if grad else None)
        off = float((loss.double() / -(logp - old.double()).exp() - 1).mean())
        assert abs(off) <= bound, (grad, off, bound)


@pytest.mark.parametrize("dtype", [F32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("vocab", [3, 1000, 4097, 30_000, 50_001, 140_000])
def test_confident_rows_keep_their_digits(dtype, vocab):
    """Labels 10 to 40 above the rest, so that 1 - p goes down to e^-28 and
    less, in chunks and at the row's edges: logp = -log(1 + r), r the others'
    sum over the label's exponential, to the digits of r; likewise the label's
    gradient c (1 - p).

    The bound: an exponential is off by 3 u |y| + 2 u (|y| < 50 here), a
    lane's chain by its length, logp and the gradient are rounded (close) and
    the factor of the gradient is an FP32 value."""
    announce(f"confident {dtype} vocab={vocab}")
    n = 24
    x = torch.randn((n, vocab), generator=gen(vocab)).to(dtype)
    labels = (torch.arange(n) * (vocab // n) + torch.arange(n) % 3) % vocab
    labels[-1], labels[-2] = vocab - 1, 0
    x[torch.arange(n), labels] = torch.linspace(10, 40, n).to(dtype)
    z = x.double()
    others = z.clone()
    others[torch.arange(n), labels] = float("-inf")
    r = (others - z.gather(1, labels[:, None])).exp().sum(1)
    logp, less = -r.log1p(), r / (1 + r)
    chain = math.ceil(math.ceil(vocab / 256) / 4) + 8
    rel = (3 * 50 + 2 + chain) * U
    d = "cuda"
    adv = torch.linspace(0.5, 2, n)
    for grad in (False, True):
        total, loss, out = (torch.empty(s, device=d) for s in ((), n, n))
        stats, g = torch.empty((n, 4), device=d), torch.empty((n, vocab), dtype=dtype, device=d)
        xd, ld = x.to(d), labels.to(d)
        ra.radamw_policy_loss(xd, ld, None, adv.to(d), ra.policy_options(), total, loss, out, row_stats=stats,
                              grad=g if grad else None, grad_scale=1024.0)
        close(out, logp, rel * logp.abs(), f"logp, grad={grad}")
        if not grad:
            ra.radamw_logits_grad(xd, ld, stats, g, grad_scale=1024.0)
        want = -1024 * adv.double() * less
        close(g.gather(1, ld[:, None])[:, 0], want, (rel + 4 * U) * want.abs(), f"label's gradient, fused={grad}")
    loss, seq, lp = torch.empty(n // 2, device=d), torch.empty(n, device=d), torch.empty(n, device=d)
    ra.radamw_preference_loss(x.to(d), labels.to(d), torch.arange(n + 1, device=d), torch.zeros(n, device=d),
                              ra.preference_options(), torch.empty((), device=d), loss, seq, lp, stats)
    close(seq, logp, rel * logp.abs(), "seq_logp")


@pytest.mark.parametrize("dtype,vocab", [(F32, 30_000), (torch.bfloat16, 100_000), (torch.float16, 12_000),
                                         (torch.bfloat16, 140_000)])
def test_rows_whose_maximum_is_far_from_every_early_column(dtype, vocab):
    """The first columns and those around the label are masked by -inf or lie
    45 to 3000 below the others: the exponentials relative to the largest of
    them leave the range, and the row's maximum is found first."""
    announce(f"far maximum {dtype} {vocab}")
    lows = [-45.0, -60.0, -100.0, -3000.0]
    n = len(lows) + 1
    x = torch.randn((n, vocab), generator=gen(vocab)).to(dtype)
    labels = torch.full((n,), vocab - 20)
    for i, low in enumerate(lows):
        x[i, :9000] = low
        x[i, vocab - 40:] = low
    x[4, :9000] = float("-inf")
    x[4, vocab - 40:] = float("-inf")
    x[4, labels[4]] = -70.0
    adv = torch.randn(n, generator=gen(18))
    taken = torch.ones(n, dtype=torch.bool)
    check_policy(x, labels, taken, None, adv, ra.policy_options(), scale=8.0)
    check_preference(x, labels, taken, [0, 2, n], torch.tensor([-40.0, -50.0]), ra.preference_options(0.01, 0.1))
