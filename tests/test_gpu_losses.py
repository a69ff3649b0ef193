"""GPU tests of the clipped policy loss, the preference loss and the logits'
gradient from saved records, against plain 64-bit forms (bounds in
vocab_helpers.py)."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from gpu_helpers import DEV, announce
from vocab_helpers import U, Rows, close, policy, preference

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def place(t, pad=0):
    """t on the GPU as the leading columns of wider rows of NaN, and the whole."""
    whole = torch.full((t.shape[0], t.shape[1] + pad), NAN, dtype=t.dtype, device=DEV)
    whole[:, :t.shape[1]] = t.to(DEV)
    return whole[:, :t.shape[1]], whole


def make_rows(n, vocab, dtype, seed, std=2.0, share=0.7, index=torch.int64):
    g = gen(seed)
    x = (torch.randn((n, vocab), generator=g) * std).to(dtype)
    labels = torch.randint(0, vocab, (n,), generator=g)
    x.scatter_add_(1, labels[:, None], torch.full((n, 1), 3.0, dtype=dtype))
    taken = torch.rand(n, generator=g) < share
    if n:
        taken[-1] = True
    labels[~taken] = torch.where(torch.rand(int((~taken).sum()), generator=g) < 0.5, -100, vocab)
    return x, labels.to(index), taken


def outputs(n):
    f = lambda k: torch.full((k,), NAN, device=DEV)  # noqa: E731
    return dict(total=torch.full((), NAN, device=DEV), loss=f(n), logp=f(n))


def run_policy(x, labels, old, adv, opts, ref=None, w=None, grad=True, scale=1.0, pad=0, in_place=False, stats=True):
    n = x.shape[0]
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    xd, whole = place(x, pad)
    o = outputs(n)
    st = torch.full((n, 4), NAN, device=DEV) if stats else None
    gd = gwhole = None
    if grad:
        gd, gwhole = (xd, whole) if in_place else place(torch.full_like(x, NAN), pad + 1 if pad else 0)
    ra.radamw_policy_loss(xd, d(labels), d(old), d(adv), opts, o["total"], o["loss"], o["logp"], ref_logp=d(ref),
                          weights=d(w), row_stats=st, grad=gd, grad_scale=scale)
    if gwhole is not None and pad:
        assert bool(gwhole[:, x.shape[1]:].isnan().all())
    return o, gd, st, xd


def check_policy(x, labels, taken, old, adv, opts, ref=None, w=None, scale=1.0, pad=0, in_place=False):
    if w is not None:
        taken = taken & (w != 0)
    r = Rows(x, labels, taken)
    loss, loss_err, coef, coef_err = policy(r, old, ref, adv, w, opts.clip_low, opts.clip_high, opts.kl_coef)
    want, slack = r.grad(coef, coef_err, scale)
    zero = torch.zeros(())
    o, gd, st, xd = run_policy(x, labels, old, adv, opts, ref, w, True, scale, pad, in_place)
    close(o["logp"], torch.where(taken, r.logp, zero), torch.where(taken, r.err, zero), "logp")
    close(o["loss"], loss, loss_err, "loss")
    ww = torch.ones_like(loss) if w is None else torch.where(taken, w.double(), zero)
    # the total sums the rounded losses
    close(o["total"], (loss * ww).sum(), ((loss_err + U * loss.abs()) * ww.abs()).sum().item(), "total")
    close(gd, want, slack, "gradient")
    # the loss alone, and the gradient from the records, of another scale
    o2, _, st2, xd2 = run_policy(x, labels, old, adv, opts, ref, w, False, scale, pad)
    twice = dict(logp=2 * r.err, loss=2 * loss_err, total=2 * ((loss_err + U * loss.abs()) * ww.abs()).sum())
    for k in o:
        close(o2[k], o[k].double(), twice[k], k)
    g2, _ = place(torch.full_like(x, NAN), pad)
    up = torch.tensor(0.75, device=DEV)
    ra.radamw_logits_grad(xd2, labels.to(DEV), st2, g2, upstream=up, grad_scale=scale)
    want2, slack2 = r.grad(coef, coef_err + U * coef.abs(), scale * 0.75)
    close(g2, want2, slack2 + 2 * U * want2.abs(), "gradient from records")
    return o, gd


def policy_inputs(r, n, seed, spread=0.3):
    """old, ref, advantages, weights: no ratio within 1e-3 of a clip bound of the defaults used here."""
    g = gen(seed)
    logp = r.logp.float()
    old = logp + spread * torch.randn(n, generator=g)
    for edge in (0.8, 1.28, 1.2):
        near = ((logp - old).exp() - edge).abs() < 2e-3
        old = torch.where(near, old + 0.02, old)
    ref = logp + 0.5 * torch.randn(n, generator=g)
    return old, ref, torch.randn(n, generator=g), torch.rand(n, generator=g) + 0.1


# one lane's chunk and less, each row size the kernels tell apart, odd ones, and rows held by two reads
VOCABS = [1, 2, 3, 7, 8, 9, 127, 1000, 1025, 8191, 8193, 16385, 32003, 65536, 65537]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy_vocabularies(vocab, dtype):
    announce(f"policy vocab={vocab} {dtype}")
    n = 9
    x, labels, taken = make_rows(n, vocab, dtype, vocab)
    old, ref, adv, w = policy_inputs(Rows(x, labels, taken), n, vocab + 1)
    check_policy(x, labels, taken, old, adv, ra.policy_options(0.2, 0.28, 0.05), ref, w, 64.0, pad=3)


@pytest.mark.parametrize("dtype,vocab", [(F32, 65539), (F32, 100_003), (BF16, 131_072), (BF16, 131_081), (F16, 160_001)])
def test_policy_large_rows(dtype, vocab):
    announce(f"policy vocab={vocab} {dtype}")
    n = 5
    x, labels, taken = make_rows(n, vocab, dtype, vocab)
    old, ref, adv, w = policy_inputs(Rows(x, labels, taken), n, vocab + 1)
    check_policy(x, labels, taken, old, adv, ra.policy_options(0.2, 0.28, 0.05), ref, w, 1024.0)


@pytest.mark.parametrize("n", [0, 1, 2, 1000])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_policy_lengths(n, index):
    announce(f"policy n={n}")
    x, labels, taken = make_rows(n, 200, BF16, n, index=index)
    old, ref, adv, w = policy_inputs(Rows(x, labels, taken), n, n + 1) if n else (torch.empty(0),) * 4
    if n == 0:
        o, *_ = run_policy(x, labels, old, adv, ra.policy_options(), grad=True)
        assert float(o["total"]) == 0.0
        return
    check_policy(x, labels, taken, old, adv, ra.policy_options(0.2, 0.2, 0.0), None, w)
    check_policy(x, labels, taken, old, adv, ra.policy_options(0.2, 0.2, 0.1), ref, None)


@pytest.mark.parametrize("dtype,vocab", [(F32, 1003), (BF16, 40_001), (F16, 150_000)])
def test_policy_in_place(dtype, vocab):
    """The gradient in the logits' own storage is the one beside them, bit for bit."""
    announce(f"policy in place {dtype}")
    n = 6
    x, labels, taken = make_rows(n, vocab, dtype, 3)
    old, ref, adv, w = policy_inputs(Rows(x, labels, taken), n, 4)
    opts = ra.policy_options(0.2, 0.28, 0.05)
    _, g, *_ = run_policy(x, labels, old, adv, opts, ref, w, pad=1)
    _, h, st, _ = run_policy(x, labels, old, adv, opts, ref, w, pad=1, in_place=True)
    assert torch.equal(g, h)
    xd, _ = place(x, 1)
    gd, _ = place(torch.full_like(x, NAN), 2)
    ra.radamw_logits_grad(xd, labels.to(DEV), st, gd)
    ra.radamw_logits_grad(xd, labels.to(DEV), st, xd)
    assert torch.equal(xd, gd)


def test_policy_on_policy_ratio_is_one():
    """No old_logp: the ratio is exactly 1 and inside clips of any width, 0 too."""
    announce("policy on policy")
    n, vocab = 20, 501
    x, labels, taken = make_rows(n, vocab, F32, 1, share=1.0)
    adv = torch.randn(n, generator=gen(2))
    o, _ = check_policy(x, labels, taken, None, adv, ra.policy_options(0.0, 0.0, 0.0))
    assert torch.equal(o["loss"].cpu(), -adv)


def test_policy_clip_sides():
    """Four signs: the gradient is exactly zero where clipping holds the loss."""
    announce("policy clip")
    vocab = 300
    x, labels, taken = make_rows(4, vocab, F32, 5, share=1.0)
    lp = Rows(x, labels, taken).logp.float()
    old = lp - torch.tensor([0.5, 0.5, -0.5, -0.5])
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0])
    _, g = check_policy(x, labels, taken, old, adv, ra.policy_options(0.2, 0.2, 0.0))
    assert [bool((g[i] == 0).all()) for i in range(4)] == [True, False, False, True]


@pytest.mark.parametrize("dtype,vocab", [(F32, 1000), (BF16, 5000), (BF16, 140_000), (F16, 9001)])
def test_policy_masked_logits(dtype, vocab):
    """Vocabulary entries masked by the type's lowest value or -inf; a row
    whose every entry is the lowest value is uniform; a row that is all -inf,
    holds +inf or NaN gives NaN, and only that row."""
    announce(f"policy masked logits {dtype} {vocab}")
    low = torch.finfo(dtype).min
    n = 7
    x, labels, taken = make_rows(n, vocab, dtype, 8, share=1.0)
    labels[:] = vocab // 2
    keep = torch.arange(vocab) % 3 == (vocab // 2) % 3
    x[0, ~keep] = low
    x[1, ~keep] = float("-inf")
    x[2] = low
    x[3] = float("-inf")
    x[4, 1] = float("inf")
    x[5, vocab - 1] = NAN
    if dtype != F16:
        x[6, :] = -1e4
        x[6, labels[6]] = 3e38
    adv = torch.randn(n, generator=gen(9))
    o, g = check_policy(x, labels, taken, None, adv, ra.policy_options())
    assert o["logp"].isnan().cpu().tolist() == [False, False, False, True, True, True, False]
    assert abs(float(o["logp"][2]) + torch.log(torch.tensor(float(vocab)))) < 1e-5
    assert g.isnan().any(1).cpu().tolist() == [False, False, False, True, True, True, False]


@pytest.mark.parametrize("dtype,vocab", [(F32, 30_000), (BF16, 100_000), (F16, 12_000), (BF16, 140_000)])
def test_policy_rows_whose_leading_columns_mislead(dtype, vocab):
    """The first columns are masked (-inf or the lowest value), far below the
    rest, or hold a value so small that the others' exponentials relative to
    it leave FP32's range; large maxima on either side of 2^24."""
    announce(f"policy leading columns {dtype} {vocab}")
    lead = 9000
    n = 7
    x, labels, taken = make_rows(n, vocab, dtype, 17, share=1.0)
    labels[:] = vocab - 5
    x[0, :lead] = float("-inf")
    x[1, :lead] = torch.finfo(dtype).min
    x[2, :lead] = -3000.0
    x[3, :lead] = -90.0
    if dtype != F16:
        x[4] += 2.0 ** 23
        x[5, :lead] = -(2.0 ** 25)
        x[6, lead:] += 2.0 ** 26
    adv = torch.randn(n, generator=gen(18))
    check_policy(x, labels, taken, None, adv, ra.policy_options())
    bounds = [0, 4, n]
    check_preference(x, labels, taken, bounds, torch.tensor([-40.0, -50.0]), ra.preference_options(0.1, 0.1))


@pytest.mark.parametrize("vocab", [777, 140_001])
def test_policy_absent_rows_may_hold_anything(vocab):
    """Rows that take no part: NaN logits, old and reference values, any
    advantage, reach nothing; every row absent gives a total of 0."""
    announce("policy absent rows")
    n = 8
    x, labels, taken = make_rows(n, vocab, BF16, 11, share=1.0)
    old, ref, adv, w = policy_inputs(Rows(x, labels, taken), n, 12)
    taken[:] = True
    labels[2], labels[5] = -100, vocab + 3
    w[6] = 0.0
    for i in (2, 5, 6):
        x[i], old[i], ref[i], adv[i] = NAN, NAN, float("inf"), NAN
    w[2] = NAN  # a label outside is enough
    taken[[2, 5]] = False
    clean = torch.where(taken, w, torch.zeros(()))
    opts = ra.policy_options(0.2, 0.28, 0.1)
    o, g, *_ = run_policy(x, labels, old, adv, opts, ref, w)
    assert bool((g[[2, 5, 6]] == 0).all()) and bool((o["loss"][[2, 5, 6]] == 0).all())
    assert bool(o["total"].isfinite()) and bool(g.isfinite().all())
    check_policy(torch.where((taken & (w != 0))[:, None], x, torch.zeros((), dtype=BF16)), labels, taken,
                 old.nan_to_num(0), adv.nan_to_num(0), opts, ref.nan_to_num(0, 0), clean)
    o, g, *_ = run_policy(x, torch.full_like(labels, -1), old, adv, opts, ref, None)
    assert float(o["total"]) == 0.0 and bool((g == 0).all()) and bool((o["logp"] == 0).all())


@pytest.mark.parametrize("vocab", [60, 20_000, 140_000])
def test_impossible_labels(vocab):
    """Labels whose own logit is -inf: their probability is 0, the ratio with
    itself 1, a rejected sequence with one is infinitely far away."""
    announce(f"impossible labels {vocab}")
    x, labels, taken = make_rows(6, vocab, F32, 71, share=1.0)
    for i in (1, 4):
        x[i, labels[i]] = float("-inf")
    adv = torch.tensor([1.0, -2.0, 0.5, 1.0, 1.0, 1.0])
    o, g, *_ = run_policy(x, labels, None, adv, ra.policy_options())
    assert bool(o["logp"][[1, 4]].isneginf().all()) and torch.equal(o["loss"].cpu(), -adv)
    assert bool(g.isfinite().all()) and float(g[1, labels[1]]) == 2.0 and float(g[4, labels[4]]) == -1.0
    old = torch.full((6,), -3.0)
    o, g, *_ = run_policy(x, labels, old, adv.abs(), ra.policy_options())
    assert bool((o["loss"][[1, 4]] == 0).all()) and bool((g[[1, 4]] == 0).all())
    # chosen 0..3, rejected 3..6, which holds row 4
    o, g, *_ = run_preference(x[[0, 2, 3, 5, 4, 1]], labels[[0, 2, 3, 5, 4, 1]], [0, 3, 5], torch.zeros(2),
                              ra.preference_options())
    assert o["seq_logp"].isneginf().tolist() == [False, True] and float(o["loss"]) == 0.0 and bool((g == 0).all())
    o, g, *_ = run_preference(x[[4, 0, 2]], labels[[4, 0, 2]], [0, 1, 3], torch.zeros(2), ra.preference_options())
    assert float(o["loss"]) == float("inf") and bool(g.isfinite().all())
    assert abs(float(g[0, labels[4]]) + 0.1) < 1e-6


def test_more_rows_than_a_launch_holds():
    """2^21 rows and some: every kernel goes on with the next launch."""
    announce("rows over launches")
    n, vocab = (1 << 21) + 5, 8
    x, labels, taken = make_rows(n, vocab, F32, 81)
    taken[-3:] = True
    labels[-3:] = torch.tensor([7, 0, 3])
    adv = torch.randn(n, generator=gen(82))
    check_policy(x, labels, taken, None, adv, ra.policy_options(), None, torch.full((n,), 1.0 / n))
    bounds = [1, 1 << 20, (1 << 20) + 7, (1 << 21) - 1, n - 1]
    check_preference(x, labels, taken, bounds, torch.zeros(4), ra.preference_options(1e-6, 0.1))


def test_policy_gradient_against_differences():
    """The gradient against central differences of the 64-bit loss."""
    announce("policy differences")
    n, vocab = 3, 11
    x, labels, taken = make_rows(n, vocab, F32, 21, share=1.0)
    old, ref, adv, w = policy_inputs(Rows(x, labels, taken), n, 22)
    opts = ra.policy_options(0.2, 0.28, 0.3)
    _, g, *_ = run_policy(x, labels, old, adv, opts, ref, w)

    def total(z):
        lp = z.log_softmax(1).gather(1, labels[:, None])[:, 0]
        r = (lp - old.double()).exp()
        a = adv.double()
        d = ref.double() - lp
        loss = -torch.minimum(r * a, r.clamp(0.8, 1.28) * a) + 0.3 * (d.exp() - d - 1)
        return float((loss * w.double()).sum())

    h = 1e-5
    for i in range(n):
        for j in range(vocab):
            z = x.double()
            z[i, j] += h
            up = total(z)
            z[i, j] -= 2 * h
            # the difference's own error: h^2 times a third derivative of order 10, and 2^-52 / h
            assert abs((up - total(z)) / (2 * h) - float(g[i, j])) < 1e-5


def test_policy_total_is_reproducible():
    announce("policy reproducible")
    n, vocab = 3000, 257
    x, labels, taken = make_rows(n, vocab, BF16, 31)
    old, ref, adv, w = policy_inputs(Rows(x, labels, taken), n, 32)
    opts = ra.policy_options(0.2, 0.28, 0.1)
    first = run_policy(x, labels, old, adv, opts, ref, w)
    again = run_policy(x, labels, old, adv, opts, ref, w)
    assert all(torch.equal(first[0][k], again[0][k]) for k in first[0]) and torch.equal(first[1], again[1])


def test_policy_rows_past_32_bit_offsets():
    """Rows that begin beyond 2^31 elements and 2^32 bytes."""
    announce("policy far rows")
    vocab, n = 65_536, 33_000
    x = torch.zeros((n, vocab), dtype=BF16, device=DEV)
    labels = torch.full((n,), -100, device=DEV)
    at = [0, 16_384, 32_767, 32_768, n - 1]
    g = gen(40)
    rows = torch.randn((len(at), vocab), generator=g).to(BF16)
    for k, i in enumerate(at):
        x[i] = rows[k].to(DEV)
        labels[i] = 100 * k
    o = outputs(n)
    adv = torch.ones(n, device=DEV)
    ra.radamw_policy_loss(x, labels, None, adv, ra.policy_options(), o["total"], o["loss"], o["logp"], grad=x)
    r = Rows(rows, torch.tensor([100 * k for k in range(len(at))]), torch.ones(len(at), dtype=torch.bool))
    close(o["logp"][at], r.logp, r.err, "logp")
    want, slack = r.grad(-torch.ones(len(at), dtype=torch.float64), torch.zeros(len(at), dtype=torch.float64), 1.0)
    close(x[at], want, slack, "gradient")
    x[at] = 0
    assert not bool(x.any())


# -------------------------------------------------------------- preference --

def run_preference(x, labels, bounds, ref, opts, w=None, grad=True, scale=1.0, in_place=False, pad=0):
    n, pairs = x.shape[0], (len(bounds) - 1) // 2
    xd, _ = place(x, pad)
    f = lambda k: torch.full((k,), NAN, device=DEV)  # noqa: E731
    o = dict(total=f(1), loss=f(pairs), seq_logp=f(2 * pairs), logp=f(n))
    st = torch.full((n, 4), NAN, device=DEV)
    gd = None if not grad else xd if in_place else place(torch.full_like(x, NAN), pad)[0]
    ra.radamw_preference_loss(xd, labels.to(DEV), torch.tensor(bounds, dtype=labels.dtype, device=DEV), ref.to(DEV),
                              opts, o["total"], o["loss"], o["seq_logp"], o["logp"], st,
                              weights=None if w is None else w.to(DEV), grad=gd, grad_scale=scale)
    return o, gd, st, xd


def check_preference(x, labels, taken, bounds, ref, opts, w=None, scale=1.0, pad=0):
    r = Rows(x, labels, taken)
    loss, loss_err, sums, sum_err, coef, coef_err = preference(r, bounds, ref, w, opts.beta, opts.label_smoothing)
    want, slack = r.grad(coef, coef_err, scale)
    o, gd, st, xd = run_preference(x, labels, bounds, ref, opts, w, True, scale, pad=pad)
    zero = torch.zeros(())
    close(o["logp"], torch.where(taken, r.logp, zero), torch.where(taken, r.err, zero), "logp")
    close(o["seq_logp"], sums, sum_err, "seq_logp")
    close(o["loss"], loss, loss_err, "loss")
    ww = torch.ones_like(loss) if w is None else w.double()
    close(o["total"][0], (loss * ww).sum(), ((loss_err + U * loss.abs()) * ww.abs()).sum().item(), "total")
    close(gd, want, slack + 2 * U * want.abs(), "gradient")
    o2, _, st2, _ = run_preference(x, labels, bounds, ref, opts, w, False, scale, pad=pad)
    assert all(torch.equal(o[k], o2[k]) for k in o) and torch.equal(st, st2)
    g2 = place(torch.full_like(x, NAN), 0)[0]
    ra.radamw_logits_grad(xd, labels.to(DEV), st, g2, upstream=torch.tensor([-2.0], device=DEV), grad_scale=scale)
    close(g2, -2 * want, 2 * slack + 4 * U * want.abs(), "gradient from records")
    return o, gd


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", [1, 7, 1001, 16385, 40_000, 131_075])
def test_preference_vocabularies(vocab, dtype):
    announce(f"preference vocab={vocab} {dtype}")
    bounds = [0, 4, 5, 9, 12]
    x, labels, taken = make_rows(12, vocab, dtype, vocab)
    ref = preference(Rows(x, labels, taken), bounds, torch.zeros(4), None, 0.1, 0.0)[2].float() + 3 * torch.randn(
        4, generator=gen(1))
    check_preference(x, labels, taken, bounds, ref, ra.preference_options(0.1, 0.1), torch.tensor([0.7, 0.2]), 64.0,
                     pad=3)


@pytest.mark.parametrize("bounds", [[0, 1, 2], [0, 0, 0], [0, 0, 5], [3, 7, 20], [0, 300, 301, 301, 700, 1000, 1000],
                                    [5, 5, 5, 5, 900]])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_preference_sequences(bounds, index):
    """Empty sequences, sequences of one row, rows before the first and
    behind the last, sequences longer than a workgroup."""
    announce(f"preference {bounds}")
    n = bounds[-1] + 6
    x, labels, taken = make_rows(n, 97, BF16, n, index=index)
    pairs = (len(bounds) - 1) // 2
    ref = torch.randn(2 * pairs, generator=gen(3))
    r = Rows(x, labels, taken)
    sums = preference(r, bounds, torch.zeros(2 * pairs), None, 0.1, 0.0)[2]
    o, g = check_preference(x, labels, taken, bounds, sums.float() + 5 * ref, ra.preference_options(0.2, 0.0))
    assert bool((g[:bounds[0]] == 0).all()) and bool((g[bounds[-1]:] == 0).all())


@pytest.mark.parametrize("pairs", [1, 2, 8, 9, 40, 1100])
def test_preference_pair_counts(pairs):
    """One workgroup for up to 8 pairs, one each beyond, with and without weights."""
    announce(f"preference pairs={pairs}")
    g = gen(pairs)
    lengths = torch.randint(0, 6, (2 * pairs,), generator=g)
    bounds = [2] + (2 + lengths.cumsum(0)).tolist()
    x, labels, taken = make_rows(bounds[-1] + 3, 33, F32, pairs)
    r = Rows(x, labels, taken)
    sums = preference(r, bounds, torch.zeros(2 * pairs), None, 0.1, 0.0)[2].float()
    ref = sums + 3 * torch.randn(2 * pairs, generator=g)
    check_preference(x, labels, taken, bounds, ref, ra.preference_options(0.3, 0.2))
    check_preference(x, labels, taken, bounds, ref, ra.preference_options(0.3, 0.0), torch.rand(pairs, generator=g))


def test_preference_far_margins():
    """h of +-1000: the loss is linear or zero, without overflow; weight 0."""
    announce("preference margins")
    x, labels, taken = make_rows(6, 50, F32, 2, share=1.0)
    bounds = [0, 1, 2, 3, 4, 5, 6]
    ref = torch.tensor([-1000.0, 1000.0, 0.0, 0.0, 0.0, float("inf")])
    w = torch.tensor([1.0, 1.0, 0.0])
    opts = ra.preference_options(1.0, 0.0)
    o, g, *_ = run_preference(x, labels, bounds, ref, opts, w)
    loss = o["loss"].cpu()
    assert loss[0] == 0 and abs(loss[1] - 1000) < 20 and bool(o["total"].isfinite())
    assert bool(g.isfinite().all()) and bool((g[[2, 5]] == 0).all()) and bool((g[[0, 3]] == 0).all())
    assert abs(float(g[1, labels[1]]) + float(1 - o["logp"][1].exp())) < 1e-5


def test_preference_pair_of_weight_zero_may_hold_nan():
    announce("preference nan pair")
    x, labels, taken = make_rows(8, 300, BF16, 19, share=1.0)
    x[2] = NAN
    x[6, 7] = float("inf")
    x[7] = float("-inf")
    o, g, *_ = run_preference(x, labels, [0, 2, 4, 6, 8], torch.zeros(4), ra.preference_options(),
                              torch.tensor([1.0, 0.0]))
    assert bool(o["total"].isfinite()) and o["loss"].isnan().tolist() == [False, True]
    assert bool(g.isfinite().all()) and bool((g[[2, 3, 6, 7]] == 0).all()) and bool((g[:2] != 0).any())


def test_preference_in_place_and_differences():
    announce("preference differences")
    x, labels, taken = make_rows(7, 9, F32, 13, share=1.0)
    labels[2] = -100
    bounds, ref = [0, 3, 7], torch.tensor([-5.0, -6.0])
    opts = ra.preference_options(0.5, 0.1)
    _, g, *_ = run_preference(x, labels, bounds, ref, opts)
    _, h, *_ = run_preference(x, labels, bounds, ref, opts, in_place=True)
    assert torch.equal(g, h)
    ls = torch.nn.functional.logsigmoid

    def total(z):
        lp = z.log_softmax(1).gather(1, labels.clamp(min=0)[:, None])[:, 0] * (labels >= 0)
        m = 0.5 * ((lp[:3].sum() + 5.0) - (lp[3:].sum() + 6.0))
        return float(-0.9 * ls(m) - 0.1 * ls(-m))

    step = 1e-5
    for i in range(7):
        for j in range(9):
            z = x.double()
            z[i, j] += step
            up = total(z)
            z[i, j] -= 2 * step
            assert abs((up - total(z)) / (2 * step) - float(g[i, j])) < 1e-5


def test_preference_offsets_outside_are_held():
    """Offsets outside 0 .. n (a caller's error) touch nothing outside."""
    announce("preference bad offsets")
    x, labels, taken = make_rows(10, 40, BF16, 17, share=1.0)
    big = 2 ** 62
    for bounds in ([-big, 3, big], [big, -big, 4], [-1, 2 * big - 1 + big // 2 - big, 10]):
        o, g, *_ = run_preference(x, labels, bounds, torch.zeros(2), ra.preference_options())
        assert bool(o["loss"].isfinite().all()) and bool(g.isfinite().all())


def test_loss_refusals():
    announce("loss refusals")
    n, vocab = 6, 32
    x = torch.randn((n, vocab), device=DEV)
    labels = torch.zeros(n, dtype=torch.int64, device=DEV)
    adv = torch.ones(n, device=DEV)
    o = outputs(n)
    st = torch.full((n, 4), NAN, device=DEV)
    args = (x, labels, None, adv)
    outs = (o["total"], o["loss"], o["logp"])

    def refused(status, f):
        with pytest.raises(ra.RadamwError) as e:
            f()
        assert e.value.status == status, e.value

    before = ra.radamw_launch_count()
    pol, pre = ra.radamw_policy_loss, ra.radamw_preference_loss
    for bad in (ra.policy_options(-0.1), ra.policy_options(1.1), ra.policy_options(0.2, -1.0),
                ra.policy_options(0.2, float("inf")), ra.policy_options(kl_coef=-1.0),
                ra.policy_options(kl_coef=NAN), ra.policy_options(kl_coef=0.1)):
        refused(-1, lambda: pol(*args, bad, *outs))  # the last: no reference
    opts = ra.policy_options()
    refused(-1, lambda: pol(*args, opts, *outs, grad=torch.empty_like(x), grad_scale=NAN))
    refused(-3, lambda: pol(*args, opts, o["total"], o["loss"], o["loss"]))
    refused(-3, lambda: pol(*args, opts, *outs, weights=o["loss"]))
    wide = torch.randn((n, 2 * vocab), device=DEV)
    refused(-3, lambda: pol(wide[:, :vocab], labels, None, adv, opts, *outs, grad=wide[:, vocab:]))
    refused(-4, lambda: pol(*args, opts, *outs, row_stats=torch.empty(4 * n + 1, device=DEV)[1:]))
    p = (torch.zeros(1, device=DEV), torch.zeros(1, device=DEV), torch.zeros(2, device=DEV), torch.zeros(n, device=DEV))
    off = torch.tensor([0, 3, 6], device=DEV)
    for bad in (ra.preference_options(-1.0), ra.preference_options(NAN), ra.preference_options(0.1, 1.5)):
        refused(-1, lambda: pre(x, labels, off, torch.zeros(2, device=DEV), bad, *p, st))
    refused(-1, lambda: pre(x, labels, off[:1], torch.zeros(0, device=DEV), ra.preference_options(), p[0],
                            torch.zeros(0, device=DEV), torch.zeros(0, device=DEV), p[3], st))
    for bad in (lambda: pol(x.double(), labels, None, adv, opts, *outs), lambda: pol(x, labels[:-1], None, adv, opts, *outs),
                lambda: pol(x, labels, None, adv.double(), opts, *outs), lambda: pol(x.t(), labels, None, adv, opts, *outs),
                lambda: pol(*args, opts, *outs, grad=torch.empty_like(x, dtype=BF16)),
                lambda: pol(*args, opts, *outs, row_stats=st[:-1]), lambda: pol(x.cpu(), labels, None, adv, opts, *outs),
                lambda: pre(x, labels, off.int(), torch.zeros(2, device=DEV), ra.preference_options(), *p, st),
                lambda: ra.radamw_logits_grad(x, labels, st, None)):
        with pytest.raises(ValueError):
            bad()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.capture_begin(capture_error_mode="relaxed")
        try:
            refused(-1, lambda: pol(*args, opts, *outs))
            refused(-1, lambda: pre(x, labels, off, torch.zeros(2, device=DEV), ra.preference_options(), *p, st))
            refused(-1, lambda: ra.radamw_logits_grad(x, labels, st, torch.empty_like(x)))
            adv.add_(0)
        finally:
            graph.capture_end()
    torch.cuda.synchronize()
    assert ra.radamw_launch_count() == before
    assert all(bool(v.isnan().all()) for v in o.values())
