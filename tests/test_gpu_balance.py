"""GPU tests of radamw_balance_loss and radamw_balance_grad against their
plain 64-bit form."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from block_helpers import balance
from gpu_helpers import DEV, announce
from vocab_helpers import close

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inputs(n, experts, k, dtype=F32, ids=torch.int64, masked=0.0, stray=False, std=2.0):
    x = (std * torch.randn((n, experts), generator=gen(1))).to(dtype)
    i = torch.randint(-2 if stray else 0, experts + (3 if stray else 0), (n, k), generator=gen(2)).to(ids)
    mask = torch.rand(n, generator=gen(3)) >= masked if masked else None
    return x, i, mask


def run(x, ids, mask=None, bounds=None, weights=None, coef=0.01, z=0.0, score="softmax", scale=1.0, grad=True, pad=0,
        in_place=False):
    """One call; its outputs by name."""
    n, experts = x.shape
    groups = 1 if bounds is None else len(bounds) - 1
    buf = torch.full((n, experts + pad), 7.0, dtype=x.dtype, device=DEV)
    xd = buf[:, :experts]
    xd.copy_(x)
    out = {"total": torch.empty((), device=DEV), "loss": torch.empty(groups, device=DEV),
           "counts": torch.full((groups, experts), -7, dtype=torch.int32, device=DEV),
           "tokens": torch.full((groups,), -7, dtype=torch.int32, device=DEV),
           "mean_prob": torch.empty((groups, experts), device=DEV)}
    g = xd if in_place else torch.empty((n, experts), dtype=x.dtype, device=DEV) if grad else None
    ws = torch.full((ra.radamw_balance_workspace_bytes(n, experts, groups),), 255, dtype=torch.uint8, device=DEV)
    extra = dict(mask=None if mask is None else mask.to(DEV),
                 offsets=None if bounds is None else torch.tensor(bounds, dtype=ids.dtype, device=DEV),
                 weights=None if weights is None else weights.to(DEV))
    o = ra.balance_options(coef, z, score)
    ra.radamw_balance_loss(xd, ids.to(DEV), o, out["total"], out["loss"], out["counts"], out["tokens"], out["mean_prob"],
                           ws, grad=g, grad_scale=scale, **extra)
    if grad:
        out["grad"] = g
    elif not in_place:
        # the backward pass's gradient, its scale from the device
        g2 = torch.empty((n, experts), dtype=x.dtype, device=DEV)
        ra.radamw_balance_grad(xd, ids.shape[1], o, out["counts"], out["tokens"], g2, grad_scale=scale / 4,
                               upstream=torch.tensor(4.0, device=DEV), **extra)
        out["grad"] = g2
    if pad:
        assert bool((buf[:, experts:] == 7).all())
    return out


def check(got, ref):
    assert torch.equal(got["counts"].cpu().long(), ref["counts"]) and torch.equal(got["tokens"].cpu().long(), ref["tokens"])
    for k in ("mean_prob", "loss", "total", "grad"):
        close(got[k], *ref[k], k)


CASES = [
    dict(n=1, experts=1, k=1), dict(n=3, experts=4, k=2, dtype=BF16), dict(n=256, experts=8, k=2, dtype=BF16, z=0.001),
    dict(n=100, experts=5, k=1, dtype=F16, ids=torch.int32, scale=65536.0), dict(n=333, experts=16, k=4, masked=0.4, z=0.1),
    dict(n=1000, experts=64, k=6, stray=True), dict(n=700, experts=160, k=6, score="sigmoid", masked=0.2),
    dict(n=515, experts=256, k=8, z=0.001, dtype=F32), dict(n=515, experts=255, k=8, dtype=BF16, pad=3),
    dict(n=2000, experts=384, k=8, score="sigmoid", ids=torch.int32), dict(n=60, experts=513, k=3, z=0.01),
    dict(n=60, experts=1024, k=3, dtype=F16, scale=65536.0), dict(n=60, experts=1030, k=3, score="sigmoid"),
    dict(n=40, experts=2048, k=8, z=0.01), dict(n=40, experts=4096, k=8), dict(n=33, experts=4091, k=8, dtype=BF16),
    dict(n=70_001, experts=32, k=2, masked=0.1, z=0.001), dict(n=5000, experts=96, k=4, std=40.0),
    dict(n=5000, experts=96, k=4, std=40.0, score="sigmoid")]
# one workgroup's batch and the next larger ones
CASES += [dict(n=n, experts=e, k=3, dtype=d, z=0.01, masked=0.3) for n, e, d in
          ((2048, 8, F32), (2049, 8, F32), (32, 512, BF16), (33, 512, F32), (103, 160, F32), (5461, 3, F16), (16384, 1, BF16))
          if e >= 3 or d == BF16]
GROUPED = [dict(n=300, experts=24, k=2, bounds=[0, 100, 100, 101, 300], z=0.01),
           dict(n=5000, experts=64, k=6, bounds=[7, 8, 2000, 2000, 4900], masked=0.3, score="sigmoid", weighted=True),
           dict(n=4096, experts=128, k=8, bounds=list(range(0, 4097, 64)), dtype=BF16, ids=torch.int32, weighted=True),
           dict(n=64, experts=8, k=2, bounds=list(range(65)), z=0.1), dict(n=10, experts=9, k=2, bounds=[4] * 40 + [5])]


def case(kw):
    kw = dict(kw)
    x, ids, mask = inputs(kw.pop("n"), kw.pop("experts"), kw.pop("k"), kw.pop("dtype", F32), kw.pop("ids", torch.int64),
                          kw.pop("masked", 0.0), kw.pop("stray", False), kw.pop("std", 2.0))
    if kw.pop("weighted", False):
        kw["weights"] = torch.randn(len(kw["bounds"]) - 1, generator=gen(4))
    pad = kw.pop("pad", 0)
    return x, ids, mask, kw, pad


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("kw", CASES + GROUPED, ids=lambda kw: "-".join(str(v)[:24] for v in kw.values()))
def test_balance(kw, grad):
    announce(f"balance {str(kw)[:200]} grad={grad}")
    x, ids, mask, kw, pad = case(kw)
    check(run(x, ids, mask, grad=grad, pad=pad, **kw), balance(x, ids, mask, **kw))


def test_equal_calls_and_in_place():
    announce("balance in place")
    x, ids, mask = inputs(3000, 40, 3, BF16, masked=0.2)
    kw = dict(bounds=[0, 1000, 2900], z=0.01)
    a, b = (run(x, ids, mask, **kw) for _ in range(2))
    c = run(x, ids, mask, in_place=True, **kw)
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


def test_rows_that_take_no_part_hold_anything():
    """NaN logits and stray ids in masked rows and outside the groups."""
    announce("balance masked garbage")
    x, ids, mask = inputs(500, 20, 2, masked=0.5)
    kw = dict(bounds=[50, 200, 450], z=0.1)
    ref = balance(x, ids, mask, **kw)
    dead = ~mask
    dead[:50] = dead[450:] = True
    x[dead] = float("nan")
    ids[dead] = 1 << 40
    for grad in (True, False):
        got = run(x, ids, mask, grad=grad, **kw)
        check(got, ref)
        assert bool((got["grad"].cpu()[dead] == 0).all())


def test_infinite_logits():
    """Experts that are masked with -inf have no probability and no gradient;
    a row of them alone adds nothing; the types' lowest values are numbers."""
    announce("balance -inf")
    x, ids, _ = inputs(200, 12, 2)
    x[:, 3] = -float("inf")
    x[17] = -float("inf")
    x[18] = torch.finfo(F32).min
    x[19, :5] = torch.finfo(F32).min
    for score, z in (("softmax", 0.0), ("sigmoid", 0.0)):
        ref = balance(x, ids, None, score=score, z=z)
        got = run(x, ids, None, score=score, z=z)
        check(got, ref)
        inf = x == -float("inf")  # row 18 holds the lowest value there
        assert bool((got["grad"].cpu()[inf] == 0).all()) and int(inf.sum()) == 12 + 198 - 1
        assert bool(got["grad"].isfinite().all())
    # the z-loss of such a row is left out, the others' is there
    x[18] = 1.0
    x[19, :5] = -3.0
    check(run(x, ids, None, z=0.1), balance(x, ids, None, z=0.1))


def test_nan_stays_in_its_row():
    announce("balance NaN")
    x, ids, _ = inputs(64, 8, 2)
    x[5, 2] = float("nan")
    got = run(x, ids)
    assert bool(got["grad"][5].isnan().all()) and bool(got["total"].isnan())
    rows = [i for i in range(64) if i != 5]
    close(got["grad"][rows], balance(x.nan_to_num(0.0), ids)["grad"][0][rows],
          balance(x.nan_to_num(0.0), ids)["grad"][1][rows], "grad")


@pytest.mark.parametrize("groups", [1, 3])
def test_no_rows(groups):
    announce(f"balance no rows, {groups} groups")
    x, ids = torch.empty((0, 6)), torch.empty((0, 2), dtype=torch.int64)
    got = run(x, ids, bounds=None if groups == 1 else [0] * (groups + 1))
    assert float(got["total"]) == 0 and bool((got["loss"] == 0).all())
    assert bool((got["counts"] == 0).all()) and bool((got["tokens"] == 0).all()) and bool((got["mean_prob"] == 0).all())


def test_all_rows_masked():
    announce("balance all masked")
    x, ids, _ = inputs(130, 16, 2)
    got = run(x, ids, torch.zeros(130, dtype=torch.bool), z=0.5)
    assert float(got["total"]) == 0 and not got["counts"].any() and not got["grad"].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_balanced_router_has_no_gradient(score):
    """Experts that are chosen equally often cost the same: the gradient is a
    difference of equal terms, and exactly zero."""
    announce(f"balance of a balanced router {score}")
    x, _, _ = inputs(1557, 6, 1)
    ids = torch.arange(6).expand(1557, 6).contiguous()
    for grad in (True, False):
        got = run(x, ids, None, bounds=[0, 500, 1557], score=score, grad=grad)
        assert not got["grad"].any() and bool((got["counts"] == got["tokens"][:, None]).all())
    # one choice more of one expert: the difference has all its digits, up to the probabilities' own error.  It is 1 /
    # 1557 of the count, and the bound of the sum over all of it 1557 times as large as what is asked for here.
    ids = ids.clone()
    ids[0, 0] = 1
    ref = balance(x, ids, score=score)["grad"][0]
    got = run(x, ids, score=score)["grad"].cpu().double()
    # probabilities: 80 u (3 u |x| and 70 u of the sum among them), twice in a product, and the products' roundings
    assert float((got - ref).abs().max()) <= 400 * 2.0 ** -24 * float(ref.abs().max())


def test_counts_summed_over_ranks():
    """Gradients from counts and tokens that two halves of a batch summed are
    the whole batch's."""
    announce("balance two halves")
    x, ids, _ = inputs(600, 32, 4)
    whole = run(x, ids, z=0.01)
    halves = [run(x[s], ids[s], z=0.01, grad=False) for s in (slice(0, 250), slice(250, 600))]
    counts, tokens = (halves[0][k] + halves[1][k] for k in ("counts", "tokens"))
    assert torch.equal(counts, whole["counts"]) and torch.equal(tokens, whole["tokens"])
    grad = torch.empty((600, 32), device=DEV)
    for s in (slice(0, 250), slice(250, 600)):
        ra.radamw_balance_grad(x[s].to(DEV), 4, ra.balance_options(0.01, 0.01), counts, tokens, grad[s])
    assert torch.equal(grad, whole["grad"])


def test_bad_offsets_stay_in_bounds():
    """Offsets outside 0 .. n are clamped for every access."""
    announce("balance bad offsets")
    x, ids, _ = inputs(300, 8, 2)
    got = run(x, ids, bounds=[-100, 50, 10_000_000])
    ref = balance(x, ids, None, bounds=[0, 50, 300])
    check(got, ref)


def test_refusals_on_the_device():
    announce("balance refusals")
    x, ids = torch.zeros((8, 4), device=DEV), torch.zeros((8, 2), dtype=torch.int64, device=DEV)
    o = ra.balance_options()

    def call(**kw):
        a = dict(logits=x, ids=ids, total=torch.empty((), device=DEV), loss=torch.empty(1, device=DEV),
                 counts=torch.empty((1, 4), dtype=torch.int32, device=DEV),
                 tokens=torch.empty(1, dtype=torch.int32, device=DEV), mean_prob=torch.empty((1, 4), device=DEV),
                 workspace=torch.empty(ra.radamw_balance_workspace_bytes(8, 4), dtype=torch.uint8, device=DEV))
        extra = {k: kw.pop(k) for k in list(kw) if k not in a}
        a.update(kw)
        ra.radamw_balance_loss(a["logits"], a["ids"], o, a["total"], a["loss"], a["counts"], a["tokens"], a["mean_prob"],
                               a["workspace"], **extra)

    call()
    for kw in (dict(ids=ids[:7]), dict(ids=ids.float()), dict(ids=ids.reshape(-1)), dict(counts=torch.empty((1, 4), device=DEV)),
               dict(mask=torch.ones(8, device=DEV)), dict(mask=torch.ones(7, dtype=torch.bool, device=DEV)),
               dict(loss=torch.empty(2, device=DEV)), dict(weights=torch.ones(2, device=DEV)),
               dict(offsets=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(grad=x.half())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw, status in ((dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV)), -5),
                       (dict(mean_prob=x[:1]), -3), (dict(grad=x[:, :]), 0)):
        if status == 0:
            call(**kw)
            continue
        with pytest.raises(ra.RadamwError) as e:
            call(**kw)
        assert e.value.status == status
