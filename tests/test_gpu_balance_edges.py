"""GPU tests of the balance loss where its values are far from ordinary:
sigmoid scores below FP32's range."""
import math

import pytest
import torch

from block_helpers import balance
from gpu_helpers import announce
from test_gpu_balance import check, gen, inputs, run

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# the last FP32 number whose score 1 / (1 + exp(-x)) is a number in 64 bits, and the next
LAST, BEYOND = -709.78265380859375, -709.78271484375


def far(n, experts, k, dtype, lo, hi):
    x, ids, mask = inputs(n, experts, k, dtype, masked=0.2)
    x = (torch.rand((n, experts), generator=gen(7)) * (hi - lo) + lo).to(dtype)
    return x, ids, mask


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("n,experts,dtype", [(40, 2, F32), (500, 16, F32), (3000, 160, F32), (3001, 37, BF16), (700, 96, F16),
                                             (60, 1030, F32), (33, 4091, BF16), (40, 2048, F32)])
@pytest.mark.parametrize("lo,hi", [(-92.0, -89.0), (-700.0, -88.0), (-8.0, -3.0), (-104.0, -80.0), (-500.0, -490.0)])
def test_rows_of_far_negative_logits(n, experts, dtype, lo, hi, grad):
    """Scores that FP32 holds as zeros have shares all the same."""
    announce(f"balance sigmoid {n} x {experts} {dtype} logits {lo} .. {hi} grad={grad}")
    x, ids, mask = far(n, experts, 2, dtype, lo, hi)
    ref = balance(x, ids, mask, score="sigmoid", coef=1.0)
    assert abs(float(ref["mean_prob"][0].sum()) - 1.0) < 1e-9
    check(run(x, ids, mask, grad=grad, score="sigmoid", coef=1.0), ref)


def test_shares_of_a_pair():
    announce("balance sigmoid pair")
    x, ids = torch.tensor([[-90.0, -92.0]]), torch.tensor([[0]])
    p = 1 / (1 + math.exp(-2.0))
    got = run(x, ids, score="sigmoid")["mean_prob"].cpu().double()
    assert float((got - torch.tensor([[p, 1 - p]])).abs().max()) < 1e-6


def test_far_rows_beside_ordinary_ones_and_in_place():
    """Rows of both kinds side by side in a wave, in groups, with experts that
    are masked; the gradient over the logits has the same bits."""
    announce("balance sigmoid far rows beside others")
    x, ids, mask = inputs(1000, 24, 3, F32, masked=0.1)
    x[::3] -= 120.0
    x[1::5] -= 400.0
    x[:, 5] = -math.inf
    kw = dict(bounds=[3, 400, 400, 990], score="sigmoid", weights=torch.tensor([0.5, 1.0, -2.0]))
    ref = balance(x, ids, mask, **kw)
    got = run(x, ids, mask, **kw)
    check(got, ref)
    assert bool((got["grad"][:, 5] == 0).all())
    again = run(x, ids, mask, in_place=True, **kw)
    for k in got:
        assert torch.equal(got[k], again[k]), k


def test_scores_of_zero():
    """A score that is 0 in 64 bits is 0: such a row has no probabilities, such
    an expert no part of a row's."""
    announce("balance sigmoid zero scores")
    x, ids, _ = inputs(64, 12, 2)
    x[4] = BEYOND
    x[5] = LAST
    x[6] = -1e30
    x[7] = torch.finfo(F32).min
    x[8] = torch.linspace(-712.0, -708.0, 12)
    x[9, 1:] = -720.0
    ref = balance(x, ids, score="sigmoid", coef=1.0)
    got = run(x, ids, score="sigmoid", coef=1.0)
    check(got, ref)
    grad = got["grad"].cpu()
    assert not grad[4].any() and not grad[6].any() and not grad[7].any() and bool(grad[5].any())
    for row in (8, 9):
        assert bool((grad[row, x[row] <= BEYOND] == 0).all()) and bool(grad.isfinite().all())
    # a NaN beside them stays in its row
    x[8, 3] = float("nan")
    assert bool(run(x, ids, score="sigmoid")["grad"][8].isnan().all())
