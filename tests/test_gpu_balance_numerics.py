"""GPU tests of the balance loss's exponentials: errors to one side add up over
a batch, where roundings average out."""
import pytest
import torch

from gpu_helpers import announce
from test_gpu_balance import gen, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score,top", [("softmax", 0.0), ("softmax", 3.0), ("sigmoid", 0.0), ("sigmoid", -20.0), ("sigmoid", -300.0)])
def test_probabilities_lean_to_no_side(score, top):
    """The mean relative error of 65536 probabilities of exp(-d), d from 40 to
    60, each of a row and a group of its own.

    The exponent d log2 e is below 87: its roundings (of the difference, of two
    products) are at most three halves of a step of 2^-17, evenly spread, ln 2
    times that in the probability, and their mean over 65536 of them 256 times
    less: 3.1e-8, five times the standard deviation of evenly spread ones.
    v_exp_f32 is within 1 ulp, 1.2e-7, to whatever side, which the sums,
    reciprocals and products (7 roundings of at most 6e-8, even) leave as it
    is.  log2 e rounded to FP32 would move the mean by 50 * 1.3e-8 = 6.7e-7."""
    announce(f"balance numerics {score} top={top}")
    n = 65536
    x = torch.zeros((n, 2))
    x[:, 0] = top
    x[:, 1] = top - (40 + 20 * torch.rand(n, generator=gen(1)))
    ids = torch.zeros((n, 1), dtype=torch.int64)
    got = run(x, ids, bounds=list(range(n + 1)), score=score)["mean_prob"].cpu().double()
    z = x.double()
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)
    error = got[:, 1] / s[:, 1] - 1
    assert abs(float(error.mean())) < 1.2e-7 + 3.1e-8 + 7 * 6e-8 / 256
    assert float(error.abs().max()) < 87 * 2.0 ** -22
