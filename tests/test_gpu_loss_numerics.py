"""GPU tests of the losses where a row's exponents or its sum are hard to
hold: against the plain 64-bit forms, with and without the gradient (which
take different kernels)."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from gpu_helpers import announce
from test_gpu_losses import check_policy, check_preference, gen

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
