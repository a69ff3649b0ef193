"""GPU tests of the balance loss over groups that are switched off."""
import pytest
import torch

from block_helpers import balance
from gpu_helpers import announce
from test_gpu_balance import inputs, run
from vocab_helpers import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zero", [0.0, -0.0])
@pytest.mark.parametrize("score,z", [("softmax", 0.1), ("softmax", 0.0), ("sigmoid", 0.0)])
@pytest.mark.parametrize("grad", [True, False])
def test_a_group_of_weight_zero_has_a_zero_gradient(score, z, grad, zero):
    """Whatever its logits are; what is counted of it stays, and its own loss
    is what they make it."""
    announce(f"balance weight {zero} {score} z={z} grad={grad}")
    x, ids, mask = inputs(400, 20, 2, masked=0.2)
    kw = dict(bounds=[0, 100, 250, 400], z=z, score=score, weights=torch.tensor([0.75, zero, -0.5]))
    ref = balance(x, ids, mask, **kw)
    x[100:250:3, 4] = float("nan")
    x[101:250:3, 7] = float("inf")
    got = run(x, ids, mask, grad=grad, **kw)
    assert bool(got["loss"][1].isnan()) and not got["grad"][100:250].any()
    assert torch.equal(got["counts"].cpu().long(), ref["counts"]) and torch.equal(got["tokens"].cpu().long(), ref["tokens"])
    for k in ("loss", "mean_prob"):
        close(got[k][[0, 2]], ref[k][0][[0, 2]], ref[k][1][[0, 2]], k)
    for k in ("total", "grad"):
        close(got[k], *ref[k], k)


def test_a_batch_of_weight_zero():
    announce("balance weight 0, one group")
    for n in (100, 9000):  # one workgroup, several
        x, ids, _ = inputs(n, 16, 2)
        x[3, 5] = float("nan")
        for grad in (True, False):
            got = run(x, ids, weights=torch.zeros(1), z=0.1, grad=grad)
            assert float(got["total"]) == 0 and not got["grad"].any()
