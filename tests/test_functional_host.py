"""CPU tests of the autograd forms: what they hand to the library, with the
library's calls replaced by recorders."""
import pytest
import torch

from optimizer_step_dl_amd import _abi, functional

F32 = torch.float32


@pytest.fixture
def default_dtype(request):
    before = torch.get_default_dtype()
    torch.set_default_dtype(request.param)
    yield request.param
    torch.set_default_dtype(before)


@pytest.mark.parametrize("default_dtype", [torch.float64, torch.bfloat16, torch.float16, F32], indirect=True)
def test_losses_under_any_default_dtype(default_dtype, monkeypatch):
    """Totals, losses, log-probabilities, records and default weights are
    FP32, whatever torch's default is."""
    seen = []

    def record(logits, *args, **kw):
        values = [a for a in (*args, *kw.values()) if torch.is_tensor(a) and a.is_floating_point()]
        seen.append([v.dtype for v in values if v is not kw.get("grad")])
        for v in values:
            v.zero_()

    monkeypatch.setattr(_abi, "radamw_policy_loss", record)
    monkeypatch.setattr(_abi, "radamw_preference_loss", record)
    monkeypatch.setattr(_abi, "radamw_logits_grad", lambda logits, labels, stats, grad, upstream: seen.append(
        [stats.dtype, upstream.dtype]))
    x = torch.zeros((6, 5), dtype=F32, requires_grad=True)
    labels = torch.tensor([0, 1, -100, 4, 2, 3])
    total, loss, logp = functional.policy_loss(x, labels, torch.zeros(6))
    total.backward()
    assert total.dtype == loss.dtype == logp.dtype == F32
    total, loss, seq = functional.preference_loss(x, labels, torch.tensor([0, 2, 6]), torch.zeros(2))
    total.backward()
    assert total.dtype == loss.dtype == seq.dtype == F32
    # advantages, total, loss, logp, weights, records; the records and the upstream value;
    # the reference's sums, total, loss, seq_logp, logp, records, weights; the same two
    assert [len(d) for d in seen] == [6, 2, 7, 2]
    assert all(d == F32 for call in seen for d in call), seen
