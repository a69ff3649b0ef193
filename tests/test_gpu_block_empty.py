"""GPU tests of the autograd forms on batches without rows, as a micro-batch
may be."""
import pytest
import torch

from gpu_helpers import DEV, announce
from optimizer_step_dl_amd.functional import balance_loss, dropout, embedding, policy_loss, residual_norm

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("shape", [(0, 24), (3, 0, 24), (0, 5, 24)])
def test_gradients_without_rows(shape):
    """A sum hands its gradient on with strides of zero."""
    announce(f"gradients without rows {shape}")
    x, y = (torch.empty(shape, device=DEV, requires_grad=True) for _ in range(2))
    w, table = torch.ones(24, device=DEV, requires_grad=True), torch.ones((7, 24), device=DEV, requires_grad=True)
    ids = torch.empty(shape[:-1], dtype=torch.int64, device=DEV)
    for out, leaves in ((lambda: dropout(x, 0.5, seed=1), [x]), (lambda: residual_norm(x, y), [x, y]),
                        (lambda: residual_norm(x, y, post_weight=w), [x, y, w]),
                        (lambda: residual_norm(x, None, pre_weight=w), [x, w]), (lambda: embedding(ids, table), [table])):
        got = out()
        assert got.shape == x.shape
        for g, t in zip(torch.autograd.grad(got.sum(), leaves), leaves):
            assert g.shape == t.shape and bool((g == 0).all())


def test_inputs_without_rows():
    """Of a transposed tensor's none."""
    announce("inputs without rows")
    x = torch.ones((24, 9), device=DEV, requires_grad=True)
    none, labels, values = x.t()[:0], torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
    total = policy_loss(none, labels, values)[0] + balance_loss(none, labels[:, None].expand(0, 2))[0] + \
        residual_norm(none, none).sum() + dropout(none, 0.5, seed=1).sum()
    total.backward()
    assert float(total.detach()) == 0 and bool((x.grad == 0).all())


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("shape,gate_shape", [((0, 24), (24,)), ((0, 24), (1, 24)), ((3, 0, 24), (24,)), ((3, 0, 24), (3, 1, 24)),
                                              ((0, 5, 24), (24,)), ((0, 5, 24), (0, 1, 24)), ((0, 24), (0, 24)),
                                              ((3, 0, 24), (3, 0, 24))])
def test_gates_of_an_empty_batch(shape, gate_shape, post, pre):
    announce(f"residual_norm empty {shape} gate {gate_shape} post={post} pre={pre}")
    x = torch.empty(shape, device=DEV, requires_grad=True)
    y = torch.empty(shape, dtype=BF16, device=DEV, requires_grad=True)
    gate = torch.ones(gate_shape, dtype=BF16, device=DEV, requires_grad=True)
    weights = {k: torch.ones(24, device=DEV, requires_grad=True)
               for k, given in (("post_weight", post), ("pre_weight", pre)) if given}
    torch.full((1 << 20,), float("nan"), device=DEV)  # freed memory that gradients may be given
    got = residual_norm(x, y, gate=gate, p=0.1, seed=1, **weights)
    got = got if pre else (got,)
    assert [t.shape for t in got] == [x.shape] * len(got)
    assert [t.dtype for t in got] == [F32, BF16][:len(got)]
    sum(t.float().sum() for t in got).backward()
    for t in (x, y, gate, *weights.values()):
        assert t.grad.shape == t.shape and t.grad.dtype == t.dtype and bool((t.grad == 0).all())


def test_an_empty_batch_beside_others():
    """The gate's gradient of a step is that of the other micro-batches."""
    announce("residual_norm empty micro-batch")
    gate = torch.full((24,), 0.5, device=DEV, requires_grad=True)
    w = torch.ones(24, device=DEV, requires_grad=True)
    g = torch.Generator().manual_seed(1)
    x, y = (torch.randn((6, 24), generator=g).to(DEV) for _ in range(2))
    residual_norm(x, y, gate=gate, pre_weight=w)[1].square().sum().backward()
    want = gate.grad.clone(), w.grad.clone()
    residual_norm(x[:0], y[:0], gate=gate, pre_weight=w)[1].square().sum().backward()
    assert torch.equal(gate.grad, want[0]) and torch.equal(w.grad, want[1])
