"""CPU tests of how the autograd forms lay out their rows."""
import pytest
import torch

from optimizer_step_dl_amd.functional import _rows


@pytest.mark.parametrize("t", [torch.ones(()).expand(0, 24), torch.ones((24, 9)).t()[:0], torch.ones(()).expand(3, 0, 24),
                               torch.ones(()).expand(5, 24), torch.ones((24, 9)).t(), torch.ones((24, 1)).t(),
                               torch.ones((6, 24))[:, ::2], torch.ones((1, 24))[:, ::2], torch.ones((2, 3, 24)).permute(1, 0, 2),
                               torch.ones((0, 24)), torch.ones(24)], ids=lambda t: f"{tuple(t.shape)} {t.stride()}")
def test_rows_have_unit_columns_and_do_not_overlap(t):
    r = _rows(t)
    rows, cols = r.shape
    assert rows * cols == t.numel() and cols == t.shape[-1]
    assert r.stride(1) == 1 and (rows <= 1 or r.stride(0) >= cols)
    assert torch.equal(r.reshape(t.shape), t)


def test_rows_that_fit_are_not_copied_and_copies_carry_gradients():
    x = torch.ones((6, 40), requires_grad=True)
    part = x[:, 3:27]
    assert _rows(part).data_ptr() == part.data_ptr()
    (2 * _rows(x.t())).sum().backward()
    assert bool((x.grad == 2).all())
