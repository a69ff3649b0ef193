"""GPU tests of the residual norms where dropout leaves nothing of a row."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from block_helpers import Residual, keep_mask
from gpu_helpers import DEV, announce
from test_gpu_residual import COUNTER, SEED, Case
from vocab_helpers import close

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("n,dim,stream,branch,p", [
    (400, 3, F32, F32, 0.6), (400, 3, BF16, BF16, 0.6), (400, 8, F32, BF16, 0.9), (400, 8, F32, F32, 0.9),
    (400, 9, F16, F16, 0.9), (2100, 8, F32, BF16, 0.9), (2100, 5, F16, F16, 0.8), (2100, 12, F32, F16, 0.9),
    (64, 8200, F32, BF16, 1.0), (64, 8193, BF16, BF16, 1.0), (64, 4100, F32, F32, 1.0)])
def test_rows_that_are_dropped_whole(n, dim, stream, branch, p):
    """A branch of NaN whose row is dropped in every column: nothing of it
    reaches the stream, nor the norm before the next block."""
    announce(f"residual dropped rows {n} x {dim} {stream} {branch} p={p}")
    c = Case(n, dim, stream=stream, branch=branch, p=p)
    whole = ~keep_mask(n, dim, p, SEED, COUNTER).any(1)
    assert 20 <= int(whole.sum()) and (p == 1.0 or not bool(whole.all()))
    clean = Residual(c.x, c.y, None, **c.ref).forward()
    c.y[whole] = float("nan")
    h = torch.empty((n, dim), dtype=stream, device=DEV)
    out = torch.empty((n, dim), dtype=branch, device=DEV)
    ra.radamw_residual_norm(c.x.to(DEV), c.y.to(DEV), c.options(), h=h, out=out, post_weight=c.post.to(DEV),
                            pre_weight=c.pre.to(DEV))
    assert torch.equal(h.cpu()[whole], c.x[whole])
    for got, k in ((h, "h"), (out, "out")):
        close(got, *clean[k], k)
