"""GPU tests of the residual norms and their gradient where many rows meet:
several rows to a worker at every shape of a row's lanes, more rows than one
launch has, more than 2^31 elements."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from block_helpers import Residual
from gpu_helpers import DEV, announce
from test_gpu_residual import COUNTER, SEED, Case, normal
from vocab_helpers import U, close

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


# three rows and more to a worker, at every shape of a row's lanes, with and without the parts that are known at compile
# time, gate rows that end inside a worker
WORKERS = [dict(n=n, dim=d, stream=s, branch=BF16, weight=w, gate=g, gate_type=BF16, per=per, post=post, p=p)
           for n, d in ((1300, 512), (1100, 2048), (1030, 4096), (771, 8192)) for s in (F32, BF16)
           for w, g, per, post, p in ((F32, "column", None, True, 0.1), (BF16, "sequence", 7, True, 0.0),
                                      (F32, "element", None, True, 0.1), (F32, None, None, False, 0.0))]
WORKERS += [dict(n=515, dim=d, stream=s, branch=BF16, weight=F32, gate=g, gate_type=F32, per=per, post=post, p=0.1)
            for d, s in ((8200, F32), (8193, BF16), (16384, BF16), (16383, F32))
            for g, per, post in (("sequence", 5, True), ("element", None, True), (None, None, False))]
WORKERS += [dict(n=515, dim=d, stream=s, branch=BF16, weight=F32, gate=g, gate_type=F32, per=per, post=post, p=0.1)
            for d, s, g, per, post in ((16392, F32, "sequence", 5, True), (16385, BF16, None, None, False),
                                       (32768, BF16, "column", None, True))]


@pytest.mark.parametrize("kw", WORKERS, ids=lambda kw: "-".join(str(v).replace("torch.", "") for v in kw.values()))
def test_workers_of_several_rows(kw):
    announce(f"residual backward {kw}")
    Case(**kw).backward()


@pytest.mark.parametrize("stream", [F32, BF16])
def test_more_rows_than_a_launch(stream):
    """2^21 + 5 rows: those on both sides of the launches' border are what a
    call of their own gives, which is held to the plain form."""
    announce(f"residual 2^21 + 5 rows {stream}")
    n, dim, border = (1 << 21) + 5, 8, 1 << 21
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.empty((n, dim), dtype=stream, device=DEV).normal_(generator=g)
    y = torch.empty((n, dim), dtype=BF16, device=DEV).normal_(generator=g)
    w, gate = (normal((dim,), F32, s, 0.1, 1.0) for s in (1, 2))
    per = border - 3  # the second gate row begins before the border
    gates = torch.stack([gate, -gate])
    h, out, rstd = torch.empty_like(x), torch.empty_like(y), torch.full((2, n), 7.0, device=DEV)

    def call(a, b, gate_rows, per, h, out, rstd):
        ra.radamw_residual_norm(x[a:b], y[a:b], ra.residual_options(p=0.2, seed=SEED, offset=COUNTER, first_row=a),
                                gate=gate_rows.to(DEV), rows_per_gate=per, post_weight=w.to(DEV), pre_weight=w.to(DEV),
                                h=h, out=out, rstd=rstd)

    call(0, n, gates, per, h, out, rstd)
    assert bool(h.isfinite().all()) and bool((rstd != 7).all())
    for a, b, row in ((0, 5, 0), (border - 6, border - 3, 0), (border - 3, border, 1), (border, n, 1)):
        h2, out2, r2 = torch.empty_like(x[a:b]), torch.empty_like(y[a:b]), torch.empty((2, b - a), device=DEV)
        call(a, b, gates[row:row + 1], n, h2, out2, r2)
        assert torch.equal(h[a:b], h2) and torch.equal(out[a:b], out2) and torch.equal(rstd[:, a:b], r2), (a, b)
        ref = Residual(x[a:b].cpu(), y[a:b].cpu(), gates[row:row + 1], per=n, post=w, pre=w, p=0.2, seed=SEED,
                       counter=COUNTER, first_row=a).forward()
        close(h2, *ref["h"], "h")
        close(out2, *ref["out"], "out")


def test_gradient_of_long_arrays():
    """More than 2^31 elements, in place: the last rows are those of a call of
    their own, and the sums over rows are those of the parts."""
    announce("residual gradient 70000 x 32768 bf16")
    n, dim, k = 70000, 32768, 64
    new = lambda seed: torch.empty((n, dim), dtype=BF16, device=DEV).normal_(  # noqa: E731
        generator=torch.Generator("cuda").manual_seed(seed))
    h, y, dh, dout = (new(s) for s in range(4))
    w = torch.ones(dim, device=DEV)
    gate = torch.full((1, dim), 0.5, device=DEV)
    rstd = torch.rand((2, n), device=DEV, generator=torch.Generator("cuda").manual_seed(9)) + 0.5

    def call(a, b, dh, dout, gx, gb):
        sums = [torch.empty(dim, device=DEV), torch.empty(dim, device=DEV), torch.empty((1, dim), device=DEV)]
        ws = torch.empty(ra.radamw_residual_grad_workspace_bytes(b - a, dim, n), dtype=torch.uint8, device=DEV)
        ra.radamw_residual_norm_grad(h[a:b], y[a:b], ra.residual_options(p=0.1, seed=1, offset=2, first_row=a),
                                     rstd[:, a:b].contiguous(), ws, grad_h=dh, grad_out=dout, grad_x=gx, grad_branch=gb,
                                     gate=gate, rows_per_gate=n, post_weight=w, pre_weight=w, grad_post_weight=sums[0],
                                     grad_pre_weight=sums[1], grad_gate=sums[2])
        return [s.reshape(-1).double() for s in sums]

    last = torch.empty((k, dim), dtype=BF16, device=DEV), torch.empty((k, dim), dtype=BF16, device=DEV)
    call(n - k, n, dh[-k:], dout[-k:], *last)
    parts = [0.0, 0.0, 0.0]
    step = 17500
    gx, gb = torch.empty((step, dim), dtype=BF16, device=DEV), torch.empty((step, dim), dtype=BF16, device=DEV)
    for a in range(0, n, step):
        parts = [p + s for p, s in zip(parts, call(a, a + step, dh[a:a + step], dout[a:a + step], gx, gb))]
    sums = call(0, n, dh, dout, dh, dout)
    assert torch.equal(dh[-k:], last[0]) and torch.equal(dout[-k:], last[1])
    # A worker adds its rows in FP32, each sum rounded by half a step of what it has become: n / 256 = 274 rows here and
    # 69 in a part.  A term is a product of values whose squares average 1 or less of which the root of the sum of
    # squares is at most 5 sqrt(n) times their size, a worker's sum 5 sqrt(274) of it: 4 is more than any of those sizes'
    # root mean square (rstd up to 1.5, twice; dropout's factor 1.12).
    worker = 274
    bound = 4.0 * 5 * worker ** 0.5 * U * worker * 256 * 1.3
    for name, whole, part in zip(("post", "pre", "gate"), sums, parts):
        assert bool(whole.isfinite().all()) and float(whole.abs().max()) > 10
        assert float((whole - part).abs().max()) <= bound, name
