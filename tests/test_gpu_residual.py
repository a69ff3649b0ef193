"""GPU tests of radamw_residual_norm and its gradient against their plain
64-bit forms."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from block_helpers import Residual
from gpu_helpers import DEV, announce
from vocab_helpers import close

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
SEED, COUNTER = 0x0123456789ABCDEF, (3 << 32) + 17


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, dtype, seed, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen(seed)) * std + mean).to(dtype)


def spread(t, stride, start):
    """A device copy of t [n, dim] whose rows are `stride` elements apart, and
    its memory."""
    n, dim = t.shape
    buf = torch.full((start + max(1, n) * stride,), 7.0, dtype=t.dtype, device=DEV)
    view = buf.as_strided((n, dim), (stride, 1), start)
    view.copy_(t)
    return view, buf


class Case:
    def __init__(self, n, dim, stream=F32, branch=F32, weight=F32, gate=None, gate_type=F32, per=None, post=True, pre=True,
                 p=0.0, scale=1.0, offset=0.0, eps=1e-6, pad=0, start=0, first=0, grad_h=True):
        self.n, self.dim, self.pad, self.start = n, dim, pad, start
        self.branch_type = branch
        per = {None: None, "column": max(1, n), "element": 1}.get(gate, per)
        self.per = per
        self.x = normal((n, dim), stream, 1, 3.0)
        self.y = normal((n, dim), branch, 2) if gate is not None or post or branch is not None else None
        rows = 0 if gate is None else -(-n // per)
        self.gate = None if gate is None else normal((rows, dim), gate_type, 3, 0.3, 0.5)
        self.post = normal((dim,), weight, 4, 0.1, 1.0 - offset) if post else None
        self.pre = normal((dim,), weight, 5, 0.1, 1.0 - offset) if pre else None
        self.dh = normal((n, dim), stream, 6) if grad_h else None
        self.dout = normal((n, dim), branch, 7) if pre else None
        self.kw = dict(eps=eps, residual_scale=scale, weight_offset=offset, p=p, seed=SEED, offset=COUNTER,
                       first_row=first)
        self.ref = dict(per=per, post=self.post, pre=self.pre, eps=eps, offset=offset, scale=scale, p=p, seed=SEED,
                        counter=COUNTER, first_row=first)

    def options(self):
        kw = dict(self.kw)
        return ra.residual_options(**kw)

    def put(self, t):
        return None if t is None else spread(t, self.dim + self.pad, self.start)[0]

    def shared(self):
        return dict(gate=self.put(self.gate), rows_per_gate=self.per,
                    post_weight=None if self.post is None else self.post.to(DEV),
                    pre_weight=None if self.pre is None else self.pre.to(DEV))

    def forward(self):
        n, dim = self.n, self.dim
        empty = torch.empty((n, dim))
        h, hbuf = spread(empty.to(self.x.dtype), dim + self.pad + 1, self.start)
        out, obuf = (None, None) if self.pre is None else spread(empty.to(self.branch_type), dim + self.pad, self.start + 1)
        rstd = torch.full((2, n), 7.0, device=DEV)
        ra.radamw_residual_norm(self.put(self.x), self.put(self.y), self.options(), h=h, out=out, rstd=rstd,
                                **self.shared())
        ref = Residual(self.x, self.y, self.gate, **self.ref).forward()
        got = {"h": h, "out": out, "rstd_branch": rstd[0], "rstd_h": rstd[1]}
        for k, (v, slack) in ref.items():
            close(got[k], v, slack, k)
        if self.post is None:
            assert bool((rstd[0] == 7).all())
        # nothing between the rows is written
        for t, buf in ((h, hbuf), (out, obuf)):
            if t is not None:
                t.fill_(7.0)
                assert bool((buf == 7).all())

    def backward(self, in_place=False):
        n, dim = self.n, self.dim
        r = Residual(self.x, self.y, self.gate, **self.ref)
        rstd = torch.stack([(v.double().square().mean(1) + self.kw["eps"]).rsqrt().float() for v in (self.y, self.x)])
        ref = r.backward(self.dh, self.dout, rstd.reshape(-1))
        dh, dout = self.put(self.dh), self.put(self.dout)
        gx = dh if in_place else spread(torch.empty((n, dim), dtype=self.x.dtype), dim + 1, 0)[0]
        gb = dout if in_place and dout is not None else self.put(torch.empty((n, dim), dtype=self.y.dtype))
        got = {"x": gx, "branch": gb,
               "gate": None if self.gate is None else self.put(torch.empty_like(self.gate)),
               "post": None if self.post is None else torch.empty_like(self.post, device=DEV),
               "pre": None if self.pre is None else torch.empty_like(self.pre, device=DEV)}
        need = ra.radamw_residual_grad_workspace_bytes(n, dim, self.per or 1)
        workspace = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN, to be read nowhere

        def call():
            ra.radamw_residual_norm_grad(self.put(self.x), self.put(self.y), self.options(), rstd.to(DEV), workspace,
                                         grad_h=dh, grad_out=dout, grad_x=gx, grad_branch=gb, grad_gate=got["gate"],
                                         grad_post_weight=got["post"], grad_pre_weight=got["pre"], **self.shared())

        call()
        for k, (v, slack) in ref.items():
            close(got[k], v, slack, "grad_" + k)
        if not in_place:  # equal calls give equal bits
            first = {k: v.clone() for k, v in got.items() if v is not None}
            call()
            assert all(torch.equal(first[k], got[k]) for k in first)


TYPES = [(F32, F32, F32, F32), (F32, BF16, F32, BF16), (F32, F16, F16, F32), (BF16, BF16, BF16, BF16),
         (F16, F16, F32, F16)]
CASES = [dict(n=37, dim=200, stream=s, branch=b, weight=w, gate="column", gate_type=g, p=0.3, scale=0.5)
         for s, b, w, g in TYPES]
# every width of a row's lanes, multiples of eight and others
CASES += [dict(n=5, dim=d, stream=F32, branch=BF16, weight=BF16, gate="element", gate_type=BF16, p=0.2, offset=1.0)
          for d in (1, 7, 8, 9, 63, 511, 512, 513, 1024, 1025, 2047, 2048, 2050, 4096, 4104, 5000, 8192, 8193, 16384,
                    16390, 32768, 32761)]
CASES += [
    # sums over many rows: several rows per worker, one gate row for all, per sequence, ragged sequences
    dict(n=1300, dim=64, gate="column", p=0.1), dict(n=1300, dim=264, gate="sequence", per=100),
    dict(n=4100, dim=72, stream=BF16, branch=BF16, weight=BF16, gate="sequence", gate_type=BF16, per=7),
    dict(n=2500, dim=136, gate="sequence", per=2, p=0.5), dict(n=2048, dim=520, gate="sequence", per=1999),
    dict(n=1025, dim=1024, stream=F32, branch=F16, weight=F32, gate="sequence", per=1024),
    dict(n=300, dim=2048, gate="element", gate_type=BF16), dict(n=1, dim=4096, gate="column", p=0.1),
    dict(n=255, dim=96, gate="column"), dict(n=257, dim=96, gate="column"),
    # norms that are absent
    dict(n=300, dim=130, post=False), dict(n=300, dim=130, pre=False, gate="column"),
    dict(n=300, dim=130, post=False, pre=False, gate="sequence", per=40, p=0.4), dict(n=9, dim=256, post=False, pre=False),
    dict(n=600, dim=512, post=False, p=0.9), dict(n=600, dim=768, pre=False, p=0.1, scale=-2.0),
    # no gradient from the stream, rows apart and unaligned, another first row, large eps
    dict(n=50, dim=100, grad_h=False), dict(n=50, dim=99, pad=3, start=1, stream=BF16, branch=BF16, weight=BF16, p=0.1),
    dict(n=50, dim=104, pad=5, start=3, stream=F32, branch=BF16, gate="element", gate_type=F16),
    dict(n=50, dim=64, first=2 ** 32 - 50, p=0.5), dict(n=20, dim=33, eps=0.5, offset=0.25, scale=0.0),
    dict(n=3, dim=40, p=1.0, gate="column")]


# rows that fill their lanes, with the parts that the gradient knows at compile time, and rows in pairs
CASES += [dict(n=n, dim=d, stream=s, branch=b, weight=F32, gate=g, gate_type=b, per=7 if g == "sequence" else None, post=post,
               p=p)
          for n, d in ((70, 512), (300, 1024), (33, 2048), (20, 4096), (9, 8192))
          for s, b in ((BF16, BF16), (F32, F16))
          for g, post, p in (("element", True, 0.3), (None, True, 0.0), ("sequence", True, 0.2), ("column", False, 0.1))]
CASES += [dict(n=2049, dim=d, stream=s, branch=b, weight=w, gate=g, gate_type=F32, per=3, p=0.2)
          for d, s, b, w, g in ((100, F16, F16, F16, "sequence"), (1003, F32, BF16, F32, "column"), (260, F32, F32, F32, None),
                                (2048, BF16, BF16, BF16, "element"))]


@pytest.mark.parametrize("kw", CASES, ids=lambda kw: "-".join(str(v).replace("torch.", "") for v in kw.values()))
def test_forward(kw):
    announce(f"residual forward {kw}")
    Case(**kw).forward()


@pytest.mark.parametrize("kw", CASES, ids=lambda kw: "-".join(str(v).replace("torch.", "") for v in kw.values()))
def test_backward(kw):
    announce(f"residual backward {kw}")
    Case(**kw).backward()


@pytest.mark.parametrize("kw", [dict(n=70, dim=520, stream=BF16, branch=BF16, weight=BF16, gate="column", p=0.2),
                                dict(n=70, dim=8200, stream=F32, branch=BF16), dict(n=70, dim=521, pre=False)])
def test_gradients_in_place(kw):
    announce(f"residual backward in place {kw}")
    Case(**kw).backward(in_place=True)


@pytest.mark.parametrize("dim", [96, 97, 8192])
def test_forward_in_place(dim):
    """h over x and out over the branch: the same bits."""
    announce(f"residual forward in place {dim}")
    c = Case(33, dim, stream=BF16, branch=BF16, weight=F32, gate="column", p=0.1)
    x, y = c.put(c.x), c.put(c.y)
    h, out = torch.empty_like(x), torch.empty_like(y)
    ra.radamw_residual_norm(x, y, c.options(), h=h, out=out, **c.shared())
    ra.radamw_residual_norm(x, y, c.options(), h=x, out=y, **c.shared())
    assert torch.equal(h, x) and torch.equal(out, y)


@pytest.mark.parametrize("stream,out_type", [(F32, F32), (F32, BF16), (F16, F16)])
def test_norm_without_a_branch(stream, out_type):
    """The first norm of a model: out and x's gradient alone."""
    announce(f"norm alone {stream} {out_type}")
    n, dim = 400, 200
    x, w = normal((n, dim), stream, 1, 2.0), normal((dim,), F32, 2, 0.1, 1.0)
    dh, dout = normal((n, dim), stream, 3), normal((n, dim), out_type, 4)
    o = ra.residual_options(eps=1e-5)
    out, rstd = torch.empty((n, dim), dtype=out_type, device=DEV), torch.full((2, n), 7.0, device=DEV)
    ra.radamw_residual_norm(x.to(DEV), None, o, pre_weight=w.to(DEV), out=out, rstd=rstd)
    r = Residual(x, None, pre=w, eps=1e-5)
    ref = r.forward()
    close(out, *ref["out"], "out")
    close(rstd[1], *ref["rstd_h"], "rstd")
    gx, gw = torch.empty((n, dim), dtype=stream, device=DEV), torch.empty(dim, device=DEV)
    ws = torch.empty(ra.radamw_residual_grad_workspace_bytes(n, dim), dtype=torch.uint8, device=DEV)
    ra.radamw_residual_norm_grad(x.to(DEV), None, o, rstd, ws, grad_h=dh.to(DEV), grad_out=dout.to(DEV),
                                 pre_weight=w.to(DEV), grad_x=gx, grad_pre_weight=gw)
    want = r.backward(dh, dout, rstd.cpu().reshape(-1))
    close(gx, *want["x"], "grad_x")
    close(gw, *want["pre"], "grad_pre")


def test_no_rows():
    """n = 0: the weights' gradients are zeros, nothing else is written."""
    announce("residual no rows")
    x, w = torch.empty((0, 24), device=DEV), torch.ones(24, device=DEV)
    o = ra.residual_options()
    ra.radamw_residual_norm(x, x, o, post_weight=w, pre_weight=w, h=x, out=x)
    ws = torch.empty(ra.radamw_residual_grad_workspace_bytes(0, 24), dtype=torch.uint8, device=DEV)
    a, b = torch.full((24,), 7.0, device=DEV), torch.full((24,), 7.0, device=DEV)
    ra.radamw_residual_norm_grad(x, x, o, x, ws, post_weight=w, pre_weight=w, grad_h=x, grad_out=x, grad_x=x,
                                 grad_branch=x, grad_post_weight=a, grad_pre_weight=b)
    assert bool((a == 0).all()) and bool((b == 0).all())


def test_zero_rows_and_values_that_are_not_numbers():
    """A row of zeros has finite norms and gradients; a NaN or an infinity
    stays in its row; a dropped one in a branch without a norm is nowhere."""
    announce("residual zeros and NaN")
    n, dim = 12, 80
    c = Case(n, dim, gate="column", p=0.5)
    c.x[2], c.y[2] = 0.0, 0.0
    c.y[5, 3], c.x[7, 11], c.y[9, 0] = float("nan"), float("nan"), float("inf")
    h, out, rstd = torch.empty((n, dim), device=DEV), torch.empty((n, dim), device=DEV), torch.empty((2, n), device=DEV)
    ra.radamw_residual_norm(c.x.to(DEV), c.y.to(DEV), c.options(), h=h, out=out, rstd=rstd, **c.shared())
    good = [i for i in range(n) if i not in (5, 7, 9)]
    assert bool(h[good].isfinite().all()) and bool(out[good].isfinite().all()) and bool((out[2] == 0).all())
    assert bool(out[[5, 7]].isnan().all())
    gx, gb = torch.empty((n, dim), device=DEV), torch.empty((n, dim), device=DEV)
    ra.radamw_residual_norm_grad(h, c.y.to(DEV), c.options(), rstd, None, grad_h=c.dh.to(DEV), grad_out=c.dout.to(DEV),
                                 grad_x=gx, grad_branch=gb, **c.shared())
    assert bool(gx[good].isfinite().all()) and bool(gb[good].isfinite().all())
    # without a norm behind the branch, what is dropped is never seen
    c = Case(n, dim, gate="column", post=False, p=0.5)
    clean = Residual(c.x, c.y, c.gate, **c.ref)
    c.y[~clean.keep] = float("nan")
    c.forward()
    c.backward()


def test_long_arrays():
    """More than 2^31 elements: the last rows are those of a call of their
    own, and the sums are those of the parts."""
    announce("residual 70000 x 32768 bf16")
    n, dim, k = 70000, 32768, 64
    y = torch.empty((n, dim), dtype=BF16, device=DEV).normal_(generator=torch.Generator("cuda").manual_seed(1))
    x = torch.empty((n, dim), dtype=BF16, device=DEV).normal_(generator=torch.Generator("cuda").manual_seed(2))
    w = torch.ones(dim, device=DEV)
    tail_x, tail_y = x[-k:].clone(), y[-k:].clone()
    rstd = torch.empty((2, n), device=DEV)
    o = ra.residual_options(p=0.1, seed=1, offset=2)
    ra.radamw_residual_norm(x, y, o, post_weight=w, pre_weight=w, h=x, out=y, rstd=rstd)
    h, out, r = torch.empty_like(tail_x), torch.empty_like(tail_y), torch.empty((2, k), device=DEV)
    ra.radamw_residual_norm(tail_x, tail_y, ra.residual_options(p=0.1, seed=1, offset=2, first_row=n - k),
                            post_weight=w, pre_weight=w, h=h, out=out, rstd=r)
    assert torch.equal(x[-k:], h) and torch.equal(y[-k:], out) and torch.equal(rstd[:, -k:], r)


def test_refusals_on_the_device():
    announce("residual refusals")
    x, w = torch.ones((6, 16), device=DEV), torch.ones(16, device=DEV)
    o = ra.residual_options()
    big = torch.ones((12, 16), device=DEV)
    new = lambda: torch.empty((6, 16), device=DEV)  # noqa: E731
    for kw in (dict(h=new().half()), dict(h=new()[:5]), dict(post_weight=w[:8]), dict(pre_weight=w.half(), post_weight=w),
               dict(gate=x[:2], rows_per_gate=2), dict(gate=x[:2], rows_per_gate=0), dict(rstd=w[:11]),
               dict(out=new().double())):
        with pytest.raises(ValueError):
            ra.radamw_residual_norm(x, x.clone(), o, **{**dict(h=new(), out=new(), pre_weight=w), **kw})
    for kw, status in ((dict(h=big[1:7], out=big[6:12]), -3), (dict(h=None, out=new()), -1),
                       (dict(h=new(), out=None), -1)):
        with pytest.raises(ra.RadamwError) as e:
            ra.radamw_residual_norm(big[:6], x, o, pre_weight=w, **kw)
        assert e.value.status == status, kw
    with pytest.raises(ra.RadamwError) as e:  # a workspace that is asked for
        ra.radamw_residual_norm_grad(x, x, o, new()[:2].reshape(-1)[:12], None, pre_weight=w, grad_h=x, grad_out=x,
                                     grad_x=new(), grad_branch=new(), grad_pre_weight=torch.empty_like(w))
    assert e.value.status == -5
    assert bool((big == 1).all())
