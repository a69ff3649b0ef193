"""GPU tests of radamw_dropout against its plain 64-bit form."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from block_helpers import dropout
from gpu_helpers import DEV, announce
from vocab_helpers import close

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(n, dim, dtype, seed, stride=None, start=0):
    """(CPU values, device tensor) [n, dim], rows `stride` apart from element
    `start` on."""
    x = torch.randn((n, dim), generator=gen(seed)).to(dtype)
    stride = stride or dim
    buf = torch.full((start + n * stride,), 7.0, dtype=dtype, device=DEV)
    view = buf[start:].as_strided((n, dim), (stride, 1), start)
    view.copy_(x)
    return x, view, buf


CASES = [  # n, dim, dtype, p, stride, start
    (1, 1, F32, 0.5, None, 0), (1, 7, BF16, 0.5, None, 0), (3, 8, F16, 0.1, None, 0), (2, 9, F32, 0.9, 17, 1),
    (129, 1111, F32, 0.25, None, 0), (77, 1000, BF16, 0.1, 1003, 3), (65, 4096, F16, 0.6, 4100, 0),
    (33, 16385, BF16, 0.3, None, 1), (1, 100_003, F32, 0.4, None, 0), (4099, 640, BF16, 0.2, None, 0),
    (5, 24, F32, 0.0, None, 0), (5, 24, BF16, 1.0, None, 0), (5, 24, F16, 2.0 ** -18, None, 0),
    (5, 24, F16, 1 - 2.0 ** -16, None, 0)]


@pytest.mark.parametrize("n,dim,dtype,p,stride,start", CASES)
def test_dropout(n, dim, dtype, p, stride, start):
    announce(f"dropout {n} x {dim} {dtype} p={p} stride={stride} start={start}")
    x, xd, _ = rows(n, dim, dtype, 1, stride, start)
    _, out, buf = rows(n, dim, dtype, 2, dim + 5, 2)
    before = buf.clone()
    seed, offset, first = 0xDEADBEEFCAFEF00D, (1 << 40) + 77, 12345
    ra.radamw_dropout(xd, out, ra.dropout_options(p, seed, offset, first))
    ref, slack = dropout(x, p, seed, offset, first)
    close(out, ref, slack, "out")
    # dropped exactly, and nothing between the rows is written
    assert torch.equal(out.cpu() == 0, (ref == 0) | (x == 0))
    before.as_strided((n, dim), (dim + 5, 1), 2).copy_(out)
    assert torch.equal(before, buf)


def test_long_batch_and_large_rows():
    """Several pieces per lane; the last rows of a call that begins at 2^32 - n."""
    announce("dropout 2049 x 8200 bf16")
    n, dim = 2049, 8200
    x = torch.randn((n, dim), generator=gen(3)).to(BF16)
    out = torch.empty((n, dim), dtype=BF16, device=DEV)
    ra.radamw_dropout(x.to(DEV), out, ra.dropout_options(0.1, 5, 6, 2 ** 32 - n))
    ref, slack = dropout(x, 0.1, 5, 6, 2 ** 32 - n)
    close(out, ref, slack, "out")


def test_offsets_beyond_32_bits():
    """An array of more than 2^31 elements: its last rows have the numbers of
    a call of their own."""
    announce("dropout 70000 x 32768 bf16")
    n, dim = 70000, 32768
    x = torch.ones((n, dim), dtype=BF16, device=DEV)
    ra.radamw_dropout(x, x, ra.dropout_options(0.5, 1, 2))
    tail = torch.ones((100, dim), dtype=BF16, device=DEV)
    ra.radamw_dropout(tail, tail, ra.dropout_options(0.5, 1, 2, n - 100))
    assert torch.equal(x[-100:], tail)
    kept = float((x != 0).float().mean(1).mean())
    assert abs(kept - 0.5) < 5 * 0.5 / (n * dim) ** 0.5


def test_in_place_and_dropped_values():
    """In place; a dropped NaN or infinity is 0, a kept one stays."""
    announce("dropout in place")
    x = torch.randn((50, 100), generator=gen(4))
    x[::3] = float("nan")
    x[1::3] = float("inf")
    xd = x.to(DEV)
    ra.radamw_dropout(xd, xd, ra.dropout_options(0.5, 9, 9))
    keep = dropout(torch.ones(50, 100), 0.5, 9, 9)[0] != 0
    want = torch.where(keep, x * 2, 0.0)
    assert torch.equal(xd.cpu().nan_to_num(123.0), want.nan_to_num(123.0))


def test_gradient_is_the_same_call():
    announce("dropout gradient")
    x, g = torch.randn((40, 72), generator=gen(5)), torch.randn((40, 72), generator=gen(6))
    o = ra.dropout_options(0.3, 11, 12)
    out, gx = torch.empty((40, 72), device=DEV), torch.empty((40, 72), device=DEV)
    ra.radamw_dropout(x.to(DEV), out, o)
    ra.radamw_dropout(g.to(DEV), gx, o)
    # out = m x elementwise, so that the gradient is m g
    m = dropout(torch.ones(40, 72), 0.3, 11, 12)[0]
    close(gx, m * g.double(), 2.0 ** -24 * (m * g).abs().double(), "gradient")
    assert torch.equal(out != 0, gx != 0)


def test_refusals_on_the_device():
    announce("dropout refusals")
    x = torch.ones((4, 8), device=DEV)
    o = ra.dropout_options(0.5, 1, 2)
    for out, what in ((x[1:], ValueError), (x.t(), ValueError), (x.half(), ValueError), (x[:, ::2], ValueError)):
        with pytest.raises(what):
            ra.radamw_dropout(x, out, o)
    buf = torch.ones(100, device=DEV)
    with pytest.raises(ra.RadamwError) as e:
        ra.radamw_dropout(buf[:32].view(4, 8), buf[8:40].view(4, 8), o)  # a shifted overlap
    assert e.value.status == -3
    assert bool((buf == 1).all())
    launches = ra.radamw_launch_count()
    ra.radamw_dropout(x[:0], x[:0], o)
    assert ra.radamw_launch_count() == launches
