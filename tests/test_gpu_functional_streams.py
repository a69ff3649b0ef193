"""GPU tests of the autograd embedding's grad_buffer where the forward passes
of one table ran on several streams."""
import pytest
import torch

from gpu_helpers import DEV, announce
from optimizer_step_dl_amd.functional import embedding

pytestmark = pytest.mark.gpu

SPIN = 5_000_000  # cycles: some milliseconds, against microseconds of work


def uses(table, buffer, ids, streams):
    """One embedding per stream, each with a gradient of its own, summed."""
    total = 0
    for k, (i, s) in enumerate(zip(ids, streams)):
        with torch.cuda.stream(s):
            x = embedding(i, table, scale=0.5 + k, grad_buffer=buffer)
            part = x.float().square().sum()
        torch.cuda.current_stream().wait_stream(s)
        total = total + part
    return total


def inputs(dtype, n=60_000, rows=300, dim=256):
    g = torch.Generator().manual_seed(1)
    table = torch.randn((rows, dim), generator=g).to(dtype).to(DEV).requires_grad_()
    ids = [torch.randint(0, rows, (n,), generator=g).to(DEV) for _ in range(3)]
    start = torch.randn((rows, dim), generator=g).to(dtype).to(DEV)
    return table, ids, start


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("late", [0, 1, 2])
def test_buffer_of_three_streams(dtype, late):
    """The sums are those of one stream, bit for bit, and the caller's stream
    reads them behind backward(), whichever stream is late."""
    announce(f"buffer of three streams {dtype} late={late}")
    table, ids, start = inputs(dtype)
    main = torch.cuda.current_stream()
    want = start.clone()
    uses(table, want, ids, [main] * 3).backward()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    buffer = start.clone()
    torch.cuda.synchronize()
    total = uses(table, buffer, ids, streams)
    with torch.cuda.stream(streams[late]):
        torch.cuda._sleep(SPIN)
    total.backward()
    got = buffer.clone()  # on the caller's stream, with nothing waited for
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(buffer, want)


@pytest.mark.parametrize("late", [0, 1])
def test_buffer_that_torch_adds_to_as_well(late):
    """table.grad as the buffer of a table that is also an output head: the
    head's gradient is added to the same memory on the stream of its own
    node."""
    announce(f"tied buffer late={late}")
    table, ids, start = inputs(torch.float32)
    main = torch.cuda.current_stream()
    x = torch.randn((64, 256), generator=torch.Generator().manual_seed(2)).to(DEV)

    def step(streams):
        table.grad = start.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):  # the node of the table belongs to this stream
            head = (x @ table.t()).square().sum()
        main.wait_stream(streams[0])
        total = head + uses(table, table.grad, ids[:1], streams[1:])
        with torch.cuda.stream(streams[late]):
            torch.cuda._sleep(SPIN)
        total.backward()
        got = table.grad.clone()
        torch.cuda.synchronize()
        return got

    want = step([main, main])
    got = step([torch.cuda.Stream(), torch.cuda.Stream()])
    assert torch.equal(got, want)


def test_buffer_and_backward_on_a_side_stream():
    """backward() called on a stream of its own goes on behind the writes."""
    announce("buffer, backward on a side stream")
    table, ids, start = inputs(torch.float32)
    want = start.clone()
    uses(table, want, ids, [torch.cuda.current_stream()] * 3).backward()
    buffer = start.clone()
    forward, caller = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    total = uses(table, buffer, ids, [forward] * 3)
    with torch.cuda.stream(forward):
        torch.cuda._sleep(SPIN)
    with torch.cuda.stream(caller):
        caller.wait_stream(torch.cuda.default_stream())
        total.backward()
        got = buffer.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_buffer_with_a_copy_that_takes_the_gradient():
    """A frozen table read through a copy: the buffer is still written."""
    announce("buffer, frozen table")
    table, ids, start = inputs(torch.float32, n=50)
    copy = table.detach().to(torch.bfloat16).requires_grad_()
    buffer = torch.zeros_like(start)
    embedding(ids[0], table.detach(), model_copy=copy, grad_buffer=buffer).sum().backward()
    want = torch.zeros_like(start).index_add_(0, ids[0], torch.ones((50, 256), device=DEV))
    assert torch.equal(buffer, want)
