"""GPU tests of the embedding lookup and its gradient against plain 64-bit
forms (bounds in vocab_helpers.py)."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from gpu_helpers import DEV, announce
from vocab_helpers import close, embedding_grad, f32

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def randn(shape, seed, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def randint(lo, hi, shape, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g).to(dtype)


def strided(t, pad, fill=float("nan")):
    """t on the GPU as the leading columns of wider rows, and the whole."""
    whole = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=DEV)
    whole[:, :t.shape[1]] = t.to(DEV)
    return whole[:, :t.shape[1]], whole


def workspace(n, rows, dim, fill=0xA5):
    need = ra.radamw_embedding_grad_workspace_bytes(n, rows, dim)
    return torch.full((need,), fill, dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------ lookup --

@pytest.mark.parametrize("dim", [1, 7, 8, 64, 65, 513, 2048, 4101])
@pytest.mark.parametrize("table_dtype,out_dtype", [(F32, F32), (F32, BF16), (F32, F16), (F16, F16), (F16, F32),
                                                   (F16, BF16), (BF16, BF16), (BF16, F32), (BF16, F16)])
def test_lookup(dim, table_dtype, out_dtype):
    n, rows, scale = 37, 301, 5.3
    announce(f"lookup {dim} {table_dtype} {out_dtype}")
    table = randn((rows, dim), dim, 0.02, table_dtype)
    ids = randint(0, rows, (n,), dim + 1, torch.int32 if dim % 2 else torch.int64)
    ids[5], ids[6] = 0, rows - 1
    t, _ = strided(table, 3)
    out, whole = strided(torch.zeros(n, dim, dtype=out_dtype), 5)
    ra.radamw_embedding_lookup(t, ids.to(DEV), out, scale=scale)
    want = (table.float() * torch.tensor(f32(scale)))[ids.long()].to(out_dtype)
    same = torch.equal(out.cpu(), want)
    assert same, (out.cpu() - want).abs().max()
    assert bool(whole[:, dim:].isnan().all())  # columns behind the row are left


@pytest.mark.parametrize("n,dim", [(70_000, 40), (70_001, 33), (9000, 516), (5000, 2051), (5000, 4101), (3001, 8200)])
@pytest.mark.parametrize("table_dtype,out_dtype", [(F32, BF16), (BF16, BF16), (F16, F32)])
def test_lookup_long_lists(n, dim, table_dtype, out_dtype):
    """Lists long enough for four pieces per lane."""
    announce(f"lookup n={n} dim={dim}")
    rows = 700
    table = randn((rows, dim), dim, 1.0, table_dtype)
    ids = randint(-1, rows, (n,), dim)
    out = torch.full((n, dim), float("nan"), dtype=out_dtype, device=DEV)
    ra.radamw_embedding_lookup(table.to(DEV), ids.to(DEV), out)
    t = table.float().to(out_dtype).to(DEV)
    want = torch.where((ids >= 0).to(DEV)[:, None], t[ids.clamp(min=0).to(DEV)], torch.zeros((), dtype=out_dtype, device=DEV))
    assert torch.equal(out, want)


@pytest.mark.parametrize("n", [0, 1, 2, 63, 4097])
def test_lookup_lengths_and_ids_outside(n):
    announce(f"lookup n={n}")
    rows, dim = 17, 96
    table = randn((rows, dim), 3, 1.0, BF16)
    ids = randint(0, rows, (n,), 4)
    ids[::3] = torch.tensor([-100, rows, -1, 2 ** 40])[torch.arange(len(ids[::3])) % 4]
    out = torch.full((n, dim), float("nan"), dtype=F32, device=DEV)
    before = ra.radamw_launch_count()
    ra.radamw_embedding_lookup(table.to(DEV), ids.to(DEV), out)
    assert ra.radamw_launch_count() - before == (1 if n else 0)
    inside = (ids >= 0) & (ids < rows)
    want = torch.where(inside[:, None], table.float()[ids.clamp(0, rows - 1)], torch.zeros(()))
    assert torch.equal(out.cpu(), want)


def test_lookup_keeps_special_values_and_shapes():
    announce("lookup special values")
    table = torch.tensor([[float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 65504.0, 1e-7, 1.0]], dtype=F16)
    ids = torch.zeros((2, 3), dtype=torch.int64, device=DEV)
    out = torch.empty((6, 8), dtype=F16, device=DEV)
    ra.radamw_embedding_lookup(table.to(DEV), ids, out, scale=-1.0)
    want = (-table).expand(6, 8)
    assert torch.equal(out.cpu().nan_to_num(7), want.nan_to_num(7))
    assert torch.equal(out.cpu().signbit()[:, 3:5], want.signbit()[:, 3:5])


def test_lookup_past_32_bit_offsets():
    """A table of more than 2^32 bytes and 2^31 elements."""
    announce("lookup far rows")
    rows, dim = 280_000, 8192
    table = torch.zeros((rows, dim), dtype=BF16, device=DEV)
    far = [0, 131_072, 262_143, 262_144, rows - 1]
    for i, r in enumerate(far):
        table[r] = i + 1
    ids = torch.tensor(far, device=DEV)
    out = torch.empty((len(far), dim), dtype=BF16, device=DEV)
    ra.radamw_embedding_lookup(table, ids, out)
    want = torch.arange(1, len(far) + 1).to(BF16)[:, None].expand(-1, dim)
    assert torch.equal(out.cpu(), want)


# ---------------------------------------------------------------- gradient --

def check_grad(n, rows, dim, grad_dtype, into, ids, scale=1.0, padding_id=None, accumulate=False, seed=0, pad=0):
    grad = randn((n, dim), seed + 1, 1e-2, grad_dtype)
    old = randn((rows, dim), seed + 2, 1e-2, into) if accumulate else None
    g, _ = strided(grad, pad)
    start = old if accumulate else torch.full((rows, dim), float("nan"), dtype=into)
    t, whole = strided(start, pad)
    ws = workspace(n, rows, dim)
    ra.radamw_embedding_grad(g, ids.to(DEV), t, ws, scale=scale, padding_id=padding_id, accumulate=accumulate)
    ref, slack = embedding_grad(grad, ids, rows, scale, padding_id, old)
    close(t, ref, slack, f"gradient n={n} rows={rows} dim={dim}")
    if pad:
        assert bool(whole[:, dim:].isnan().all())
    # rows no token names: left bit for bit when adding, zeros otherwise
    named = torch.zeros(rows, dtype=torch.bool)
    flat = ids.reshape(-1).long()
    keep = (flat >= 0) & (flat < rows) & (flat != (-1 if padding_id is None else padding_id))
    named[flat[keep]] = True
    got = t.cpu()
    assert torch.equal(got[~named], old[~named] if accumulate else torch.zeros_like(got[~named]))
    # the same bits again, from a workspace of other contents
    t2, _ = strided(start, pad)
    ra.radamw_embedding_grad(g, ids.to(DEV), t2, workspace(n, rows, dim, 0x5A), scale=scale, padding_id=padding_id,
                             accumulate=accumulate)
    assert torch.equal(t2.cpu().nan_to_num(7), got.nan_to_num(7))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("grad_dtype,into", [(F32, F32), (BF16, F32), (F16, F16), (BF16, BF16), (F32, BF16),
                                             (F16, F32), (F32, F16), (F16, BF16), (BF16, F16)])
def test_grad_types(grad_dtype, into, accumulate):
    announce(f"grad {grad_dtype} {into} {accumulate}")
    n, rows, dim = 300, 97, 520
    check_grad(n, rows, dim, grad_dtype, into, randint(0, rows, (n,), 5), 1.7, None, accumulate)


@pytest.mark.parametrize("dim", [1, 5, 8, 24, 63, 64, 65, 255, 511, 513, 1029])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_dims(dim, accumulate):
    announce(f"grad dim={dim}")
    n, rows = 211, 50
    check_grad(n, rows, dim, BF16, F32, randint(0, rows, (n,), dim, torch.int32), 1.0, 3, accumulate, dim, pad=3)


@pytest.mark.parametrize("n", [0, 1, 2, 7, 8, 9, 64, 1023, 1025, 4095, 4096, 4097, 8191, 8192, 8193, 12289, 40_001])
@pytest.mark.parametrize("rows", [1, 2, 513, 40_000])
def test_grad_lengths(n, rows):
    """One workgroup's sort up to 8192 tokens, the tiled sort beyond; chunks
    of 8, 16 and 32 tokens; one, two and three passes' worth of digits."""
    announce(f"grad n={n} rows={rows}")
    ids = randint(-2, rows + 2, (n,), n + rows)
    check_grad(n, rows, 16, F32, F32, ids, 0.5, None, False, n)


@pytest.mark.parametrize("rows", [255, 256, 511, 512, 65_535, 65_536, 119_102, 262_143, 262_144])
@pytest.mark.parametrize("n", [5, 254, 1024, 1025, 8200])
def test_grad_digit_widths(rows, n):
    """Digits of every width, up to 512 of them with four waves and with
    sixteen, and 1024 in the tiled sort; ids from the whole range."""
    announce(f"grad rows={rows} n={n}")
    ids = torch.linspace(0, rows - 1, n).long()
    ids = ids[torch.randperm(n, generator=torch.Generator().manual_seed(n))]
    check_grad(n, rows, 8, F32, BF16, ids, 1.0, None, False, n)
    check_grad(n, rows, 8, F32, BF16, ids.int(), 1.0, None, True, n)


@pytest.mark.parametrize("rows", [600_000, 1_100_000])
@pytest.mark.parametrize("n", [3000, 20_000])
def test_grad_wide_vocabulary(rows, n):
    """Three passes of the small sort, three of the tiled one above 2^20."""
    announce(f"grad rows={rows} n={n}")
    ids = randint(0, rows, (n,), n)
    ids[n // 2:] = ids[:n - n // 2]
    check_grad(n, rows, 8, F32, F32, ids, 1.0, int(ids[0]), False, n)


@pytest.mark.parametrize("kind", ["one id", "two ids", "all padding", "all outside", "heavy", "sorted", "runs at edges"])
@pytest.mark.parametrize("n", [65, 5000, 20_000])
def test_grad_uneven_ids(kind, n):
    announce(f"grad {kind} n={n}")
    rows, dim, pad = 1000, 72, None
    if kind == "one id":
        ids = torch.full((n,), 7)
    elif kind == "two ids":
        ids = torch.arange(n) % 2 * 999
    elif kind == "all padding":
        ids, pad = torch.full((n,), 7), 7
    elif kind == "all outside":
        ids = torch.full((n,), -100)
    elif kind == "heavy":
        ids = randint(0, rows, (n,), n)
        ids[torch.rand(n, generator=torch.Generator().manual_seed(1)) < 0.6] = 400
        pad = 0
    elif kind == "sorted":
        ids = randint(0, rows, (n,), n).sort().values
    else:  # runs that end exactly where a chunk of 8, 16 or 32 does, and one token later
        ids = torch.arange(n) // 32
        ids[1::64] = ids[0::64][:len(ids[1::64])]
        ids = ids.clamp(max=rows - 1)
    check_grad(n, rows, dim, BF16, F32, ids, 1.0, pad, False, n)
    check_grad(n, rows, dim, BF16, BF16, ids, 1.0, pad, True, n)


@pytest.mark.parametrize("n", [8000, 16_000, 30_000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_chunk_lengths(n, accumulate):
    """Lists long enough for chunks of 16, 32 and 64 tokens, runs that end at
    every place of a chunk, one that crosses dozens."""
    announce(f"grad chunks n={n}")
    rows, dim = 900, 4100
    ids = randint(0, rows, (n,), n)
    ids[n // 4:n // 2] = 17
    ids[-200:] = rows - 1
    check_grad(n, rows, dim, BF16, BF16, ids, 1.0, 0, accumulate, n)


@pytest.mark.parametrize("kind", ["one id", "pairs", "heavy", "each once", "all outside"])
@pytest.mark.parametrize("n", [1, 9, 64, 65, 255, 256, 257, 511, 512, 513])
def test_grad_few(kind, n):
    """Up to 512 tokens are summed without a sort: lists on both sides of a
    wave's and a workgroup's tokens, ids with one token, two, more than eight
    and all."""
    announce(f"grad few {kind} n={n}")
    rows, dim, pad = 1000, 1032, 3
    if kind == "one id":
        ids = torch.full((n,), 7)
    elif kind == "pairs":  # a token and the one half a list behind it
        ids = (torch.arange(n) % max(1, n // 2)) + 5
    elif kind == "heavy":
        ids = randint(-3, rows + 3, (n,), n)
        ids[torch.rand(n, generator=torch.Generator().manual_seed(n)) < 0.4] = 400
    elif kind == "each once":
        ids = torch.randperm(rows, generator=torch.Generator().manual_seed(n))[:n]
    else:
        ids, pad = torch.full((n,), rows), 0
    check_grad(n, rows, dim, BF16, F32, ids, 0.5, pad, False, n)
    check_grad(n, rows, dim, F32, BF16, ids.int(), 0.5, pad, True, n)


@pytest.mark.parametrize("dim", [4096, 4104])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_few_widest(dim, accumulate):
    """512 tokens at the widest rows summed without a sort, and one more
    column tile."""
    announce(f"grad few dim={dim}")
    n, rows = 512, 700
    check_grad(n, rows, dim, F16, F16, randint(0, rows // 4, (n,), dim), 1.0, None, accumulate, dim)


@pytest.mark.parametrize("rows,dim", [(1, 3), (20_000, 1), (4_500_000, 2), (9000, 33), (3, 70_000)])
def test_grad_few_clears(rows, dim):
    """The rows without a token among few tokens: many rows to a workgroup,
    the largest number of rows to one, and rows longer than its share."""
    announce(f"grad few rows={rows} dim={dim}")
    n = 20
    ids = torch.linspace(0, rows - 1, n).long()
    check_grad(n, rows, dim, F32, BF16, ids, 1.0, None, False, dim)
    check_grad(0, rows, dim, F32, F32, ids[:0], 1.0, None, False, dim)


def test_grad_sums_in_token_order():
    """Equal ids keep their tokens' order: values whose FP32 sum depends on
    it give the sum taken in order (one chunk of eight tokens)."""
    announce("grad order")
    vals = torch.tensor([1.0, 2.0 ** 24, -(2.0 ** 24), 2.0 ** -10, 3.0, -3.0, 2.0 ** 23, 0.5])
    ids = torch.full((8,), 2, device=DEV)
    out = torch.empty((4, 8), device=DEV)
    ra.radamw_embedding_grad(vals[:, None].repeat(1, 8).to(DEV), ids, out, workspace(8, 4, 8))
    acc = torch.zeros(())
    for v in vals:
        acc = acc + v
    assert torch.equal(out[2].cpu(), acc.expand(8))


def test_grad_nan_and_padding():
    """NaN in a padding token's row reaches nothing; in a live one, its row only."""
    announce("grad nan")
    n, rows, dim = 100, 20, 33
    grad = randn((n, dim), 1)
    ids = randint(1, rows, (n,), 2)
    ids[10:20] = 0
    grad[10:20] = float("nan")
    live = int(torch.nonzero(ids == 5)[0])
    grad[live, 4] = float("nan")
    out = torch.empty((rows, dim), device=DEV)
    ra.radamw_embedding_grad(grad.to(DEV), ids.to(DEV), out, workspace(n, rows, dim), padding_id=0)
    bad = out.cpu().isnan()
    assert bad[5, 4] and int(bad.sum()) == 1


def test_grad_into_bucket_view():
    """Adding into a table's part of a flattened gradient bucket leaves the rest."""
    announce("grad bucket")
    rows, dim, n, off = 40, 31, 64, 1001
    bucket = torch.full((off + rows * dim + 77,), 2.0, dtype=F16, device=DEV)
    before = bucket.clone()
    view = bucket[off:off + rows * dim].view(rows, dim)
    ids = randint(0, rows, (n,), 9)
    grad = randn((n, dim), 8, 1.0, F16)
    ra.radamw_embedding_grad(grad.to(DEV), ids.to(DEV), view, workspace(n, rows, dim), accumulate=True)
    ref, slack = embedding_grad(grad, ids, rows, 1.0, None, torch.full((rows, dim), 2.0))
    close(view, ref, slack, "bucket view")
    assert torch.equal(bucket[:off], before[:off]) and torch.equal(bucket[off + rows * dim:], before[off + rows * dim:])


def test_grad_on_side_streams_at_once():
    """Two calls on two streams, each with its own workspace."""
    announce("grad two streams")
    n, rows, dim = 9000, 500, 256
    grads = [randn((n, dim), s, 1.0, BF16).to(DEV) for s in (1, 2)]
    ids = [randint(0, rows, (n,), s).to(DEV) for s in (3, 4)]
    alone = []
    for g, i in zip(grads, ids):
        out = torch.empty((rows, dim), device=DEV)
        ra.radamw_embedding_grad(g, i, out, workspace(n, rows, dim))
        alone.append(out)
    outs = [torch.empty((rows, dim), device=DEV) for _ in range(2)]
    spaces = [workspace(n, rows, dim) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, g, i, o, w in zip(streams, grads, ids, outs, spaces):
            with torch.cuda.stream(s):
                ra.radamw_embedding_grad(g, i, o, w)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert torch.equal(a, o)


def test_refusals_leave_outputs():
    announce("embedding refusals")
    rows, dim, n = 20, 16, 10
    table = randn((rows, dim), 1).to(DEV)
    ids = randint(0, rows, (n,), 2).to(DEV)
    out = torch.full((n, dim), 3.0, device=DEV)
    grad = torch.full((rows, dim), 3.0, device=DEV)
    ws = workspace(n, rows, dim)

    def refused(status, f, *a, **k):
        with pytest.raises(ra.RadamwError) as e:
            f(*a, **k)
        assert e.value.status == status

    before = ra.radamw_launch_count()
    lookup, gradient = ra.radamw_embedding_lookup, ra.radamw_embedding_grad
    refused(-1, lookup, table, ids, out, scale=float("nan"))
    refused(-1, lookup, table, ids, out, scale=1e39)
    refused(-3, lookup, table, ids, table[:n])
    refused(-5, gradient, out, ids, grad, ws[:-1])
    refused(-4, gradient, out, ids, grad, torch.empty(ws.numel() + 16, dtype=torch.uint8, device=DEV)[1:])
    refused(-5, gradient, out, ids, grad, ws, padding_id=rows)
    refused(-1, gradient, out, ids, grad, ws, padding_id=-7)
    refused(-3, gradient, grad[:n], ids, grad, ws)
    for bad in (lambda: lookup(table.cpu(), ids, out), lambda: lookup(table, ids.float(), out),
                lambda: lookup(table, ids, out[:, :-1]), lambda: lookup(table.t(), ids, out),
                lambda: lookup(table.double(), ids, out), lambda: lookup(table, ids[::2], out),
                lambda: gradient(out[:-1], ids, grad, ws), lambda: gradient(out, ids, grad.t().contiguous().t(), ws)):
        with pytest.raises(ValueError):
            bad()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.capture_begin(capture_error_mode="relaxed")
        try:
            refused(-1, lookup, table, ids, out)
            refused(-1, gradient, out, ids, grad, ws)
            grad.add_(0)
        finally:
            graph.capture_end()
    torch.cuda.synchronize()
    assert ra.radamw_launch_count() == before
    assert bool((out == 3).all()) and bool((grad == 3).all())
