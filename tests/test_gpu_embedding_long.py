"""GPU tests of the embedding gradient beyond 524288 tokens, where one
workgroup sums the sort's counts first, with chunks of every length under
uneven ids, and with rows beyond 2^31 elements."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from gpu_helpers import DEV, announce
from test_gpu_embedding import check_grad, randint, randn, workspace
from vocab_helpers import close, embedding_grad

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows", [3, 900, 70_000, 1_100_000])
@pytest.mark.parametrize("n", [524_287, 524_288, 524_289, 1_100_003])
def test_grad_on_both_sides_of_256_tiles(n, rows, accumulate):
    """256 tiles sum the counts by themselves, more are summed by one
    workgroup in several rounds; one pass of few digits up to three of 512;
    a last tile of one token."""
    announce(f"grad n={n} rows={rows} {accumulate}")
    ids = randint(-2, rows + 2, (n,), n + rows, torch.int32)
    ids[-1] = rows - 1
    ids[n // 3:n // 3 + 5000] = rows // 2
    check_grad(n, rows, 8, F32, F32, ids, 0.5, None, accumulate, n)


@pytest.mark.parametrize("kind", ["one id", "each once", "descending"])
def test_grad_long_uneven_ids(kind):
    announce(f"grad long {kind}")
    n, rows = 600_001, 700_000
    if kind == "one id":
        ids = torch.full((n,), rows - 1)
    elif kind == "each once":
        ids = torch.randperm(rows, generator=torch.Generator().manual_seed(3))[:n]
    else:
        ids = torch.arange(n - 1, -1, -1)
    check_grad(n, rows, 9, BF16, BF16, ids, 1.0, None, False, 5)


@pytest.mark.parametrize("kind,accumulate", [("one id", False), ("runs at edges", True), ("runs past edges", False),
                                             ("runs past edges", True), ("heavy", True)])
@pytest.mark.parametrize("n,dim,chunk", [(4000, 12_300, 16), (9000, 8200, 32), (30_000, 4100, 64)])
def test_grad_uneven_ids_in_longer_chunks(n, dim, chunk, kind, accumulate):
    """Chunks of 16, 32 and 64 sorted tokens: runs that end where a chunk
    does, one token later, one that crosses hundreds."""
    announce(f"grad chunks n={n} dim={dim} {kind}")
    tiles = (dim + 511) // 512
    share = n * tiles // 4096
    assert chunk == (8 if share < 16 else 16 if share < 32 else 32 if share < 64 else 64)
    rows = 400
    if kind == "one id":
        ids = torch.full((n,), 7)
    elif kind == "runs at edges":
        ids = torch.arange(n) // chunk % rows
    elif kind == "runs past edges":
        ids = (torch.arange(n) + chunk - 1) // chunk % rows
    else:
        ids = randint(0, rows, (n,), n)
        ids[torch.rand(n, generator=torch.Generator().manual_seed(1)) < 0.6] = 200
    check_grad(n, rows, dim, BF16, BF16, ids, 1.0, None, accumulate, n)


@pytest.mark.parametrize("n", [6, 700])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_past_32_bit_offsets(n, accumulate):
    """Rows of the table and of the gradient beyond 2^31 elements and 2^32
    bytes, among few tokens and many."""
    announce(f"grad far rows n={n} {accumulate}")
    rows, dim = 280_000, 8192
    stride = (1 << 31) // (n - 2) + 8
    src = randn((n, dim), 1, 1.0, BF16)
    whole = torch.full(((n - 1) * stride + dim,), float("nan"), dtype=BF16, device=DEV)
    grad = whole.as_strided((n, dim), (stride, 1))
    grad.copy_(src)
    table = torch.full((rows, dim), 2.0 if accumulate else float("nan"), dtype=BF16, device=DEV)
    far = torch.tensor([0, 131_072, 262_143, 262_144, rows - 1])
    ids = far[torch.arange(n) % 5]
    ra.radamw_embedding_grad(grad, ids.to(DEV), table, workspace(n, rows, dim), accumulate=accumulate)
    where = torch.arange(n) % 5
    ref, slack = embedding_grad(src, where, 5, 1.0, None, torch.full((5, dim), 2.0) if accumulate else None)
    close(table[far.to(DEV)], ref, slack, "far rows")
    table[far.to(DEV)] = 2.0 if accumulate else 0.0
    assert bool((table == (2.0 if accumulate else 0.0)).all())
