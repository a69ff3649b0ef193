"""GPU tests of the balance loss over more groups than one grid holds and over
more than 2^31 logits."""
import pytest
import torch

import optimizer_step_dl_amd as ra
from gpu_helpers import DEV, announce
from test_gpu_balance import gen, inputs, run
from vocab_helpers import U, close

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_more_groups_than_a_grid_holds():
    """65541 groups, some of them empty, among them those on both sides of the
    65536th: every group against the sums over its rows."""
    announce("balance 65541 groups")
    groups, experts, k = 65541, 8, 2
    lengths = torch.randint(0, 4, (groups,), generator=gen(11))
    lengths[65533:65540] = torch.tensor([2, 0, 3, 1, 2, 0, 3])
    bounds = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    n = int(bounds[-1])
    x, ids, mask = inputs(n, experts, k, masked=0.2)
    weights = torch.randn(groups, generator=gen(12))
    weights[::7] = 0.0
    group = torch.repeat_interleave(torch.arange(groups), lengths)

    def sums(v):
        return torch.zeros((groups,) + v.shape[1:], dtype=v.dtype).index_add_(0, group, v)

    # the plain form of block_helpers, with its loop over the groups as sums by index
    live = mask.double()[:, None]
    tokens = sums(mask.long())
    counts = sums((ids[:, :, None] == torch.arange(experts)).sum(1) * mask.long()[:, None])
    t = tokens.clamp(min=1).double()[:, None]
    p = torch.softmax(x.double(), 1) * live
    lse = torch.logsumexp(x.double(), 1) * live[:, 0]
    mean = sums(p) / t
    f = 0.01 * experts / k * counts / t
    loss = (f * mean).sum(1) + 0.01 * sums(lse.square()) / t[:, 0]
    up = (weights.double()[:, None] / t)[group]
    cost = f[group] * up
    zl = 0.02 * up * lse[:, None]
    away = cost - (cost * p).sum(1, keepdim=True) + zl
    grad = p * away * live
    got = run(x, ids, mask, bounds=bounds.tolist(), weights=weights, z=0.01)
    assert torch.equal(got["counts"].cpu().long(), counts) and torch.equal(got["tokens"].cpu().long(), tokens)
    # a probability: 3 u |x - max| + 2 u, 8 + 6 additions and 3 roundings, at |x - max| < 24; three rows of a group 3
    # more.  The loss adds the rounding of the mean and half a step; a log-sum is off by 2 u of its exponentials' sum, the
    # additions, and 4 u of its size, squared.
    rel = (3 * 24 + 2 + 8 + 6 + 3 + 3) * U
    close(got["mean_prob"], mean, rel * mean, "mean_prob")
    slack = 2 * rel * (f * mean).sum(1) + 0.01 * sums(2 * lse.abs() * (rel + 4 * U * (x.abs().amax(1) + 3)) + 6 * U * lse.square()) / t[:, 0]
    close(got["loss"], loss, slack, "loss")
    close(got["total"], (weights * loss).sum(), (weights.abs() * (slack + U * loss)).sum(), "total")
    close(got["grad"], grad, 4 * rel * (p * (cost.abs() + (cost * p).sum(1, keepdim=True).abs() + zl.abs())) +
          p * 0.02 * up.abs() * (rel + 4 * U * (x.abs().amax(1, keepdim=True) + 3)), "grad")


def test_long_batch():
    """More than 2^31 logits: the last rows' gradient is that of a call of
    their own with the whole's counts, the sums are those of the parts."""
    announce("balance 600000 x 4096 bf16")
    n, experts, k, tail = 600_000, 4096, 2, 100
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty((n, experts), dtype=BF16, device=DEV).normal_(generator=g)
    ids = torch.randint(0, experts, (n, k), generator=g, device=DEV)
    o = ra.balance_options(0.01, 0.001)

    def call(x, ids, grad=None):
        out = dict(total=torch.empty((), device=DEV), loss=torch.empty(1, device=DEV),
                   counts=torch.empty((1, experts), dtype=torch.int32, device=DEV),
                   tokens=torch.empty(1, dtype=torch.int32, device=DEV), mean_prob=torch.empty((1, experts), device=DEV))
        ws = torch.empty(ra.radamw_balance_workspace_bytes(len(x), experts), dtype=torch.uint8, device=DEV)
        ra.radamw_balance_loss(x, ids, o, *out.values(), ws, grad=grad)
        return out

    part = [call(x[a:b], ids[a:b]) for a, b in ((0, 200_000), (200_000, 590_000), (590_000, n))]
    keep = x[-tail:].clone()
    whole = call(x, ids, x)
    counts = torch.bincount(ids.reshape(-1), minlength=experts)
    assert torch.equal(whole["counts"][0].long(), counts) and int(whole["tokens"]) == n
    assert torch.equal(sum(v["counts"] for v in part), whole["counts"])
    mean = sum(v["mean_prob"].double() * int(v["tokens"]) for v in part) / n
    # a piece's rows are added in FP32, 586 of them by four lanes in turn, and each mean is rounded
    assert float(((whole["mean_prob"] - mean).abs() / mean).max()) < (2 * 160 + 4) * U
    grad = torch.empty_like(keep)
    ra.radamw_balance_grad(keep, k, o, whole["counts"], whole["tokens"], grad)
    assert torch.equal(grad, x[-tail:])
