"""CPU tests of the block operators' largest sizes: what radamw.h says fits is
refused by no range check, and a workspace is named for nothing that is."""
import os

import pytest

import optimizer_step_dl_amd as ra
from test_block_host import loss, loss_grad

RANGE = -5
P = 0x10000  # a pointer that is refused before anything reads it
MOST = 2 ** 24 - 2048


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ra.LIB_PATH):
        from optimizer_step_dl_amd import build
        build.build()
    return ra.load()


@pytest.mark.parametrize("n", [1, 1000, 2 ** 20, 2 ** 20 + 1, 2 ** 30 - 8])
@pytest.mark.parametrize("experts", [1, 8, 4096])
def test_most_groups(lib, n, experts):
    for groups in (MOST, MOST + 1, 2 ** 24 - 1):
        refused = [loss(lib, n=n, experts=experts, st=experts, gs=experts, off=P, groups=groups) == RANGE,
                   loss_grad(lib, n=n, experts=experts, st=experts, gs=experts, off=P, groups=groups) == RANGE,
                   lib.radamw_balance_workspace_bytes(n, experts, groups) == RANGE]
        assert refused == [groups > MOST] * 3, groups
