"""CPU tests of the vocabulary operators' largest sizes: what radamw.h says
fits is refused by no range check."""
import os

import pytest

import optimizer_step_dl_amd as ra

RANGE = -5
P = 0x10000  # a pointer that is refused before anything reads it


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ra.LIB_PATH):
        from optimizer_step_dl_amd import build
        build.build()
    return ra.load()


def grad(lib, n, dim, rows=100):
    return lib.radamw_embedding_grad(P, 2, dim, P, 0, n, rows, dim, 1.0, -1, 1, P, 2, dim, P, 1 << 60, None)


@pytest.mark.parametrize("dim", [1, 8, 257, 512, 513, 1023])
@pytest.mark.parametrize("n", [2 ** 30 - 1, 2 ** 30 - 63, 2 ** 30 - 64, 2 ** 30 - 65])
def test_gradient_of_just_below_2_30_tokens(lib, n, dim):
    assert n * dim < 2 ** 40
    assert grad(lib, n, dim) != RANGE


@pytest.mark.parametrize("n,dim", [((2 ** 40 - 1) // d, d) for d in (1029, 4096, 4097, 131_072, 2 ** 24)])
def test_gradient_of_just_below_2_40_values(lib, n, dim):
    assert grad(lib, n, dim) != RANGE


def test_limits_that_stay(lib):
    assert grad(lib, 2 ** 31 - 15, 1) == RANGE
    # column tiles of 512 x chunks of 64 tokens, four to a workgroup: 2^24 workgroups
    assert grad(lib, 2 ** 30, 2048) == RANGE and grad(lib, 2 ** 30 - 64, 2048) != RANGE
    assert lib.radamw_embedding_lookup(P, 0, 8, 8, 8, P, 0, 2 ** 24 - 1, 1.0, P, 0, 8, None) != RANGE
