"""The sizes the scan takes and refuses, by the workspace it asks for (no GPU
needed): rows of up to 2^31 - 4096 tokens are no matter of how many values B and
C have, and the limits are those the header names."""
import os

import pytest

FWD, BWD = 0, 1
LONGEST = 2 ** 31 - 4096


@pytest.fixture(scope="module")
def size():
    from varlen_depthwise_causal_amd import _build, _lib
    if not os.path.exists(_build.LIBRARY):
        _build.build()
    return _lib.load().selective_scan_workspace_bytes


@pytest.mark.parametrize("S,C,N,G", [(2 ** 28 + 1, 1, 16, 1), (2 ** 26 + 1, 1, 64, 1), (2 ** 28 + 1, 64, 13, 1),
                                     (2 ** 20, 4096, 16, 512), (LONGEST, 1, 8, 1), (LONGEST, 1, 64, 1),
                                     (LONGEST, 4096, 16, 1)])
def test_forward_takes_long_rows(size, S, C, N, G):
    M = 8 if N <= 8 else 16 if N <= 16 else 32 if N <= 32 else 64
    need = size(FWD, S, C, N, G)
    # room for the copies of B and C, and for a state of each chunk of 2048 tokens, twice
    assert need >= S * G * M * 4 + 2 * (S // 2048) * N * C * 4


@pytest.mark.parametrize("d,S,C,N,G", [(FWD, LONGEST + 1, 64, 16, 1), (FWD, LONGEST, 8192, 16, 1),
                                       (FWD, 1000, 2 ** 17, 64, 2 ** 17), (BWD, 1000, 2 ** 17, 64, 2 ** 17),
                                       (BWD, 2 ** 29, 1, 16, 1), (BWD, 2 ** 27, 1, 64, 1)])
def test_sizes_that_are_refused(size, d, S, C, N, G):
    assert size(d, S, C, N, G) == 0


@pytest.mark.parametrize("S,C,N,G", [(2 ** 28, 1, 16, 1), (2 ** 26, 1, 64, 1)])
def test_backward_below_its_limit(size, S, C, N, G):
    assert size(BWD, S, C, N, G) > 0
