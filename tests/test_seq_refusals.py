"""What the sequence layer's calls refuse before any GPU work (every call here
returns before a kernel is launched, and the addresses are never read)."""

import ctypes

import pytest

INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    from recommender_sparse_embedding_amd import _lib

    return _lib.load()


def _mat(addr, stride):
    from recommender_sparse_embedding_amd._lib import RseSeqMat

    return ctypes.byref(RseSeqMat(addr, stride))


@pytest.mark.parametrize("dtype,rows,cols", [(0, 64, 64), (1, 128, 128)])
def test_gated_tiles_past_one_launch(lib, dtype, rows, cols):
    """Blocks of 256 threads for tiles of rows by cols: 2^24 of them are 2^32
    threads, one more than a launch numbers."""
    m = _mat(0x10000, 4096)
    for n in (rows << 24, rows << 26, (rows << 30) + 1):
        assert lib.seq_gated_linear_fwd(m, m, m, n, 64, cols, dtype, 1, m, None) == UNSUPPORTED
        assert lib.seq_gated_linear_bwd(m, m, m, m, n, 64, cols, dtype, 1, m, m, m, 0x100000, 1 << 62, None) == UNSUPPORTED
