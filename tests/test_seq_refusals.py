"""What the sequence layer's calls refuse before any GPU work (every call here
returns before a kernel is launched, and the addresses are never read)."""

import ctypes
import math
import types

import pytest
import torch

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


class _Far:
    """What the bindings look at of a contiguous tensor on some GPU."""

    is_cuda = True

    def __init__(self, device, dtype, *shape):
        self.dtype, self.shape, self.at = dtype, shape, device
        self.device = f"cuda:{device}"

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def stride(self):
        return tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def rse(monkeypatch):
    import recommender_sparse_embedding_amd as m
    from recommender_sparse_embedding_amd import sequence

    monkeypatch.setattr(sequence, "_current_device", lambda: 0)
    return m


@pytest.mark.parametrize("far", ["x", "weight", "bias", "residual", "out"])
def test_norm_of_another_device(rse, far):
    """A tensor on another device than the rows, or all of them on another than
    the current one, is refused before anything is allocated."""
    on = lambda name: 1 if name == far else 0  # noqa: E731
    f = torch.float32
    with pytest.raises((ValueError, TypeError), match="cuda:1"):
        rse.seq_layer_norm_fwd(_Far(on("x"), f, 4, 64), _Far(on("weight"), f, 64), _Far(on("bias"), f, 64),
                               residual=_Far(on("residual"), f, 4, 64), out=_Far(on("out"), f, 4, 64),
                               sum_out=_Far(0, f, 4, 64))


@pytest.mark.parametrize("far", ["x", "dy", "weight", "stats"])
def test_norm_backward_of_another_device(rse, far):
    on = lambda name: 1 if name == far else 0  # noqa: E731
    f = torch.float32
    with pytest.raises((ValueError, TypeError), match="cuda:1"):
        rse.seq_layer_norm_bwd(_Far(on("x"), f, 4, 64), _Far(on("dy"), f, 4, 64), _Far(on("weight"), f, 64),
                               _Far(on("stats"), f, 4, 2))


@pytest.mark.parametrize("far", ["x", "w_gate", "w_up", "out"])
def test_gated_of_another_device(rse, far):
    on = lambda name: 1 if name == far else 0  # noqa: E731
    f = torch.float32
    with pytest.raises((ValueError, TypeError), match="cuda:1"):
        rse.seq_gated_linear_fwd(_Far(on("x"), f, 4, 64), _Far(on("w_gate"), f, 40, 64), _Far(on("w_up"), f, 40, 64),
                                 out=_Far(on("out"), f, 4, 40))


@pytest.mark.parametrize("far", ["q", "k", "v", "pos", "bias", "offsets", "table", "lens", "cache", "attn", "out"])
def test_chunk_of_another_device(rse, far):
    at = lambda name, dtype, *shape: _Far(1 if name == far else 0, dtype, *shape)  # noqa: E731
    b16, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    attn = types.SimpleNamespace(torch_dtype=b16, n_heads=4, n_kv_heads=2, dim=32, n_buckets=3, handle=None,
                                 mem=at("attn", torch.uint8, 2048), chunk_bytes=((5, 2, 5, 64), 0))
    cache = types.SimpleNamespace(handle=None, page_size=16, k=at("cache", b16, 8, 16, 2, 32))
    with pytest.raises(ValueError, match="cuda:1"):
        rse.seq_attention_chunk(attn, cache, at("q", b16, 5, 4, 32), at("k", b16, 5, 2, 32), at("v", b16, 5, 2, 32),
                                at("pos", i32, 5), at("bias", torch.float32, 4, 3), at("offsets", i64, 3),
                                at("table", i32, 2, 4), at("lens", i64, 2), out=at("out", b16, 5, 4, 32))


def test_stream_of_another_device(rse):
    f, stream = torch.float32, types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="cuda:1"):
        rse.seq_layer_norm_fwd(_Far(0, f, 4, 64), None, None, out=_Far(0, f, 4, 64), stream=stream)
    with pytest.raises(ValueError, match="cuda:1"):
        rse.seq_gated_linear_fwd(*(_Far(0, f, 64, 64) for _ in range(3)), out=_Far(0, f, 64, 64), stream=stream)
