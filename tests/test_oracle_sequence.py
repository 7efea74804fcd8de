"""Pins of the sequence attention's oracle: torch autograd in float64, finite
differences, closed forms; and the binding's and library's refusals, which
need no GPU."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import sequence as oseq


def _case(rng, lens, H, Hk, D, nb):
    N = int(sum(lens))
    off = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = rng.standard_normal((N, H, D)), rng.standard_normal((N, Hk, D)), rng.standard_normal((N, Hk, D))
    pos = np.cumsum(rng.integers(0, 9, N)).astype(np.int32)
    bounds = np.unique(rng.integers(-5, 60, nb))
    bias = rng.standard_normal((H, len(bounds) + 1))
    return q, k, v, pos, bias, off, [int(b) for b in bounds]


@pytest.mark.parametrize("causal", [True, False])
def test_oracle_matches_autograd(causal):
    rng = np.random.default_rng(5)
    q, k, v, pos, bias, off, bounds = _case(rng, [3, 0, 1, 7], 4, 2, 5, 6)
    key_off = np.where(rng.random(len(q)) < 0.3, -1, 7)
    key_off[3] = -1                                  # the one-event sequence sees nothing
    do = rng.standard_normal(q.shape)
    got = oseq.attention(q, k, v, pos, bias, off, bounds, causal, 0.3, key_off, do)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v, bias)]
    loss = torch.zeros((), dtype=torch.float64)
    for a, e in zip(off[:-1], off[1:]):
        for i in range(a, e):
            for h in range(4):
                js = [j for j in range(a, e) if key_off[j] >= 0 and (j <= i or not causal)]
                if not js:
                    assert np.all(got["out"][0][i, h] == 0) and got["lse"][h, i] == -np.inf
                    continue
                s = torch.stack([0.3 * t[0][i, h] @ t[1][j, h // 2]
                                 + t[3][h, int(np.searchsorted(bounds, pos[i] - pos[j], side="right"))] for j in js])
                o = torch.softmax(s, 0) @ torch.stack([t[2][j, h // 2] for j in js])
                np.testing.assert_allclose(got["out"][0][i, h], o.detach().numpy(), rtol=1e-12, atol=1e-13)
                np.testing.assert_allclose(got["lse"][h, i], torch.logsumexp(s, 0).item(), rtol=1e-12)
                loss = loss + (o * torch.tensor(do[i, h])).sum()
    loss.backward()
    for name, x in zip(("dq", "dk", "dv", "dbias"), t):
        np.testing.assert_allclose(got[name][0], x.grad.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("low", [-np.inf, float(np.finfo(np.float32).min), -1e30])
def test_oracle_bias_that_hides(low):
    """Distances of 0 and of 3 or more hidden by their bias: each event sees the
    two before it, the first one nothing."""
    rng = np.random.default_rng(8)
    q, k, v, do = (rng.standard_normal((6, 1, 4)) for _ in range(4))
    bias = np.array([[0.5, low, 0.25, low]])
    got = oseq.attention(q, k, v, np.arange(6), bias, [0, 6], [0, 1, 3], True, 0.5, None, do)
    assert np.all(got["out"][0][0] == 0) and got["lse"][0, 0] == -np.inf and np.all(got["dq"][0][0] == 0)
    for i in range(1, 6):
        js = list(range(max(i - 2, 0), i))
        e = np.exp(0.5 * k[js, 0] @ q[i, 0] + 0.25)
        np.testing.assert_allclose(got["out"][0][i, 0], e @ v[js, 0] / e.sum(), rtol=1e-12)
        np.testing.assert_allclose(got["lse"][0, i], np.log(e.sum()), rtol=1e-12)
    assert got["dbias"][0][0, 1] == 0 and got["dbias"][0][0, 3] == 0
    assert all(np.all(np.isfinite(x)) for n in ("out", "dq", "dk", "dv", "dbias") for x in got[n])


def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(6)
    q, k, v, pos, bias, off, bounds = _case(rng, [6, 2], 2, 1, 3, 5)
    do = rng.standard_normal(q.shape)
    loss = lambda *x: float((oseq.attention(*x[:3], pos, x[3], off, bounds, True, 0.5)["out"][0] * do).sum())  # noqa: E731
    got = oseq.attention(q, k, v, pos, bias, off, bounds, True, 0.5, None, do)
    base = [q, k, v, bias]
    for at, name in enumerate(("dq", "dk", "dv", "dbias")):
        way = rng.standard_normal(base[at].shape)
        hi, lo = list(base), list(base)
        hi[at], lo[at] = base[at] + 1e-5 * way, base[at] - 1e-5 * way
        assert abs((loss(*hi) - loss(*lo)) / 2e-5 - (got[name][0] * way).sum()) < 1e-8


def test_oracle_buckets_and_saturation():
    bounds = [-3, 0, 1, 1, 50, 2**31 - 1]
    assert oseq.bucket(np.array([0, -4, 1, 50, 49]), 0, bounds).tolist() == [2, 0, 4, 5, 4]
    assert oseq.bucket(np.array([2**31 - 1]), np.array([-1]), bounds).tolist() == [6]       # saturates upwards
    assert oseq.bucket(np.array([-2**31]), np.array([5]), bounds).tolist() == [0]


def test_oracle_step_is_the_last_row():
    rng = np.random.default_rng(7)
    q, k, v, pos, bias, off, bounds = _case(rng, [9], 4, 2, 6, 4)
    full = oseq.attention(q, k, v, pos, bias, off, bounds, True, 0.4)["out"][0]
    out, _ = oseq.step([(k, v, pos), None], np.stack([q[-1], q[-1]]), bias, bounds, 0.4)
    np.testing.assert_allclose(out[0], full[-1], rtol=1e-12)
    assert np.all(out[1] == 0)


def test_oracle_assign_by_hand():
    slots, off, taken, table = oseq.assign([3, 0, 2], [7, 1, 0], [[4, -1], [2, -1], [-1, -1]], [9, 5, 6], 8)
    assert (slots, off, taken) == ([39, 72, 73, 40, 41], [0, 3, 3, 5], 2)
    assert table == [[4, 9], [2, -1], [5, -1]]


# ---------------------------------------------------------------- refusals --
INV, UNSUP, WS = -1, -2, -3
MEM = ctypes.c_void_p(1 << 20)        # never touched: every call below is refused before


@pytest.fixture(scope="module")
def lib():
    from recommender_sparse_embedding_amd import _lib

    return _lib.load()


def test_attention_handle_refuses(lib):
    def create(H=4, Hk=2, D=64, dtype=1, scale=0.1, bounds=(1, 2), mem=MEM, size=1 << 20, n=None):
        arr = (ctypes.c_int32 * max(1, len(bounds)))(*bounds)
        h = ctypes.c_void_p()
        return lib.rse_seqattn_create(ctypes.byref(h), mem, size, H, Hk, D, dtype, 1, scale, arr,
                                      len(bounds) if n is None else n, None)

    assert create(H=5) == INV and create(H=0) == INV and create(H=512, Hk=1) == INV and create(Hk=0) == INV
    assert create(D=48) == UNSUP and create(D=256) == UNSUP
    assert create(dtype=2) == INV
    assert create(scale=float("nan")) == INV and create(scale=float("inf")) == INV
    assert create(bounds=(2, 1)) == INV and create(bounds=(-2**31, 1)) == INV and create(bounds=(1,) * 128) == INV
    assert create(n=-1) == INV
    assert create(mem=None) == INV and create(mem=ctypes.c_void_p((1 << 20) + 16)) == INV
    assert create(size=64) == WS
    assert lib.rse_seqattn_mem_size(None) == INV
    assert lib.seq_attention_fwd(None, None, None, None, None, None, None, 0, None) == INV
    assert lib.seq_attention_bwd(None, None, None, None, None, None, 0, None, None, None, None, None, None, 0, None) == INV
    assert lib.rse_seqattn_status(None, None, None) == INV and lib.rse_seqattn_clear_status(None, None) == INV


def test_cache_handle_refuses(lib):
    def create(pages=10, size=16, Hk=2, D=64, dtype=1, meta=MEM, k=MEM, meta_bytes=1 << 20):
        h = ctypes.c_void_p()
        return lib.rse_seqcache_create(ctypes.byref(h), meta, meta_bytes, k, MEM, MEM, pages, size, Hk, D, dtype, None)

    assert create(size=24) == UNSUP and create(size=4) == UNSUP and create(size=2048) == UNSUP
    assert create(D=16) == UNSUP and create(dtype=5) == INV and create(pages=0) == INV and create(Hk=0) == INV
    assert create(k=None) == INV and create(k=ctypes.c_void_p((1 << 20) + 8)) == INV
    assert create(meta=ctypes.c_void_p((1 << 20) + 16)) == INV and create(meta_bytes=8) == WS
    sz = ctypes.c_size_t()
    assert lib.rse_seqcache_assign_workspace_size(-1, ctypes.byref(sz)) == INV
    assert lib.rse_seqcache_assign_workspace_size(5, ctypes.byref(sz)) == 0 and sz.value >= 40
    assert lib.seq_cache_assign(None, None, None, 0, None, 0, None, 0, 0, None, None, None, None, 0, None) == INV
    assert lib.seq_cache_write(None, None, 0, None, None, None, None) == INV
    assert lib.seq_attention_step(None, None, None, None, None, None, None, None, 0, None, 0, 0, None, None, 0, None) == INV
    assert lib.rse_seqcache_status(None, None, None) == INV


def test_binding_refuses_before_any_call():
    import recommender_sparse_embedding_amd as rse
    from recommender_sparse_embedding_amd import sequence

    with pytest.raises(ValueError, match="int32"):
        rse.SeqAttention(2, 1, 64, boundaries=[2**31], device="cpu")
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        sequence._rows(x, torch.bfloat16, 3, 2, 64, "q")
    with pytest.raises(TypeError):
        rse.SeqCache(torch.zeros((3, 8, 64)), None, None)


def test_cache_handle_refuses_too_many_slots(lib):
    """The stated limit of 2^40 events; refused before the memory is touched."""
    h = ctypes.c_void_p()
    for pages, size in ((2**30 + 1, 1024), (2**31 - 1, 1024), (2**31, 8)):
        assert lib.rse_seqcache_create(ctypes.byref(h), MEM, 1 << 20, MEM, MEM, MEM, pages, size, 1, 32, 1, None) == INV
