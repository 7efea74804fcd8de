"""The oracle of the layer around the sequence attention against torch's float64
operations and central differences, and what the calls refuse before any GPU
work."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import seqlayer as olayer


def _inputs(n, D, H, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((n, D)), r.standard_normal((H, D)) * D**-0.5, r.standard_normal((H, D)) * D**-0.5, \
        r.standard_normal((n, H))


def _slope(f, x, v, dout, h=1e-5):
    """Central difference of sum(dout f(x)) along v."""
    return ((f(x + h * v) - f(x - h * v)) * dout).sum() / (2 * h)


@pytest.mark.parametrize("n,D", [(1, 1), (3, 7), (5, 64)])
def test_norm_matches_torch(n, D):
    r = np.random.default_rng(D)
    x, w, b = r.standard_normal((n, D)) * 3 + 2, r.standard_normal(D), r.standard_normal(D)
    got = olayer.norm(x, w, b, 1e-5, "f32")["y"][0]
    ref = torch.nn.functional.layer_norm(*(torch.from_numpy(a) for a in (x,)), (D,), torch.from_numpy(w),
                                         torch.from_numpy(b), 1e-5)
    assert np.allclose(got, ref.numpy(), rtol=1e-12, atol=1e-12)


def test_norm_gradients_are_slopes():
    r = np.random.default_rng(5)
    n, D = 6, 17
    x, w, b, dy = r.standard_normal((n, D)), r.standard_normal(D), r.standard_normal(D), r.standard_normal((n, D))
    got = olayer.norm_backward(x, dy, w, 1e-5, None, "f32")
    y = lambda x_, w_, b_: olayer.norm(x_, w_, b_, 1e-5, "f32")["y"][0]  # noqa: E731
    for name, f, at in (("dx", lambda t: y(t, w, b), x), ("dweight", lambda t: y(x, t, b), w), ("dbias", lambda t: y(x, w, t), b)):
        v = r.standard_normal(at.shape)
        assert abs(_slope(f, at, v, dy) - (got[name][0] * v).sum()) < 1e-7, name
    s = r.standard_normal((n, D))
    assert np.allclose(olayer.norm_backward(x, dy, w, 1e-5, s, "f32")["dx"][0], got["dx"][0] + s)


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
def test_gated_matches_torch_and_its_gradients_are_slopes(act):
    x, wg, wu, dout = _inputs(5, 12, 9, 1)
    f = {"sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act]
    t = [torch.from_numpy(a).requires_grad_() for a in (x, wg, wu)]
    out = f(t[0] @ t[1].T) * (t[0] @ t[2].T)
    assert np.allclose(olayer.gated(x, wg, wu, act, "f32")[0], out.detach().numpy(), rtol=1e-12, atol=1e-14)
    got = olayer.gated_backward(x, wg, wu, dout, act, "f32")
    out.backward(torch.from_numpy(dout))
    r = np.random.default_rng(2)
    for i, name in enumerate(("dx", "dw_gate", "dw_up")):
        assert np.allclose(got[name][0], t[i].grad.numpy(), rtol=1e-11, atol=1e-13), name
        at = [x, wg, wu]
        v = r.standard_normal(at[i].shape)
        put = lambda y: olayer.gated(*at[:i], y, *at[i + 1:], act, "f32")[0]  # noqa: E731
        assert abs(_slope(put, at[i], v, dout) - (got[name][0] * v).sum()) < 1e-7, name


def test_bounds_cover_rounded_arithmetic():
    """fp32 numpy stays inside the bounds, which are not loose by orders: a
    projection's is 65 u sum |x| |w|, 65 * 6e-8 * 5 = 2e-5, and the product of two
    of median size 0.6 is off by some 1e-4 of itself."""
    x, wg, wu, dout = _inputs(40, 64, 48, 3)
    x, wg, wu, dout = (a.astype(np.float32) for a in (x, wg, wu, dout))
    wide = [a.astype(np.float64) for a in (x, wg, wu, dout)]
    g, u = x @ wg.T, x @ wu.T
    s = np.float32(1) / (np.float32(1) + np.exp(-g))
    ref, bound = olayer.gated(*wide[:3], "silu", "f32")
    assert np.all(np.abs(g * s * u - ref) <= bound) and np.median(bound / np.abs(ref)) < 1e-3


# ------------------------------------------------------------ refusals (CPU) --
@pytest.fixture(scope="module")
def lib():
    from recommender_sparse_embedding_amd import _lib

    return _lib.load()


INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def _mat(addr, stride):
    from recommender_sparse_embedding_amd._lib import RseSeqMat

    return ctypes.byref(RseSeqMat(addr, stride))


def test_norm_refusals(lib):
    """Every call here returns before a kernel is launched (the addresses are
    never read)."""
    m = _mat(0x10000, 64)

    def fwd(x=m, res=None, s=None, eps=1e-5, n=4, dim=64, dtype=0, y=m):
        return lib.seq_layer_norm_fwd(x, res, s, None, None, eps, n, dim, dtype, y, None, None)

    assert fwd(n=-1) == INVALID and fwd(dim=0) == INVALID and fwd(dtype=2) == INVALID
    assert fwd(dim=8193) == UNSUPPORTED
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(res=m) == INVALID and fwd(s=m) == INVALID
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID and fwd(y=_mat(None, 64)) == INVALID
    assert fwd(x=_mat(0x10002, 64)) == INVALID                  # not an element's address
    assert fwd(y=_mat(0x10000, 63)) == INVALID and fwd(y=_mat(0x10000, -63)) == INVALID     # rows overlap
    assert fwd(y=_mat(0x10000, 0)) == INVALID
    assert fwd(res=m, s=_mat(0x10000, 10)) == INVALID
    assert fwd(n=0, x=None, y=None) == 0

    sz = ctypes.c_size_t()
    size = lib.rse_seq_layer_norm_bwd_workspace_size
    assert size(-1, 64, 0, ctypes.byref(sz)) == INVALID and size(4, 64, 0, None) == INVALID
    assert size(4, 8193, 0, ctypes.byref(sz)) == UNSUPPORTED
    assert size(10**6, 64, 0, ctypes.byref(sz)) == 0 and sz.value >= 2 * 64 * 4
    need = sz.value

    def bwd(x=m, dy=m, stats=0x20000, n=10**6, dx=m, dw=0x30000, db=0x40000, ws=0x50000, size=need):
        return lib.seq_layer_norm_bwd(x, dy, None, stats, None, n, 64, 0, dx, dw, db, ws, size, None)

    assert bwd(size=need - 1) == WORKSPACE
    assert bwd(ws=None) == INVALID and bwd(ws=0x50010) == INVALID
    assert bwd(stats=None) == INVALID and bwd(dy=None) == INVALID and bwd(dx=_mat(0x10000, 1)) == INVALID


def test_gated_refusals(lib):
    m = _mat(0x10000, 64)

    def fwd(x=m, wg=m, wu=m, n=4, dim=64, hidden=64, dtype=0, act=1, out=m):
        return lib.seq_gated_linear_fwd(x, wg, wu, n, dim, hidden, dtype, act, out, None)

    assert fwd(n=-1) == INVALID and fwd(dim=0) == INVALID and fwd(hidden=-8) == INVALID and fwd(dtype=3) == INVALID
    assert fwd(act=-1) == INVALID and fwd(act=3) == INVALID
    assert fwd(dim=6) == UNSUPPORTED and fwd(hidden=6) == UNSUPPORTED and fwd(dtype=1, dim=12) == UNSUPPORTED
    assert fwd(dim=65540) == UNSUPPORTED
    assert fwd(x=None) == INVALID and fwd(wg=None) == INVALID and fwd(wu=None) == INVALID and fwd(out=None) == INVALID
    assert fwd(x=_mat(0x10008, 64)) == INVALID and fwd(x=_mat(0x10000, 66)) == INVALID
    assert fwd(out=_mat(0x10000, 60)) == INVALID and fwd(out=_mat(0x10000, 0)) == INVALID
    assert fwd(n=0, x=None, out=None) == 0
    assert fwd(n=1 << 38) == UNSUPPORTED                        # more tiles than a launch holds

    sz = ctypes.c_size_t()
    size = lib.rse_seq_gated_linear_bwd_workspace_size
    assert size(4, 64, 64, 0, None) == INVALID and size(4, 65, 64, 0, ctypes.byref(sz)) == UNSUPPORTED
    assert size(1000, 64, 64, 0, ctypes.byref(sz)) == 0 and sz.value >= 1000 * 128 * 4
    need = sz.value

    def bwd(dout=m, dx=m, dg=m, du=m, ws=0x50000, size=need):
        return lib.seq_gated_linear_bwd(m, m, m, dout, 1000, 64, 64, 0, 1, dx, dg, du, ws, size, None)

    assert bwd(size=need - 1) == WORKSPACE and bwd(ws=None) == INVALID and bwd(ws=0x50010) == INVALID
    assert bwd(dout=None) == INVALID and bwd(dx=_mat(0x10000, 4)) == INVALID and bwd(dg=_mat(0x10000, 0)) == INVALID
    assert bwd(du=None) == INVALID


def test_binding_refuses_host_tensors():
    import recommender_sparse_embedding_amd as rse

    x = torch.zeros((4, 16))
    with pytest.raises(TypeError):
        rse.seq_layer_norm_fwd(x, None, None)
    with pytest.raises(TypeError):
        rse.seq_gated_linear_fwd(x, x, x)
