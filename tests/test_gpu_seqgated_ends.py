"""The gated projections' activations far from zero, in fp32: element by element
relative to themselves, not to the projections' sums.

One of x's elements is g and another 1, one weight of each matrix 1 and the others
0, so the products are exact: out = act(g), and dx holds act'(g) and act(g).  With
u = 2^-24, the hardware's exponential and reciprocal within one unit in the last
place (2 u), every other operation within u:
 - e^-|g|: 2 u, and u for what its exponent's rounding takes back in: 3 u.
 - sigmoid: 1 + e^-|g| is off by u and 3 u e / (1 + e) <= 1.5 u, its reciprocal
   by 2 u more: 4.5 u; for g < 0 times e: 8.5 u.  SiLU: 9.5 u.
 - sigmoid' = e / (1 + e)^2: 3 u + 2 * 4.5 u + 2 u = 14 u.
 - Phi(-x), x >= 0: e^(-x^2 / 2) 3 u; t = 1 / (1 + 0.32 x) 3 u, to which t P(t)
   is sensitive up to 2.5 times, 7.5 u; the polynomial's rounded coefficients 1.7 u
   and steps 3 u, its fit 0.5 u; two products 2 u: 18 u.  1 - Phi(-x): less.
 - sums of two terms: both terms' errors and u of the sum."""

import math

import numpy as np
import pytest
import torch

from oracle import seqlayer as olayer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def rse():
    import recommender_sparse_embedding_amd as m

    return m


def _values(most):
    at = np.concatenate([np.linspace(-most, most, 8191), np.geomspace(1e-6, most, 500), -np.geomspace(1e-6, most, 500)])
    return np.float32(np.random.default_rng(0).permutation(at))


def _bounds(act, g):
    """(act(g), act'(g)) with how far they may be off."""
    a, da = olayer.activation(act, g)
    if act == "gelu":
        cdf = 0.5 * np.vectorize(math.erfc)(-g / math.sqrt(2.0))
        phi = np.exp(-0.5 * g * g) / np.sqrt(2 * np.pi)
        return (a, 20 * U * np.abs(a)), (da, 19 * U * cdf + 6 * U * np.abs(g) * phi + U * np.abs(da))
    s, t = olayer.activation("sigmoid", g)
    t = s * olayer.activation("sigmoid", -g)[0]             # (1 - s loses what is small)
    if act == "sigmoid":
        return (s, 8.5 * U * s), (t, 14 * U * t)
    return (a, 9.5 * U * np.abs(a)), (s + g * t, 8.5 * U * s + 15 * U * np.abs(g) * t + U * np.abs(s + g * t))


# (past these the exponential is below the least normal number)
@pytest.mark.parametrize("act,most", [("sigmoid", 85.0), ("silu", 85.0), ("gelu", 12.0)])
@pytest.mark.parametrize("dim", [4, 64])
def test_activations_relative_to_themselves(rse, act, most, dim):
    g = _values(most)
    for part in (slice(0, 40), slice(0, None)):             # few rows, whose tiles differ, and all
        v = torch.from_numpy(g[part]).cuda()
        x, wg, wu = torch.zeros((len(v), dim), device="cuda"), *(torch.zeros((4, dim), device="cuda") for _ in range(2))
        x[:, 0], x[:, 1] = v, 1.0
        wg[2, 0], wu[2, 1] = 1.0, 1.0
        code = {"sigmoid": rse.SIGMOID, "silu": rse.SILU, "gelu": rse.GELU}[act]
        dout = torch.zeros((len(v), 4), device="cuda")
        dout[:, 2] = 1.0
        out = rse.seq_gated_linear_fwd(x, wg, wu, code)
        dx, _, _ = rse.seq_gated_linear_bwd(x, wg, wu, dout, code)
        (a, ea), (da, eda) = _bounds(act, np.float64(g[part]))
        for got, ref, bound, what in ((out[:, 2], a, ea, "out"), (dx[:, 1], a, ea, "du"), (dx[:, 0], da, eda, "dg")):
            off = np.abs(got.double().cpu().numpy() - ref)
            bad = off > bound
            i = np.argmax(bad)
            assert not bad.any(), (what, act, g[part][i], off[i] / U / abs(ref[i]), bound[i] / U / abs(ref[i]))


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
def test_activations_past_the_exponential(rse, act):
    """Largest, smallest and not finite projections: the limits, and NaN where the
    formula multiplies infinity by 0."""
    g = torch.tensor([3e38, -3e38, 1e20, -1e20, 200.0, -200.0, 0.0, -0.0, 1e-38, float("nan"), float("inf"), -float("inf")]).cuda()
    x, wg, wu = torch.zeros((12, 4), device="cuda"), *(torch.zeros((4, 4), device="cuda") for _ in range(2))
    x[:, 0], x[:, 1] = g, 1.0
    wg[0, 0], wu[0, 1] = 1.0, 1.0
    code = {"sigmoid": rse.SIGMOID, "silu": rse.SILU, "gelu": rse.GELU}[act]
    dout = torch.zeros((12, 4), device="cuda")
    dout[:, 0] = 1.0
    out = rse.seq_gated_linear_fwd(x[:9], wg, wu, code)[:, 0].cpu()
    dx = rse.seq_gated_linear_bwd(x[:9], wg, wu, dout[:9], code)[0].cpu()
    v = g[:9].cpu()
    half = torch.tensor([1.0, 0, 1, 0, 1, 0, 0.5, 0.5, 0.5])
    want = half if act == "sigmoid" else v * half
    slope = half * (1 - half) if act == "sigmoid" else half
    assert torch.allclose(out, want, rtol=1e-6, atol=0) and torch.allclose(dx[:, 1], want, rtol=1e-6, atol=0)
    assert torch.allclose(dx[:, 0], slope, rtol=1e-6, atol=1e-38)
    odd = rse.seq_gated_linear_fwd(x[9:], wg, wu, code)[:, 0].cpu()
    assert torch.isnan(odd[0])


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_sigmoid_ends_in_bf16(rse, act):
    """Results within a bf16 rounding, 2^-8 of themselves, and the exponent's one
    (up to 122 in base 2, 2^-18 of it and as much of its constant: 2^-16 of e^-|g|); of
    a sum of two terms that of the larger."""
    v = torch.from_numpy(_values(80.0)).bfloat16()
    g = v.double().numpy()
    x, wg, wu = torch.zeros((len(v), 8), dtype=torch.bfloat16), *(torch.zeros((8, 8), dtype=torch.bfloat16) for _ in range(2))
    x[:, 0], x[:, 1] = v, 1.0
    wg[2, 0], wu[2, 1] = 1.0, 1.0
    dout = torch.zeros((len(v), 8), dtype=torch.bfloat16)
    dout[:, 2] = 1.0
    code = {"sigmoid": rse.SIGMOID, "silu": rse.SILU}[act]
    x, wg, wu, dout = (t.cuda() for t in (x, wg, wu, dout))
    out, (dx, _, _) = rse.seq_gated_linear_fwd(x, wg, wu, code), rse.seq_gated_linear_bwd(x, wg, wu, dout, code)
    s, t = olayer.activation("sigmoid", g)[0], olayer.activation("sigmoid", g)[0] * olayer.activation("sigmoid", -g)[0]
    a, da, terms = (s, t, t) if act == "sigmoid" else (g * s, s + g * t, s + np.abs(g) * np.maximum(t, U))
    for got, ref, size in ((out[:, 2], a, np.abs(a)), (dx[:, 1], a, np.abs(a)), (dx[:, 0], da, terms)):
        off = np.abs(got.double().cpu().numpy() - ref)
        bad = off > 2.0 ** -8 * np.abs(ref) + 1.01 * 2.0 ** -16 * size
        assert not bad.any(), (act, g[np.argmax(bad)], off[np.argmax(bad)])
