"""The layer norm and the gated projections at the limits of their sizes: the
widest rows, and rows whose elements lie past 32 bits."""

import numpy as np
import pytest
import torch
from test_gpu_seqlayer import DT, _check, _check_gated, _gated_case, _np, rse  # noqa: F401  (rse: the fixture)

from oracle import seqlayer as olayer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,dim,hidden", [(3, 65536, 8), (3, 8, 65536), (200, 32768, 16), (200, 16, 32768)])
def test_gated_widest(rse, kind, n, dim, hidden):  # noqa: F811
    _check_gated(rse, kind, *_gated_case(kind, n, dim, hidden), "silu")


def test_gated_rows_past_32_bits(rse):  # noqa: F811
    """2^32 elements of x and dx and more, and of dg and du beside each other: the
    first and the last rows against the oracle, dW against that of all rows summed in
    64 bits, where a weight's row sees few of them (dout is 0 but in both ends)."""
    n, dim, hidden = (1 << 23) + 77, 512, 264
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((n, dim), generator=g, device="cuda", dtype=torch.bfloat16)
    wg, wu = (torch.randn((hidden, dim), generator=g, device="cuda").mul(dim ** -0.5).bfloat16() for _ in range(2))
    dout = torch.zeros((n, hidden), device="cuda", dtype=torch.bfloat16)
    ends = torch.cat([torch.arange(200), torch.arange(n - 200, n)]).cuda()
    dout[ends] = torch.randn((400, hidden), generator=g, device="cuda").bfloat16()
    out = rse.seq_gated_linear_fwd(x, wg, wu)
    dx, dg, du = rse.seq_gated_linear_bwd(x, wg, wu, dout)
    wide = [_np(t) for t in (x[ends], wg, wu, dout[ends])]
    _check(out[ends], olayer.gated(*wide[:3], "silu", "bf16"), "out")
    ref = olayer.gated_backward(*wide, "silu", "bf16")
    _check(dx[ends], ref["dx"], "dx")
    _check(dg, ref["dw_gate"], "dw_gate")          # (rows without a gradient add 0)
    _check(du, ref["dw_up"], "dw_up")
    assert torch.all(dx[200:n - 200] == 0)


def test_norm_rows_past_32_bits(rse):  # noqa: F811
    """More than 2^31 rows of two elements."""
    n = (1 << 31) + 1003
    x = torch.zeros((n, 2), dtype=torch.bfloat16, device="cuda")
    ends = torch.cat([torch.arange(500), torch.arange((1 << 31) - 250, (1 << 31) + 250), torch.arange(n - 500, n)]).cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    x[ends], w, b = torch.randn((1500, 2), generator=g, device="cuda").bfloat16(), *torch.randn((2, 2), generator=g, device="cuda")
    got = rse.seq_layer_norm_fwd(x, w, b, for_backward=True)
    s = _np(x[ends])
    ref = olayer.norm(s, _np(w), _np(b), 1e-5, "bf16")
    _check(got.y[ends], ref["y"], "y")
    _check(got.stats[ends, :1], ref["mean"], "mean")
    _check(got.stats[ends, 1:], ref["r"], "r")
    dy = torch.zeros_like(x)
    dy[ends] = torch.randn((1500, 2), generator=g, device="cuda").bfloat16()
    exact = torch.from_numpy(np.concatenate(olayer.norm_stats(s, 1e-5), 1)).float().cuda()
    got.stats[ends] = exact
    dx, dw, db = rse.seq_layer_norm_bwd(x, dy, w, got.stats)
    ref = olayer.norm_backward(s, _np(dy[ends]), _np(w), 1e-5, None, "bf16")
    for t, name in ((dx[ends], "dx"), (dw, "dweight"), (db, "dbias")):
        _check(t, ref[name], name)
