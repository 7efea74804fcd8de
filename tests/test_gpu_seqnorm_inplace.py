"""The layer norm in the place of its inputs where a row's odd end is loaded
by another wave than the piece that it overlaps: rows of one piece more than
whole waves hold, shared by a block."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def rse():
    import recommender_sparse_embedding_amd as m

    return m


# pieces of 16 bytes: 193 (backward: a block, the last one in its fourth wave),
# 257, 321, 385 and 449 (both: the last one in the first to the fourth wave), 513, 833
@pytest.mark.parametrize("pieces", [193, 257, 321, 385, 449, 513, 833])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_norm_in_place_of_odd_ends(rse, kind, pieces):
    per = 4 if kind == "f32" else 8
    for dim in (per * (pieces - 1) + 1, per * pieces - 1):
        g, n = torch.Generator().manual_seed(dim), 2500         # more rows than the blocks take at once
        x, res, dy, dsum = (torch.randn((n, dim), generator=g).to(DT[kind]).cuda() for _ in range(4))
        w, b = torch.randn(dim, generator=g).cuda(), torch.randn(dim, generator=g).cuda()
        ref = rse.seq_layer_norm_fwd(x, w, b, residual=res, for_backward=True)
        back = rse.seq_layer_norm_bwd(ref.sum, dy, w, ref.stats, dsum)
        for y_in, sum_in in ((0, 1), (1, 0), (None, 0), (None, 1), (0, None), (1, None)):
            ins = [x.clone(), res.clone()]
            got = rse.seq_layer_norm_fwd(ins[0], w, b, residual=ins[1], out=None if y_in is None else ins[y_in],
                                         sum_out=None if sum_in is None else ins[sum_in])
            assert torch.equal(got.y, ref.y) and torch.equal(got.sum, ref.sum), (dim, y_in, sum_in)
        alone = x.clone()
        assert torch.equal(rse.seq_layer_norm_fwd(alone, w, b, out=alone).y, rse.seq_layer_norm_fwd(x, w, b).y), dim
        for place in (0, 1):
            ins = [dy.clone(), dsum.clone()]
            got = rse.seq_layer_norm_bwd(ref.sum, ins[0], w, ref.stats, ins[1], out=ins[place])
            assert all(torch.equal(a, c) for a, c in zip(got, back)), (dim, place)
