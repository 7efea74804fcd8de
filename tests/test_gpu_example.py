"""The behaviour-attention example: it trains, and its single-event answers
are the forward's rows."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_behaviour_attention_example():
    spec = importlib.util.spec_from_file_location("behaviour_attention",
                                                  os.path.join(ROOT, "examples", "behaviour_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, off = mod.main(users=60, steps=20)
    assert losses[-1] < losses[0]
    # outputs of magnitude below 4, rounded to bf16 twice (spacing 2^-6 there),
    # the same sums in another order
    assert off <= 2**-5


def test_example_serves_what_it_trains():
    """Events whose id has no row are hidden in training: serving answers the
    other events as the forward that hides them does."""
    import torch

    import recommender_sparse_embedding_amd as rse

    spec = importlib.util.spec_from_file_location("behaviour_attention",
                                                  os.path.join(ROOT, "examples", "behaviour_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    model = mod.Recommender()
    g = torch.Generator().manual_seed(3)
    counts = torch.tensor([1, 2, 40, 17, 100, 33, 9, 3]).cuda()
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    n = int(offsets[-1])
    ids = torch.randint(0, 50, (n,), generator=g).cuda()
    times = torch.randint(1, 900, (n,), generator=g).cumsum(0).to(torch.int32).cuda()
    target = torch.randn((n, mod.HEADS, mod.HEAD_DIM), generator=g).cuda()
    for _ in range(3):
        model.train(ids, times, offsets, target, 100)
    last = offsets[1:] - 1
    ids[torch.rand(n, generator=g).cuda() < 0.3] = 10**9
    ids[last] = torch.tensor([1, 2, 10**9, 3, 4, 5, 10**9, 6]).cuda()
    ids[offsets[7]:last[7]] = 10**9              # a user of whose history nothing is known
    rows, _, x = model.lookup(ids, train=False)
    want = rse.seq_attention_fwd(model.attn, *model.project(x), times, model.bias, offsets, key_off=rows)[last]
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[last] = False
    cache, table, lens, free = model.cache(ids[keep], times[keep].contiguous(), counts - 1, 64, 8)
    got, free = model.answer(cache, table, lens, free, ids[last], times[last].contiguous())
    found = rows[last] >= 0
    assert found.tolist() == [True, True, False, True, True, True, False, True]
    # outputs of magnitude below 4, rounded to bf16 twice (spacing 2^-6 there)
    assert (got[found].float() - want[found].float()).abs().max() <= 2**-5
    assert torch.all(got[~found] == 0)
    assert model.attn.status() == 0 and cache.status() == 0
    visible = [int((rows[a:b] >= 0).sum()) for a, b in zip(offsets[:-1].tolist(), offsets[1:].tolist())]
    assert lens.tolist() == visible
