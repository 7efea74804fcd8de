"""Attention of several new events per user at the limits of its arguments:
offsets that no batch has, histories in more parts than the usual sizes make,
calls that a launch does not hold."""

import numpy as np
import pytest
import torch
from test_gpu_seqchunk import BF16, F32, Users, _np, rse  # noqa: F401  (rse: the fixture)

pytestmark = pytest.mark.gpu

BAD = -9


def _left_or_right(out, ref, what):
    """Every event's rows are the call's without the fault, or as they were."""
    same, kept = (torch.all((out == x).flatten(1), 1) for x in (ref, torch.full_like(out, 7.0)))
    assert torch.all(same | kept), what


# One user with many more new events than the others: tiles are found by a
# search; and users alike, few and many columns.
FOUND = {"search": [(5, 1)] * 40 + [(9, 400)], "many": [(20, 70), (3, 66), (8, 80)], "few": [(20, 3), (3, 2), (8, 1)]}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("users", FOUND)
def test_offsets_at_the_ends_of_64_bits(rse, users, dtype):  # noqa: F811
    """The lowest offset, multiplied by a tile's events, is 0 in 64 bits."""
    users = FOUND[users]
    ref = Users(rse, users, 4, 2, 32, dtype).call()
    for at in (0, len(users) // 2, len(users)):
        for value in (-2**63, -2**63 + 1, -2**62, -2**58, -1, 2**58, 2**62, 2**63 - 1):
            u = Users(rse, users, 4, 2, 32, dtype)
            u.off[at] = value
            out = torch.full_like(ref, 7.0)
            u.call(out=out)
            assert u.attn.status() == BAD, (at, value)
            _left_or_right(out, ref, (at, value))


def test_more_blocks_than_a_launch_holds(rse):  # noqa: F811
    """2^22 users of 4 heads are 2^24 blocks of 256 threads: refused by name, in
    every call over users or events, and nothing is written."""
    n, H, D = 1 << 22, 4, 32
    attn = rse.SeqAttention(H, H, D, BF16)
    row = torch.zeros((1, H, D), dtype=torch.bfloat16, device="cuda").expand(n, H, D)
    out = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ints = torch.zeros(n, dtype=torch.int32, device="cuda")
    off, lens = torch.arange(n + 1, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")
    bias = torch.zeros((H, 1), device="cuda")
    cache = rse.SeqCache.empty(4, 8, H, D)
    saved = torch.empty(1 << 32, dtype=torch.uint8, device="cuda")
    grads = [torch.empty_like(out) for _ in range(3)]
    for call in (lambda: rse.seq_attention_chunk(attn, cache, row, row, row, ints, bias, off, ints.view(n, 1), lens, max_new=1, out=out),
                 lambda: rse.seq_attention_step(attn, cache, row, row, row, ints, bias, ints.view(n, 1), lens, out=out),
                 lambda: rse.seq_attention_fwd(attn, row, row, row, ints, bias, off, max_len=200, out=out),
                 lambda: rse.seq_attention_bwd(attn, row, row, row, ints, bias, off, saved, row, max_len=200, grads=grads)):
        with pytest.raises(rse.RseError, match="UNSUPPORTED"):
            call()
    assert torch.all(out == 7)
    assert attn.status() == 0 and cache.status() == 0
