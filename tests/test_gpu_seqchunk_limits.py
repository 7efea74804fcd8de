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
