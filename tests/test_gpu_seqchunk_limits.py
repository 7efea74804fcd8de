"""Attention of several new events per user at the limits of its arguments:
offsets that no batch has, blocks that are more than the parts of the keys aim
at, lengths that grow under a captured call, calls that a launch does not hold."""

import numpy as np
import pytest
import torch
from test_gpu_seqchunk import BF16, F32, KIND, Users, _np, rse  # noqa: F401  (rse: the fixture)

from oracle import sequence as oseq

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


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ranges_that_overlap(rse, dtype):  # noqa: F811
    """Offsets that go up and down between the ends, so that every other user has
    all events: reported, and rows are left or written, never read past the ends;
    where that makes more blocks than the parts' list holds, all are skipped."""
    for cached, last in ((0, 1961), (600, 1961), (600, 200)):
        users = [(0, 1)] * 39 + [(cached, last)]
        n = sum(c for _, c in users)
        u = Users(rse, users, 4, 4, 32, dtype, spare=n // 16 + 1)
        u.off.copy_(torch.tensor([0, n] * 20 + [n]))
        before = [t.clone() for t in u.cache_tensors()]
        out = torch.full_like(u.q, 7.0)
        u.call(out=out, max_new=n, max_len=cached + n)
        torch.cuda.synchronize()
        assert u.attn.status() == BAD and u.cache.status() == 0
        assert torch.all(torch.isfinite(out))
        if last > 1000:
            assert torch.all(out == 7.0)
            assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(u.cache_tensors(), before))


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


# Histories in parts where the calls' own blocks, heads by tiles of new events, are
# more than twice the parts aimed at (256 of fp32 rows of 128, else 512), and the
# histories ragged: (users, cached at most, by which power of the user's number).
CROWDED = {"all heads apart": (20, 400, 1, 16, 128, F32), "a few long ones": (100, 500, 4, 4, 128, F32),
           "narrow rows": (150, 500, 3, 4, 32, BF16), "wide batch": (40, 1000, 1, 16, 64, BF16)}


@pytest.mark.parametrize("case", CROWDED)
def test_parts_of_crowded_calls(rse, case):  # noqa: F811
    B, cached, power, H, D, dtype = CROWDED[case]
    u = Users(rse, [(int(cached * ((i + 1) / B) ** power), 130) for i in range(B)], H, H, D, dtype)
    assert u.most >= 512, "in parts"
    u.check(out=torch.full_like(u.q, 7.0))


def test_parts_of_crowded_calls_of_few_columns(rse):  # noqa: F811
    """Two tiles of new events a user, histories past 4096 events: oracle of the
    users of up to 1000, and of the longest one's last events."""
    B, H, D = 150, 2, 128
    users = [(int(4100 * ((i + 1) / B) ** 4), 64) for i in range(B)]
    u = Users(rse, users, H, H, D, F32)
    out = torch.full((B * 64, H, D), 7.0, device="cuda")
    u.call(out=out)
    assert u.attn.status() == 0 and u.cache.status() == 0
    got, q = _np(out), _np(u.q)
    assert np.all(np.isfinite(got)) and not np.any(np.all(got == 7.0, axis=(1, 2)))
    for b, (k, v, t, n) in enumerate(u.hist):
        if len(t) > 1000 and b < B - 1:
            continue
        at = slice(b * 64, (b + 1) * 64)
        value, bound = oseq.chunk([(_np(k), _np(v), t.numpy(), n)], q[at], _np(u.bias), u.bounds, True, u.attn.scale, KIND[F32])
        assert np.all(np.abs(got[at] - value) <= bound), b


@pytest.mark.parametrize("new", [3, 40])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_replays_follow_the_lengths(rse, new, dtype):  # noqa: F811
    """A captured call in parts whose lengths grow and shrink between replays,
    each replay against the oracle of what the pages hold."""
    u = Users(rse, [(600, new), (20, new), (100, new)], 4, 2, 64, dtype, spare=40)
    for pool in u.cache_tensors()[:2]:
        pool.nan_to_num_(0.5)
    graph, most = torch.cuda.CUDAGraph(), u.most + 600
    u.call(max_len=most)
    torch.cuda.synchronize()
    lens = u.lens.clone()
    with torch.cuda.graph(graph):
        out = u.call(max_len=most)
    for step in (0, 1, 5, 2):
        u.lens.copy_(lens)
        u.lens[1:] += 100 * step
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        hist = []
        for b, had in enumerate(u.lens.tolist()):
            e = torch.arange(had + new, device="cuda")
            at = u.table[b].long()[e // u.page], e % u.page
            hist.append((*(_np(pool[at]) for pool in u.cache_tensors()[:2]), u.cache.pos[at].cpu().numpy(), new))
        value, bound = oseq.chunk(hist, _np(u.q), _np(u.bias), u.bounds, True, u.attn.scale, KIND[dtype])
        assert np.all(np.abs(_np(out) - value) <= bound), step
    assert u.cache.status() == 0 and u.attn.status() == 0


@pytest.mark.parametrize("users", [[(40, 3), (0, 2)], [(40, 70), (0, 66)], [(900, 3)], [(900, 70)]])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bounds", [(5,), (-2**31 + 1, -7, 0, 2**31 - 1)])
def test_times_at_the_ends_of_32_bits(rse, users, dtype, bounds):  # noqa: F811
    """Distances saturate: times at both ends of int32, in cached and new events."""
    u = Users(rse, users, 4, 2, 32, dtype, bounds=bounds)
    g = np.random.default_rng(3)
    at = np.array([-2**31, -2**31 + 1, -9, 0, 4, 2**31 - 2, 2**31 - 1])
    first = 0
    for b, (had, new) in enumerate(users):
        k, v, t, n = u.hist[b]
        t = torch.from_numpy(g.choice(at, had + new)).to(torch.int32)
        u.hist[b] = (k, v, t, n)
        e = torch.arange(had)
        page = u.table[b].cpu().long()[e // u.page]
        u.pos_pages[page, e % u.page] = t[:had]
        u.cache.pos[page.cuda(), (e % u.page).cuda()] = t[:had].cuda()
        u.pos[first:first + new] = t[had:].cuda()
        first += new
    u.check()


@pytest.mark.parametrize("new", [3, 70])
def test_tables_without_pages(rse, new):  # noqa: F811
    """No history fits: reported, out is 0, nothing is stored; idle users are none."""
    u = Users(rse, [(0, new), (-1, 2), (0, 1)], 4, 2, 32, BF16)
    before = [t.clone() for t in u.cache_tensors()]
    out = rse.seq_attention_chunk(u.attn, u.cache, u.q, u.k, u.v, u.pos, u.bias, u.off, u.table[:, :0].contiguous(), u.lens)
    assert u.cache.status() == BAD and u.attn.status() == 0 and torch.all(out == 0)
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(u.cache_tensors(), before))
