"""Attention of several new events per user over the paged history on the GPU
against the float64 oracle, what it stores, and what it reports."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import sequence as oseq

pytestmark = pytest.mark.gpu

F32, BF16 = 0, 1
KIND = {F32: "f32", BF16: "bf16 pairs"}      # (probabilities enter their product as pairs of bf16 values)
DT = {F32: torch.float32, BF16: torch.bfloat16}
BOUNDS = (0, 1, 2, 4, 8, 16, 32, 64)


@pytest.fixture(scope="module")
def rse():
    import recommender_sparse_embedding_amd as m

    return m


def _np(t):
    return t.detach().double().cpu().numpy()


class Users:
    """Users (events cached, new events) over a pool whose slots that no user
    holds are NaN, q, k and v as views of a joint projection."""

    def __init__(self, rse, users, H, Hk, D, dtype, causal=True, bounds=BOUNDS, page=16, seed=0, times="gaps", scale=None,
                 spare=0):
        self.rse, self.users, self.H, self.Hk, self.D, self.dtype, self.page = rse, users, H, Hk, D, dtype, page
        self.bounds, self.causal, dt = list(bounds), causal, DT[dtype]
        g = torch.Generator().manual_seed(seed + 31 * len(users) + sum(max(a, 0) + 7 * n for a, n in users))
        B, N = len(users), sum(n for _, n in users)
        self.most = max([max(a, 0) + n for a, n in users] + [1])
        self.max_new = max([n for _, n in users] + [1])
        per = -(-self.most // page) + spare
        n_pages = B * per + 2
        order = torch.randperm(n_pages, generator=g)[:B * per].view(B, per)
        self.table = order.to(torch.int32).cuda()
        self.k_pages, self.v_pages = (torch.full((n_pages, page, Hk, D), math.nan, dtype=dt) for _ in range(2))
        self.pos_pages = torch.full((n_pages, page), 12345, dtype=torch.int32)
        qkv = torch.randn((N, H + 2 * Hk, D), generator=g).to(dt)
        pos = torch.zeros(N, dtype=torch.int32)
        self.hist, at = [], 0
        for b, (a, n) in enumerate(users):
            if a < 0:
                self.hist.append((None, None, None, n))
                at += n
                continue
            k, v = (torch.randn((a, Hk, D), generator=g).to(dt) for _ in range(2))
            step = torch.randint(0, 30, (a + n,), generator=g) if times == "gaps" else torch.ones(a + n, dtype=torch.int64)
            t = step.cumsum(0)
            if times == "any":
                t = t[torch.randperm(a + n, generator=g)]
            t = t.to(torch.int32)
            for e in range(a):
                pg = int(order[b, e // page])
                self.k_pages[pg, e % page], self.v_pages[pg, e % page], self.pos_pages[pg, e % page] = k[e], v[e], t[e]
            pos[at:at + n] = t[a:]
            new = slice(at, at + n)
            self.hist.append((torch.cat([k, qkv[new, H:H + Hk]]), torch.cat([v, qkv[new, H + Hk:]]), t, n))
            at += n
        qkv = qkv.cuda()
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        self.pos = pos.cuda()
        self.bias = torch.randn((H, len(bounds) + 1), generator=g).cuda()
        self.off = torch.tensor(np.concatenate([[0], np.cumsum([n for _, n in users])]), dtype=torch.int64).cuda()
        self.lens = torch.tensor([a for a, _ in users], dtype=torch.int64).cuda()
        self.pools = [t.cuda() for t in (self.k_pages, self.v_pages, self.pos_pages)]
        self.cache = rse.SeqCache(*self.pools)
        self.attn = rse.SeqAttention(H, Hk, D, dtype, self.bounds, causal=causal, scale=scale)

    def call(self, **kw):
        kw = {"max_new": self.max_new, "max_len": self.most, **kw}
        return self.rse.seq_attention_chunk(self.attn, self.cache, self.q, self.k, self.v, self.pos, self.bias, self.off,
                                            self.table, self.lens, **kw)

    def oracle(self):
        hist = [(None if k is None else _np(k), None if k is None else _np(v), None if k is None else t.numpy(), n)
                for k, v, t, n in self.hist]
        return oseq.chunk(hist, _np(self.q), _np(self.bias), self.bounds, self.causal, self.attn.scale, KIND[self.dtype])

    def expected_pools(self):
        k, v, t = (x.clone() for x in (self.k_pages, self.v_pages, self.pos_pages))
        for b, ((a, n), (hk, hv, ht, _)) in enumerate(zip(self.users, self.hist)):
            for e in range(max(a, 0), a + n if a >= 0 else 0):
                pg = int(self.table[b, e // self.page])
                k[pg, e % self.page], v[pg, e % self.page], t[pg, e % self.page] = hk[e], hv[e], ht[e]
        return k, v, t

    def check(self, **kw):
        out = self.call(**kw)
        value, bound = self.oracle()
        got = _np(out)
        assert np.all(np.isfinite(got))
        off = np.abs(got - value)
        if np.any(off > bound):
            at = np.unravel_index(np.argmax(off / bound), off.shape)
            raise AssertionError(f"out at {at}: {got[at]} for {value[at]}, bound {bound[at]:.3g}")
        for name, x, y in zip("kvt", self.cache_tensors(), self.expected_pools()):
            x = x.cpu()
            assert torch.equal(torch.nan_to_num(x.double(), nan=-9.0), torch.nan_to_num(y.double(), nan=-9.0)), name
        assert self.attn.status() == 0 and self.cache.status() == 0
        return out

    def cache_tensors(self):
        return self.cache.k, self.cache.v, self.cache.pos


USERS = {"one event": [(0, 1)], "first events": [(0, 5), (0, 1), (0, 33)], "few": [(60, 3), (1, 2), (33, 1), (31, 4)],
         "idle and none": [(-1, 0), (20, 0), (-1, 3), (40, 2), (-1, 0), (7, 1)], "tile edges": [(31, 1), (32, 32), (33, 31), (63, 2)],
         "page edges": [(15, 1), (16, 1), (14, 4), (16, 16), (15, 18)], "many new": [(10, 200), (0, 65), (129, 1), (100, 128)],
         "long": [(700, 9), (3, 300), (650, 0)], "unequal": [(5, 1)] * 20 + [(90, 150)]}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("users", USERS)
def test_chunk_lengths(rse, users, D, dtype):
    Users(rse, USERS[users], 4, 2, D, dtype).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (4, 4), (6, 2), (8, 1), (24, 1), (40, 1), (96, 2)])
def test_chunk_heads_and_directions(rse, H, Hk, causal, dtype):
    """Among them heads that leave columns empty, and more than fill a tile."""
    Users(rse, [(40, 3), (3, 1), (77, 20), (150, 7)], H, Hk, 32, dtype, causal=causal).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bounds", [(), (5,), tuple(range(-20, 107)), (0, 0, 3, 3, 3), (-2**31 + 1, 2**31 - 1)])
@pytest.mark.parametrize("times", ["gaps", "any"])
def test_chunk_boundaries(rse, bounds, times, dtype):
    for users in ([(70, 3), (5, 2)], [(70, 40), (5, 90)]):
        Users(rse, users, 4, 2, 32, dtype, bounds=bounds, times=times).check()


@pytest.mark.parametrize("page", [8, 64, 1024])
def test_chunk_pages(rse, page):
    Users(rse, [(100, 9), (7, 60), (64, 64)], 4, 1, 64, BF16, page=page).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("users", [[(1300, 2)], [(1300, 70), (900, 5)], [(0, 600)]])
def test_chunk_histories_in_parts(rse, users, dtype):
    """Few users with long histories: parts on several blocks, joined."""
    u = Users(rse, users, 2, 1, 64, dtype)
    size = ctypes.c_size_t()
    rse.lib.rse_seqattn_chunk_workspace_size(u.attn.handle, u.q.shape[0], len(users), u.max_new, u.most, ctypes.byref(size))
    assert size.value > 0
    u.check()


def test_chunk_bounds_are_only_bounds(rse):
    """max_new and max_len may be larger than the data, and default."""
    users = [(50, 3), (9, 1)]
    a = Users(rse, users, 4, 2, 64, BF16, spare=3)
    ref = a.check()
    for kw in ({"max_new": None, "max_len": None}, {"max_new": 500, "max_len": 100}, {"max_new": 2**40, "max_len": 2**40}):
        b = Users(rse, users, 4, 2, 64, BF16, spare=3)
        got = b.check(**kw)
        assert got.shape == ref.shape


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_chunk_scale(rse, scale):
    for dtype in (F32, BF16):
        for users in ([(40, 3)], [(40, 50)]):
            Users(rse, users, 4, 2, 32, dtype, scale=scale).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_chunk_bias_that_hides(rse, dtype):
    """A bias of the type's lowest value hides its pairs; an event all of whose
    pairs are hidden gets 0."""
    for users in ([(40, 3)], [(40, 50)]):
        u = Users(rse, users, 4, 2, 32, dtype)
        u.bias[:, 3] = torch.finfo(torch.float32).min
        u.bias[2, :] = -math.inf
        u.check()
        assert torch.all(u.call()[:, 2] == 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("users", [[(40, 3), (30, 2)], [(40, 50), (30, 7)]])
def test_chunk_not_finite(rse, users, dtype):
    """A NaN or infinite key reaches the events that see it and no others."""
    u, clean = Users(rse, users, 4, 2, 32, dtype), Users(rse, users, 4, 2, 32, dtype)
    ref = clean.call()
    pg = int(u.table[0, 0])
    u.cache.k[pg, 5] = math.nan
    got = u.call()
    n = users[0][1]
    assert torch.all(torch.isnan(got[:n])) and torch.equal(got[n:], ref[n:])
    v = Users(rse, users, 4, 2, 32, dtype)
    v.k[n - 1] = math.nan                   # the first user's last new event: seen by itself only
    got = v.call()
    assert torch.all(torch.isnan(got[n - 1])) and torch.equal(got[n:], ref[n:])
    if n > 1:
        assert torch.equal(got[:n - 1], ref[:n - 1])


def test_chunk_equals_steps_and_forward(rse):
    """Events one by one through the step, in chunks, and all at once through
    the forward: the same arithmetic in another order."""
    g = torch.Generator().manual_seed(4)
    for dtype in (F32, BF16):
        n, H, Hk, D, page = 150, 4, 2, 64, 16
        dt = DT[dtype]
        q, k, v = (torch.randn((n, h, D), generator=g).to(dt).cuda() for h in (H, Hk, Hk))
        pos = torch.randint(0, 9, (n,), generator=g).cumsum(0).to(torch.int32).cuda()
        bias = torch.randn((H, len(BOUNDS) + 1), generator=g).cuda()
        attn = rse.SeqAttention(H, Hk, D, dtype, BOUNDS)
        ref = rse.seq_attention_fwd(attn, q, k, v, pos, bias, torch.tensor([0, n]).cuda())
        table = torch.arange(10, dtype=torch.int32).view(1, 10).cuda()
        cache = rse.SeqCache.empty(10, page, Hk, D, dtype)
        at, got = 0, []
        for size in (1, 40, 3, 100, 1, 5):
            lens = torch.tensor([at]).cuda()
            part = slice(at, at + size)
            if size == 1:
                got.append(rse.seq_attention_step(attn, cache, q[part], k[part], v[part], pos[part], bias, table, lens))
            else:
                got.append(rse.seq_attention_chunk(attn, cache, q[part], k[part], v[part], pos[part], bias,
                                                   torch.tensor([0, size]).cuda(), table, lens))
            at += size
        assert at == n
        off = (torch.cat(got).double() - ref.double()).abs().max()
        # two fp32 computations of values below 4 with relative errors of some
        # 150 terms (2 * 150 * 2^-24 * 4 < 2^-13), in bf16 rounded once each
        # (half of a spacing of 2^-6 on either side)
        assert off <= (2**-13 if dtype == F32 else 2**-6 + 2**-13)


def test_chunk_pool_past_32_bits(rse):
    """Slots whose elements lie past 2^32 bytes of the pool."""
    D, Hk, page = 128, 8, 64
    n_pages = (1 << 32) // (page * Hk * D * 2) + 20         # 4.3 GB each for k and v
    k, v = (torch.zeros((n_pages, page, Hk, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.zeros((n_pages, page), dtype=torch.int32, device="cuda")
    far = Users(rse, [(100, 3), (60, 40)], 8, Hk, D, BF16, page=page)
    big = rse.SeqCache(k, v, pos)
    shift = n_pages - far.cache.n_pages
    for x, y in zip((k, v, pos), far.cache_tensors()):
        x[shift:] = y
    ref = far.call()
    far.table += shift
    far.cache, small = big, far.cache
    got = far.call()
    assert torch.equal(got, ref)
    for x, y in zip((k, v, pos), (small.k, small.v, small.pos)):
        assert torch.equal(torch.nan_to_num(x[shift:].double()), torch.nan_to_num(y.double()))
    assert big.status() == 0


@pytest.mark.parametrize("users", [[(20, 3), (35, 2), (8, 1)], [(20, 3), (35, 60), (8, 1)]])
def test_chunk_bad_input_is_reported(rse, users):
    ref = Users(rse, users, 4, 2, 32, BF16).call()
    n = [0, *np.cumsum([x for _, x in users])]

    def run(change, **kw):
        u = Users(rse, users, 4, 2, 32, BF16)
        kw = change(u) or kw
        out = torch.full_like(ref, 7.0)
        u.call(out=out, **kw)
        return u, out

    BAD = -9
    # a history that does not fit max_len, or the table: that user's events are 0
    u, out = run(lambda u: {"max_len": users[1][0] + users[1][1] - 1})
    assert u.cache.status() == BAD and torch.all(out[n[1]:n[2]] == 0)
    assert torch.equal(out[:n[1]], ref[:n[1]]) and torch.equal(out[n[2]:], ref[n[2]:])
    u, out = run(lambda u: u.lens.__setitem__(0, 2**62))
    assert u.cache.status() == BAD and torch.all(out[:n[1]] == 0) and torch.equal(out[n[1]:], ref[n[1]:])
    # (another max_len may split the histories otherwise: its own reference)
    wide = Users(rse, users, 4, 2, 32, BF16).call(max_len=2**63 - 1)
    u, out = run(lambda u: u.lens.__setitem__(0, 2**63 - 1) or {"max_len": 2**63 - 1})
    assert u.cache.status() == BAD and torch.all(out[:n[1]] == 0) and torch.equal(out[n[1]:], wide[n[1]:])
    u, out = run(lambda u: u.lens.__setitem__(2, -5))           # idle, no error
    assert u.cache.status() == 0 and torch.all(out[n[2]:] == 0) and torch.equal(out[:n[2]], ref[:n[2]])
    # pages out of the pool: only what they hold is left out, nothing is written elsewhere
    for page in (-1, 10**6):
        u, out = run(lambda u: u.table.__setitem__((1, 0), page))
        assert u.cache.status() == BAD and torch.all(torch.isfinite(out))
        assert torch.equal(out[:n[1]], ref[:n[1]]) and torch.equal(out[n[2]:], ref[n[2]:])
        u, out = run(lambda u: u.table.__setitem__((1, u.table.shape[1] - 1), page))
        assert torch.equal(out[:n[1]], ref[:n[1]])
    # offsets: the sequences concerned are left as they were
    u, out = run(lambda u: u.off.__setitem__(1, n[2] + 1))
    assert u.attn.status() == BAD
    u, out = run(lambda u: u.off.__setitem__(3, n[3] - 1))
    assert u.attn.status() == BAD and torch.equal(out[:n[2]], ref[:n[2]]) and torch.all(out[n[3] - 1:] == 7)
    if users[1][1] > 8:
        u, out = run(lambda u: {"max_new": 8})
        assert u.attn.status() == BAD and torch.all(out[n[1]:n[2]] == 7)
        assert torch.all(torch.isfinite(out[:n[1]]))


def test_chunk_refusals(rse):
    u = Users(rse, [(20, 3), (8, 1)], 4, 2, 32, BF16)
    good = dict(q=u.q, k=u.k, v=u.v, pos=u.pos, off=u.off, table=u.table, lens=u.lens, out=None)

    def call(**kw):
        a = {**good, **kw}
        return rse.seq_attention_chunk(u.attn, u.cache, a["q"], a["k"], a["v"], a["pos"], u.bias, a["off"], a["table"],
                                       a["lens"], out=a["out"])

    call()
    for kw in ({"k": u.k[:3]}, {"q": u.q[:, :3]}, {"pos": u.pos[:3]}, {"lens": u.lens[:1]}, {"table": u.table[:1]},
               {"off": u.off[:1]}, {"out": torch.empty((4, 4, 64), dtype=torch.bfloat16, device="cuda")},
               {"q": torch.empty((4, 4, 33), dtype=torch.bfloat16, device="cuda")[:, :, 1:]}):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in ({"q": u.q.float()}, {"lens": u.lens.int()}, {"table": u.table.long()}, {"off": u.off.int()}, {"k": u.k.cpu()}):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(rse.RseError):
        call(out=torch.empty((1, 4, 32), dtype=torch.bfloat16, device="cuda").expand(4, 4, 32))
    other = rse.SeqCache.empty(4, 16, 4, 32)
    with pytest.raises(rse.RseError):
        rse.seq_attention_chunk(u.attn, other, u.q, u.k, u.v, u.pos, u.bias, u.off, u.table, u.lens)
    none = torch.empty((0, 4, 32), dtype=torch.bfloat16, device="cuda")
    got = rse.seq_attention_chunk(u.attn, u.cache, none, none[:, :2], none[:, :2], u.pos[:0], u.bias, u.off[:1],
                                  u.table[:0], u.lens[:0])
    assert got.shape == (0, 4, 32)


@pytest.mark.parametrize("users", [[(200, 3), (35, 2)], [(200, 60), (35, 7)]])
def test_chunk_in_a_graph_and_on_another_stream(rse, users):
    u = Users(rse, users, 4, 2, 64, BF16)
    refs, qs = [], []
    for s in range(3):
        x = Users(rse, users, 4, 2, 64, BF16)
        q = torch.randn(x.q.shape, generator=torch.Generator().manual_seed(s)).bfloat16().cuda()
        x.q = q
        qs.append(q)
        refs.append(x.call())
    u.q = qs[0].clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = u.call(stream=st)
    st.synchronize()
    assert torch.equal(got, refs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = u.call()
    for i in (0, 1, 2, 1, 0):
        u.q.copy_(qs[i])
        graph.replay()
        eager = u.rse.seq_attention_chunk(u.attn, u.cache, qs[2 - i], u.k, u.v, u.pos, u.bias, u.off, u.table, u.lens,
                                          max_new=u.max_new, max_len=u.most)
        torch.cuda.synchronize()
        assert torch.equal(out, refs[i]) and torch.equal(eager, refs[2 - i])


def test_chunk_repeats_are_identical(rse):
    u = Users(rse, [(1300, 70), (900, 5)], 4, 2, 64, BF16)
    a = u.call()
    assert all(torch.equal(u.call(), a) for _ in range(3))


# Histories of unequal users, idle ones and ones without events among them, that
# are split into parts (whose number follows the lengths on the device).
PARTS = {"many": [(1500, 40), (0, 1), (-1, 3), (700, 0), (260, 33), (511, 1), (512, 64), (3, 70)],
         "few": [(1300, 2), (-1, 1), (700, 3), (0, 2), (255, 1), (2000, 0)],
         "one of many": [(2, 1)] * 30 + [(1800, 25)] + [(-1, 0)] * 5}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("users", PARTS)
def test_chunk_parts_of_unequal_users(rse, users, D, dtype):
    for causal in (True, False):
        Users(rse, PARTS[users], 4, 2, D, dtype, causal=causal).check()


@pytest.mark.parametrize("users", [[(900, 3), (600, 2)], [(900, 50), (600, 7)]])
def test_chunk_not_finite_in_parts(rse, users):
    """NaN in one part reaches its users' events, and a part that sees nothing
    weighs nothing."""
    for dtype in (F32, BF16):
        u, clean = Users(rse, users, 4, 2, 32, dtype), Users(rse, users, 4, 2, 32, dtype)
        ref, n = clean.call(), users[0][1]
        u.cache.k[int(u.table[0, 20]), 5] = math.nan
        got = u.call()
        assert torch.all(torch.isnan(got[:n])) and torch.equal(got[n:], ref[n:])
        far = Users(rse, users, 4, 2, 32, dtype, times="ones", bounds=(400,))
        far.bias[:, 1] = -math.inf                              # keys further back than 400
        far.check()
        far.bias[:, :] = -math.inf
        assert torch.all(far.call() == 0)


def test_chunk_parts_follow_the_lengths(rse):
    """A captured call whose lengths grow between replays, as a program adds the
    events that it stored."""
    for new in (3, 40):
        users = [(600, new), (20, new), (100, new)]
        u = Users(rse, users, 4, 2, 64, BF16, spare=40)
        graph, most = torch.cuda.CUDAGraph(), u.most + 600
        u.call(max_len=most)
        torch.cuda.synchronize()
        lens = u.lens.clone()
        with torch.cuda.graph(graph):
            out = u.call(max_len=most)
        for step in (0, 1, 5, 2):
            at = lens.clone()
            at[1:] += 100 * step                                # (over pages of zeros and NaN: filled first)
            for pool in u.cache_tensors():
                pool.nan_to_num_(0) if pool.is_floating_point() else None
            u.lens.copy_(at)
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            eager = u.call(max_len=most)
            assert torch.equal(got, eager) and torch.all(torch.isfinite(got))
        assert u.cache.status() == 0 and u.attn.status() == 0


def test_chunk_long_table_windows(rse):
    """A part over more pages than a block keeps of the table at a time: the
    same keys in small and in large pages give the same bits."""
    H = 256                                                     # all heads apart: too many blocks for parts
    users = [(4300, 70)] + [(3, 66)] * 8                        # more than two tiles of 32 columns
    small = Users(rse, users, H, H, 32, BF16, page=8)
    large = Users(rse, users, H, H, 32, BF16, page=64)
    for name in ("q", "k", "v", "pos", "bias"):
        setattr(large, name, getattr(small, name))
    for b, (had, _) in enumerate(users):
        for pool, other in zip(large.cache_tensors(), small.cache_tensors()):
            pool.view(-1, *pool.shape[2:])[_slots(large, b, had)] = other.view(-1, *other.shape[2:])[_slots(small, b, had)]
    a, b = small.call(), large.call()
    assert torch.equal(a, b) and torch.all(torch.isfinite(a))


def _slots(u, b, n):
    e = torch.arange(n, device="cuda")
    return u.table[b].long()[e // u.page] * u.page + e % u.page


@pytest.mark.parametrize("new", [3, 40])
def test_chunk_bad_input_in_parts(rse, new):
    """What is reported of calls without parts is of those with them."""
    users = [(600, new), (700, new), (90, new)]
    ref = Users(rse, users, 4, 2, 32, BF16).call()
    for change, status, kept in ((lambda u: u.lens.__setitem__(1, 10**7), "cache", None),
                                 (lambda u: u.table.__setitem__((1, 30), -1), "cache", None),
                                 (lambda u: u.table.__setitem__((1, 30), 10**6), "cache", None),
                                 (lambda u: u.off.__setitem__(2, new - 1), "attn", 7.0),
                                 (lambda u: u.off.__setitem__(1, 10**9), "attn", 7.0),
                                 (lambda u: u.off.copy_(torch.tensor([0, 3 * new, 0, 3 * new])), "attn", None)):
        u = Users(rse, users, 4, 2, 32, BF16)
        change(u)
        out = torch.full_like(ref, 7.0)
        u.call(out=out)
        assert getattr(u, status).status() == -9
        if status == "cache":
            assert torch.equal(out[:new], ref[:new]) and torch.equal(out[2 * new:], ref[2 * new:])
        if kept is not None:
            assert torch.all(out[new:2 * new] == kept)
