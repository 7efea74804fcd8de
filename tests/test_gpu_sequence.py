"""Attention over behaviour sequences on the GPU against the float64 oracle:
forward, every gradient, the single-event step over the paged history, page
tables and slots.  An element may be off by the oracle's bound for it (sums in
fp32, bf16 products where the type is bf16), no more."""

import math

import numpy as np
import pytest
import torch

from oracle import sequence as oseq

pytestmark = pytest.mark.gpu

F32, BF16 = 0, 1
KIND = {F32: "f32", BF16: "bf16"}
DT = {F32: torch.float32, BF16: torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(got, ref, what):
    value, bound = ref
    got = _np(got)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    off = np.abs(got - value)
    at = np.unravel_index(np.argmax(off / bound), off.shape) if off.size else ()
    assert np.all(off <= bound), f"{what} at {at}: {got[at]} for {value[at]}, bound {bound[at]:.3g}"


class Case:
    """Inputs of one jagged batch, as views of a joint [N, H + 2 Hk, D] tensor."""

    def __init__(self, lens, H, Hk, D, dtype, causal=True, bounds=(0, 1, 2, 4, 8, 16, 32, 64), times=True, missing=0.0,
                 seed=0, size=1.0):
        import recommender_sparse_embedding_amd as rse

        self.rse, self.causal, self.bounds, self.dtype = rse, causal, list(bounds), dtype
        g = torch.Generator().manual_seed(seed + 1000 * len(lens) + sum(lens))
        N = sum(lens)
        qkv = (torch.randn((N, H + 2 * Hk, D), generator=g) * size).to(DT[dtype]).cuda()
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        self.dout = torch.randn((N, H, D), generator=g).to(DT[dtype]).cuda()
        gaps = torch.randint(0, 30, (N,), generator=g) if times else torch.ones(N, dtype=torch.int64)
        self.pos = gaps.cumsum(0).to(torch.int32).cuda()
        self.bias = torch.randn((H, len(bounds) + 1), generator=g).cuda()
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int64).cuda()
        self.key_off = None
        if missing:
            self.key_off = torch.where(torch.rand(N, generator=g) < missing, -1, 5).cuda()
        self.max_len = max(lens, default=0)
        self.attn = rse.SeqAttention(H, Hk, D, dtype, bounds, causal=causal)

    def oracle(self, dout=True):
        return oseq.attention(_np(self.q), _np(self.k), _np(self.v), self.pos.cpu().numpy(), _np(self.bias),
                              self.off.cpu().numpy(), self.bounds, self.causal, self.attn.scale,
                              None if self.key_off is None else self.key_off.cpu().numpy(),
                              _np(self.dout) if dout else None, KIND[self.dtype])

    def run(self, **kw):
        kw = {"key_off": self.key_off, "max_len": self.max_len, **kw}
        where = (self.attn, self.q, self.k, self.v, self.pos, self.bias, self.off)
        out, saved = self.rse.seq_attention_fwd(*where, for_backward=True, **kw)
        dq, dk, dv, db = self.rse.seq_attention_bwd(*where, saved, self.dout, **kw)
        assert self.attn.status() == 0
        return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dbias": db}

    def forward(self, **kw):
        kw = {"key_off": self.key_off, "max_len": self.max_len, **kw}
        return self.rse.seq_attention_fwd(self.attn, self.q, self.k, self.v, self.pos, self.bias, self.off, **kw)

    def check(self):
        got, ref = self.run(), self.oracle()
        for name in got:
            _check(got[name], ref[name], name)
        assert torch.equal(self.forward(), got["out"])
        return got


LENS = {"one": [1], "empties": [0, 1, 0, 0, 2, 0], "tile edges": [31, 32, 33, 63, 64, 65], "blocks": [127, 128, 129],
        "long": [300, 5], "longer": [513], "none": [0, 0], "many": [(7 * i) % 41 for i in range(60)]}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_attention_lengths(lens, D, dtype):
    Case(LENS[lens], 4, 2, D, dtype).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (4, 4), (6, 2), (8, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_heads_and_directions(H, Hk, causal, dtype):
    Case([40, 3, 77, 150], H, Hk, 64, dtype, causal=causal, missing=0.3).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bounds", [(), (5,), tuple(range(-63, 64)), tuple(2**m for m in range(31)),
                                    (0, 0, 3, 3, 3, 2**31 - 1)])
def test_attention_boundaries(bounds, dtype):
    if not bounds:
        # one bucket: its gradient is the sum of all ds, 0 but for rounding
        got, ref = (c := Case([50, 140], 2, 1, 32, dtype, bounds=bounds)).run(), c.oracle()
        assert np.all(np.abs(_np(got["dbias"])) <= ref["dbias"][1])
    Case([50, 140], 2, 1, 32, dtype, bounds=bounds, causal=False).check()
    Case([50, 140], 2, 1, 32, dtype, bounds=bounds, times=False).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_any_order_of_times(dtype):
    c = Case([60, 130], 2, 2, 32, dtype, bounds=(-100, -1, 0, 7, 2**20, 2**30, 2**31 - 1), causal=False)
    g = torch.Generator().manual_seed(1)
    c.pos = torch.randint(-2**31, 2**31, c.pos.shape, generator=g).to(torch.int32).cuda()
    c.pos[::7] = -2**31
    c.pos[1::7] = 2**31 - 1
    c.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing_and_what_they_hide(causal, dtype):
    """Every key of one sequence and the first keys of the others have no row;
    their keys and values hold NaN and infinities, which nothing may see."""
    c = Case([70, 33, 1, 140, 64], 4, 2, 64, dtype, causal=causal)
    off = torch.zeros(c.pos.numel(), dtype=torch.int64)
    off[70:103] = -1                  # the whole second sequence
    off[103] = -9
    off[104:110] = -1                 # its first events see nothing when causal
    off[150:170] = -(2**62)
    c.key_off = off.cuda()
    hide = c.key_off < 0
    c.k[hide] = float("nan")
    c.v[hide] = torch.tensor(float("inf")).to(c.v.dtype)
    got = c.check()
    assert torch.all(got["out"][70:104] == 0) and torch.all(got["dq"][70:104] == 0)
    assert torch.all(got["dk"][hide] == 0) and torch.all(got["dv"][hide] == 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_neighbours_do_not_leak(dtype):
    """A sequence of NaN between two others, and rows before and after the batch."""
    c = Case([37, 20, 45], 2, 1, 64, dtype)
    ref = c.oracle()
    for t in (c.q, c.k, c.v, c.dout):
        t[37:57] = float("nan")
    got = c.run()
    keep = torch.ones(102, dtype=torch.bool)
    keep[37:57] = False
    for name in ("out", "dq", "dk", "dv"):
        _check(got[name][keep.cuda()], tuple(x[keep.numpy()] for x in ref[name]), name)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(dtype):
    """Scores of some hundreds: probabilities of 0 and 1, no overflow."""
    Case([90, 150], 2, 1, 64, dtype, size=6.0).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bias_of_the_lowest_value(dtype):
    """A bucket's bias at the type's lowest value acts as a mask; a row with
    nothing else takes the plain average of equal scores."""
    c = Case([40, 90], 2, 2, 32, dtype, bounds=(1, 2, 4))
    c.bias[:, 2] = torch.finfo(torch.float32).min
    c.bias[0, 0] = -1e30
    got = c.run()
    off, lo = c.oracle(), c.bias[:, 2].cpu().numpy()
    assert np.all(lo < -3e38)
    # the bounds hold wherever the row has a finite-scale score; those rows
    # are the ones whose best score is ordinary
    ordinary = off["lse"].T > -1e4
    out = _np(got["out"])
    assert np.all(np.isfinite(out))
    err = np.abs(out - off["out"][0])
    scale = np.abs(_np(c.v)).max() * (4e-3 if dtype == F32 else 2e-2)
    assert np.all(err[ordinary] <= scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeat_runs_are_identical(dtype):
    c = Case([200, 31, 129, 64], 4, 2, 64, dtype, missing=0.1)
    a, b = c.run(), c.run()
    for name in a:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_match_differences(dtype):
    """The directional derivative of sum(out * dout) along random directions,
    by central differences of the float64 oracle."""
    c = Case([20, 140], 2, 1, 32, dtype, bounds=(1, 2, 4, 8, 40))
    got, ref = c.run(), c.oracle()
    rng = np.random.default_rng(3)
    base = [_np(c.q), _np(c.k), _np(c.v), _np(c.bias)]
    do = _np(c.dout)

    def loss(x):
        o = oseq.attention(*x[:3], c.pos.cpu().numpy(), x[3], c.off.cpu().numpy(), c.bounds, True, c.attn.scale)
        return float((o["out"][0] * do).sum())

    for at, name in enumerate(("dq", "dk", "dv", "dbias")):
        way = rng.choice([-1.0, 1.0], base[at].shape)
        hi, lo = list(base), list(base)
        hi[at], lo[at] = base[at] + 1e-5 * way, base[at] - 1e-5 * way
        slope = (loss(hi) - loss(lo)) / 2e-5
        # every element may be off by its bound; differences by 1e-6
        assert abs((_np(got[name]) * way).sum() - slope) <= ref[name][1].sum() + 1e-6 * (1 + abs(slope)), name


def test_strides_past_32_bits():
    """Events 2^28 elements apart: byte offsets far past 2^32."""
    c = Case([3, 9], 2, 1, 32, BF16)
    far = torch.empty((12, 1 << 28), dtype=torch.bfloat16, device="cuda")
    q, k, v = (far[:, a:a + h * 32].view(12, h, 32) for a, h in ((0, 2), (64, 1), (96, 1)))
    for t, x in ((q, c.q), (k, c.k), (v, c.v)):
        t.copy_(x)
    ref, want = c.oracle(), c.run()
    c.q, c.k, c.v = q, k, v
    got = c.run()
    for name in got:
        assert torch.equal(got[name], want[name])
        _check(got[name], ref[name], name)


def test_joint_gradient_views_and_another_stream():
    c = Case([30, 80], 4, 2, 64, BF16)
    want = c.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        joint = torch.full((110, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    where = (c.attn, c.q, c.k, c.v, c.pos, c.bias, c.off)
    out, saved = c.rse.seq_attention_fwd(*where, max_len=80, for_backward=True, stream=side)
    views = (joint[:, :4], joint[:, 4:6], joint[:, 6:])
    got = c.rse.seq_attention_bwd(*where, saved, c.dout, max_len=80, grads=views, stream=side)
    side.synchronize()
    assert torch.equal(out, want["out"]) and torch.equal(got[3], want["dbias"])
    for x, name in zip(views, ("dq", "dk", "dv")):
        assert torch.equal(x, want[name]), name


def test_max_len_is_only_a_bound():
    """A looser max_len may take other kernels: the results keep their bounds."""
    for dtype in (F32, BF16):
        c = Case([20, 100, 3], 4, 2, 64, dtype)
        ref = c.oracle()
        for most in (100, 123, None, 10**12):
            got = c.run(max_len=most)
            for name in got:
                _check(got[name], ref[name], f"{name} at max_len {most}")


def test_malformed_offsets_are_reported():
    c = Case([20, 30], 2, 1, 64, BF16)
    for bad in ([0, 20, 49], [0, 60, 50], [1, 20, 50], [0, -5, 50]):
        c.off = torch.tensor(bad, dtype=torch.int64).cuda()
        c.forward(max_len=50)
        assert c.attn.status() == -9, bad
        c.attn.clear_status()
    c.off = torch.tensor([0, 20, 50], dtype=torch.int64).cuda()
    c.forward(max_len=29)                        # the second sequence is longer
    assert c.attn.status() == -9
    c.attn.clear_status()
    _check(c.forward(max_len=30), c.oracle(False)["out"], "after the status was cleared")


def test_refusals_of_tensors():
    c = Case([20, 30], 2, 1, 64, BF16)
    rse = c.rse
    where = [c.attn, c.q, c.k, c.v, c.pos, c.bias, c.off]

    def call(at, x):
        return rse.seq_attention_fwd(*where[:at], x, *where[at + 1:])

    with pytest.raises(TypeError):
        call(1, c.q.float())
    with pytest.raises(ValueError):
        call(1, c.q[:, :1])
    with pytest.raises(ValueError, match="16 bytes"):
        call(2, torch.zeros((50, 1, 68), dtype=torch.bfloat16, device="cuda")[:, :, 1:65])
    with pytest.raises(ValueError, match="16 bytes"):
        call(2, torch.zeros((50, 64, 2), dtype=torch.bfloat16, device="cuda")[:, :, :1].transpose(1, 2))
    with pytest.raises(TypeError):
        call(4, c.pos.long())
    with pytest.raises(ValueError):
        call(5, c.bias[:, 1:].contiguous())
    with pytest.raises(TypeError):
        call(6, c.off.int())
    with pytest.raises(ValueError):
        call(6, c.off[:1])
    with pytest.raises(rse.RseError) as e:
        rse.seq_attention_fwd(*where, max_len=-1)
    assert e.value.code == -1
    out, saved = rse.seq_attention_fwd(*where, for_backward=True)
    with pytest.raises(rse.RseError) as e:
        rse.seq_attention_bwd(*where, saved[:8].contiguous(), c.dout)
    assert e.value.code == -3


# ------------------------------------------------------------------- serving --
class Serving:
    def __init__(self, lens, H, Hk, D, dtype, page=16, bounds=(1, 2, 4, 8, 16, 32, 64, 128), extra=0, seed=0):
        import recommender_sparse_embedding_amd as rse

        self.rse, self.lens, self.page, self.dtype, self.bounds = rse, lens, page, dtype, list(bounds)
        g = torch.Generator().manual_seed(seed + sum(lens))
        B, most = len(lens), max(max(lens) // page + 1, 1)
        n_pages = B * most + 2 + extra
        self.table = (torch.randperm(B * most, generator=g) + 2 + extra).view(B, most).to(torch.int32)
        norm = lambda *s: torch.randn(s, generator=g).to(DT[dtype]).cuda()  # noqa: E731
        self.cache = rse.SeqCache.empty(n_pages, page, Hk, D, dtype)
        if extra < 1000:                         # what nobody cached is NaN
            self.cache.k.fill_(float("nan"))
            self.cache.v.fill_(float("nan"))
            self.cache.pos.fill_(-2**31)
        self.q, self.nk, self.nv = norm(B, H, D), norm(B, Hk, D), norm(B, Hk, D)
        self.hist = []
        for b, n in enumerate(lens):
            if n < 0:
                self.hist.append(None)
                continue
            k, v = norm(n, Hk, D), norm(n, Hk, D)
            t = torch.randint(0, 40, (n + 1,), generator=g).cumsum(0).to(torch.int32).cuda()
            slot = self.table[b].long()[torch.arange(n) // page] * page + torch.arange(n) % page
            at = slot.cuda()
            self.cache.k.view(-1, Hk, D)[at] = k
            self.cache.v.view(-1, Hk, D)[at] = v
            self.cache.pos.view(-1)[at] = t[:n]
            self.hist.append((torch.cat([k, self.nk[b:b + 1]]), torch.cat([v, self.nv[b:b + 1]]), t))
        self.pos = torch.tensor([0 if h is None else int(h[2][-1]) for h in self.hist], dtype=torch.int32).cuda()
        self.bias = torch.randn((H, len(bounds) + 1), generator=g).cuda()
        self.attn = rse.SeqAttention(H, Hk, D, dtype, bounds)
        self.t_lens = torch.tensor(lens, dtype=torch.int64).cuda()
        self.table = self.table.cuda()

    def run(self, **kw):
        kw = {"max_len": max(self.lens) + 1, **kw}
        return self.rse.seq_attention_step(self.attn, self.cache, self.q, self.nk, self.nv, self.pos, self.bias,
                                           self.table, self.t_lens, **kw)

    def oracle(self):
        hist = [None if h is None else (_np(h[0]), _np(h[1]), h[2].cpu().numpy()) for h in self.hist]
        return oseq.step(hist, _np(self.q), _np(self.bias), self.bounds, self.attn.scale, KIND[self.dtype])

    def check(self):
        out = self.run()
        _check(out, self.oracle(), "step")
        assert self.cache.status() == 0
        for b, n in enumerate(self.lens):
            if n >= 0:
                p = int(self.table[b, n // self.page])
                assert torch.equal(self.cache.k[p, n % self.page], self.nk[b])
                assert torch.equal(self.cache.v[p, n % self.page], self.nv[b])
                assert int(self.cache.pos[p, n % self.page]) == int(self.pos[b])
            else:
                assert torch.all(out[b] == 0)
        assert torch.equal(self.run(), out)      # the lengths did not move: the same again
        return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("lens,page", [([0], 16), ([0, -1, 1, 15, 16, 17], 16), ([31, 32, 33, 63, 64, 65, -1], 8),
                                       ([300], 64), ([1500, 3, 700], 32), ([5], 1024)])
def test_step_lengths(lens, page, D, dtype):
    Serving(lens, 4, 2, D, dtype, page).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (8, 1), (12, 4), (16, 1), (40, 2)])
def test_step_heads(H, Hk, dtype):
    Serving([100, 37, 0], H, Hk, 64, dtype).check()


@pytest.mark.parametrize("bounds", [(), tuple(range(-60, 67)), tuple(2**m for m in range(31))])
def test_step_boundaries(bounds):
    Serving([100, 260], 4, 2, 32, BF16, bounds=bounds).check()


def test_step_pool_past_32_bits():
    """Pages past 2^32 bytes and 2^31 elements of the pool."""
    extra = (1 << 31) // (64 * 2 * 128) + 100
    Serving([70, 10], 4, 2, 128, BF16, 64, extra=extra).check()


def test_step_bad_input_is_reported():
    s = Serving([20, 40], 4, 2, 64, BF16)
    good = s.run()
    s.run(max_len=30)                            # the second history is longer
    assert s.cache.status() == -9
    s.cache.clear_status()
    table = s.table.clone()
    s.table[1, 0] = 10**6
    out = s.run()
    assert s.cache.status() == -9 and torch.equal(out[0], good[0]) and torch.all(torch.isfinite(out))
    s.cache.clear_status()
    s.table = table
    s.t_lens = torch.tensor([20, 10**9], dtype=torch.int64).cuda()
    out = s.run()
    assert s.cache.status() == -9 and torch.equal(out[0], good[0]) and torch.all(out[1] == 0)


def test_step_in_a_graph():
    s = Serving([20, 400, -1, 0], 4, 2, 64, BF16)
    want = s.check().clone()
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run(out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(out=out)
    for _ in range(4):
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(s.run(), want)


def test_training_in_a_graph():
    c = Case([20, 130, 0, 64], 4, 2, 64, BF16)
    want = c.run()
    torch.cuda.synchronize()
    where = (c.attn, c.q, c.k, c.v, c.pos, c.bias, c.off)

    def once():
        out, saved = c.rse.seq_attention_fwd(*where, max_len=c.max_len, for_backward=True)
        return (out, *c.rse.seq_attention_bwd(*where, saved, c.dout, max_len=c.max_len))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once()
    for _ in range(4):
        for t in got:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for t, name in zip(got, ("out", "dq", "dk", "dv", "dbias")):
            assert torch.equal(t, want[name]), name
        c.run()


@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("B", [1, 7, 1500])
def test_assign_and_write(B, page):
    import recommender_sparse_embedding_amd as rse

    rng = np.random.default_rng(B + page)
    lens = rng.integers(0, 40, B)
    counts = np.where(rng.random(B) < 0.2, 0, rng.integers(0, 90, B))
    most = int((lens + counts).max()) // page + 1
    n_pages = B * most + 5
    ids = rng.permutation(n_pages).astype(np.int32)
    held = np.arange(most)[None, :] < -(-lens[:, None] // page)
    table = np.where(held, ids[:B * most].reshape(B, most), -1).astype(np.int32)
    free = np.setdiff1d(ids, table[held])
    rng.shuffle(free)
    ref = oseq.assign(counts, lens, table, free, page)
    cache = rse.SeqCache.empty(n_pages, page, 2, 32)
    for t in (cache.k, cache.v, cache.pos):
        t.zero_()
    cuda = lambda x, dt: torch.tensor(x, dtype=dt).cuda()  # noqa: E731
    t_table, N = cuda(table, torch.int32), int(counts.sum())
    args = (cache, cuda(counts, torch.int64), cuda(lens, torch.int64), t_table)
    slots, off, taken = rse.seq_cache_assign(*args, cuda(free, torch.int32), N)
    assert slots.tolist() == ref[0] and off.tolist() == ref[1] and taken.item() == ref[2]
    assert t_table.tolist() == ref[3] and cache.status() == 0
    joint = torch.randn((N, 4, 32), device="cuda").bfloat16()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    rse.seq_cache_write(cache, slots, joint[:, :2], joint[:, 2:], pos)
    assert torch.equal(cache.k.view(-1, 2, 32)[slots], joint[:, :2])
    assert torch.equal(cache.v.view(-1, 2, 32)[slots], joint[:, 2:])
    assert torch.equal(cache.pos.view(-1)[slots], pos)
    rest = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert torch.all(cache.k.view(-1, 64)[rest] == 0) and torch.all(cache.pos.view(-1)[rest] == 0)
    if ref[2] == 0:
        return
    # a free list one page short: nothing is assigned
    before = cuda(table, torch.int32)
    again = before.clone()
    slots, _, taken = rse.seq_cache_assign(*args[:3], again, cuda(free[:ref[2] - 1], torch.int32), N)
    assert cache.status() == -5 and torch.all(slots == -1) and taken.item() == 0 and torch.equal(again, before)
    cache.clear_status()
    # a count that does not fit the table, a negative one, a wrong sum
    for bad in ((0, most * page + 1), (0, -1), (0, int(counts[0]) + 1)):
        c = counts.copy()
        c[bad[0]] = bad[1]
        _, _, taken = rse.seq_cache_assign(cache, cuda(c, torch.int64), args[2], again, cuda(free, torch.int32), N)
        assert cache.status() == -9 and taken.item() == 0 and torch.equal(again, before)
        cache.clear_status()
    # slots: negative ones are skipped, one past the pool is reported
    kept = cache.k.clone()
    odd = torch.tensor([-1, n_pages * page], dtype=torch.int64, device="cuda")
    two = torch.ones((2, 2, 32), dtype=torch.bfloat16, device="cuda")
    rse.seq_cache_write(cache, odd, two, two, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert cache.status() == -9 and torch.equal(cache.k, kept)


def test_prompt_then_steps_equal_one_pass():
    """A session's events through the forward, their keys stored, then events
    one by one: each step's output is the causal forward's row."""
    import recommender_sparse_embedding_amd as rse

    g = torch.Generator().manual_seed(4)
    lens, more, H, Hk, D, P = [5, 40, 0, 33], 3, 4, 2, 64, 16
    B, full = len(lens), [n + more for n in lens]
    N = sum(full)
    q, k, v = (torch.randn((N, h, D), generator=g).bfloat16().cuda() for h in (H, Hk, Hk))
    pos = torch.randint(0, 20, (N,), generator=g).cumsum(0).to(torch.int32).cuda()
    bias = torch.randn((H, 6), generator=g).cuda()
    attn = rse.SeqAttention(H, Hk, D, rse.BF16, [1, 5, 25, 125, 625])
    off = torch.tensor(np.concatenate([[0], np.cumsum(full)]), dtype=torch.int64).cuda()
    want = rse.seq_attention_fwd(attn, q, k, v, pos, bias, off)
    cache = rse.SeqCache.empty(64, P, Hk, D)
    table = torch.full((B, 4), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(64, generator=g).to(torch.int32).cuda()
    first = torch.cat([torch.arange(int(off[b]), int(off[b]) + n) for b, n in enumerate(lens)]).cuda()
    held = torch.zeros(B, dtype=torch.int64, device="cuda")
    counts = torch.tensor(lens, dtype=torch.int64).cuda()
    slots, _, taken = rse.seq_cache_assign(cache, counts, held, table, free, len(first))
    rse.seq_cache_write(cache, slots, k[first], v[first], pos[first])
    held, free = counts.clone(), free[int(taken):].contiguous()
    one = torch.ones(B, dtype=torch.int64, device="cuda")
    for _ in range(more):
        _, _, taken = rse.seq_cache_assign(cache, one, held, table, free, B)
        at = off[:-1] + held
        out = rse.seq_attention_step(attn, cache, q[at], k[at], v[at], pos[at], bias, table, held)
        # both round the same sums in another order
        assert torch.allclose(out.float(), want[at].float(), rtol=2**-6, atol=2**-8)
        held += 1
        free = free[int(taken):].contiguous()
    assert cache.status() == 0 and attn.status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal", [True, False])
def test_many_boundaries_on_both_sides(causal, dtype):
    """Every power of two and its negative, distances over all of int32: tiles
    that span dozens of buckets, with at most one boundary to a cell."""
    bounds = sorted([2**m for m in range(31)] + [-(2**m) for m in range(31)])
    for seed in (0, 1):
        c = Case([70, 190], 4, 4 if seed else 1, 32, dtype, bounds=bounds, causal=causal, seed=seed)
        g = torch.Generator().manual_seed(seed)
        span = torch.randint(-2**31, 2**31, c.pos.shape, generator=g)
        c.pos = (span >> torch.randint(0, 31, c.pos.shape, generator=g)).to(torch.int32).cuda()
        c.pos[::11] = 2**31 - 1
        c.pos[5::11] = -2**31
        c.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 4), (5, 5), (8, 2)])
def test_many_short_sequences(H, Hk, dtype):
    """More sequences than blocks: each block goes through several, of lengths
    from none to the limit, some of them hidden."""
    lens = [(37 * i) % 129 for i in range(700)]
    c = Case(lens, H, Hk, 32, dtype, missing=0.1)
    got = c.run()
    sample = [0, 1, 3, 7, 100, 350, 501, 698, 699]
    off = np.concatenate([[0], np.cumsum(lens)])
    keep = np.concatenate([np.arange(off[b], off[b + 1]) for b in sample])
    part = [lens[b] for b in sample]
    q, k, v, do = (_np(t)[keep] for t in (c.q, c.k, c.v, c.dout))
    ref = oseq.attention(q, k, v, c.pos.cpu().numpy()[keep], _np(c.bias), np.concatenate([[0], np.cumsum(part)]),
                         c.bounds, True, c.attn.scale, c.key_off.cpu().numpy()[keep], do, KIND[dtype])
    at = torch.from_numpy(keep).cuda()
    for name in ("out", "dq", "dk", "dv"):
        _check(got[name][at], ref[name], name)
    # the bias gradient against the sum over sequence pieces, each run alone
    total, slack = np.zeros_like(ref["dbias"][0]), np.zeros_like(ref["dbias"][0])
    for a in range(0, 700, 100):
        ids = np.arange(off[a], off[a + 100])
        r = oseq.attention(*(_np(t)[ids] for t in (c.q, c.k, c.v)), c.pos.cpu().numpy()[ids], _np(c.bias),
                           off[a:a + 101] - off[a], c.bounds, True, c.attn.scale, c.key_off.cpu().numpy()[ids],
                           _np(c.dout)[ids], KIND[dtype])["dbias"]
        total, slack = total + r[0], slack + r[1]
    _check(got["dbias"], (total, slack), "dbias")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_negative_and_zero_scale(dtype):
    for scale in (-0.3, 0.0):
        c = Case([50, 200], 4, 1, 64, dtype)
        c.attn = c.rse.SeqAttention(4, 1, 64, dtype, c.bounds, scale=scale)
        c.check()


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min, -1e30])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bias_that_hides(low, dtype):
    """Buckets whose bias is -infinity, the lowest value or -1e30 hide their
    pairs: each event sees the two before it, the first ones nothing."""
    c = Case([1, 40, 150], 2, 1, 32, dtype, bounds=(0, 1, 3), times=False)
    c.bias[:, 1] = low                           # the event itself
    c.bias[:, 3] = low                           # three events back and further
    c.check()
    got = c.run()
    first = torch.tensor([0, 1, 41]).cuda()
    assert all(torch.all(torch.isfinite(got[n])) for n in ("out", "dq", "dk", "dv", "dbias"))
    assert torch.all(got["out"][first] == 0) and torch.all(got["dq"][first] == 0)
    assert torch.all(got["dbias"][:, [1, 3]] == 0)


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min])
@pytest.mark.parametrize("lens", [[0, 40, 5], [0, 2000]])
def test_step_bias_that_hides(lens, low):
    """The event itself and what is long past hidden: nothing is left of a user
    without history, and whole parts of a long one."""
    c = Serving(lens, 4, 1, 64, BF16, bounds=(0, 1, 300))
    c.bias[:, 1] = low
    c.bias[:, 3] = low
    out = c.check()
    assert torch.all(out[0] == 0) and torch.all(torch.isfinite(out))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(4, 1), (3, 3)])
def test_most_buckets_and_wide_rows(H, Hk, D, dtype):
    """127 boundaries with the widest rows: the largest use of LDS."""
    Case([20, 170], H, Hk, D, dtype, bounds=tuple(range(1, 128)), times=False).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hk", [(64, 1), (33, 1), (8, 8)])
def test_step_most_buckets_and_heads(H, Hk, dtype):
    Serving([150, 700, 0], H, Hk, 128, dtype, bounds=tuple(range(1, 128))).check()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (3, 1), (4, 1), (5, 1)])
@pytest.mark.parametrize("lens", [[0, 1, -1, 7, 8, 15, 16, 17], [31, 32, 33, 63, 64, 65, 127], [1500, 3, 300]])
def test_step_fp32_few_heads(lens, H, Hk, D):
    """Up to 4 heads a key/value head have a kernel of their own, 5 the other."""
    Serving(lens, H, Hk, D, F32, page=8).check()


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_step_fp32_scale(scale):
    s = Serving([90, 0, 700], 4, 2, 64, F32)
    s.attn = s.rse.SeqAttention(4, 2, 64, F32, s.bounds, scale=scale)
    s.check()


@pytest.mark.parametrize("D", [32, 64, 128])
def test_step_fp32_many_parts_and_hidden(D):
    s = Serving([9000, 40, 0], 2, 1, D, F32, page=64, bounds=(0, 1, 3000))
    s.bias[:, 1] = float("-inf")
    s.bias[:, 3] = torch.finfo(torch.float32).min
    out = s.check()
    assert torch.all(out[2] == 0)


# ------------------------------------------------------------ bf16 accuracy --
KIND["pairs"] = "bf16 pairs"


@pytest.mark.parametrize("lens", [[1, 2, 40, 128], [300, 5, 33]])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (4, 1)])
def test_bf16_forward_rounds_once(H, Hk, D, lens):
    """bf16 outputs are fp32 arithmetic rounded once: the probabilities enter
    their product as pairs of bf16 values."""
    for causal in (True, False):
        c = Case(lens, H, Hk, D, BF16, causal=causal, missing=0.2)
        c.dtype = "pairs"
        ref = c.oracle(False)["out"]
        _check(c.forward(), ref, "out")
        _check(c.run()["out"], ref, "out before a backward")


@pytest.mark.parametrize("lens", [[1, 2, 40, 128], [300, 5, 33]])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (4, 1)])
def test_bf16_gradients_round_once(H, Hk, D, lens):
    for causal in (True, False):
        c = Case(lens, H, Hk, D, BF16, causal=causal, missing=0.2)
        c.dtype = "pairs"
        got, ref = c.run(), c.oracle()
        for name in got:
            _check(got[name], ref[name], name)


@pytest.mark.parametrize("lens", [[0, 1, 31, 65], [1500, -1, 300]])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (16, 1)])
def test_bf16_step_rounds_once(H, Hk, D, lens):
    s = Serving(lens, H, Hk, D, BF16)
    s.dtype = "pairs"
    s.check()


# --------------------------------------------------- values that are not finite --
@pytest.mark.parametrize("dtype,H,Hk", [(F32, 4, 2), (F32, 5, 1), (BF16, 4, 2), (BF16, 5, 1)])
@pytest.mark.parametrize("lens", [[40, 0, 33], [1500, 3, 700]])
def test_step_keeps_what_is_not_finite(lens, dtype, H, Hk):
    """NaN in a query, a cached key or value or a bias, and scores that
    overflow, give NaN where the formula does, and nowhere else."""
    def fresh():
        return Serving(lens, H, Hk, 64, dtype, bounds=(1, 2, 4, 8, 16, 32, 64, 128))

    def check(s, want_nan, what):
        out = _np(s.run())
        ref, bound = s.oracle()
        assert np.array_equal(np.isnan(out), want_nan), what
        assert np.all(np.abs(out - ref)[~want_nan] <= bound[~want_nan]), what
        assert s.cache.status() == 0

    none = np.zeros((3, H, 64), bool)
    nan = float("nan")
    group = H // Hk
    s = fresh()                                  # one head's query
    want = none.copy()
    ref = s.oracle()
    s.q[0, 1, 5] = nan
    want[0, 1] = True
    s.oracle = lambda: ref
    check(s, want, "q")
    for at in (2, lens[0] - 1, lens[0]):         # a key: cached early, cached last, new
        s = fresh()
        ref = s.oracle()
        s.oracle = lambda: ref  # noqa: B023
        if at < lens[0]:
            s.cache.k[s.table[0, at // s.page], at % s.page, Hk - 1, 7] = nan
        else:
            s.nk[0, Hk - 1, 7] = nan
        want = none.copy()
        want[0, (Hk - 1) * group:] = True
        check(s, want, f"k {at}")
    s = fresh()                                  # one element of a value
    ref = s.oracle()
    s.oracle = lambda: ref
    s.cache.v[s.table[2, 0], 3, 0, 11] = nan
    want = none.copy()
    want[2, :group, 11] = True
    check(s, want, "v")
    s = fresh()                                  # the bias of the event itself
    ref = s.oracle()
    s.oracle = lambda: ref
    s.bias[H - 1, 0] = nan
    want = none.copy()
    want[:, H - 1] = True
    check(s, want, "bias")
    s = fresh()                                  # a score that overflows: infinity less infinity
    ref = s.oracle()
    s.oracle = lambda: ref
    s.q[2, 0, 0] = 3e38
    s.cache.k[s.table[2, 0], 1, 0, 0] = 3e38
    out = _np(s.run())
    assert np.all(np.isnan(out[2, 0])) and np.all(np.isfinite(out[:2]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens,most", [([20, 90, 7], 90), ([150, 290, 33], 290)])
@pytest.mark.parametrize("H,Hk", [(2, 1), (4, 1)])
def test_training_keeps_what_is_not_finite(H, Hk, lens, most, dtype):
    """A row with a score that is NaN or +infinity has no log-sum: its output,
    its gradient and what it sends to the keys that it sees are NaN; the other
    sequences keep their values."""
    a, b = lens[0], lens[0] + lens[1]
    for what in ("q", "k", "overflow"):
        c = Case(lens, H, Hk, 64, dtype)
        ref = c.oracle()
        i = a + 60                               # of the second sequence
        if what == "q":
            c.q[i, 0, 3] = float("nan")
        elif what == "k":
            c.k[i, 0, 3] = float("nan")
        else:
            c.q[i, 0], c.k[i, 0] = 3e38, 3e38
        got = c.run(max_len=most)
        rows = [i] if what != "k" else list(range(i, b))
        heads = [0] if what != "k" else list(range(H // Hk))
        for name in ("out", "dq"):
            assert torch.all(torch.isnan(got[name][rows][:, heads])), (what, name)
        last = rows[-1] + 1                      # the keys that the last such row sees
        for name in ("dk", "dv"):
            assert torch.all(torch.isnan(got[name][a:last, 0])), (what, name)
        keep = torch.ones(sum(lens), dtype=torch.bool)
        keep[a:b] = False
        for name in ("out", "dq", "dk", "dv"):
            _check(got[name][keep.cuda()], tuple(x[keep.numpy()] for x in ref[name]), name)
        if what == "q":                          # later keys are not seen by it
            assert torch.all(torch.isfinite(got["dv"][last:b]))


def test_assign_reports_bad_pages():
    """Held pages and free pages outside the pool: their events get slot -1,
    the table keeps its entry and the status says so; the others are assigned."""
    import recommender_sparse_embedding_amd as rse

    P, n_pages = 8, 10
    cuda = lambda x, dt: torch.tensor(x, dtype=dt).cuda()  # noqa: E731
    cache = rse.SeqCache.empty(n_pages, P, 1, 32)
    for bad in (-1, -7, n_pages, 2**31 - 1):
        for where in ("held", "free"):
            # users: 3 cached in page 4, 2 new; 5 cached in `held`, 6 new; none cached, 9 new
            held, free = [4, 2], [5, 6, 7]
            if where == "held":
                held[1] = bad
            else:
                free[1] = bad
            table = cuda([[held[0], -3, -3], [held[1], -3, -3], [-3, -3, -3]], torch.int32)
            slots, off, taken = rse.seq_cache_assign(cache, cuda([2, 6, 9], torch.int64), cuda([3, 5, 0], torch.int64),
                                                     table, cuda(free, torch.int32), 17)
            assert cache.status() == -9, (bad, where)
            cache.clear_status()
            second = held[1] * P + np.arange(5, 8) if where == "held" else 2 * P + np.arange(5, 8)
            third = 6 * P + np.arange(8) if where == "held" else np.full(8, -1)
            if where == "held":
                second = np.full(3, -1)
            want = [4 * P + 3, 4 * P + 4, *second, *(5 * P + np.arange(3)), *third, 7 * P]
            assert slots.tolist() == want, (bad, where)
            assert off.tolist() == [0, 2, 8, 17] and taken.item() == 3
            first = -3 if where == "free" else 6
            assert table.tolist() == [[4, -3, -3], [held[1], 5, -3], [first, 7, -3]], (bad, where)
            # what is written is what has a slot
            cache.k.zero_()
            x = torch.ones((17, 1, 32), dtype=torch.bfloat16, device="cuda")
            rse.seq_cache_write(cache, slots, x, x, torch.zeros(17, dtype=torch.int32, device="cuda"))
            assert int((cache.k.view(-1, 32)[:, 0] != 0).sum()) == sum(w >= 0 for w in want) and cache.status() == 0


def test_outputs_that_overlap_are_refused():
    """Outputs whose heads or events share memory are refused before anything
    is written; other layouts, and inputs that overlap themselves, are not."""
    c = Case([2, 1], 3, 1, 32, BF16)
    rse, where = c.rse, (c.attn, c.q, c.k, c.v, c.pos, c.bias, c.off)
    want, saved = rse.seq_attention_fwd(*where, for_backward=True)
    grads = rse.seq_attention_bwd(*where, saved, c.dout)
    new = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    flat = new(4096)
    bad = [new(1, 3, 32).expand(3, 3, 32), new(3, 1, 32).expand(3, 3, 32), flat.as_strided((3, 3, 32), (96, 16, 1)),
           flat.as_strided((3, 3, 32), (24, 1024, 1)), flat.as_strided((3, 3, 32), (32, 64, 1)),
           flat.as_strided((3, 3, 32), (64, 40, 1))]
    for t in bad:
        with pytest.raises(rse.RseError) as e:
            rse.seq_attention_fwd(*where, out=t)
        assert e.value.code == -1
        with pytest.raises(rse.RseError):
            rse.seq_attention_bwd(*where, saved, c.dout, grads=(t, new(3, 1, 32), new(3, 1, 32)))
    with pytest.raises(rse.RseError):
        rse.seq_attention_bwd(*where, saved, c.dout, grads=(new(3, 3, 32), new(1, 1, 32).expand(3, 1, 32), new(3, 1, 32)))
    assert torch.all(flat == 0)
    one = Case([1], 3, 1, 32, BF16)
    for shape in ((8, 16, 1), (4096, 24, 1), (0, 0, 1)):
        with pytest.raises(rse.RseError):
            one.forward(out=flat.as_strided((1, 3, 32), shape))
    assert torch.equal(one.forward(out=flat.as_strided((1, 3, 32), (8, 40, 1))), one.forward())
    flat.zero_()
    good = [new(3, 3, 32).transpose(0, 1), flat.as_strided((3, 3, 32), (32, 96, 1)),
            flat.as_strided((3, 3, 32), (256, 64, 1)), flat.as_strided((3, 3, 32), (160, 64, 1))]
    for t in good:
        assert torch.equal(rse.seq_attention_fwd(*where, out=t), want)
        got = rse.seq_attention_bwd(*where, saved, c.dout, grads=(t, new(3, 1, 32), new(3, 1, 32)))
        assert torch.equal(got[0], grads[0])
    # one key and one gradient given for all events or heads
    k, do = c.k[:1].expand(3, 1, 32), c.dout[:, :1].expand(3, 3, 32)
    out, saved = rse.seq_attention_fwd(c.attn, c.q, k, *where[3:], for_backward=True)
    got = rse.seq_attention_bwd(c.attn, c.q, k, *where[3:], saved, do)
    full = rse.seq_attention_bwd(c.attn, c.q, k.contiguous(), *where[3:], saved, do.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(got, full))

    s = Serving([5, 9], 4, 2, 64, BF16)
    with pytest.raises(rse.RseError):
        s.run(out=new(1, 4, 64).expand(2, 4, 64))
    assert torch.equal(s.run(out=new(4, 2, 64).transpose(0, 1)), s.run())


def test_steps_keep_nothing_per_length():
    """A server whose longest history grows by one a step: the layer holds no
    more afterwards than before."""
    s = Serving([20, 40], 4, 2, 64, BF16)
    s.run()
    held = lambda: sum(len(x) for x in vars(s.attn).values() if isinstance(x, (dict, list, set, tuple)))  # noqa: E731
    before = held()
    want = s.run()
    for most in range(41, 141):
        assert torch.equal(s.run(max_len=most), want)
    assert held() <= before


# ------------------------------------------------- batches past one grid's size --
def _grid_fit(head_blocks, waves):
    """Sequences that a grid of the short form takes side by side (short_grid);
    with more, each block goes on to further ones."""
    return -(-(8192 // waves) // head_blocks)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hk,batch", [(1, 1, 8207), (8, 8, 1301), (32, 32, 555), (64, 16, 301)])
def test_blocks_that_go_on_to_further_sequences(H, Hk, batch, dtype):
    """More sequences than the short form's blocks, by an uneven amount, of
    lengths from none to the limit: the grouped (64 on 16 heads) and the plain
    kernels of dk and dv, and those of the forward and dq."""
    wh = 4 if H > 1 else 1
    grouped = H // Hk % 4 == 0 and H > 1
    dkv_blocks = Hk if grouped else -(-Hk // wh)
    for fit in (_grid_fit(-(-H // wh), wh), _grid_fit(dkv_blocks, wh)):
        assert fit < batch and batch % fit       # each block takes one or more, not all as many
    lens = [(37 * i) % 129 if i % 9 == 4 else (5 * i) % 8 for i in range(batch)]
    Case(lens, H, Hk, 32, dtype, causal=H != 8, missing=0.1).check()


def _searched(lens, tile, most):
    """Whether tiles of that many events are numbered by the offsets and found
    by a search (tile_grid)."""
    n, batch = sum(lens), len(lens)
    return -(-min(most, n) // tile) > 4 * (n // tile + batch) // batch


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (4, 1), (8, 2)])
def test_tiles_found_by_a_search(H, Hk, D, dtype):
    """One long sequence among many short ones and empty ones, first, between
    and last; and a usual batch without max_len."""
    short = [(7 * i) % 10 for i in range(40)]
    for at, causal in ((0, True), (17, False), (40, True)):
        lens = short[:at] + [600] + short[at:]
        assert all(_searched(lens, tile, 600) for tile in (32, 64, 128))
        Case(lens, H, Hk, D, dtype, causal=causal, missing=0.1).check()
    lens = [0, 0] + [11 + (13 * i) % 20 for i in range(58)]
    c = Case(lens, H, Hk, D, dtype, causal=H != 3)
    assert all(_searched(lens, tile, sum(lens)) for tile in (32, 64, 128))
    ref, got = c.oracle(), c.run(max_len=None)
    for name in got:
        _check(got[name], ref[name], name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,H,Hk", [(32, 4, 4), (64, 2, 1), (128, 4, 1)])
def test_malformed_offsets_of_searched_tiles(D, H, Hk, dtype):
    """Reported, forward and backward, and the call after them is right."""
    lens = [(7 * i) % 10 for i in range(40)] + [600]
    c = Case(lens, H, Hk, D, dtype)
    good, n = c.off.clone(), sum(lens)
    dout = c.dout
    for at, x in ((1, n + 5), (20, -3), (40, 0), (0, 2), (41, n - 1), (30, 2**62), (7, -2**62)):
        c.off = good.clone()
        c.off[at] = x
        where = (c.attn, c.q, c.k, c.v, c.pos, c.bias, c.off)
        out, saved = c.rse.seq_attention_fwd(*where, max_len=600, for_backward=True)
        assert c.attn.status() == -9, (at, x)
        c.attn.clear_status()
        c.rse.seq_attention_bwd(*where, saved, dout, max_len=600)
        assert c.attn.status() == -9, (at, x)
        c.attn.clear_status()
    c.off = good
    c.forward(max_len=599)                       # the long one is longer
    assert c.attn.status() == -9
    c.attn.clear_status()
    c.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_malformed_offsets_of_many_short_sequences(dtype):
    lens = [(5 * i) % 8 for i in range(1301)]
    c = Case(lens, 8, 8, 32, dtype)
    good, n = c.off.clone(), sum(lens)
    for at, x in ((1, n + 5), (1200, -3), (1300, 0), (0, 2), (1301, n - 1), (700, 2**62)):
        c.off = good.clone()
        c.off[at] = x
        where = (c.attn, c.q, c.k, c.v, c.pos, c.bias, c.off)
        out, saved = c.rse.seq_attention_fwd(*where, max_len=100, for_backward=True)
        assert c.attn.status() == -9, (at, x)
        c.attn.clear_status()
        c.rse.seq_attention_bwd(*where, saved, c.dout, max_len=100)
        assert c.attn.status() == -9, (at, x)
        c.attn.clear_status()
    c.off = good
    c.check()


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min, -1e30])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bias_that_hides_from_both_key_heads(low, dtype):
    """A hidden bucket in the middle, and for one head also that of the event
    itself: rows with nothing left are 0 in out and dq and send nothing."""
    c = Case([1, 40, 90], 2, 2, 32, dtype, bounds=(1, 2, 4), times=False)
    c.bias[:, 2] = low
    c.bias[0, 0] = low
    got = c.check()
    first = torch.tensor([0, 1, 41]).cuda()      # of head 0: the event itself hidden
    assert torch.all(got["out"][first, 0] == 0) and torch.all(got["dq"][first, 0] == 0)
    assert torch.equal(got["out"][first, 1], c.v[first, 1])      # of head 1: only itself
    assert torch.all(got["dbias"][:, 2] == 0) and got["dbias"][0, 0] == 0


@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (4, 4)])
def test_many_small_probabilities_count(H, Hk):
    """One key of probability almost 1, then 4095 of 2^-25 of it: added one by
    one to a running sum of 1 in fp32 each would be lost.  Summed by tiles of
    32 the sum errs by at most 2^-24 for each of 128 tiles and of some 20 steps
    within and after them; a row's out is what the small ones bring (exact in
    fp32, the bias being -25 in base 2), over it."""
    n, D = 4096, 32
    c = Case([n], H, Hk, D, F32, causal=False, bounds=(10**5,))
    c.pos = torch.arange(n, dtype=torch.int32).cuda()
    c.pos[0] = -10**6                            # far from every other event: bucket 1
    low, log2e = np.float32(-25 * math.log(2.0)), np.float32(1.4426950408889634)
    while low * log2e < -25:
        low = np.nextafter(low, np.float32(0))
    while low * log2e > -25:
        low = np.nextafter(low, np.float32(-30))
    assert low * log2e == -25
    c.bias[:, 0], c.bias[:, 1] = float(low), 0.0
    c.q.zero_()
    c.v.fill_(1.0)
    c.v[0] = 0.0
    small = (n - 1) * math.exp(float(low))
    want = small / (1 + small)
    got = _np(c.run()["out"])[1:]
    u = 2.0**-24
    # the bias in base 2 is off by 4 u of 25 or less, its power by as much
    bound = want * (128 + 20 + 100) * u
    assert np.all(np.abs(got - want) <= bound), np.abs(got / want - 1).max()
