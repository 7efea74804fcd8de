"""Workloads of the sequence operators: attention over behaviour sequences
with a learned relative bias by buckets of distance (forward, and a training
step with every gradient), its single-event form over a paged history, and
the page tables and slot maps of that history.

Every case is a dict of plain values; ``prepare`` draws its inputs from the
seed, ``run`` makes one pass (in elementary torch operations, or with
``own`` through the library), ``exact`` is the definition in float64 and
``work`` the bytes and operations that the pass cannot do without.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --
def _attn(name, op, batch, longest, heads, kv, dim, dtype, *, causal=True, buckets=32, times=True, missing=False,
          lengths="uniform"):
    return {"name": name, "op": op, "batch": batch, "longest": longest, "heads": heads, "kv": kv, "dim": dim,
            "dtype": dtype, "causal": causal, "buckets": buckets, "times": times, "missing": missing,
            "lengths": lengths}


def _step(name, batch, longest, heads, kv, dim, dtype, *, page=32, buckets=32, lengths="uniform"):
    return {"name": name, "op": "step", "batch": batch, "longest": longest, "heads": heads, "kv": kv, "dim": dim,
            "dtype": dtype, "page": page, "buckets": buckets, "times": True, "lengths": lengths}


def _fill(name, batch, longest, kv, dim, dtype, *, page=32):
    return {"name": name, "op": "fill", "batch": batch, "longest": longest, "kv": kv, "dim": dim, "dtype": dtype,
            "page": page, "lengths": "uniform"}


def listed():
    return [
        # training on the behaviour-sequence workload: 8192 users' last 1..100
        # events, four fields of dim 64 as four heads, some events' rows missing
        _attn("train clicks", "train", 8192, 100, 4, 4, 64, "bf16", missing=True),
        # training on long histories, shared key heads, event times
        _attn("train long", "train", 12, 2048, 8, 2, 64, "bf16", buckets=64),
        # the same layer on fp32 rows as the pooled lookup gives them, sessions
        # of medium length, both directions (masked-event training)
        _attn("train fp32 both ways", "train", 512, 203, 4, 2, 32, "f32", causal=False, times=False, missing=True),
        # a debugging batch: three short sequences
        _attn("train tiny", "train", 3, 17, 2, 1, 128, "bf16", buckets=16),
        # scoring whole histories (no gradient): a large batch of long ones
        _attn("forward histories", "fwd", 16, 4096, 8, 2, 64, "bf16", buckets=64),
        # scoring a serving batch of recent sessions
        _attn("forward sessions", "fwd", 96, 333, 4, 4, 128, "bf16", times=False, missing=True),
        # one user's next event after a short history
        _step("step one user", 1, 60, 4, 4, 64, "bf16"),
        # a serving batch in mid-session
        _step("step sessions", 256, 1000, 8, 2, 64, "bf16", page=16),
        # few users with very long histories, wide shared heads
        _step("step lifelong", 24, 32768, 16, 2, 128, "bf16", page=64, buckets=64, lengths="long"),
        # histories held in fp32
        _step("step fp32", 128, 2048, 4, 4, 64, "f32"),
        # a burst of new sessions moved into the cache
        _fill("fill sessions", 300, 90, 2, 64, "bf16", page=16),
        # many users' histories moved into the cache
        _fill("fill histories", 4096, 400, 2, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("train", "fwd", "step", "step", "train", "fill"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    dim = rng.choice((32, 64, 128))
    kv = rng.choice((1, 2, 4))
    if op == "fill":
        longest = _log(rng, 1, 2000)
        batch = _log(rng, 1, max(1, min(4096, 800_000 // longest)))
        return {"op": "fill", "batch": batch, "longest": longest, "kv": kv, "dim": dim, "dtype": dtype,
                "page": rng.choice((16, 32, 64, 128)), "lengths": "uniform"}
    heads = kv * rng.choice((1, 1, 2, 3, 4))
    case = {"op": op, "heads": heads, "kv": kv, "dim": dim, "dtype": dtype,
            "buckets": rng.choice((8, 31, 32, 64, 128)), "times": rng.random() < 0.7}
    if op == "step":
        longest = _log(rng, 1, 20000)
        batch = _log(rng, 1, max(1, min(512, 600_000 // (longest * kv))))
        return {**case, "batch": batch, "longest": longest, "page": rng.choice((16, 32, 64, 128)),
                "lengths": rng.choice(("uniform", "long"))}
    # a training sequence has two events at least: over a single one the
    # probabilities are constant and their gradients zero
    longest = _log(rng, 2 if op == "train" else 1, 2000)
    # pairs x heads x dim at most those of a tenth of the largest case
    room = (16 * 8 * 4096 * 4096 * 64) // 10 // (longest * longest * heads * dim)
    batch = _log(rng, 1, max(1, min(4000, 400_000 // longest, room)))
    return {**case, "batch": batch, "longest": longest, "causal": rng.random() < 0.7,
            "missing": rng.random() < 0.5, "lengths": "uniform"}


# ----------------------------------------------------------------- inputs --
def _boundaries(case):
    """buckets - 1 ascending distances, evenly spaced in their logarithm: from
    one event to the longest history, or from a second to a year."""
    n = case["buckets"] - 1
    top = 31_536_000 if case["times"] else 4 * case["longest"]
    got, last = [], 0
    for m in range(n):
        last = max(last + 1, int(round(top ** (m / max(1, n - 1)))))
        got.append(last)
    return got


def _host_lengths(case):
    """The batch's lengths, ascending in evenly spaced steps over 1..longest
    (or its upper half), every 17th sequence empty: the same for every seed."""
    lo = 1 if case["lengths"] == "uniform" else (case["longest"] + 1) // 2
    B, span = case["batch"], case["longest"] - lo
    n = [case["longest"] - (span * (B - 1 - i)) // max(1, B - 1) for i in range(B)]
    n[1:-1:17] = [0] * len(n[1:-1:17])
    return n


def _lengths(case, g):
    """The lengths in an order of the seed's, and that order."""
    order = torch.randperm(case["batch"], generator=g, device="cuda")
    return torch.tensor(_host_lengths(case), device="cuda")[order], order


def _host_cached(case):
    """(length, events of it cached already) of every sequence of a fill."""
    return [(n, (n * (i % 97)) // 97 if i % 2 == 0 else 0) for i, n in enumerate(_host_lengths(case))]


def _times(case, n, g):
    """Ascending event times of one row of n events: seconds with gaps from
    within a session to days, or plain indexes."""
    if not case.get("times", True):
        return torch.arange(n[1], device="cuda", dtype=torch.int32).expand(n).contiguous()
    gap = torch.exp(torch.randn(n, generator=g, device="cuda") * 2.0 + 4.0).clamp(1, 86_400.0)
    return gap.to(torch.int64).cumsum(1).clamp(max=2**31 - 1).to(torch.int32)


def _index(case, offsets):
    """Rows of the padded form: [batch, longest] event numbers, and which are real."""
    at = torch.arange(case["longest"], device="cuda")
    real = at[None, :] < (offsets[1:] - offsets[:-1])[:, None]
    return torch.where(real, offsets[:-1, None] + at[None, :], 0), real


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, Hk, D = DTYPES[case["dtype"]], case["batch"], case["kv"], case["dim"]
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    lens, order = _lengths(case, g)
    s = {"case": case, "lens": lens}
    if case["op"] in ("train", "fwd"):
        N, H = sum(_host_lengths(case)), case["heads"]
        offsets = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = lens.cumsum(0)
        # one projection gives q, k and v side by side: they are views of it
        qkv = normal(N, H + 2 * Hk, D)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        _, real = _index(case, offsets)
        s["pos"] = _times(case, (B, case["longest"]), g)[real].contiguous()
        s["offsets"] = offsets
        s["bias"] = torch.randn((H, case["buckets"]), generator=g, device="cuda")
        s["key_off"] = None
        if case["missing"]:      # row offsets of the lookup; -1 where no row was found
            off = torch.randint(0, 1 << 40, (N,), generator=g, device="cuda")
            s["key_off"] = torch.where(torch.rand(N, generator=g, device="cuda") < 0.05, -1, off)
        if case["op"] == "train":
            s["dout"] = normal(N, H, D)
    else:
        P, most = case["page"], case["longest"] // case["page"] + 1
        n_pages = B * most + 3
        table = torch.randperm(n_pages, generator=g, device="cuda")[:B * most].to(torch.int32).view(B, most)
        if case["op"] == "step":
            H = case["heads"]
            s["lens"] = torch.where(lens == 0, -1, lens - 1)      # events cached; -1: the slot is idle
            s["table"] = table.contiguous()
            s["q"], s["k"], s["v"] = normal(B, H, D), normal(B, Hk, D), normal(B, Hk, D)
            s["k_pages"], s["v_pages"] = normal(n_pages, P, Hk, D), normal(n_pages, P, Hk, D)
            t = _times(case, (B, most * P), g)
            s["pos_pages"] = torch.zeros((n_pages, P), dtype=torch.int32, device="cuda")
            s["pos_pages"][table.reshape(-1).long()] = t.view(B * most, P)
            s["pos"] = t.gather(1, s["lens"].clamp(min=0)[:, None])[:, 0].contiguous()
            s["bias"] = torch.randn((H, case["buckets"]), generator=g, device="cuda")
        else:
            # half of the users have some history cached already
            had = torch.where(order % 2 == 0, (lens * (order % 97)) // 97, 0)
            s["lens"], s["counts"] = had, lens - had
            held = torch.arange(most, device="cuda")[None, :] < ((had + P - 1) // P)[:, None]
            s["table"] = torch.where(held, table, -1).contiguous()
            s["free"] = table[~held].contiguous()
            N = sum(n - had for n, had in _host_cached(case))
            s["k"], s["v"] = normal(N, Hk, D), normal(N, Hk, D)
            s["pos"] = torch.randint(0, 1 << 30, (N,), generator=g, device="cuda").to(torch.int32)
            s["k_pages"], s["v_pages"] = normal(n_pages, P, Hk, D), normal(n_pages, P, Hk, D)
            s["pos_pages"] = torch.zeros((n_pages, P), dtype=torch.int32, device="cuda")
    if own and "k_pages" in s:   # the cache's and the layer's handles, made once by a program
        import recommender_sparse_embedding_amd as rse
        s["cache"] = rse.SeqCache(s["k_pages"], s["v_pages"], s["pos_pages"])
    if "buckets" in case:
        s["boundaries"] = torch.tensor(_boundaries(case), dtype=torch.int64, device="cuda")
        if own:
            import recommender_sparse_embedding_amd as rse
            s["attn"] = rse.SeqAttention(case["heads"], Hk, D, rse.BF16 if dt == torch.bfloat16 else rse.F32,
                                         _boundaries(case), causal=case.get("causal", True))
    return s


# -------------------------------------------------------------- plain form --
def _padded(x, index, real):
    """[N, H, D] in its type -> [batch, H, longest, D] in 32 bits, 0 past each end."""
    return (x.float()[index] * real[:, :, None, None]).transpose(1, 2).contiguous()


def _plain_attention(s, train):
    c = s["case"]
    H, Hk, D = c["heads"], c["kv"], c["dim"]
    index, real = _index(c, s["offsets"])
    group = H // Hk
    q = _padded(s["q"], index, real)
    k = _padded(s["k"], index, real).repeat_interleave(group, 1)
    v = _padded(s["v"], index, real).repeat_interleave(group, 1)
    at = s["pos"][index].long()
    bucket = torch.bucketize(at[:, :, None] - at[:, None, :], s["boundaries"], right=True)     # [B, L, L]
    keep = real[:, None, :] & real[:, :, None]
    if c["causal"]:
        keep = keep & torch.ones((c["longest"],) * 2, dtype=torch.bool, device="cuda").tril()
    if s["key_off"] is not None:
        keep = keep & (s["key_off"][index] >= 0)[:, None, :]
    keep = keep[:, None]
    scale = 1.0 / math.sqrt(D)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * scale
    x = x + s["bias"][:, bucket].transpose(0, 1)
    x = x.masked_fill(~keep, -math.inf)
    top = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    del x
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, v)
    back = lambda y: y.transpose(1, 2)[real].to(s["q"].dtype)  # noqa: E731
    if not train:
        return back(out)
    do = _padded(s["dout"], index, real)
    dp = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds = p * (dp - (p * dp).sum(3, keepdim=True))
    del dp
    dq = torch.matmul(ds, k) * scale
    B, L = c["batch"], c["longest"]
    dk = (torch.matmul(ds.transpose(2, 3).contiguous(), q) * scale).view(B, Hk, group, L, D).sum(2)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do).view(B, Hk, group, L, D).sum(2)
    rows = torch.zeros((B, H, L, c["buckets"]), device="cuda")
    rows.scatter_add_(3, bucket[:, None].expand(B, H, L, L), ds)
    return {"out": back(out), "dq": back(dq), "dk": back(dk), "dv": back(dv), "dbias": rows.sum((0, 2))}


def _plain_step(s):
    c = s["case"]
    P, H, Hk, D, L = c["page"], c["heads"], c["kv"], c["dim"], c["longest"]
    lens, B = s["lens"], c["batch"]
    live = lens >= 0
    kp, vp, tp = s["k_pages"].view(-1, Hk, D), s["v_pages"].view(-1, Hk, D), s["pos_pages"].view(-1)
    table = s["table"].long()
    n = lens.clamp(min=0)
    slot = table.gather(1, (n // P)[:, None])[:, 0] * P + n % P
    kp[slot] = torch.where(live[:, None, None], s["k"], kp[slot])
    vp[slot] = torch.where(live[:, None, None], s["v"], vp[slot])
    tp[slot] = torch.where(live, s["pos"], tp[slot])
    at = torch.arange(L, device="cuda")
    keep = at[None, :] <= lens[:, None]
    slots = torch.where(keep, table[:, at // P] * P + at % P, 0)
    k = (kp[slots].float() * keep[:, :, None, None]).repeat_interleave(H // Hk, 2)              # [B, L, H, D]
    v = (vp[slots].float() * keep[:, :, None, None]).repeat_interleave(H // Hk, 2)
    bucket = torch.bucketize(s["pos"].long()[:, None] - tp[slots].long(), s["boundaries"], right=True)
    x = (k * s["q"].float()[:, None]).sum(3) / math.sqrt(D) + s["bias"].t()[bucket]
    x = x.masked_fill(~keep[:, :, None], -math.inf)
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(1)
    out = (p[:, :, :, None] * v).sum(1) / torch.where(total == 0, 1.0, total)[:, :, None]
    return {"out": out.to(s["q"].dtype), "k": s["k_pages"], "v": s["v_pages"], "pos": s["pos_pages"]}


def _plain_fill(s):
    c = s["case"]
    P, Hk, D, B = c["page"], c["kv"], c["dim"], c["batch"]
    had, count, N = s["lens"], s["counts"], s["k"].shape[0]
    offsets = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = count.cumsum(0)
    first, last = (had + P - 1) // P, (had + count + P - 1) // P
    taken = (last - first).cumsum(0)
    column = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    fresh = (column >= first[:, None]) & (column < last[:, None])
    which = (taken - (last - first))[:, None] + column - first[:, None]
    if s["free"].numel():
        s["table"].copy_(torch.where(fresh, s["free"][torch.where(fresh, which, 0)], s["table"]))
    event = torch.arange(N, device="cuda")
    user = torch.searchsorted(offsets, event, right=True) - 1
    at = had[user] + event - offsets[user]
    slots = s["table"][user, at // P].long() * P + at % P
    s["k_pages"].view(-1, Hk, D)[slots] = s["k"]
    s["v_pages"].view(-1, Hk, D)[slots] = s["v"]
    s["pos_pages"].view(-1)[slots] = s["pos"]
    return {"slots": slots, "offsets": offsets, "taken": taken[-1:], "table": s["table"], "k": s["k_pages"],
            "v": s["v_pages"], "pos": s["pos_pages"]}


# --------------------------------------------------------------------- run --
def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "step":
            return _plain_step(s)
        if c["op"] == "fill":
            return _plain_fill(s)
        return _plain_attention(s, c["op"] == "train")
    import recommender_sparse_embedding_amd as rse
    if c["op"] in ("step", "fill"):
        cache = s["cache"]
    if c["op"] == "step":
        out = rse.seq_attention_step(s["attn"], cache, s["q"], s["k"], s["v"], s["pos"], s["bias"], s["table"],
                                     s["lens"], max_len=c["longest"])
        return {"out": out, "k": cache.k, "v": cache.v, "pos": cache.pos}
    if c["op"] == "fill":
        slots, offsets, taken = rse.seq_cache_assign(cache, s["counts"], s["lens"], s["table"], s["free"],
                                                     s["k"].shape[0])
        rse.seq_cache_write(cache, slots, s["k"], s["v"], s["pos"])
        return {"slots": slots, "offsets": offsets, "taken": taken, "table": s["table"], "k": cache.k,
                "v": cache.v, "pos": cache.pos}
    where = (s["q"], s["k"], s["v"], s["pos"], s["bias"], s["offsets"])
    if c["op"] == "fwd":
        return rse.seq_attention_fwd(s["attn"], *where, key_off=s["key_off"], max_len=c["longest"])
    out, saved = rse.seq_attention_fwd(s["attn"], *where, key_off=s["key_off"], max_len=c["longest"],
                                       for_backward=True)
    dq, dk, dv, dbias = rse.seq_attention_bwd(s["attn"], *where, saved, s["dout"], key_off=s["key_off"],
                                              max_len=c["longest"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dbias": dbias}


# -------------------------------------------------------------------- work --
def work(case):
    B, Hk, D = case["batch"], case["kv"], case["dim"]
    e = 2 if case["dtype"] == "bf16" else 4
    lens = _host_lengths(case)
    N = sum(lens)
    if case["op"] == "fill":
        P = case["page"]
        new = sum(n - had for n, had in _host_cached(case))
        pages = sum(-(-n // P) - -(-had // P) for n, had in _host_cached(case))
        return {"bytes": 2 * new * (2 * Hk * D * e + 4) + 16 * new + 24 * B + 8 * pages, "flops": 0}
    H = case["heads"]
    if case["op"] == "step":
        live = sum(n > 0 for n in lens)
        return {"bytes": N * (2 * Hk * D * e + 4) + live * D * e * (2 * H + 2 * Hk)
                + sum(4 * -(-n // case["page"]) for n in lens) + 12 * B + 4 * H * case["buckets"],
                "flops": 4 * N * H * D}
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
    qs, ks = N * H * D * e, N * Hk * D * e
    small = 4 * N + 8 * B + (8 * N if case["missing"] else 0) + 4 * H * case["buckets"]
    if case["op"] == "fwd":
        return {"bytes": 2 * qs + 2 * ks + small, "flops": 4 * D * H * pairs}
    return {"bytes": 4 * qs + 4 * ks + small + 4 * H * case["buckets"], "flops": 14 * D * H * pairs}


# ------------------------------------------------------------------- exact --
def _exact_attention(s, train):
    """Sequence by sequence in float64."""
    c = s["case"]
    H, Hk, D = c["heads"], c["kv"], c["dim"]
    dev = "cuda"
    N = s["q"].shape[0]
    new = lambda h: torch.zeros((N, h, D), dtype=torch.float64, device=dev)  # noqa: E731
    out, dq, dk, dv = new(H), new(H), new(Hk), new(Hk)
    dbias = torch.zeros((H, c["buckets"]), dtype=torch.float64, device=dev)
    edges = s["boundaries"].to(torch.int64)
    offsets = s["offsets"].tolist()
    kv_of = torch.arange(H, device=dev) // (H // Hk)
    for a, b in zip(offsets[:-1], offsets[1:]):
        n = b - a
        if not n:
            continue
        heads = lambda y: y[a:b].double().permute(1, 0, 2).contiguous()  # noqa: E731
        q, k, v = heads(s["q"]), heads(s["k"])[kv_of], heads(s["v"])[kv_of]
        t = s["pos"][a:b].to(torch.int64)
        cell = torch.searchsorted(edges, (t.view(n, 1) - t.view(1, n)).reshape(-1), side="right").view(n, n)
        logit = torch.bmm(q, k.mT.contiguous()) / D**0.5 + torch.stack([row[cell] for row in s["bias"].double()])
        bad = torch.zeros((n, n), dtype=torch.bool, device=dev)
        if c["causal"]:
            bad |= torch.ones((n, n), dtype=torch.bool, device=dev).triu(1)
        if s["key_off"] is not None:
            bad |= (s["key_off"][a:b] < 0).view(1, n)
        logit[:, bad] = -math.inf
        w = torch.nan_to_num(torch.softmax(logit, dim=2), nan=0.0)
        out[a:b] = torch.bmm(w, v).permute(1, 0, 2)
        if not train:
            continue
        do = heads(s["dout"])
        dw = torch.bmm(do, v.mT.contiguous())
        dl = w * dw - w * (w * dw).sum(2, keepdim=True)
        dq[a:b] = (torch.bmm(dl, k) / D**0.5).permute(1, 0, 2)
        dk[a:b].index_add_(1, kv_of, (torch.bmm(dl.mT.contiguous(), q) / D**0.5).permute(1, 0, 2))
        dv[a:b].index_add_(1, kv_of, torch.bmm(w.mT.contiguous(), do).permute(1, 0, 2))
        flat = torch.arange(H, device=dev).view(H, 1) * c["buckets"] + cell.view(1, -1)
        dbias += torch.bincount(flat.reshape(-1), weights=dl.reshape(-1),
                                minlength=H * c["buckets"]).view(H, c["buckets"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dbias": dbias} if train else out


def _exact_step(s):
    c = s["case"]
    P, H, Hk, D = c["page"], c["heads"], c["kv"], c["dim"]
    kp, vp, tp = s["k_pages"].clone(), s["v_pages"].clone(), s["pos_pages"].clone()
    out = torch.zeros((c["batch"], H, D), dtype=torch.float64, device="cuda")
    edges = s["boundaries"].to(torch.int64)
    for b, n in enumerate(s["lens"].tolist()):
        if n < 0:
            continue
        pages = s["table"][b, :n // P + 1].long()
        kp[pages[-1], n % P], vp[pages[-1], n % P], tp[pages[-1], n % P] = s["k"][b], s["v"][b], s["pos"][b]
        k, v = kp[pages].view(-1, Hk, D)[:n + 1].double(), vp[pages].view(-1, Hk, D)[:n + 1].double()
        cell = torch.searchsorted(edges, s["pos"][b].long() - tp[pages].view(-1)[:n + 1].long(), side="right")
        q = s["q"][b].double().view(Hk, H // Hk, D)
        w = torch.bmm(q, k.permute(1, 2, 0).contiguous()).view(H, -1) / D**0.5 + s["bias"].double()[:, cell]
        w = torch.softmax(w, dim=1).view(Hk, H // Hk, -1)
        out[b] = torch.bmm(w, v.permute(1, 0, 2).contiguous()).view(H, D)
    return {"out": out, "k": kp.double(), "v": vp.double(), "pos": tp}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "fill":
        return None              # whole numbers and copies
    if case["op"] == "step":
        return _exact_step(s)
    return _exact_attention(s, case["op"] == "train")
