"""A small sequence recommender on the library's calls: a user's events are
looked up one row each, projected, attended over within the user's sequence
(with a learned bias for the time between two events), and trained end to end:
the attention's gradients go through the projection into the sparse update of
the rows.  Then the trained layer serves: histories are moved into the paged
cache and every user's next event is answered by one step.

    python examples/behaviour_attention.py        (needs an MI355X GPU)
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import recommender_sparse_embedding_amd as rse  # noqa: E402

DIM, HEADS, KV_HEADS, HEAD_DIM, PAGE = 64, 4, 2, 32, 16
BOUNDARIES = [1, 10, 60, 600, 3600, 86400, 7 * 86400]        # seconds between two events


class Recommender:
    def __init__(self, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.idmap = rse.IdMap([1 << 14], max_load=0.8, device=device)
        self.blocks = rse.EmbeddingBlocks(DIM, rse.F32, rse.ADAGRAD, rows_per_chunk_log2=12, seed=seed,
                                          device=device).grow(4)
        self.optim = rse.Optim(rse.ADAGRAD, lr=0.05)
        self.attn = rse.SeqAttention(HEADS, KV_HEADS, HEAD_DIM, rse.BF16, BOUNDARIES)
        self.bias = torch.zeros((HEADS, self.attn.n_buckets), device=device)
        self.proj = torch.randn((DIM, (HEADS + 2 * KV_HEADS) * HEAD_DIM), generator=g, device=device) * DIM**-0.5
        self.steps = 0

    def lookup(self, ids: torch.Tensor, train: bool):
        """Row offsets and rows [n, DIM] of events, one bag per event; an id
        that has no row (never trained on) gives offset -1 and a zero row."""
        n = ids.numel()
        ends = torch.tensor([0, n], dtype=torch.int64, device=ids.device)
        bags = torch.arange(n + 1, dtype=torch.int64, device=ids.device)
        rows = torch.empty_like(ids)
        n_new = torch.zeros(1, dtype=torch.int64, device=ids.device)
        rse.idmap_find_or_insert(self.idmap, self.blocks, ids, ends, 1, 1, rows, n_new, insert_missing=train)
        x = torch.empty((n, 1, DIM), device=ids.device)
        rse.embedding_bag_fwd(self.blocks, rows, bags, 1, n, rse.SUM, x)
        return rows, bags, x.view(n, DIM)

    def project(self, x: torch.Tensor):
        """q, k, v as views of one joint projection."""
        qkv = (x @ self.proj).bfloat16().view(len(x), HEADS + 2 * KV_HEADS, HEAD_DIM)
        return qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]

    def train(self, ids, times, offsets, target, max_len) -> torch.Tensor:
        """One step towards `target` [n, HEADS, HEAD_DIM]; returns the loss."""
        rows, bags, x = self.lookup(ids, train=True)
        q, k, v = self.project(x)
        where = (self.attn, q, k, v, times, self.bias, offsets)
        out, saved = rse.seq_attention_fwd(*where, key_off=rows, max_len=max_len, for_backward=True)
        diff = out.float() - target
        n = len(ids)
        joint = torch.empty((n, HEADS + 2 * KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=ids.device)
        grads = (joint[:, :HEADS], joint[:, HEADS:HEADS + KV_HEADS], joint[:, HEADS + KV_HEADS:])
        *_, dbias = rse.seq_attention_bwd(*where, saved, diff.bfloat16(), key_off=rows, max_len=max_len, grads=grads)
        dqkv = joint.view(n, -1).float()
        dx = dqkv @ self.proj.t()
        self.steps += 1
        n_unique = torch.zeros(1, dtype=torch.int64, device=ids.device)
        rse.embedding_bag_bwd_update(self.blocks, rows, bags, 1, n, rse.SUM, dx.view(n, 1, DIM).contiguous(),
                                     self.optim, self.steps, n_unique)
        self.proj -= 1e-4 * (x.t() @ dqkv)
        self.bias -= 1e-4 * dbias
        return diff.square().mean()

    def cache(self, ids, times, counts, n_pages: int, max_pages: int):
        """Users' histories in a new cache: (cache, page table, lengths, free
        pages).  Training hides events whose id has no row; here they are not
        cached, which is the same to every later event (distances are by time)."""
        rows, _, x = self.lookup(ids, train=False)
        seen = rows >= 0
        user = torch.repeat_interleave(torch.arange(counts.numel(), device=ids.device), counts)
        lens = torch.bincount(user[seen], minlength=counts.numel())
        _, k, v = self.project(x[seen])
        cache = rse.SeqCache.empty(n_pages, PAGE, KV_HEADS, HEAD_DIM)
        table = torch.full((counts.numel(), max_pages), -1, dtype=torch.int32, device=ids.device)
        free = torch.arange(n_pages, dtype=torch.int32, device=ids.device)
        slots, _, taken = rse.seq_cache_assign(cache, lens, torch.zeros_like(lens), table, free, len(k))
        rse.seq_cache_write(cache, slots, k, v, times[seen].contiguous())
        return cache, table, lens, free[int(taken):].contiguous()

    def answer(self, cache, table, lens, free, ids, times):
        """One new event per user: its attention over the user's history.  An
        id without a row is neither answered (0) nor cached: a step's event
        always sees itself."""
        rows, _, x = self.lookup(ids, train=False)
        seen = rows >= 0
        one = seen.long()
        _, _, taken = rse.seq_cache_assign(cache, one, lens, table, free, int(one.sum()))
        q, k, v = self.project(x)
        at = torch.where(seen, lens, -1)
        out = rse.seq_attention_step(self.attn, cache, q, k, v, times, self.bias, table, at)
        lens += one
        return out, free[int(taken):].contiguous()


def main(users: int = 200, longest: int = 100, steps: int = 30, device="cuda"):
    g = torch.Generator(device=device).manual_seed(1)
    model = Recommender(device=device)
    counts = torch.randint(1, longest + 1, (users,), generator=g, device=device)
    offsets = torch.zeros(users + 1, dtype=torch.int64, device=device)
    offsets[1:] = counts.cumsum(0)
    n = int(offsets[-1])
    ids = (torch.rand(n, generator=g, device=device) ** 3 * 3000).long()        # a few ids make most of the events
    times = torch.randint(1, 900, (n,), generator=g, device=device).cumsum(0).to(torch.int32)
    target = torch.randn((n, HEADS, HEAD_DIM), generator=g, device=device) * 0.3
    losses = [model.train(ids, times, offsets, target, longest) for _ in range(steps)]
    losses = [round(float(x), 5) for x in losses]
    print("loss", losses[0], "->", losses[-1])

    # some events of ids that training never met, which have no row; then the
    # histories without their last event, and that event as the next one: the
    # answer is the forward's row of it
    last = offsets[1:] - 1
    ids = torch.where(torch.rand(n, generator=g, device=device) < 0.05, ids + 10**6, ids)
    rows, _, x = model.lookup(ids, train=False)
    want = rse.seq_attention_fwd(model.attn, *model.project(x), times, model.bias, offsets, key_off=rows,
                                 max_len=longest)[last]
    keep = torch.ones(n, dtype=torch.bool, device=device)
    keep[last] = False
    cache, table, lens, free = model.cache(ids[keep], times[keep].contiguous(), counts - 1, users * 8, 8)
    got, free = model.answer(cache, table, lens, free, ids[last], times[last].contiguous())
    found = rows[last] >= 0
    off = float((got[found].float() - want[found].float()).abs().max())
    print("one step against the whole forward: largest difference", off)
    assert model.attn.status() == 0 and cache.status() == 0
    return losses, off


if __name__ == "__main__":
    main()
