"""Ranking with event histories: the history operators beside the library's bags, Linear layers and interaction.

A user's past items are rows of an item table.  They are encoded once with windowed attention, their keys and
values go to the 8-bit cache, and at serving time

* a new event of a user is one appended row,
* every candidate item of a request is a query of the user's cached history,
* the result joins the dense features and the candidate's own row in the pairwise-dot interaction, and the
  top MLP gives the click probability,
* "what if the user had clicked this one" is a fork of the history, an append to it, and a lookup; the fork is
  freed afterwards, and the pool compacted now and then.

Every step runs in the library's kernels.  Run: python examples/history_ranking.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import dlrm_embedding_interaction_amd as dl  # noqa: E402


class HistoryRanker:
    def __init__(self, items=5000, dim=64, heads=2, n_dense=13, window=200, sinks=4, n_slots=64, max_events=512,
                 page_events=16, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device=device) * scale

        self.dim, self.heads, self.window, self.sinks, self.device = dim, heads, window, sinks, device
        self.items = draw(items, dim, scale=dim ** -0.5)
        self.w_qkv, self.b_qkv = draw(3 * dim, dim, scale=dim ** -0.5 * 4), draw(3 * dim, scale=0.1)
        self.w_bot, self.b_bot = draw(dim, n_dense, scale=n_dense ** -0.5), draw(dim, scale=0.1)
        width = dim + 3                                   # x and the dots of [x, candidate, history]
        self.w_top = [draw(32, width, scale=width ** -0.5), draw(1, 32, scale=32 ** -0.5)]
        self.b_top = [draw(32, scale=0.1), draw(1, scale=0.1)]
        pages = -(-max_events // page_events)
        self.cache = dl.HistoryCache(n_pages=n_slots * pages // 2, n_slots=n_slots, max_pages=pages,
                                     n_kv_heads=heads, head_dim=dim // heads, page_events=page_events, device=device)

    def rows(self, idx):
        """(N, dim) rows of the item table, as bags of one index."""
        off = torch.arange(idx.numel(), device=self.device)
        return dl.embbag_sum([self.items], [idx.reshape(-1).contiguous()], [off])[:, 0]

    def project(self, idx):
        """q, k, v of items, three groups of columns of one Linear layer's output."""
        qkv = dl.linear_bias_act(self.rows(idx), self.w_qkv, self.b_qkv, dl.ACT_NONE)
        return (t.unflatten(1, (self.heads, -1)) for t in qkv.split(self.dim, 1))

    def encode(self, events, offsets, slots):
        """Histories of several users: their encoded events; keys and values go to the cache."""
        q, k, v = self.project(events)
        self.cache.append(k, v, offsets, slots=slots)
        return dl.history_attention(q, k, v, offsets, window=self.window, sinks=self.sinks)

    def click(self, item, slots):
        """One new event for each of several users."""
        _, k, v = self.project(item)
        self.cache.append(k, v, torch.arange(item.numel(), device=self.device), slots=slots)

    def attend(self, candidates, slots):
        """(B, C) candidates against the histories of B slots -> (B, C, dim)."""
        q = next(self.project(candidates))
        q = q.unflatten(0, tuple(candidates.shape))
        return self.cache.lookup(q, window=self.window, sinks=self.sinks, slots=slots).flatten(2)

    def score(self, dense, candidates, slots):
        """Click probabilities (B, C)."""
        B, C = candidates.shape
        hist = self.attend(candidates, slots).reshape(B * C, self.dim)
        x = dl.linear_bias_act(dense, self.w_bot, self.b_bot, dl.ACT_RELU).repeat_interleave(C, 0)
        emb = torch.stack([self.rows(candidates), hist], 1)
        z = dl.interact_lower_tri(x, emb, concat_dense=True)
        z = dl.linear_bias_act(z, self.w_top[0], self.b_top[0], dl.ACT_RELU)
        return dl.linear_bias_act(z, self.w_top[1], self.b_top[1], dl.ACT_SIGMOID).reshape(B, C)

    def what_if(self, dense, item, candidates, slots, spare):
        """Probabilities if each user had clicked `item` first; the users' own histories stay as they are."""
        self.cache.fork(slots, spare)
        self.click(item, spare)
        p = self.score(dense, candidates, spare)
        self.cache.free(spare)
        return p


def main(users=16, candidates=8, device="cuda"):
    r = HistoryRanker(device=device)
    g = torch.Generator(device=device)
    g.manual_seed(1)
    lens = [(37 * i) % 400 for i in range(users)]         # one user is new
    offsets = torch.tensor([sum(lens[:i]) for i in range(users)], device=device)
    events = torch.randint(0, r.items.shape[0], (sum(lens),), generator=g, device=device)
    slots = torch.arange(users, dtype=torch.int32, device=device)
    encoded = r.encode(events, offsets, slots)
    dense = torch.rand((users, 13), generator=g, device=device)
    cand = torch.randint(0, r.items.shape[0], (users, candidates), generator=g, device=device)
    before = r.score(dense, cand, slots)
    click = cand[:, 0].contiguous()
    tried = r.what_if(dense, click, cand, slots, slots + users)
    again = r.score(dense, cand, slots)
    r.click(click, slots)
    after = r.score(dense, cand, slots)
    r.cache.trim(slots, window=r.window, sinks=r.sinks)
    r.cache.compact()
    trimmed = r.score(dense, cand, slots)
    torch.cuda.synchronize()
    print(f"{users} users, {sum(lens)} events encoded, {r.cache.n_free} pages free, {r.cache.n_refused} refused")
    print(f"first user's probabilities: {[round(p, 4) for p in before[0].tolist()]}")
    print(f"after the click: largest change {float((after - before).abs().max()):.4f}")
    return dict(encoded=encoded, before=before, tried=tried, again=again, after=after, trimmed=trimmed, ranker=r,
                events=events, lens=lens, slots=slots, candidates=cand, click=click)


if __name__ == "__main__":
    main()
