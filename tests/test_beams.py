"""The calls that continue event histories with beams, on the GPU, against their 64-bit forms (beams_oracle).

Bars, derived before the first run.
* Parents, items, page lists, counts and codes are compared exactly.
* Scores: exponentials off by at most 2^-28 of their value move the logarithm of their sum by 2^-28, and so do the
  factors that join the parts of a row; the score is rounded to fp32 once: 2^-24 |s| + 2^-27.
* Lookups: the bars of test_history; the shared part adds one more join to the corrections that they count for each 64
  keys of the history's length.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import beams_oracle as bo
import dlrm_embedding_interaction_amd as dl
from test_history import ALL, U, Pair, bound, f64, gen, randn, starts

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


# --- selection ----------------------------------------------------------------------


def check_select(logits, scores, keep, allowed=None, ended=None, end_item=-1, got=None):
    if got is None:
        got = dl.history_select(logits.cuda(), None if scores is None else scores.cuda(), keep,
                                None if allowed is None else allowed.cuda(), None if ended is None else ended.cuda(),
                                end_item)
    s, p, i = (t.cpu().numpy() for t in got)
    want_s, want_p, want_i = bo.select(f64(logits), None if scores is None else f64(scores), keep,
                                       None if allowed is None else allowed.numpy().astype(bool),
                                       None if ended is None else ended.numpy().astype(bool), end_item)
    assert np.array_equal(p, want_p), (p[:2], want_p[:2])
    assert np.array_equal(i, want_i), (i[:2], want_i[:2])
    some = np.isfinite(want_s)
    assert np.array_equal(s[~some], want_s[~some].astype(np.float32))
    err = np.abs(s[some] - want_s[some]) / (U * np.abs(want_s[some]) + 2.0 ** -27)
    worst = float(err.max()) if err.size else 0.0
    print(f"select {logits.dtype} {tuple(logits.shape)} keep {keep}: worst error / bar {worst:.3f}", flush=True)
    assert worst <= 1.0


def some_scores(groups, beams, seed):
    return -3 - 4 * torch.rand((groups, beams), generator=gen(seed))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("items", [1, 2, 63, 64, 65, 511, 512, 513, 1025, 5003, 20011])
@pytest.mark.parametrize("beams,keep", [(1, 1), (3, 5), (8, 8), (5, 64)])
def test_select(dtype, items, beams, keep):
    logits = randn((3, beams, items), 1, dtype, 3.0)
    check_select(logits, some_scores(3, beams, 2), keep)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("groups,beams,items,keep", [(2, 128, 700, 128), (3, 1, 70001, 100), (1, 64, 3001, 65),
                                                     (200, 2, 300, 2), (1, 1, 262147, 128), (2, 33, 130, 127)])
def test_select_shapes(dtype, groups, beams, items, keep):
    logits = randn((groups, beams, items), 3, dtype, 2.0)
    check_select(logits, None if beams == 1 else some_scores(groups, beams, 4), keep)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("items", [40, 5003, 40000])
def test_select_ties(dtype, items):
    """Equal scores: the lowest beam, then the lowest item.  Constant rows, few values, equal beams, zeros of both
    signs."""
    few = torch.randint(-2, 3, (2, 4, items), generator=gen(5)).to(dtype)
    check_select(few, torch.zeros(2, 4), 100)
    check_select(torch.full((2, 3, items), 1.5, dtype=dtype), None, 17)
    zeros = torch.zeros((1, 2, items), dtype=dtype)
    zeros[:, :, ::3] *= -1.0
    check_select(zeros, None, 64)
    row = randn((1, 1, items), 6, dtype, 2.0)
    check_select(row.expand(2, 5, items).contiguous(), torch.full((2, 5), -1.25), 33)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_sorted_rows(dtype):
    """Rising and falling rows: every item, or none behind the first, is one of the best so far."""
    up = torch.linspace(-30, 8, 9000).to(dtype)
    rows = torch.stack([up, up.flip(0), torch.cat([up[::2], up[::2].flip(0)])])[None]
    check_select(rows, torch.zeros(1, 3), 128)
    check_select(rows, torch.tensor([[0.0, -0.5, 3.0]]), 64)
    check_select(rows[:, :1], None, 3)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_values_at_the_ends_of_the_range(dtype):
    top = torch.finfo(dtype).max
    x = randn((8, 2, 600), 7, dtype, 2.0)
    x[0, 0, 5] = float("nan")
    x[0, 1, 599] = float("nan")
    x[1, 0, 7] = float("inf")
    x[2, 0] = -float("inf")
    x[2, 1, ::2] = -float("inf")
    x[3, 0] = -float("inf")
    x[3, 0, 77] = -top
    x[4, 0, 3] = top
    x[4, 1] = -top
    x[5, 0] = top
    x[5, 1, 9] = -top
    x[6] = -float("inf")
    s = torch.tensor([[0.0, 0.0]] * 7 + [[float("-inf"), float("nan")]])
    s[5, 1] = float("inf")
    check_select(x, s, 4)
    check_select(x, None, 128)
    big = torch.tensor([[-3.0e38, 3.0e38]])
    check_select(x[4:5], big, 5)


@pytest.mark.parametrize("dtype", TYPES)
def test_select_logits_far_from_zero_and_from_each_other(dtype):
    """Rows that rise, fall and jump by thousands, around 0 and around values at which exponents lose their fractions."""
    ramp = torch.linspace(-3000.0, 3000.0, 9001)
    jumps = torch.cat([ramp[::7], 20 * ramp[::5], ramp[::11] - 2900, torch.full((4000,), -50000.0)])[:9001]
    jumps = torch.cat([jumps, torch.full((9001 - len(jumps),), -1000.0)])
    rows = torch.stack([ramp, ramp.flip(0), ramp[torch.randperm(9001, generator=gen(23))], jumps, jumps.flip(0)])[None]
    s = torch.tensor([[0.0, -1.5, -0.75, -2.0, 1.0]])
    check_select(rows.to(dtype), s, 64)
    if dtype != torch.float16:                     # up to 65504
        check_select((rows + 2.0 ** 21).to(dtype), s, 9)
        check_select((rows - 2.0 ** 21).to(dtype), s, 9)
        check_select((rows * 2.0 ** 90).to(dtype), s, 9)
    check_select((rows * 2.0 ** -20).to(dtype), s, 100)


@pytest.mark.parametrize("beams,items,keep", [(1, 3000, 4), (1, 600001, 3), (24, 66000, 24), (100, 20000, 128)])
def test_select_many_parts(beams, items, keep):
    """Rows cut into 2, 256, 32 and 8 parts."""
    check_select(randn((1, beams, items), 24, torch.bfloat16, 2.0), some_scores(1, beams, 25), keep)


@pytest.mark.parametrize("items", [300, 5003])
def test_select_equal_scores_of_all_beams(items):
    """More equal candidates than the join holds at once."""
    same = torch.full((2, 128, items), 0.25)
    check_select(same, torch.zeros(2, 128), 128)
    ended = torch.zeros((2, 128), dtype=torch.bool)
    ended[:, ::3] = True
    check_select(same, torch.zeros(2, 128), 100, ended=ended)


def test_beams_refusals():
    x = torch.zeros((2, 3, 10), device="cuda")
    s = torch.zeros((2, 3), device="cuda")
    for args in ((x[0], ), (x, s[:1]), (x.transpose(1, 2), ), (x[:, :, ::2], ), (x, s, -1), (x, s, 2 ** 32 + 1),
                 (x, s, 3, s[0] > 0), (x, s, 3, None, s[0] > 0), (x, s, 3, None, None, 2 ** 31)):
        with pytest.raises(ValueError):
            dl.history_select(*args)
    for args in ((x.double(), ), (x, s.double()), (x, s, 3, x), (x, s, 3, None, s), (x.cpu(), )):
        with pytest.raises(TypeError):
            dl.history_select(*args)
    for args in ((x, s, 0), (x, s, 129), (x, s, 2 ** 31 - 1), (x[:, :0], s[:, :0], 1), (x[:, :, :0], s), (x[:0], s[:0]),
                 (x[:, :1].expand(2, 3, 10), s), (x[:1, :1].expand(2, 3, 10), s)):
        with pytest.raises((RuntimeError, ValueError)):
            dl.history_select(*args)
    h = dl.HistoryCache(20, 6, 4, 1, 32, 16)
    p = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    for parents, slots in ((p[0], None), (p, p[:1]), (p.cpu(), None)):
        with pytest.raises((ValueError, TypeError)):
            h.reorder(parents, slots)
    for parents in (p[:, :0], p[:0], torch.zeros((3, 3), dtype=torch.int32, device="cuda")):
        with pytest.raises(RuntimeError):
            h.reorder(parents)
    with pytest.raises(RuntimeError):
        h.reorder(torch.zeros((1, 129), dtype=torch.int32, device="cuda"),
                  torch.zeros((1, 129), dtype=torch.int32, device="cuda"))
    q = torch.zeros((6, 2, 32), device="cuda")
    for groups in (0, -1, 4, p, torch.zeros((2, 4), dtype=torch.int64, device="cuda")[:, 0]):
        with pytest.raises((ValueError, TypeError)):
            h.lookup_shared(q, groups)
    with pytest.raises(RuntimeError):
        h.lookup_shared(q, p[0, :0])
    assert h.n_free == 20 and h.n_refused == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("items", [3, 1003, 9001])
def test_select_allowed_and_ended(dtype, items):
    x = randn((4, 6, items), 8, dtype, 2.0)
    s = some_scores(4, 6, 9)
    one = torch.rand(items, generator=gen(10)) < 0.3
    each = torch.rand((4, 6, items), generator=gen(11)) < 0.4
    each[0, 0] = False
    each[1] = False
    x[each.logical_not()] = torch.where(torch.rand(int((~each).sum()), generator=gen(12)) < 0.5, float("nan"),
                                        float("inf")).to(dtype)
    check_select(x, s, 10, allowed=each)
    check_select(x, s, 10, allowed=each.to(torch.uint8) * 3)
    y = randn((4, 6, items), 13, dtype, 2.0)
    y[:, :, ~one] = float("nan")
    check_select(y, s, 6, allowed=one)
    ended = torch.rand((4, 6), generator=gen(14)) < 0.5
    ended[3] = True
    s[3, 2] = -float("inf")
    y[ended] = float("nan")                       # not read
    check_select(y, s, 6, allowed=one, ended=ended, end_item=items + 5)
    check_select(y, s, 64, allowed=one, ended=ended)
    s[:] = -2.0
    check_select(randn((4, 6, items), 15, dtype), s, 6, ended=ended, end_item=0)


def test_select_nothing_is_read_outside_the_rows():
    """Rows of a wider tensor whose other columns are NaN, at every alignment; masks of such rows."""
    for dtype in TYPES:
        for items, extra in ((700, 1), (513, 3), (64, 2), (1000, 8)):
            wide = torch.full((2, 3, items + 2 * extra), float("nan"), dtype=dtype)
            x = randn((2, 3, items), 16, dtype, 2.0)
            wide[:, :, extra:extra + items] = x
            may = torch.ones((2, 3, items + 2 * extra), dtype=torch.bool)
            may[:, :, extra:extra + items] = torch.rand((2, 3, items), generator=gen(17)) < 0.5
            view, mview = wide.cuda()[:, :, extra:extra + items], may.cuda()[:, :, extra:extra + items]
            s = some_scores(2, 3, 18)
            check_select(x, s, 5, got=dl.history_select(view, s.cuda(), 5))
            check_select(x, s, 5, allowed=may[:, :, extra:extra + items],
                         got=dl.history_select(view, s.cuda(), 5, allowed=mview))


def test_select_rows_beyond_32_bits():
    """Rows whose elements lie past 2^32."""
    items, ld = 1000, 1500000001
    flat = torch.empty(3 * ld + items, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(flat, (2, 2, items), (2 * ld, ld, 1))
    x = randn((2, 2, items), 19, torch.bfloat16, 2.0)
    view.copy_(x)
    s = some_scores(2, 2, 20)
    check_select(x, s, 6, got=dl.history_select(view, s.cuda(), 6))


def test_select_rows_do_not_depend_on_each_other():
    """A group's result is the same alone, with other groups beside it, and beside rows that hold NaN."""
    x = randn((6, 4, 3001), 21, torch.float16, 2.0).cuda()
    s = some_scores(6, 4, 22).cuda()
    want = dl.history_select(x, s, 7)
    x[3] = float("nan")
    got = dl.history_select(x, s, 7)
    keep = [0, 1, 2, 4, 5]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(want, got))
    assert torch.all(got[1][3] == -1) and torch.all(got[0][3] == -float("inf"))
    again = dl.history_select(x, s, 7)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_select_on_streams_and_in_a_graph():
    shape = (5, 4, 9001)
    x = randn(shape, 23, torch.bfloat16, 2.0).cuda()
    s = some_scores(5, 4, 24).cuda()
    want = dl.history_select(x, s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            got += [dl.history_select(x, s) for _ in range(4)]
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        first = dl.history_select(x, s)
        second = dl.history_select(x, first[0])           # a step behind a step
    for i in range(4):
        x.copy_(randn(shape, 100 + i, torch.bfloat16, 2.0))
        s.copy_(some_scores(5, 4, 200 + i))
        a = dl.history_select(x, s)
        b = dl.history_select(x, a[0])
        g.replay()
        torch.cuda.synchronize()
        for o, w in ((first, a), (second, b)):
            assert all(torch.equal(t, u) for t, u in zip(o, w))


# --- the cache ----------------------------------------------------------------------


class Beams(Pair):
    """test_history's pair of caches, with the calls of this file."""

    def __init__(self, n_pages, n_slots, max_pages, kv, dim, page, dtype):
        super().__init__(n_pages, n_slots, max_pages, kv, dim, page, dtype)
        self.cpu = bo.Cache(n_pages, n_slots, max_pages, kv, dim, page)

    def fork(self, src, dst):
        self.cpu.fork(src, dst)
        self.gpu.fork(self.slots(src), self.slots(dst))

    def reorder(self, slots, parents):
        self.cpu.reorder(slots, parents)
        self.gpu.reorder(self.slots(parents), slots=self.slots(slots))

    def shared(self, slots, groups, heads, queries=1, window=ALL, sinks=0, dtype=None, scale=None, q=None):
        dtype = dtype or self.dtype
        self.seed += 2
        q = randn((len(slots), queries, heads, self.dim), self.seed, dtype) if q is None else q
        got = self.gpu.lookup_shared(q.cuda(), groups, window=window, sinks=sinks, scale=scale, slots=self.slots(slots))
        scale = self.dim ** -0.5 if scale is None else scale
        out, mag, big = self.cpu.lookup(slots, f64(q), window, sinks, scale)
        n = max([0] + [self.cpu.lens[s] for s in slots if 0 <= s < len(self.cpu.lens)])
        tol = bound(out, mag, big, self.dim, n + 64, dtype, 2.0 ** -15 if dtype != torch.float32 else U, 0.0)
        err = np.abs(f64(got) - out)
        worst = float((err / tol).max())
        print(f"shared {dtype} dim {self.dim} page {self.page} groups {groups}: worst error / bar {worst:.3f}", flush=True)
        assert worst <= 1.0
        return got


def roomy(page):
    """Pages of a table so wide that a lookup without a window reads shared tiles once however small it is: calls
    whose tables and windows hold little are looked up history by history."""
    return 400000 // page


def family(dtype, dim, page, kv=2, shared=150, beams=5, users=2, tails=(3, 1, 9, 2, 70), room=None):
    """`users` histories of `shared` events and more, each forked into `beams`, with events of their own behind."""
    most = -(-(shared + 40 * users + max(tails) + 8) // page)
    p = Beams(users * (most + beams * 8) + 40, users * beams + 3, room or roomy(page), kv, dim, page, dtype)
    firsts = [u * beams for u in range(users)]
    p.append(firsts, [shared + 40 * u for u in range(users)])
    p.fork([f for f in firsts for _ in range(beams - 1)], [f + 1 + i for f in firsts for i in range(beams - 1)])
    every = list(range(users * beams))
    p.append(every, [tails[i % len(tails)] for i in every])
    return p, every


@pytest.mark.parametrize("page", [16, 64])
def test_reorder(page):
    p, every = family(torch.bfloat16, 32, page, room=400 // page)
    groups = [every[:5], every[5:]]
    p.reorder(groups, [[1, 0, 2, 4, 3], [0, 0, 0, 3, 0]])          # a permutation; one beam takes over
    p.same()
    p.append(every, [1] * 10)
    p.same()
    p.lookup(every, 4)
    p.reorder(groups, [[4, 4, -1, 0, 2], [-1, -1, -1, -1, -1]])    # beams that die, a whole group
    p.same()
    p.append(every, [1, 0, 2, 1, 1, 3, 0, 17, 1, 1])
    p.same()
    p.reorder([[3, 77, 4, 3, 0, -5]], [[0, 1, 1, 2, 9, 0]])        # slots and parents that are none, a slot twice
    p.same()
    p.reorder([[1], [2], [8]], [[0], [-1], [-2]])
    p.same()
    p.gpu.compact()
    p.cpu.compact()
    p.same()


@pytest.mark.parametrize("beams", [1, 2, 63, 64, 65, 128])
def test_reorder_wide(beams):
    """Groups of up to 128, page lists of more than one block's columns."""
    p = Beams(900, beams + 2, 150, 1, 32, 16, torch.float16)
    p.append([0], [1700])
    p.fork([0] * (beams - 1) or [0], list(range(1, beams)) or [beams])
    every = list(range(beams))
    p.append(every, [1 + i % 19 for i in every])
    p.same()
    r = np.random.RandomState(beams)
    for _ in range(3):
        parents = [int(x) for x in r.randint(-1, beams, beams)]
        parents[0] = int(r.randint(0, beams))
        p.reorder([every], [parents])
        p.same()
        p.append(every, [1] * beams)
        p.same()


@pytest.mark.parametrize("n_pages", [9000, 40000])
def test_reorder_large_pools(n_pages):
    p = Beams(n_pages, 40, 30, 1, 32, 16, torch.bfloat16)
    every = list(range(40))
    p.append(every, [(i * 37) % 400 for i in every])
    r = np.random.RandomState(1)
    p.reorder([every[:20], every[20:]], r.randint(-1, 20, (2, 20)).tolist())
    p.same()


def test_reorder_without_slots():
    p, every = family(torch.bfloat16, 32, 16, room=25)
    parents = [[2, 2, 1, 0, 4], [1, 0, 0, 1, 1]]
    p.cpu.reorder([every[:5], every[5:]], parents)
    p.gpu.reorder(p.slots(parents))
    p.same()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("dim", [32, 64, 128])
def test_shared(dtype, page, dim):
    p, every = family(dtype, dim, page)
    for heads, queries in ((2, 1), (8, 1), (6, 5), (40, 1)):
        p.shared(every, 5, heads, queries)
    for window, sinks in ((1, 0), (5, 3), (64, 1), (100, 70), (130, 64), (150, 16), (ALL, 3)):
        p.shared(every, 5, 4, 1, window, sinks)


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_shared_ragged_groups(itype):
    """Offsets of groups: one history, none, many; groups that cut through families or hold several; an offset before
    the first group."""
    p, every = family(torch.bfloat16, 64, 16, shared=300, users=3)
    every = every + [16, 15]                       # empty histories
    for offs in ([0], [0, 5, 10], [0, 1, 1, 1, 7, 12, 17], [3, 3, 10], list(range(17)), [0, 17], [0, 14, 15, 16]):
        p.shared(every, torch.tensor(offs, dtype=itype, device="cuda"), 8)
        p.shared(every, torch.tensor(offs, dtype=itype, device="cuda"), 2, 3, 200, 70)
    other = [5, 0, 10, 1, 99, 6, 11, -1, 2]        # another order, slots that are none
    refused = p.gpu.n_refused
    got = p.shared(other, torch.tensor([0, 4], dtype=itype, device="cuda"), 4)
    assert p.gpu.n_refused == refused + 2
    assert torch.all(got[4] == 0) and torch.all(got[7] == 0)
    p.shared([2, 2, 2, 1], 4, 4)                   # a history several times


@pytest.mark.parametrize("dtype,dim,page,users,shared,beams,heads,kv,queries", [
    (torch.bfloat16, 64, 32, 1, 9000, 3, 4, 2, 1),         # one group cut into many runs
    (torch.float16, 128, 64, 1, 5000, 20, 8, 1, 2),        # many chunks of rows
    (torch.float32, 128, 16, 2, 1500, 4, 2, 1, 1),
    (torch.bfloat16, 32, 16, 70, 100, 2, 3, 3, 1),         # many groups, few tiles each
    (torch.float32, 64, 64, 9, 640, 7, 5, 1, 5)])
def test_shared_shapes(dtype, dim, page, users, shared, beams, heads, kv, queries):
    p, every = family(dtype, dim, page, kv, shared, beams, users, tails=(1, 2, 0, 5))
    p.shared(every, beams, heads, queries)
    p.shared(every, beams, heads, queries, window=shared // 2, sinks=7)


def test_shared_histories_without_anything_in_common():
    p = Beams(200, 6, roomy(32), 2, 64, 32, torch.bfloat16)
    p.append(list(range(6)), [300, 301, 64, 1, 0, 500])
    p.shared(list(range(6)), 6, 4)
    p.shared(list(range(6)), 2, 4, 1, 100, 4)
    p.fork([5], [4])
    p.cpu.truncate([4], [130])
    p.gpu.truncate(p.slots([4]), p.slots([130]))
    p.append([4], [400])                           # shares its first pages alone
    p.shared([5, 4], 2, 8)


def test_shared_trimmed_histories():
    p, every = family(torch.bfloat16, 64, 16, shared=400)
    p.cpu.trim(every[:3], 100, 20)
    p.gpu.trim(p.slots(every[:3]), 100, 20)
    p.same()
    p.shared(every, 5, 4, 1, 100, 20)
    p.shared(every, 5, 4, 1, 40, 0)
    p.shared(every, 5, 4)                          # some pages are there for one history and gone for the next


@pytest.mark.parametrize("room", [30, 60])
def test_shared_one_by_one(room):
    """Tables and windows of few events: history by history, whatever the groups."""
    p, every = family(torch.bfloat16, 64, 16, shared=200, room=room)
    for window, sinks in ((ALL, 0), (100, 20), (1, 0)):
        a = p.shared(every, 5, 4, 2, window, sinks)
        p.seed -= 2
        assert torch.equal(a, p.shared(every, torch.tensor([0, 3], device="cuda"), 4, 2, window, sinks))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,members,rows", [
    (32, 16, 4, 4), (32, 64, 8, 4), (32, 32, 8, 8), (32, 16, 40, 4), (64, 32, 4, 4), (64, 64, 8, 4), (64, 16, 8, 8),
    (64, 64, 40, 4), (128, 64, 4, 4), (128, 16, 8, 4), (128, 32, 8, 8), (128, 16, 40, 4), (128, 64, 40, 5)])
def test_shared_windows(dtype, dim, page, members, rows):
    """Windows and sinks that end in shared tiles, at another event for each row, and NaN events that some rows see and
    others do not.  Histories stand in the batch many times, each time with other queries."""
    kv, users = 8, 3
    p = Beams(users * (700 // page + members * 8), users * members, 1000 // page, kv, dim, page, dtype)
    firsts = [u * members for u in range(users)]

    def edit(k, v):
        v[180:190] = float("nan")                 # the first user's
    p.append(firsts, [300, 410, 333], edit=edit)
    p.fork([f for f in firsts for _ in range(members - 1)], [f + 1 + i for f in firsts for i in range(members - 1)])
    every = list(range(users * members))
    p.append(every, [(3, 1, 9, 2, 70, 0, 131)[i % 7] for i in every])
    batch = every * (4400 // (kv * len(every)) + 1)
    some = list(range(0, len(batch), 41)) + list(range(7))
    for window, sinks in ((290, 0), (260, 10), (300, 70), (340, 1), (200, 181)):
        p.seed += 2
        q = randn((len(batch), 1, rows * kv, dim), p.seed, dtype)
        got = p.gpu.lookup_shared(q.cuda(), members, window=window, sinks=sinks, slots=p.slots(batch))
        got = f64(got)[some]
        out, mag, big = p.cpu.lookup([batch[i] for i in some], f64(q)[some], window, sinks, dim ** -0.5)
        seen = np.isnan(out)
        assert np.array_equal(np.isnan(got), seen)
        tol = bound(np.nan_to_num(out), np.nan_to_num(mag), big, dim, 700, dtype,
                    2.0 ** -15 if dtype != torch.float32 else U, 0.0)
        worst = float((np.abs(got - out)[~seen] / tol[~seen]).max())
        print(f"window {window} sinks {sinks}: worst error / bar {worst:.3f}, {seen.mean():.2f} not numbers", flush=True)
        assert worst <= 1.0


@pytest.mark.parametrize("dtype", TYPES)
def test_shared_events_that_a_row_does_not_see_do_not_reach_it(dtype):
    """NaN events that some rows' windows have passed and others' have not."""
    p = Beams(200, 4, 30, 1, 32, 16, dtype)
    clean = Beams(200, 4, 30, 1, 32, 16, dtype)

    def edit(k, v):
        k[180:200] = float("nan")
        v[180:200] = float("nan")
    for c, e in ((p, edit), (clean, None)):
        c.append([0], [400], edit=e)
        c.fork([0, 0, 0], [1, 2, 3])
        c.append([0, 1, 2, 3], [1, 21, 40, 90])
    q = randn((4, 2, 2, 32), 30, dtype).cuda()
    for window in (201, 222, 240, 260, 300):       # rows see [len - window, len)
        args = dict(window=window, sinks=10, slots=p.slots([0, 1, 2, 3]))
        got, want = (c.gpu.lookup_shared(q, 4, **args) for c in (p, clean))
        for b, n in enumerate(p.cpu.lens):         # 401, 421, 440, and 400: 490 events pass 30 pages and are refused
            if n - window >= 200:
                assert torch.equal(got[b], want[b])
            else:
                assert torch.isnan(got[b]).all()


def test_shared_offsets_that_are_none():
    """Offsets that fall or lie outside the batch give some result, touch nothing else and hold nothing up; more groups
    than histories are all right."""
    p, every = family(torch.bfloat16, 64, 16, shared=300, users=3)
    q = randn((15, 2, 8, 64), 33, torch.bfloat16).cuda()
    want = p.shared(every, 5, 8, 2, q=q)
    for offs in ([0, 10, 5], [7, 3, 12, 1], [0, 10 ** 6, 2], [-5, -9, 4], [2 ** 31 - 1, -2 ** 31, 3], [9, 0] * 40,
                 [0, 2 ** 40 + 3, -2 ** 60]):
        room = torch.full((17, 2, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        itype = torch.int64 if max(offs) > 2 ** 31 else torch.int32
        p.gpu.lookup_shared(q, torch.tensor(offs, dtype=itype, device="cuda"), slots=p.slots(every), out=room[1:16])
        assert torch.all(room[0] == 7) and torch.all(room[16] == 7)
        assert torch.equal(p.gpu.lookup_shared(q, 5, slots=p.slots(every)), want)
    for offs in ([0] * 100, list(range(0, 300, 3)), [0, 10 ** 6, 10 ** 6]):
        p.shared(every, torch.tensor(offs, dtype=torch.int32, device="cuda"), 8)
    p.same()


def test_shared_bad_pages_are_not_seen():
    p, every = family(torch.bfloat16, 64, 16, shared=200, users=1)
    for x, page in ((2, -1), (5, 10 ** 6), (6, -7)):
        for s in every:
            p.gpu.table[s, x] = page
            p.cpu.lists[s][x] = None
    p.shared(every, 5, 4)
    p.shared(every, 5, 4, 1, 120, 40)


def test_shared_strided_queries_and_output():
    p, every = family(torch.float16, 64, 32)
    q = randn((10, 4, 64), 31, torch.float16)
    want = p.shared(every, 5, 4, q=q[:, None])[:, 0]
    wide = torch.zeros((10, 4 * 64 + 6), dtype=torch.float16, device="cuda")
    view = wide[:, 3:259].unflatten(1, (4, 64))
    view.copy_(q)
    out_wide = torch.full((10, 4 * 64 + 10), 7.0, dtype=torch.float16, device="cuda")
    out = out_wide[:, 5:261].unflatten(1, (4, 64))
    got = p.gpu.lookup_shared(view, 5, out=out, slots=p.slots(every))
    assert got is out and torch.equal(out, want)
    assert torch.all(out_wide[:, :5] == 7) and torch.all(out_wide[:, 261:] == 7)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0 ** 100])
def test_shared_scales(scale):
    p, every = family(torch.float32, 32, 16)
    if scale > 1:                                  # the largest product alone counts, wherever it lies
        for c in (p.gpu.k_scale, ):
            c.mul_(2.0 ** -100)
        p.cpu.k *= 2.0 ** -100
    p.shared(every, 5, 4, scale=scale)


def test_shared_is_repeatable_on_streams_and_in_a_graph():
    p, every = family(torch.bfloat16, 128, 64, shared=2000, users=3)
    offs = torch.tensor([0, 4, 5, 11], dtype=torch.int32, device="cuda")
    slots = p.slots(every)
    q = randn((15, 8, 128), 32, torch.bfloat16).cuda()
    want = p.gpu.lookup_shared(q, offs, slots=slots)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got += [p.gpu.lookup_shared(q, offs, slots=slots) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    for out, groups in zip(outs, (offs, 5)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.gpu.lookup_shared(q, groups, slots=slots, out=out)
        graphs.append(g)
    for i in range(4):
        q.copy_(randn(tuple(q.shape), 300 + i, torch.bfloat16))
        for out in outs:
            out.zero_()
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):          # two graphs of one cache at once
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], p.gpu.lookup_shared(q, offs, slots=slots))
        assert torch.equal(outs[1], p.gpu.lookup_shared(q, 5, slots=slots))


# --- together -----------------------------------------------------------------------


def test_beam_search_over_histories():
    """Steps of a beam search, eager and as a replayed graph, against the 64-bit forms fed with the same numbers: lookup
    of the shared histories, logits by a Linear layer, selection, reordering, and the taken items' events behind the
    histories."""
    users, beams, kv, heads, dim, items, page = 3, 4, 2, 4, 32, 700, 16
    pairs = [Beams(400, users * beams, roomy(page), kv, dim, page, torch.float32) for _ in range(2)]
    table = randn((items, heads * dim), 40, torch.float32, 0.3).cuda()
    keys, values = (randn((items, kv, dim), s, torch.float32).cuda() for s in (41, 42))
    zero = torch.zeros(items, device="cuda")
    every = list(range(users * beams))
    firsts = [u * beams for u in range(users)]
    for p in pairs:
        p.append(firsts, [100, 64, 213])
        p.fork([f for f in firsts for _ in range(beams - 1)], [f + 1 + i for f in firsts for i in range(beams - 1)])
    offsets = torch.arange(users * beams, dtype=torch.int64, device="cuda")
    start = torch.full((users, beams), -float("inf"))
    start[:, 0] = 0                               # the first step has one live beam

    def step(c, q, scores):
        h = c.lookup_shared(q, beams)
        logits = dl.linear_bias_act(h.flatten(1), table, zero, dl.ACT_NONE).unflatten(0, (users, beams))
        s, parents, took = dl.history_select(logits, scores, beams)
        c.reorder(parents)
        at = took.flatten().clamp(min=0).long()
        k, v = keys[at], values[at]
        c.append(k, v, offsets)
        scores.copy_(s)
        q.copy_(table[at].unflatten(1, (heads, dim)))
        return logits, parents, took, k, v

    state = [(randn((users * beams, heads, dim), 43, torch.float32).cuda(), start.cuda()) for _ in pairs]
    eager, replayed = pairs
    graph = None
    for t in range(6):
        q, scores = state[0]
        before, had = q.clone(), scores.cpu()
        logits, parents, took, k, v = step(eager.gpu, q, scores)
        want, mag, big = eager.cpu.lookup(every, f64(before)[:, None], ALL, 0, dim ** -0.5)
        lin = want[:, 0].reshape(users * beams, -1) @ f64(table).T
        assert np.abs(f64(logits).reshape(lin.shape) - lin).max() < 1e-3
        check_select(logits.cpu(), had, beams, got=(scores, parents, took))
        eager.cpu.reorder([every[f:f + beams] for f in firsts], parents.tolist())
        eager.cpu.append(every, [1] * len(every), f64(k), f64(v))
        eager.same()
        if t == 0:
            step(replayed.gpu, *state[1])
        elif t == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(replayed.gpu, *state[1])
        if t:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state[0][1], state[1][1]) and torch.equal(state[0][0], state[1][0])
        for n in ("table", "lens", "refs", "counters"):
            assert torch.equal(getattr(eager.gpu, n), getattr(replayed.gpu, n)), n


def test_the_example_suggests_what_a_walk_along_the_path_scores():
    """examples/history_ranking.py: a suggested path's score is the sum of its items' log-probabilities, each looked up
    behind the items before it, and the users' own histories stay as they are."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "history_ranking.py")
    spec = importlib.util.spec_from_file_location("history_ranking", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    got = module.main(users=5)
    r, slots, likely, paths = got["ranker"], got["slots"], got["likely"], got["paths"]
    free = r.cache.n_free
    assert torch.isfinite(likely).all() and torch.all(likely[:, :-1] >= likely[:, 1:])
    total = torch.zeros(15, dtype=torch.float64, device="cuda")
    spare = torch.arange(30, 45, dtype=torch.int32, device="cuda")
    r.cache.fork(slots.repeat_interleave(3), spare)
    item = got["click"].repeat_interleave(3)         # as many rows as there, so that their projections are the same
    for t in range(paths.shape[2]):
        seen = r.cache.lookup(next(r.project(item)), window=r.window, sinks=r.sinks, slots=spare)
        logits = dl.linear_bias_act(seen.flatten(1), r.items, r.b_items, dl.ACT_NONE).double()
        item = paths[:, :, t].flatten().long()
        total += (logits - torch.logsumexp(logits, 1, keepdim=True)).gather(1, item[:, None])[:, 0]
        r.click(item, spare)
    r.cache.free(spare)
    # logits: fp32 sums of 64 products below 8 in all, in another order for the lookup's part: 2 x 64 x 2^-24 x 8 each;
    # three of them and as many of their rows' largest
    assert float((total - likely.flatten().double()).abs().max()) < 6 * 2 * 64 * 2.0 ** -24 * 8
    assert r.cache.n_free == free and r.cache.n_refused == 0
    assert len({tuple(p) for p in paths[0].tolist()}) == 3
