"""Lookups of groups where the shared tiles' own kernels run, on the GPU: odd numbers, masks, missing pages and ragged
groups, for 16 and 32 rows to a wave and blocks of one, two and four waves.

Calls of few tiles are looked up history by history, whatever the groups are, so every call here says first that it is
not one of those.  Bars as in test_beams; numbers that are none stand exactly where the 64-bit form has them.
"""
import numpy as np
import pytest
import torch

from test_beams import Beams
from test_history import ALL, U, bound, f64, randn

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
KV = 8
# head_dim, events to a page, histories of a group, heads per kv head: 16 rows to a wave; 32; blocks of two waves; of four
SHAPES = [(32, 16, 4, 4), (32, 64, 8, 4), (32, 32, 8, 8), (64, 32, 4, 4), (64, 64, 8, 4), (64, 16, 8, 8), (64, 64, 20, 8),
          (128, 64, 4, 4), (128, 16, 8, 4), (128, 32, 8, 8), (128, 16, 20, 8)]


def reaches_shared_tiles(cache, batch, rows, window, sinks):
    """The rule by which few tiles are looked up history by history."""
    span = -(-cache.table.shape[1] * cache.page_events // 64)
    tiles = span
    if window < span * 64 and sinks < span * 64:
        tiles = min(span, -(-window // 64) + 1 + -(-sinks // 64))
    return tiles > 5 and batch * tiles * cache.n_kv_heads * -(-rows // 16) > 24576


def check(p, batch, groups, q, window, sinks, some):
    """A lookup of the batch's histories against the 64-bit form at the rows `some`, and its odd numbers against those of
    the lookup of each history for itself."""
    queries, heads = q.shape[1:3]
    assert reaches_shared_tiles(p.gpu, len(batch), queries * (heads // p.kv), window, sinks)
    args = dict(window=window, sinks=sinks, slots=p.slots(batch))
    got = p.gpu.lookup_shared(q.cuda(), groups, **args)
    one = p.gpu.lookup(q.cuda(), **args)
    assert torch.equal(torch.isnan(got), torch.isnan(one))
    got = f64(got)[some]
    with np.errstate(invalid="ignore"):
        out, mag, big = p.cpu.lookup([batch[i] for i in some], f64(q)[some], window, sinks, p.dim ** -0.5)
    odd = np.isnan(out)
    assert np.array_equal(np.isnan(got), odd)
    n = max(p.cpu.lens) + 64
    tol = bound(np.nan_to_num(out), np.nan_to_num(mag), np.nan_to_num(big, posinf=0.0), p.dim, n, q.dtype,
                2.0 ** -15 if q.dtype != torch.float32 else U, 0.0)
    worst = float((np.abs(got - out)[~odd] / tol[~odd]).max(initial=0.0))
    print(f"window {window} sinks {sinks}: worst error / bar {worst:.3f}, {odd.mean():.2f} not numbers", flush=True)
    assert worst <= 1.0
    return odd


def users_of(dtype, dim, page, members, lens, edit=None, tails=(0,), room=1000):
    """One history for each length, forked into `members`, the i-th of them with tails[i] events of its own."""
    users = len(lens)
    p = Beams(users * (room // page + members * 8), users * members, room // page, KV, dim, page, dtype)
    firsts = [u * members for u in range(users)]
    p.append(firsts, lens, edit=edit)
    if members > 1:
        p.fork([f for f in firsts for _ in range(members - 1)], [f + 1 + i for f in firsts for i in range(members - 1)])
    every = list(range(users * members))
    p.append(every, [tails[i % members % len(tails)] for i in every])
    return p, every


def repeated(every):
    """The histories as often as a call with shared tiles of its own needs; each time with other queries."""
    return every * (4400 // (KV * len(every)) + 1)


def sample(batch, members):
    """Some rows of the batch, members of the first and the last group among them."""
    n = min(members, 7)
    return sorted(set(range(0, len(batch), 61)) | set(range(n)) | set(range(len(batch) - n, len(batch))))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,members,heads", SHAPES)
def test_keys_and_queries_that_are_no_numbers_reach_the_result(dtype, dim, page, members, heads):
    """Shared prefixes with a tile of NaN keys, or of nothing but NaN keys, behind which some histories have events of
    their own and others none; queries that are NaN or infinite.  No score of a run of tiles is then a number."""
    lens = [448, 448, 384]

    def edit(k, v):
        k[448 + 128:448 + 192] = float("nan")
        k[896:] = float("nan")
    p, every = users_of(dtype, dim, page, members, lens, edit, tails=(0, 70, 0, 3, 330))
    batch = repeated(every)
    q = randn((len(batch), 1, heads * KV, dim), 61, dtype)
    q[2::5, 0, 1] = float("nan")
    q[1::7, 0, -1] = float("nan")
    q[::6, 0, heads, :] = float("inf")
    q[3::4, 0, 2 * heads + 1, 5] = -float("inf")
    for window, sinks in ((ALL, 0), (300, 0), (390, 64), (320, 200)):
        odd = check(p, batch, members, q, window, sinks, sample(batch, members))
        assert 0.05 < odd.mean() < 0.95


WINDOWS = [(ALL, 0), (290, 0), (300, 70), (340, 1), (200, 181)]


def ragged(batch, members, itype):
    """Offsets of groups of no, one, many histories and one in between, which cut through families, with about `members`
    histories to a group."""
    sizes, at = (members, 0, 2 * members + 3, 1, members // 2 + 1, members), 0
    offs = []
    while at < batch:
        offs.append(at)
        at += sizes[len(offs) % len(sizes)]
    return torch.tensor(offs, dtype=itype, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,members,heads", SHAPES)
def test_windows_of_ragged_groups(dtype, dim, page, members, heads):
    """Groups that hold parts of families or several, each history with its own end of window and sinks; some have lost the
    pages that a window before had passed."""
    p, every = users_of(dtype, dim, page, members, [320, 448, 389], tails=(0, 3, 70, 1, 131, 0, 9))
    p.cpu.trim(every[1::5], 300, 70)
    p.gpu.trim(p.slots(every[1::5]), 300, 70)
    p.same()
    # a family's histories several times, then the next one's, so that groups hold few families
    batch = [s for u in range(3) for s in repeated(every[u * members:(u + 1) * members])[:4400 // (3 * KV) + 7]]
    q = randn((len(batch), 1, heads * KV, dim), 62, dtype)
    for i, (window, sinks) in enumerate(WINDOWS):
        offs = ragged(len(batch), members, (torch.int32, torch.int64)[i % 2])
        check(p, batch, offs, q, window, sinks, sample(batch, members))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,members,heads,queries", [
    (32, 64, 2, 1, 5), (64, 16, 2, 3, 7), (64, 32, 5, 2, 9), (128, 64, 1, 4, 3), (128, 32, 3, 1, 17), (128, 16, 7, 5, 4)])
def test_windows_of_several_queries(dtype, dim, page, members, heads, queries):
    """Rows of one history that share waves with those of its neighbours; NaN keys and values that some histories' windows
    have passed and others' have not."""
    def edit(k, v):
        k[60:75] = float("nan")
        v[330 + 100:330 + 230] = float("nan")
    p, every = users_of(dtype, dim, page, members, [330, 448, 389], edit, tails=(131, 0, 70, 31, 1))
    batch = repeated(every)
    q = randn((len(batch), queries, heads * KV, dim), 63, dtype)
    odd = [check(p, batch, members, q, window, sinks, sample(batch, members)).mean() for window, sinks in WINDOWS]
    assert 0.05 < np.mean(odd) < 0.95


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,page,members,heads", SHAPES)
def test_pages_that_are_not_there_in_shared_tiles(dtype, dim, page, members, heads):
    """Pages that all histories of a group have lost, by a trim before the fork, or whose entries are no pages: nothing of
    them is seen, in tiles that all rows see whole and in those where each has its own mask, also where a whole tile is gone
    and next to events that are no numbers."""
    lens = [448, 400, 640]

    def edit(k, v):
        v[448 + 20] = float("nan")
        k[848 + 300, :, 1] = float("nan")
    p = Beams(3 * (1000 // page + members * 8), 3 * members, 1000 // page, KV, dim, page, dtype)
    firsts = [u * members for u in range(3)]
    p.append(firsts, lens, edit=edit)
    p.cpu.trim([0], 250, 40)
    p.gpu.trim(p.slots([0]), 250, 40)
    p.fork([f for f in firsts for _ in range(members - 1)], [f + 1 + i for f in firsts for i in range(members - 1)])
    every = list(range(3 * members))
    p.append(every, [(0, 3, 70, 1, 131)[i % members % 5] for i in every])
    p.same()
    for first, gone in ((1, (0, 5)), (2, (-1, 2, 4, 5, 6, 7))):
        for x in gone:
            x = x if x >= 0 else lens[first] // page - 1
            for s in every[first * members:(first + 1) * members]:
                p.gpu.table[s, x] = (-1, 10 ** 6, -7)[x % 3]
                p.cpu.lists[s][x] = None
    batch = repeated(every)
    q = randn((len(batch), 1, heads * KV, dim), 64, dtype)
    for window, sinks in WINDOWS:
        check(p, batch, members, q, window, sinks, sample(batch, members))
