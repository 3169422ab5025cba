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
    worst = float((np.abs(got - out)[~odd] / tol[~odd]).max())
    print(f"window {window} sinks {sinks}: worst error / bar {worst:.3f}, {odd.mean():.2f} not numbers", flush=True)
    assert worst <= 1.0
    return odd


def users_of(dtype, dim, page, members, lens, edit=None, tails=(0,), room=1000):
    """One history for each length, forked into `members`, the i-th of them with tails[i] events of its own."""
    users = len(lens)
    p = Beams(users * (room // page + members * 8), users * members, room // page, KV, dim, page, dtype)
    firsts = [u * members for u in range(users)]
    p.append(firsts, lens, edit=edit)
    p.fork([f for f in firsts for _ in range(members - 1)], [f + 1 + i for f in firsts for i in range(members - 1)])
    every = list(range(users * members))
    p.append(every, [tails[i % members % len(tails)] for i in every])
    return p, every


def repeated(every):
    """The histories as often as a call with shared tiles of its own needs; each time with other queries."""
    return every * (4400 // (KV * len(every)) + 1)


def sample(batch, members):
    """Some rows of the batch, each member of the first and the last group among them."""
    return sorted(set(range(0, len(batch), 41)) | set(range(members)) | set(range(len(batch) - members, len(batch))))


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
