"""Launch shapes of the event-history calls that their sizes choose: each test names the rule that it meets."""
import numpy as np
import pytest
import torch

import dlrm_embedding_interaction_amd as dl
import history_oracle as ho
from test_history import ALL, Pair, check_encode, gen, randn, starts

pytestmark = pytest.mark.gpu


def strided(t, extra):
    """The rows of t inside wider ones, off by `extra` elements: no row is 16-byte aligned."""
    wide = torch.zeros((t.shape[0], t.shape[1] * t.shape[2] + 2 * extra), dtype=t.dtype, device="cuda")
    view = wide[:, extra:extra + t.shape[1] * t.shape[2]].unflatten(1, tuple(t.shape[1:]))
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("window,sinks", [(1600, 7), (ALL, 0)])
def test_encode_eight_waves_with_rows_of_their_own(dtype, padded, window, sinks):
    """Heads of 128 in groups of four, 24 tiles or more in the window, 256 blocks or more: 64 rows of four heads in a
    block of eight waves.  Four of the sixteen heads are compared."""
    lens, heads, kv, dim = [2000, 2100, 600], 16, 4, 128
    n = sum(lens)
    q, k, v = (randn((n, h, dim), s, dtype) for s, h in ((1, heads), (2, kv), (3, kv)))
    pad = (torch.rand(n, generator=gen(4)) < 0.2).to(torch.uint8) if padded else None
    if padded:
        pad[2000:2070] = 1                  # rows that see nothing
    got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), window=window, sinks=sinks,
                               padding=None if pad is None else pad.cuda())
    some = [0, 5, 10, 15]
    check_encode(q[:, some], k, v, lens, window, sinks, got[:, some], padding=pad)
    if padded:
        assert torch.all(got[2000:2070] == 0)
    # element by element: the same result
    again = dl.history_attention(strided(q, 3), strided(k, 3), strided(v, 3), starts(lens).cuda(), window=window,
                                 sinks=sinks, padding=None if pad is None else pad.cuda())
    assert torch.equal(again, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 1)])
def test_encode_shared_keys_of_any_alignment(dtype, dim, heads, kv):
    """Few long histories, whose waves share a row's keys, with rows that are read element by element, and an output
    that is written so."""
    lens = [900, 1100]
    n = sum(lens)
    q, k, v = (randn((n, h, dim), s, dtype) for s, h in ((5, heads), (6, kv), (7, kv)))
    pad = (torch.rand(n, generator=gen(8)) < 0.3).to(torch.uint8)
    wide = torch.full((n, heads * dim + 5), -7.0, dtype=dtype, device="cuda")
    out = wide[:, 2:2 + heads * dim].unflatten(1, (heads, dim))
    for p in (None, pad):
        dl.history_attention(strided(q, 1), strided(k, 1), strided(v, 1), starts(lens).cuda(), window=700, sinks=9,
                             padding=None if p is None else p.cuda(), out=out)
        check_encode(q, k, v, lens, 700, 9, out, padding=p)
        assert torch.all(wide[:, :2] == -7) and torch.all(wide[:, 2 + heads * dim:] == -7)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("histories,tiles", [(3, 33), (3, 40), (3, 48), (3, 49), (90, 32), (90, 33)])
def test_lookup_around_its_longest_blocks(dtype, histories, tiles):
    """Blocks of eight waves take histories of up to 48 tiles of 64 events, blocks of fewer (90 histories of four kv
    heads) up to 32; longer ones are cut into runs."""
    kv = 2 if histories < 10 else 4
    lens = [64 * tiles - 5] + [(i * 37) % 300 for i in range(histories - 1)]
    page = 32
    p = Pair(sum(-(-n // page) for n in lens), histories, 2 * tiles, kv, 64, page, dtype)
    p.append(list(range(histories)), lens)
    p.lookup(list(range(histories)), 2 * kv)
    p.lookup(list(range(histories)), kv, 3, window=64 * tiles - 70, sinks=5)


@pytest.mark.parametrize("n_pages", [32767, 32768, 32769])
def test_free_list_where_one_block_no_longer_writes_it(n_pages):
    """Pools of up to 32768 pages are listed and planned by one block, larger ones by many."""
    c = dl.HistoryCache(n_pages, 300, 200, 1, 32, 16)
    lens = [(i * 613) % 3200 for i in range(200)]
    k = torch.zeros((sum(lens), 1, 32), dtype=torch.bfloat16, device="cuda")
    c.append(k, k, starts(lens).cuda())
    need = sum(-(-x // 16) for x in lens)
    assert c.n_refused == 0 and c.n_free == n_pages - need
    c.free(torch.arange(0, 200, 3, dtype=torch.int32, device="cuda"))

    def check():
        want = torch.nonzero(c.refs.cpu() == 0).flatten().flip(0).to(torch.int32)
        assert c.n_free == want.numel()
        assert torch.equal(c.free_pages[:want.numel()].cpu(), want)
    check()
    table = c.table.cpu()
    c.compact()
    check()
    used = n_pages - c.n_free
    assert int(c.refs[:used].min()) == 1 and int(c.refs[used:].sum()) == 0
    held = c.table.cpu()
    assert torch.equal(held >= 0, table >= 0)
    assert torch.equal(held[held >= 0].sort()[0], torch.arange(used, dtype=torch.int32))


def test_trimmed_histories_in_a_pool_of_many_blocks():
    """Trimming, which gives back pages in the middle of histories, where many blocks write the list."""
    n_pages, lens = 40000, [(i * 97) % 900 for i in range(64)]
    c = dl.HistoryCache(n_pages, 64, 60, 1, 32, 16)
    o = ho.Cache(n_pages, 64, 60, 1, 32, 16)
    k = randn((sum(lens), 1, 32), 9, torch.bfloat16)
    c.append(k.cuda(), k.cuda(), starts(lens).cuda())
    o.append(list(range(64)), lens, k.double().numpy(), k.double().numpy())
    slots = torch.arange(64, dtype=torch.int32, device="cuda")
    for window, sinks in ((500, 40), (100, 20), (1, 0)):
        c.trim(slots, window=window, sinks=sinks)
        o.trim(range(64), window, sinks)
        torch.cuda.synchronize()
        assert c.refs.tolist() == o.refs
        assert c.free_pages[:c.n_free].tolist() == o.free[::-1]
        assert [[p for p in row if p >= 0] for row in c.table.tolist()] == \
            [[p for p in row if p is not None] for row in o.lists]
    assert np.sum([len(r) for r in o.lists]) > 0


def test_append_refused_for_want_of_pages_takes_none():
    """One history is refused for want of pages, the next needs none and is served: the list stays as it was."""
    c = dl.HistoryCache(4, 3, 8, 1, 32, 16)
    k = randn((82, 1, 32), 10, torch.bfloat16).cuda()
    c.append(k[:1], k[:1], torch.zeros(1, dtype=torch.int64, device="cuda"))
    c.append(k[1:], k[1:], starts([66, 15]).cuda(), slots=torch.tensor([1, 0], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert c.lens.tolist() == [16, 0, 0] and c.refs.tolist() == [1, 0, 0, 0]
    assert c.n_refused == 1 and c.n_free == 3 and c.free_pages[:3].tolist() == [3, 2, 1]
