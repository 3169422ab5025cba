"""The event-history operators on the GPU against their 64-bit form (history_oracle).

Bars, derived before the first run.  u = 2^-24; h(t) = half a step of type t (bf16 2^-8, fp16 2^-11).
* Logit: products are exact or lose at most 3 u each (three bf16 parts of an fp32 factor), sums of dim terms
  lose dim u, the scale and the change to base 2 three more:  d = (dim + 8) u * max_j sum |scale q k|.
* Weight: exp(s - m) is off by 2 d from its logits and by 4 u from the exponential; the running maximum's
  corrections, one for each 64 keys, and the sums by (n / 64 + n) 4 u at most; the same again for the sum
  under the fraction; P's own rounding adds w.
* Output: (4 d + (8 + 2 n) 4 u + w) sum p |v| + h(out) |o|.
w is h(bf16) / h(fp16) where the weights are rounded to the 16-bit type of the values once (encoder), u for fp32
and 2^-15 for the lookup, which keeps them in two bf16 parts (fp32: three).  fp16 weights below 2^-14 are off by 2^-25
absolute: + 2^-25 sum |v| over the row's keys.
Codes, scales, page lists, counts and lengths are compared exactly.
"""
import numpy as np
import pytest
import torch

import dlrm_embedding_interaction_amd as dl
import history_oracle as ho

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
ALL = 1 << 30


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(shape, seed, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def starts(lens, itype=torch.int64):
    o = np.concatenate([[0], np.cumsum(lens)[:-1]]) if len(lens) else np.zeros(0)
    return torch.tensor(o.astype(np.int64), dtype=itype)


def bound(out, mag, big, dim, n, dtype, w, vmax):
    d = (dim + 8) * U * big
    tol = (4 * d + (8 + 2 * n) * 4 * U + w) * mag + HALF[dtype] * np.abs(out)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * n * vmax + 2.0 ** -25      # small weights; outputs below 2^-14
    return tol + 1e-30


def check_encode(q, k, v, lens, window, sinks, got, padding=None, scale=None):
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    out, mag, big = ho.attention(f64(q), f64(k), f64(v), lens, window, sinks, scale,
                                 None if padding is None else padding.cpu().numpy())
    n = max(lens) if lens else 0
    w = HALF[q.dtype]
    tol = bound(out, mag, big, dim, n, q.dtype, w, float(v.abs().max()) if v.numel() else 0.0)
    err = np.abs(f64(got) - out)
    worst = float((err / tol).max()) if err.size else 0.0
    print(f"encode {q.dtype} dim {dim} lens {lens[:4]}: worst error / bar {worst:.3f}", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 3), (8, 1)])
def test_encode_ragged(dtype, dim, heads, kv):
    lens = [1, 0, 63, 64, 65, 2, 0, 200, 17]
    n = sum(lens)
    q, k, v = (randn((n, h, dim), s, dtype) for s, h in ((1, heads), (2, kv), (3, kv)))
    got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), window=50, sinks=3)
    check_encode(q, k, v, lens, 50, 3, got)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (64, 0), (65, 64), (63, 65), (100, 500), (ALL, 0),
                                          (33, 7), (128, 129)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_encode_windows_and_sinks(window, sinks, dtype):
    lens = [300, 128, 129, 1]
    n = sum(lens)
    q, k, v = (randn((n, 2, 64), s, dtype) for s in (4, 5, 6))
    got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens, torch.int32).cuda(), window=window,
                               sinks=sinks)
    check_encode(q, k, v, lens, window, sinks, got)


@pytest.mark.parametrize("dtype,lens", [(torch.bfloat16, [2111]), (torch.float16, [1025, 700]),
                                        (torch.float32, [900])])
def test_encode_long(dtype, lens):
    n = sum(lens)
    q, k, v = (randn((n, h, 128), s, dtype) for s, h in ((7, 4), (8, 2), (9, 2)))
    got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), window=700, sinks=70)
    check_encode(q, k, v, lens, 700, 70, got)


def test_encode_large_logits():
    """Logits in the hundreds: the running maximum moves, weights underflow."""
    lens = [150, 90]
    n = sum(lens)
    for dtype in (torch.float32, torch.bfloat16):
        q, k, v = randn((n, 2, 64), 10, dtype, 6.0), randn((n, 2, 64), 11, dtype, 6.0), randn((n, 2, 64), 12, dtype)
        got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), scale=1.0)
        check_encode(q, k, v, lens, ALL, 0, got, scale=1.0)


def test_encode_many_short_histories():
    lens = [(i * 7) % 21 for i in range(500)]
    n = sum(lens)
    q, k, v = (randn((n, 2, 32), s, torch.float32) for s in (13, 14, 15))
    got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), window=20)
    check_encode(q, k, v, lens, 20, 0, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extra", [0, 16, 3])
def test_encode_columns_of_one_projection(dtype, extra):
    """q, k and v as columns of one wide tensor; rows of any alignment; out inside a wider one."""
    lens = [70, 5]
    n, heads, kv, dim = sum(lens), 4, 2, 64
    wide = randn((n, (heads + 2 * kv) * dim + extra), 16, dtype)
    w = wide.cuda()
    cut = lambda t, a, h: t[:, extra + a * dim:extra + (a + h) * dim].unflatten(1, (h, dim))
    out = torch.full((n, heads * dim + 5), -7.0, dtype=dtype, device="cuda")
    view = out[:, 2:2 + heads * dim].unflatten(1, (heads, dim))
    dl.history_attention(cut(w, 0, heads), cut(w, heads, kv), cut(w, heads + kv, kv), starts(lens).cuda(),
                         window=40, sinks=2, out=view)
    check_encode(cut(wide, 0, heads), cut(wide, heads, kv), cut(wide, heads + kv, kv), lens, 40, 2, view)
    assert torch.all(out[:, :2] == -7) and torch.all(out[:, 2 + heads * dim:] == -7)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_encode_padding_and_rows_that_see_nothing(dtype):
    lens = [100, 70, 30]
    n = sum(lens)
    q, k, v = (randn((n, 2, 64), s, dtype) for s in (17, 18, 19))
    pad = (torch.rand(n, generator=gen(20)) < 0.5).to(torch.uint8)
    pad[:40] = 1                    # the first rows of history 0 see nothing
    pad[100:170] = 2                # history 1 sees nothing at all
    for window in (1, 16, ALL):
        got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), window=window,
                                   padding=pad.cuda())
        check_encode(q, k, v, lens, window, 0, got, padding=pad)
        assert torch.all(got[:40] == 0) and torch.all(got[100:170] == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_encode_what_is_not_seen_does_not_reach_a_row(dtype, bad):
    lens = [90, 61, 40]
    n = sum(lens)
    q, k, v = (randn((n, 2, 64), s, dtype) for s in (21, 22, 23))
    pad = torch.zeros(n, dtype=torch.uint8)
    pad[10] = pad[95] = 1
    args = dict(window=20, sinks=2)
    clean = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), padding=pad.cuda(), **args)
    k2, v2 = k.clone(), v.clone()
    for t in (k2, v2):
        t[[10, 95]] = bad           # padding events
        t[50] = bad                 # seen by rows 50..69 of history 0 alone
        t[150] = bad                # the last event of history 1: seen by itself alone
    got = dl.history_attention(q.cuda(), k2.cuda(), v2.cuda(), starts(lens).cuda(), padding=pad.cuda(), **args)
    hit = torch.zeros(n, dtype=torch.bool)
    hit[50:70] = True
    hit[150] = True
    assert torch.equal(got[~hit.cuda()], clean[~hit.cuda()])
    assert not torch.isfinite(got[hit.cuda()].float()).any()
    # values alone: rows that see an infinite value are infinite or NaN, nobody else is
    got = dl.history_attention(q.cuda(), k.cuda(), v2.cuda(), starts(lens).cuda(), padding=pad.cuda(), **args)
    assert torch.equal(got[~hit.cuda()], clean[~hit.cuda()])
    assert not torch.isfinite(got[hit.cuda()].float()).any()


def test_encode_nothing():
    q = torch.empty((0, 2, 64), device="cuda")
    assert dl.history_attention(q, q, q, torch.zeros(3, dtype=torch.int64, device="cuda")).shape == q.shape


def test_encode_on_another_stream_and_in_a_graph():
    lens = [130, 0, 64]
    n = sum(lens)
    q, k, v = (randn((n, 4, 64), s, torch.bfloat16).cuda() for s in (24, 25, 26))
    off = starts(lens).cuda()
    want = dl.history_attention(q, k, v, off, window=33, sinks=4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = dl.history_attention(q, k, v, off, window=33, sinks=4)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dl.history_attention(q, k, v, off, window=33, sinks=4, out=out)
    for i in range(4):
        q.copy_(randn(tuple(q.shape), 100 + i, torch.bfloat16))
        want = dl.history_attention(q, k, v, off, window=33, sinks=4)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# --- the cache ----------------------------------------------------------------------


class Pair:
    """A GPU cache and its oracle, driven by the same calls."""

    def __init__(self, n_pages, n_slots, max_pages, kv, dim, page, dtype):
        self.gpu = dl.HistoryCache(n_pages, n_slots, max_pages, kv, dim, page)
        # what a page held before is nobody's: not a number, so that reading it shows
        self.gpu.k.fill_(0x7F)
        self.gpu.v.fill_(0x7F)
        self.gpu.k_scale.fill_(float("nan"))
        self.gpu.v_scale.fill_(float("nan"))
        self.cpu = ho.Cache(n_pages, n_slots, max_pages, kv, dim, page)
        self.kv, self.dim, self.page, self.dtype = kv, dim, page, dtype
        self.seed = 1000

    def slots(self, s):
        return torch.tensor(s, dtype=torch.int32, device="cuda")

    def events(self, n, scale):
        self.seed += 2
        return (randn((n, self.kv, self.dim), self.seed + i, self.dtype, scale) for i in (0, 1))

    def append(self, slots, counts, scale=1.0, edit=None):
        k, v = self.events(sum(counts), scale)
        if edit:
            edit(k, v)
        self.cpu.append(slots, counts, f64(k), f64(v))
        self.gpu.append(k.cuda(), v.cuda(), starts(counts).cuda(), slots=self.slots(slots))

    def same(self):
        torch.cuda.synchronize()
        g, c = self.gpu, self.cpu
        assert g.lens.tolist() == c.lens
        assert g.refs.tolist() == c.refs
        free = g.free_pages[:g.n_free].tolist()
        assert free == c.free[::-1]
        assert g.n_refused == c.refused
        table = g.table.tolist()
        for row, want in zip(table, c.lists):
            want = [-1 if p is None else p for p in want]
            assert row == want + [-1] * (len(row) - len(want))
        k, v = (t.view(torch.float8_e4m3fn).cpu().double().numpy() for t in (g.k, g.v))
        v = v.swapaxes(2, 3)
        ks, vs = f64(g.k_scale), f64(g.v_scale)
        for row, n in zip(c.lists, c.lens):
            for i, p in enumerate(row):
                m = min(self.page, n - i * self.page)
                if p is None or m <= 0:
                    continue
                assert np.array_equal(ks[p], c.ks[p]) and np.array_equal(vs[p], c.vs[p])
                assert np.array_equal(k[p, :, :m] * ks[p][:, None, None], c.k[p, :, :m], equal_nan=True)
                assert np.array_equal(v[p, :, :m] * vs[p][:, None, None], c.v[p, :, :m], equal_nan=True)

    def lookup(self, slots, heads, queries=1, window=ALL, sinks=0, dtype=None, scale=None):
        dtype = dtype or self.dtype
        self.seed += 2
        q = randn((len(slots), queries, heads, self.dim), self.seed, dtype)
        got = self.gpu.lookup(q.cuda(), window=window, sinks=sinks, scale=scale, slots=self.slots(slots))
        scale = self.dim ** -0.5 if scale is None else scale
        out, mag, big = self.cpu.lookup(slots, f64(q), window, sinks, scale)
        n = max([0] + [self.cpu.lens[s] for s in slots if 0 <= s < len(self.cpu.lens)])
        w = 2.0 ** -15 if dtype != torch.float32 else U
        vmax = np.abs(self.cpu.v).max()
        tol = bound(out, mag, big, self.dim, n, dtype, w, 0.0)
        err = np.abs(f64(got) - out)
        worst = float((err / tol).max())
        print(f"lookup {dtype} dim {self.dim} page {self.page}: worst error / bar {worst:.3f} (vmax {vmax:.2g})",
              flush=True)
        assert worst <= 1.0
        return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("dim", [32, 64, 128])
def test_cache_append_and_lookup(dtype, page, dim):
    p = Pair(60, 7, 20, 2, dim, page, dtype)
    p.append([0, 1, 3, 5, 6], [1, page, page + 1, 150, 0])
    p.same()
    p.append([0, 1, 2, 3, 5], [1, 1, 1, 1, 1], 3.0)            # scales grow, held codes are rounded again
    p.append([6, 5, 0], [2, 7, 40], 0.01)
    p.append([6], [3], 1000.0)
    p.same()
    for heads, queries in ((2, 1), (8, 1), (6, 5), (40, 1)):
        p.lookup([0, 1, 2, 3, 4, 5, 6], heads, queries)
    for window, sinks in ((1, 0), (5, 3), (64, 1), (100, 70), (31, 16)):
        p.lookup([5, 3, 6, 4, 1], 4, 1, window, sinks)


def test_cache_values_at_the_ends_of_the_range():
    """Zeros, the largest and smallest magnitudes, values that are not finite."""
    p = Pair(20, 3, 8, 1, 32, 16, torch.float32)

    def edit(k, v):
        k[:3] = 0
        k[3] = 448.0
        k[4] = 448.1
        k[5] = 2.0 ** -118
        v[0] = 3.0e38
        v[1] = 2.0 ** -126
        v[2, 0, 5] = float("nan")
        v[3, 0, 6] = float("inf")
        v[4, 0, 7] = -float("inf")
    for n in (1, 2, 3, 5, 6, 40):
        p.append([0], [n], edit=edit if n > 5 else None)
    p.append([1], [20], edit=lambda k, v: (k.zero_(), v.zero_()))
    p.append([2], [17], edit=lambda k, v: (k.mul_(2.0 ** -125), v.mul_(2.0 ** 120)))
    p.same()
    got = p.gpu.lookup(randn((1, 4, 32), 1, torch.float32).cuda(), slots=p.slots([1]))
    assert torch.all(got == 0)
    # the element that is not finite spoils its own output element alone
    q = randn((1, 1, 32), 2, torch.float32).cuda()
    got = p.gpu.lookup(q, slots=p.slots([0]))[0, 0].cpu()
    assert torch.isnan(got[5:8]).all()
    p.lookup([2], 3, scale=2.0 ** 100)


def test_cache_masked_events_do_not_reach_a_query():
    """NaN events outside the window, and whatever lies behind a history's end, stay out."""
    p = Pair(30, 2, 8, 2, 64, 32, torch.bfloat16)

    def edit(k, v):
        k[10:20] = float("nan")
        v[10:20] = float("nan")
    p.append([0, 1], [100, 33], edit=edit)
    p.lookup([0, 1], 4, 1, window=30, sinks=10)
    p.lookup([0], 4, 3, window=80, sinks=0)
    got = p.gpu.lookup(randn((1, 4, 64), 3, torch.bfloat16).cuda(), window=81, slots=p.slots([0]))
    assert torch.isnan(got.float()).all()


def test_cache_long_lookup_and_offsets_past_32_bits():
    """A pool of more than 2^32 code bytes, the history on its last pages."""
    page, kv, dim = 64, 8, 128
    n_pages = (1 << 32) // (page * kv * dim) + 40
    c = dl.HistoryCache(n_pages, 2, 40, kv, dim, page)
    n = 2000
    c.free_pages.copy_(torch.arange(n_pages, dtype=torch.int32).cuda())       # highest first: test-only order
    k, v = (randn((n, kv, dim), s, torch.bfloat16) for s in (31, 32))
    c.append(k.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    used = c.table[0, :32].cpu()
    assert int(used.min()) * page * kv * dim > (1 << 32) - 1
    o = ho.Cache(32, 1, 40, kv, dim, page)
    o.append([0], [n], f64(k), f64(v))
    q = randn((1, 1, 16, dim), 33, torch.bfloat16)
    got = c.lookup(q.cuda())
    out, mag, big = o.lookup([0], f64(q), ALL, 0, dim ** -0.5)
    tol = bound(out, mag, big, dim, n, torch.bfloat16, 2.0 ** -15, 0.0)
    assert (np.abs(f64(got) - out) <= tol).all()


@pytest.mark.parametrize("lens,heads,kv,page", [([5000], 8, 1, 64), ([1, 3000, 0, 17], 12, 4, 32),
                                                ([400] * 40, 4, 4, 16), ([64, 128, 2048], 64, 2, 64)])
def test_lookup_splits_histories(lens, heads, kv, page):
    """One long history over many blocks, ragged batches, many rows: partial results join."""
    need = sum(-(-n // page) for n in lens)
    p = Pair(need, len(lens), -(-max(lens) // page), kv, 64, page, torch.bfloat16)
    p.append(list(range(len(lens))), lens)
    slots = list(range(len(lens)))
    p.lookup(slots, heads)
    p.lookup(slots, heads, 3, window=1000, sinks=5)
    p.lookup(slots, heads, 1, dtype=torch.float32)
    p.lookup(slots, heads, 1, dtype=torch.float16)
    # the same call gives the same bits
    q = randn((len(lens), heads, 64), 9, torch.bfloat16).cuda()
    a, b = p.gpu.lookup(q), p.gpu.lookup(q)
    assert torch.equal(a, b)


def test_lookup_strided_queries_and_slot_order():
    p = Pair(20, 4, 6, 2, 64, 16, torch.float32)
    p.append([0, 1, 2, 3], [20, 33, 1, 90])
    q = randn((4, 4, 64), 5, torch.float32)
    want = p.gpu.lookup(q.cuda())
    wide = torch.zeros((4, 4 * 64 + 3), device="cuda")
    view = wide[:, 3:].unflatten(1, (4, 64))
    view.copy_(q)
    assert torch.equal(p.gpu.lookup(view), want)
    back = p.gpu.lookup(q.flip(0).cuda(), slots=p.slots([3, 2, 1, 0]))
    assert torch.equal(back.flip(0), want)


def test_lookup_bad_pages_and_slots_are_not_seen():
    p = Pair(20, 3, 6, 1, 64, 16, torch.float32)
    p.append([0, 1], [96, 40])
    q = randn((1, 2, 64), 6, torch.float32).cuda()
    p.gpu.table[0, 1] = -1
    p.gpu.table[0, 3] = 20
    p.gpu.table[0, 4] = 1 << 30
    p.cpu.lists[0][1] = p.cpu.lists[0][3] = p.cpu.lists[0][4] = None
    p.lookup([0, 1], 2)
    p.gpu.lens[1] = 1 << 30              # a length the table cannot hold is cut to what it can
    p.gpu.lookup(q, slots=p.slots([1]))
    torch.cuda.synchronize()
    for slot in (-1, 3, 1 << 30):
        assert torch.all(p.gpu.lookup(q, slots=p.slots([slot])) == 0)


def test_append_refusals():
    p = Pair(6, 5, 3, 1, 32, 16, torch.float32)
    p.append([0, 9, 1, -1, 2], [16, 3, 49, 2, 5])     # bad slots; longer than three pages
    p.same()
    p.append([1, 2, 3, 4], [32, 3, 33, 1])            # 2 + 0 + 3 + 1 pages of 4: the third and fourth do not fit
    p.same()
    p.append([4, 0], [1, 16])
    p.same()
    assert p.cpu.refused == 5


def test_fork_copy_on_append_free_and_compact():
    p = Pair(40, 12, 6, 2, 64, 16, torch.bfloat16)
    p.append([0, 1, 2], [40, 16, 70])
    src, dst = [0, 0, 0, 1, 2, 2], [3, 4, 5, 6, 7, 8]
    p.cpu.fork(src, dst)
    p.gpu.fork(p.slots(src), p.slots(dst))
    p.same()
    p.append([3, 4, 6, 7], [1, 20, 1, 1], 4.0)        # shared tails are copied, their scales grow in the copy alone
    p.same()
    p.append([0, 5], [2, 2])                          # the last two holders of a tail append in one call
    p.same()
    p.lookup([0, 3, 4, 5, 6, 7, 8], 4)
    for gone in ([0, 4], [2, 7]):
        p.cpu.truncate(gone, [0] * len(gone))
        p.gpu.free(p.slots(gone))
        p.same()
    p.cpu.compact()
    p.gpu.compact()
    p.same()
    p.lookup([1, 3, 5, 6, 8], 4)
    src, dst = [8, 1, 50, 3], [3, 5, 6, -1]           # destinations that hold something; bad slots
    p.cpu.fork(src, dst)
    p.gpu.fork(p.slots(src), p.slots(dst))
    p.same()


def test_truncate_and_trim():
    p = Pair(40, 6, 10, 1, 32, 16, torch.float16)
    p.append([0, 1, 2, 3], [150, 64, 17, 16])
    slots, lens = [0, 1, 2, 3, 4, 77], [100, 64, 18, 0, 0, 1]
    p.cpu.truncate(slots, lens)
    p.gpu.truncate(p.slots(slots), p.slots(lens))
    p.same()
    p.cpu.fork([0], [5])
    p.gpu.fork(p.slots([0]), p.slots([5]))
    p.cpu.truncate([5], [33])                         # inside a page another history holds
    p.gpu.truncate(p.slots([5]), p.slots([33]))
    p.append([5], [1])
    p.same()
    p.cpu.trim([0, 1, -3], 20, 5)
    p.gpu.trim(p.slots([0, 1, -3]), 20, 5)
    p.same()
    p.lookup([0, 1, 5], 2, 1, window=20, sinks=5)
    p.append([0, 1], [3, 30])
    p.lookup([0, 1, 5], 2, 1, window=20, sinks=5)
    p.cpu.truncate([0, 0], [40, -1])                  # into a trimmed page; below zero
    p.gpu.truncate(p.slots([0]), p.slots([40]))
    p.gpu.truncate(p.slots([0]), p.slots([-1]))
    p.same()
    p.cpu.trim([0], 1, 0)
    p.gpu.trim(p.slots([0]), 1, 0)
    p.same()


@pytest.mark.parametrize("n_pages", [5000, 16384, 16385, 40000])
def test_free_list_of_large_pools(n_pages):
    """More pages than one block lists: the order is the pages' own."""
    c = dl.HistoryCache(n_pages, 300, 64, 1, 32, 16)
    n = 1000
    lens = [(i * 37) % (n + 1) for i in range(200)]
    k = torch.zeros((sum(lens), 1, 32), device="cuda")
    c.append(k, k, starts(lens).cuda())
    need = sum(-(-x // 16) for x in lens)
    refused = c.n_refused
    if need <= n_pages:
        assert refused == 0 and c.n_free == n_pages - need
    c.free(torch.arange(0, 200, 3, dtype=torch.int32, device="cuda"))

    def check():
        refs = c.refs.cpu()
        want = torch.nonzero(refs == 0).flatten().flip(0).to(torch.int32)
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
    live = held[held >= 0]
    assert live.numel() == used and torch.equal(live.sort()[0], torch.arange(used, dtype=torch.int32))


def test_cache_calls_in_a_graph():
    """Append, lookup, fork, free and compaction replayed against eager calls on a second cache."""
    caches = [dl.HistoryCache(300, 20, 10, 2, 64, 16) for _ in range(2)]
    k, v = (randn((500, 2, 64), s, torch.bfloat16).cuda() for s in (41, 42))
    off = torch.arange(10, dtype=torch.int64, device="cuda") * 50
    one = torch.arange(10, dtype=torch.int64, device="cuda")
    q, k1, v1 = (torch.zeros((10, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    src = torch.arange(0, 10, dtype=torch.int32, device="cuda")
    dst = src + 10
    for c in caches:
        c.append(k, v, off)

    def step(c, out):
        c.fork(src, dst)
        c.append(k1, v1, one, slots=dst)
        c.lookup(q, slots=dst, out=out)
        c.free(dst[::2].contiguous())
        c.compact()
        c.append(k1, v1, one)

    for c in caches:
        step(c, torch.empty_like(q))           # workspaces exist before the capture
    outs = [torch.empty_like(q) for _ in caches]
    torch.cuda.synchronize()
    even = dst[::2].contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = caches[0]
        c.fork(src, dst)
        c.append(k1, v1, one, slots=dst)
        c.lookup(q, slots=dst, out=outs[0])
        c.free(even)
        c.compact()
        c.append(k1, v1, one)
    for i in range(5):
        for t, s in ((q, 200), (k1, 300), (v1, 400)):
            t.copy_(randn(tuple(t.shape), s + i, torch.bfloat16))
        g.replay()
        step(caches[1], outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        for n in ("table", "lens", "refs", "counters"):
            assert torch.equal(getattr(caches[0], n), getattr(caches[1], n)), n


def test_graph_keeps_its_workspace_when_a_later_call_needs_more():
    """A captured lookup, whose runs meet in the workspace, replayed after calls of larger batches on its stream and
    after their like has been allocated anew."""
    n = 65 * 64
    c = dl.HistoryCache(2 * 65, 66, 65, 2, 64, 64)
    k, v = (randn((2 * n, 2, 64), s, torch.bfloat16).cuda() for s in (51, 52))
    c.append(k, v, torch.arange(2, dtype=torch.int64, device="cuda") * n)
    q = randn((1, 8, 64), 53, torch.bfloat16).cuda()
    large = randn((66, 30, 8, 64), 54, torch.bfloat16).cuda()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = c.lookup(q)
        out = torch.empty_like(q)
        with torch.cuda.graph(g, stream=side):
            c.lookup(q, out=out)
        c.lookup(large)
        fills = [torch.full((1 << s,), 77, dtype=torch.uint8, device="cuda") for s in range(9, 26) for _ in range(3)]
        for _ in range(3):
            out.zero_()
            g.replay()
            side.synchronize()
            assert torch.equal(out, want)
            assert all(bool((f == 77).all()) for f in fills)
            c.lookup(large)


# --- the example: all of them together ----------------------------------------------


def test_example_ranking_with_histories():
    """examples/history_ranking.py: a fork's score is the score after the click, and leaves the user's own as it
    was; trimming and compaction change nothing; the histories' vectors match the 64-bit form."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "history_ranking.py")
    spec = importlib.util.spec_from_file_location("history_ranking", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    out = mod.main()
    r, lens, slots = out["ranker"], out["lens"], out["slots"]
    assert r.cache.n_refused == 0
    for p in ("before", "tried", "after"):
        assert bool(((out[p] > 0) & (out[p] < 1)).all())
    assert torch.equal(out["before"], out["again"])
    assert torch.equal(out["tried"], out["after"])
    assert torch.equal(out["trimmed"], out["after"])
    q, k, v = r.project(out["events"])
    check_encode(q.cpu(), k.cpu(), v.cpu(), lens, r.window, r.sinks, out["encoded"])
    o = ho.Cache(400, len(lens), 40, r.heads, r.dim // r.heads, r.cache.page_events)
    o.append(list(range(len(lens))), lens, f64(k), f64(v))
    _, k1, v1 = r.project(out["click"])
    o.append(list(range(len(lens))), [1] * len(lens), f64(k1), f64(v1))
    got = r.attend(out["candidates"], slots)
    cq = f64(next(r.project(out["candidates"]))).reshape(*out["candidates"].shape, r.heads, -1)
    want, mag, big = o.lookup(list(range(len(lens))), cq, r.window, r.sinks, (r.dim // r.heads) ** -0.5)
    tol = bound(want, mag, big, r.dim // r.heads, max(lens) + 1, torch.float32, U, 0.0)
    assert (np.abs(f64(got).reshape(want.shape) - want) <= tol).all()


# --- few long histories: the waves of a block share a row's keys ---------------------


@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 32), (torch.bfloat16, 64), (torch.float16, 128),
                                       (torch.float32, 32), (torch.float32, 64), (torch.float32, 128)])
@pytest.mark.parametrize("heads,kv", [(1, 1), (2, 1)])
@pytest.mark.parametrize("window,sinks,padded", [(ALL, 0, False), (600, 5, True)])
def test_encode_few_long_histories(dtype, dim, heads, kv, window, sinks, padded):
    lens = [1300, 733]
    n = sum(lens)
    q, k, v = (randn((n, h, dim), s, dtype) for s, h in ((51, heads), (52, kv), (53, kv)))
    pad = (torch.rand(n, generator=gen(54)) < 0.3).to(torch.uint8) if padded else None
    if padded:
        pad[1300:1400] = 1              # rows that see nothing
    got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(), window=window, sinks=sinks,
                               padding=None if pad is None else pad.cuda())
    check_encode(q, k, v, lens, window, sinks, got, padding=pad)
    if padded:
        assert torch.all(got[1300:1400] == 0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_encode_few_long_histories_keep_what_is_not_seen_out(bad):
    n, window = 1500, 700
    q, k, v = (randn((n, 1, 64), s, torch.bfloat16) for s in (55, 56, 57))
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    clean = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), off, window=window)
    v[500] = bad
    k[501] = bad
    got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), off, window=window)
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[500:501 + window] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert not torch.isfinite(got[hit].float()).any()


@pytest.mark.parametrize("page", [16, 64])
def test_append_a_few_events_to_many_histories(page):
    """Fewer events than two for each history: a page's first event does the page's work, also where a history's
    few events open a second page, and where histories get none."""
    p = Pair(80, 16, 5, 2, 32, page, torch.bfloat16)
    p.append(list(range(16)), [page - 1, page, page + 1, 1, 0, 2 * page - 1, 3, page - 2] * 2)
    for counts in ([2] * 16, [1] * 16, [0, 2, 1, 3, 5, 0, 2, 2] * 2, [0] * 15 + [1], [page + 3] + [0] * 15):
        p.append(list(range(16)), counts, 2.0)
        p.same()
    p.cpu.fork([0, 1, 2], [13, 14, 15])
    p.gpu.fork(p.slots([0, 1, 2]), p.slots([13, 14, 15]))
    p.append([13, 14, 15, 3], [1, 2, 0, 1], 4.0)
    p.same()
    p.lookup(list(range(16)), 4)
