"""The event-history operators at the ends of their types' ranges, and where few bits would show.

Values that a row does not see leave it bit for bit as it was.  Where a result is compared with its formula, the bar
counts u = 2^-24 for each fp32 rounding, and half a step of the output's type.
"""
import math

import numpy as np
import pytest
import torch

import dlrm_embedding_interaction_amd as dl
import history_oracle as ho
from test_history import ALL, HALF, U, Pair, bound, f64, gen, randn, starts

MAX32 = torch.finfo(torch.float32).max


def encode(q, k, v, lens, pad=None, **kw):
    return dl.history_attention(q.cuda(), k.cuda(), v.cuda(), starts(lens).cuda(),
                                padding=None if pad is None else pad.cuda(), **kw).cpu()


# --- a row's bits are its own ----------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,dim", [([200, 61], 64), ([1300], 128)])
def test_encode_rows_do_not_depend_on_their_neighbours(dtype, lens, dim):
    """Logits of other rows, however large, move nothing in a row of ordinary ones."""
    n = sum(lens)
    q, k, v = (randn((n, 2, dim), s, dtype) for s in (17, 18, 19))
    want = encode(q, k, v, lens)
    loud = torch.arange(n) % 5 == 2
    q[loud] *= 60
    got = encode(q, k, v, lens)
    assert torch.equal(got[~loud], want[~loud])
    assert not torch.equal(got[loud], want[loud])


# --- fp32: finite values next to the largest one ------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("value", [MAX32, -MAX32, 3.3962e38, 3.3961e38])
@pytest.mark.parametrize("lens,window,dim", [([90, 61, 40], 20, 64), ([90, 61, 40], 20, 128), ([1500], 700, 32),
                                             ([1500], 700, 64), ([1300, 200], 700, 128)])
def test_encode_fp32_large_values_do_not_reach_rows_that_do_not_see_them(value, lens, window, dim):
    n, at = sum(lens), 50
    q, k, v = (randn((n, 1, dim), s, torch.float32) for s in (1, 2, 3))
    pad = torch.zeros(n, dtype=torch.uint8)
    pad[[10, 95, 96]] = 1
    clean = encode(q, k, v, lens, pad, window=window)
    k2, v2 = k.clone(), v.clone()
    for t in (k2, v2):
        t[[10, 96]] = value
        t[at] = value
    hit = torch.zeros(n, dtype=torch.bool)
    hit[at:min(at + window, lens[0])] = True
    for kk in (k2, k):
        got = encode(q, kk, v2, lens, pad, window=window)
        assert torch.equal(got[~hit], clean[~hit])
    # beside an infinity, which changes how the tile is worked on
    v2[95] = float("inf")
    assert torch.equal(encode(q, k2, v2, lens, pad, window=window)[~hit], clean[~hit])
    # a row that sees a large value feels it in that element alone
    v3 = v.clone()
    v3[at, :, 7] = value
    got = encode(q, k, v3, lens, pad, window=window)
    other = torch.arange(dim) != 7
    assert torch.equal(got[:, :, other], clean[:, :, other])
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("value", [3.3999e38, -3.3999e38, 3.3962e38])
@pytest.mark.parametrize("lens", [[70, 9], [1300]])
def test_encode_fp32_large_values_count_as_they_are(value, lens):
    n, dim = sum(lens), 64
    q, k, v = (randn((n, 2, dim), s, torch.float32) for s in (4, 5, 6))
    # a large value of q or k meets zeros: it changes nothing
    q[:, :, 3], k[:, :, 3], q[:, :, 40], k[:, :, 40] = 0, 0, 0, 0
    clean = encode(q, k, v, lens)
    q[20, :, 3] = value
    k[33, :, 40] = value
    assert torch.equal(encode(q, k, v, lens), clean)
    # a weight of 1: six products of parts, those left out (3 u), the weight, its sum and the division
    v[33] = value
    v[34, :, ::2] = -value
    got = encode(q, k, v, lens, window=1)
    assert bool(((got.double() - v.double()).abs() <= 16 * U * v.double().abs()).all())
    # beside a value that is not finite in the same tile
    v[35, :, 1] = float("inf")
    got = encode(q, k, v, lens, window=1)
    fin = torch.isfinite(v)
    assert bool(((got.double() - v.double()).abs() <= 16 * U * v.double().abs())[fin].all())
    assert not torch.isfinite(got[~fin]).any()


# --- infinite keys -------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,dim", [([90, 61], 64), ([90, 61], 128), ([1300], 32), ([1300], 128)])
@pytest.mark.parametrize("scale", [0.125, -0.125])
def test_encode_a_key_of_minus_infinity_has_no_weight(dtype, lens, dim, scale):
    """Element 3 of every query is positive, of some keys -inf (+inf where the scale is negative): their logits are
    -inf, and they count as events that nothing sees."""
    n, bad = sum(lens), -math.copysign(math.inf, scale)
    q, k, v = (randn((n, 2, dim), s, dtype) for s in (7, 8, 9))
    q[:, :, 3] = q[:, :, 3].abs() + 0.5
    q[5, :, 3] = 1                      # one part holds it whole: the other parts are zeros
    pad = torch.zeros(n, dtype=torch.uint8)
    gone = [0, 4, 40, 60, 88]
    pad[gone] = 1
    want = encode(q, k, v, lens, pad, scale=scale)
    k[gone, :, 3] = bad
    got = encode(q, k, v, lens, torch.zeros_like(pad), scale=scale)
    rows = torch.arange(n) > 0          # row 0 sees nothing else
    assert torch.equal(got[rows], want[rows])
    # against the sign of the queries: +inf, and what follows is not a number
    k[60, :, 3] = -bad
    got = encode(q, k, v, lens, torch.zeros_like(pad), scale=scale)
    assert torch.equal(got[1:60], want[1:60])
    assert torch.isnan(got[60:lens[0]].float()).all()
    assert torch.equal(got[lens[0]:], want[lens[0]:])


# --- weights and their sums ----------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("up", [3, 7])
def test_encode_large_values_behind_a_rising_maximum(dtype, up):
    """Key 40's logit passes those before it by less than the running maximum follows at once; its value is 2^127.
    The weighted mean is finite, and so is the result."""
    n, dim = 64, 64
    q, k, v = (torch.zeros((n, 1, dim), dtype=dtype) for _ in range(3))
    q[:, :, 0] = 1
    k[40, :, 0] = up
    v[40] = 2.0 ** 127
    got = encode(q, k, v, [n], scale=math.log(2))
    out, mag, big = ho.attention(f64(q), f64(k), f64(v), [n], ALL, 0, math.log(2))
    tol = bound(out, mag, big, dim, n, dtype, HALF[dtype], 0.0)
    assert bool((np.abs(f64(got) - out) <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [700, 4000])
@pytest.mark.parametrize("log2", [-25.2, -28.0])
def test_encode_fp16_small_weights_count(n, log2):
    """One key holds nearly all weight and a value of 0; the others, of 2^log2 each, make the result.  Weights are
    rounded to fp16 against a maximum of at least 2^7: those below 2^-21 of the largest are off by 2^-32 at most."""
    dim = 32
    q, k, v = (torch.zeros((n, 1, dim), dtype=torch.float16) for _ in range(3))
    q[:, :, 0] = 1
    k[1:, :, 0] = log2
    v[1:] = 1
    got = encode(q, k, v, [n], scale=math.log(2))
    out, mag, big = ho.attention(f64(q), f64(k), f64(v), [n], ALL, 0, math.log(2))
    # outputs below 2^-14 are off by half a step of 2^-24
    tol = bound(out, mag, big, dim, n, torch.float32, HALF[torch.float16], 0.0) + \
        HALF[torch.float16] * np.abs(out) + n * 2.0 ** -32 + 2.0 ** -25
    worst = (np.abs(f64(got) - out) / tol).max()
    print(f"worst error / bar {worst:.3f}, last row {float(got[-1, 0, 0]):.3e} for {out[-1, 0, 0]:.3e}", flush=True)
    assert worst <= 1


# --- scales at the ends of their range -----------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-38, -1e-38, 1e-44, 3e38, -3e38])
def test_scales_at_the_ends_of_their_range(dtype, scale):
    """A scale of 0 weighs all events alike, however large their products; a tiny one is not rounded up; a large one
    leaves products of 0 at 0."""
    n, dim = 80, 64
    big = 0.0 if abs(scale) > 1 else 2.0 ** 63
    q, k = (torch.zeros((n, 1, dim), dtype=dtype) for _ in range(2))
    q[:, :, 0] = big
    k[:, :, 0] = big * randn((n, 1), 11, torch.float32).sign().to(dtype)
    v = randn((n, 1, dim), 12, dtype)
    got = encode(q, k, v, [n], scale=scale)
    out, mag, b = ho.attention(f64(q), f64(k), f64(v), [n], ALL, 0, float(np.float32(scale)))
    tol = bound(out, mag, b, dim, n, dtype, HALF[dtype], 0.0)
    assert bool((np.abs(f64(got) - out) <= tol).all())
    p = Pair(10, 1, 6, 1, dim, 16, dtype)
    k2, v2 = k.clone(), randn((n, 1, dim), 13, dtype)
    p.cpu.append([0], [n], f64(k2), f64(v2))
    p.gpu.append(k2.cuda(), v2.cuda(), starts([n]).cuda())
    got = p.gpu.lookup(q[:1].cuda(), scale=scale)
    out, mag, b = p.cpu.lookup([0], f64(q[:1])[:, None], ALL, 0, float(np.float32(scale)))
    tol = bound(out, mag, b, dim, n, dtype, 2.0 ** -15 if dtype != torch.float32 else U, 0.0)
    assert bool((np.abs(f64(got)[:, None] - out) <= tol).all())


# --- the cache at the ends of fp32's range --------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim", [32, 128])
@pytest.mark.parametrize("count", [1, 5, 40])
def test_cache_keeps_large_finite_values_finite(dtype, dim, count):
    """From 248 x 2^120 on the nearest code at the largest scale, 256, would stand for 2^128: 240 is held."""
    p = Pair(10, 1, 6, 1, dim, 16, dtype)
    top = torch.finfo(dtype).max
    q = torch.zeros((1, 1, dim), dtype=torch.float32)
    seen = np.zeros((0, 1, dim))
    for sign in (1.0, -1.0):
        k, v = (randn((count, 1, dim), s, dtype) for s in (14, 15))
        v[0, 0, 1], v[0, 0, 2], v[0, 0, 3] = sign * 3.29e38, sign * 3.3e38, sign * top
        v[-1, 0, 4] = sign * 3.2e38
        k[0, 0, 5] = sign * top
        p.gpu.append(k.cuda(), v.cuda(), starts([count]).cuda())
        held = f64(v)
        # the block of the first event has scale 2^120: codes are multiples of 2^111 x 1, 2, 4 .. 16 there
        unit = 2.0 ** 120
        for e in (0, count - 1):
            for d in (1, 2, 3, 4):
                x = held[e, 0, d]
                if abs(x) > 1e38:
                    held[e, 0, d] = np.sign(x) * min(ho.e4m3(abs(x) / unit), 240.0) * unit
        seen = np.concatenate([seen, held])
    torch.cuda.synchronize()
    assert torch.isfinite(p.gpu.k_scale[p.gpu.refs > 0]).all()
    codes = p.gpu.v[p.gpu.refs > 0].cpu().view(torch.float8_e4m3fn).float()
    scales = p.gpu.v_scale[p.gpu.refs > 0].cpu()
    table = p.gpu.table[0].cpu()
    for j, row in enumerate(seen):
        page = int(table[j // 16])
        c = p.gpu.v[page, 0, :, j % 16].cpu().view(torch.float8_e4m3fn).double().numpy()
        s = float(p.gpu.v_scale[page, 0])
        for d in (1, 2, 3, 4):
            if abs(row[0, d]) > 1e38:
                assert c[d] * s == row[0, d], (j, d)
    assert codes.numel() and scales.numel()
    # one event alone in the window: the lookup gives its values, all finite
    one = Pair(4, 1, 2, 1, dim, 16, dtype)
    k, v = torch.zeros((1, 1, dim), dtype=dtype), torch.full((1, 1, dim), -top, dtype=dtype)
    one.gpu.append(k.cuda(), v.cuda(), starts([1]).cuda())
    got = one.gpu.lookup(q.cuda())
    assert bool((got == -240 * 2.0 ** 120).all())
    # what is not finite is still held as NaN
    v[0, 0, 0], v[0, 0, 1] = float("inf"), float("nan")
    one.gpu.append(k.cuda(), v.cuda(), starts([1]).cuda())
    got = one.gpu.lookup(q.cuda(), window=1).cpu()[0, 0]
    assert torch.isnan(got[:2]).all() and bool((got[2:] == -240 * 2.0 ** 120).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [0.0, 2.0 ** -99, -2.0 ** -92])
def test_cache_scale_grows_by_more_than_fp32_holds(dtype, first):
    """A block that held zeros or tiny values gets large ones: its scale grows from 2^-100 to 2^119, a quotient that
    fp32 does not hold; what it held becomes zeros."""
    p = Pair(20, 4, 4, 2, 64, 16, dtype)
    p.append([0, 1, 2], [3, 15, 1], edit=lambda k, v: (k.fill_(first), v.fill_(first)))
    p.same()
    p.cpu.fork([0], [3])
    p.gpu.fork(p.slots([0]), p.slots([3]))

    def edit(k, v):
        k.fill_(2.0 ** 127)
        v[:, 0] = 2.0 ** 60
        v[:, 1] = -2.0 ** 126
    p.append([0, 1, 2, 3], [1, 3, 9, 2], edit=edit)
    p.same()
    held = p.gpu.table[0, 0]
    assert torch.isfinite(p.gpu.k[held].cpu().view(torch.float8_e4m3fn).float()[:, :4]).all()


# --- refusals ------------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("events", [40, 65 * 64])
def test_lookup_counts_the_slots_it_refuses(events):
    """In one launch and in two: bad slots give zeros, and each is counted once."""
    p = Pair(70, 3, 66, 2, 64, 64, torch.bfloat16)
    p.append([0, 1], [events, 5])
    q = randn((5, 40, 4, 64), 16, torch.bfloat16).cuda()
    got = p.gpu.lookup(q, slots=p.slots([-1, 0, 3, 1 << 30, 1]))
    assert p.gpu.n_refused == 3
    assert bool((got[[0, 2, 3]] == 0).all()) and bool((got[[1, 4]] != 0).any())
    p.gpu.lookup(q, window=9, slots=p.slots([2, 0, 1, 0, -5]))
    assert p.gpu.n_refused == 4
    p.gpu.lookup(q[:3])
    assert p.gpu.n_refused == 4


# --- counters that no call wrote ---------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("count,left", [(1 << 30, 4), (7, 4), (-5, 0)])
def test_append_reads_no_place_past_the_free_list(count, left):
    """A count of free pages that passes the pool's size, or is below zero, is cut to what the list can hold."""
    c = dl.HistoryCache(6, 2, 6, 1, 32, 16)
    c.counters[0] = count
    k = randn((20, 1, 32), 24, torch.bfloat16).cuda()
    c.append(k, k, torch.zeros(1, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    assert c.n_free == left
    assert c.table[0].tolist() == ([0, 1] + [-1] * 4 if left else [-1] * 6)
    assert c.n_refused == (0 if left else 1)


# --- workspaces of captured calls ------------------------------------------------------


@pytest.mark.gpu
def test_captured_lookups_share_no_workspace():
    """Two lookups, each cut into many runs that meet in a workspace, captured on one stream and replayed side by side on
    two, beside eager ones on the stream of the capture."""
    n = 65 * 64
    c = dl.HistoryCache(8 * 65, 8, 65, 2, 64, 64)
    k, v = (randn((8 * n, 2, 64), s, torch.bfloat16).cuda() for s in (20, 21))
    c.append(k, v, torch.arange(8, dtype=torch.int64, device="cuda") * n)
    slots = [torch.arange(a, a + 4, dtype=torch.int32, device="cuda") for a in (0, 4)]
    qs = [randn((4, 8, 64), s, torch.bfloat16).cuda() for s in (22, 23)]
    want = [c.lookup(q, slots=s) for q, s in zip(qs, slots)]
    outs = [torch.empty_like(q) for q in qs]
    side = torch.cuda.Stream()
    graphs = []
    held = {s: w[0] for s, w in c._ws.items()}
    torch.cuda.synchronize()
    for q, s, out in zip(qs, slots, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            for _ in range(10):
                c.lookup(q, slots=s, out=out)
        graphs.append(g)
    # a capture neither takes a stream's workspace nor leaves one behind
    assert {s: w[0] for s, w in c._ws.items()} == held
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(side):
            eager = [c.lookup(qs[1], slots=slots[1]) for _ in range(10)]
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w)
        assert all(torch.equal(e, want[1]) for e in eager)
