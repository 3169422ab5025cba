"""That fp32 event-history calls keep all 24 bits: inputs on which a lost part of a factor, or a lost product of parts,
shows far above the bars, and on which the kernels stay below them.

Bars, u = 2^-24.  Where one weight, or two that sum to 1, meet the values: six products of parts are added (6 u), those
left out are below 4 u, the weights' sum, its reciprocal and the last product take 3 u:  16 u |v|.  Two logits of size
|s| that differ by about 1: each is off by 6 u |s| for its additions, 4 u |s| for what is left out, 2 u |s| for the scale
and the difference to the maximum, and the smaller weight moves by a quarter of the sum:  (16 + 6 |s|) u.  Values
between 1 and 2 under two weights of logits below 1:  (16 x 2 + 6) u.
"""
import numpy as np
import pytest
import torch

import dlrm_embedding_interaction_amd as dl

U = 2.0 ** -24
SIX = ((0, 2), (1, 1), (2, 0), (0, 1), (1, 0), (0, 0))


def draws(shape, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.rand(shape, generator=g)


def pair_logits(n, dim, seed):
    """Keys of even events have element 0, of odd ones element dim - 1; every query has both, with all 24 bits in use:
    a row that sees two events weighs two products near 402 whose errors have nothing in common.  bf16 steps are 1/8
    there: the products of second parts are about 0.05 x 0.05 and -0.05 x 0.025."""
    q, k = torch.zeros((n, 1, dim)), torch.zeros((n, 1, dim))
    q[:, 0, 0], q[:, 0, dim - 1] = 20.05 + draws(n, seed) / 128, 19.95 + draws(n, seed + 1) / 128
    y = draws(n, seed + 2) / 128
    even = torch.arange(n) % 2 == 0
    k[even, 0, 0], k[~even, 0, dim - 1] = 20.05 + y[even], 20.15 + y[~even]
    return q, k


def cases(n, dim):
    """(name, q, k, v, window, bar): scale 1, one history of n events."""
    zero = torch.zeros((n, 1, dim))
    v = (draws((n, 1, dim), 1) - 0.5) * 8
    q, k = pair_logits(n, dim, 2)
    odd = (torch.arange(n) % 2).float()[:, None, None].expand(n, 1, dim).contiguous()
    near = draws((n, 1, dim), 5) - 0.5
    one, y = zero.clone(), zero.clone()
    one[:, :, 0], y[:, :, 0] = 1, draws((n, 1), 6)          # logits below 1
    return [("values", zero, zero, v, 1, 16 * U * v.double().abs().numpy()),
            ("weights and values", one, y, 1 + draws((n, 1, dim), 7), 2, (16 * 2 + 6) * U),
            ("weights", near, near.flip(0) * 3, torch.ones((n, 1, dim)), 2, 16 * U),
            ("logits", q, k, odd, 2, (16 + 6 * 410) * U)]


def exact(q, k, v, window):
    q, k, v = (t[:, 0].double().numpy() for t in (q, k, v))
    return weighted(q @ k.T, window)[0] @ v


def weighted(s, window):
    i, j = np.arange(len(s))[:, None], np.arange(len(s))[None, :]
    s = np.where((j <= i) & (i - j < window), s, -np.inf)
    w = np.exp(s - s.max(1, keepdims=True))
    return w / w.sum(1, keepdims=True), w


def split(x, n, cut=False):
    """fp32 values as n bf16 parts, rounded or cut off."""
    out, r = [], torch.as_tensor(x, dtype=torch.float32)
    for _ in range(n):
        e = (r.view(torch.int32) & -65536).view(torch.float32) if cut else r.bfloat16().float()
        out.append(e.double().numpy())
        r = r - e
    return out + [np.zeros_like(out[0])] * (3 - n)


def emulate(q, k, v, window, parts=(3, 3, 3, 3), pairs=SIX, pv=SIX):
    """The products of parts alone, everything else in 64 bits; `parts` of q, k, the weights and v; `pairs` of the first
    product, `pv` of the second."""
    a, b, d = split(q[:, 0], parts[0]), split(k[:, 0], parts[1]), split(v[:, 0], parts[3])
    s = sum(a[i] @ b[j].T for i, j in pairs)
    w = weighted(s, window)[1].astype(np.float32)
    p = split(torch.from_numpy(w), parts[2])
    return sum(p[i] @ d[j] for i, j in pv) / w.astype(np.float64).sum(1, keepdims=True)


def worst(name, got, q, k, v, window, bar):
    e = np.abs(got - exact(q, k, v, window)) / (bar if np.ndim(bar) == 0 else np.maximum(bar[:, 0], 1e-30))
    print(f"{name}: worst error / bar {e.max():.3f}", flush=True)
    return e.max()


def test_bars_hold_for_all_parts_and_fail_for_a_lost_one():
    lost = {"values": [dict(parts=(3, 3, 3, 2))], "weights": [dict(parts=(3, 3, 2, 3))],
            "weights and values": [dict(pv=SIX[:x] + SIX[x + 1:]) for x in range(6)],
            "logits": [dict(parts=(2, 3, 3, 3)), dict(parts=(3, 2, 3, 3)), dict(pairs=SIX[:1] + SIX[2:]),
                       dict(pairs=SIX[1:]), dict(pairs=SIX[:2] + SIX[3:])]}
    for name, q, k, v, window, bar in cases(300, 32):
        assert worst(name, emulate(q, k, v, window), q, k, v, window, bar) <= 0.5
        for loss in lost[name]:
            assert worst(f"{name} {loss}", emulate(q, k, v, window, **loss), q, k, v, window, bar) > 2


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("n", [300, 1500])
def test_encode_fp32_keeps_its_bits(n, dim):
    """In blocks of their own rows (300) and with waves that share a row's keys (1500, all events in the window)."""
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    for name, q, k, v, window, bar in cases(n, dim):
        got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), off, window=window, scale=1.0)
        assert worst(name, got[:, 0].cpu().double().numpy(), q, k, v, window, bar) <= 1
    if n > 1000:
        # every event is seen, but all logits save two are far below: the same two weights
        q, k = torch.zeros((n, 1, dim)), torch.zeros((n, 1, dim))
        q[:, 0, 0], q[:, 0, 1] = 20 + draws(n, 7) / 32, 20 + draws(n, 8) / 32
        k[:, 0, 0] = -20
        k[3, 0, 0], k[900, 0, 0] = 20 + draws(1, 9).item() / 32, 0
        k[900, 0, 1] = 20 + draws(1, 10).item() / 32
        v = torch.zeros((n, 1, dim))
        v[900] = 1
        got = dl.history_attention(q.cuda(), k.cuda(), v.cuda(), off, scale=1.0)
        assert worst("logits far apart", got[:, 0].cpu().double().numpy(), q, k, v, n, (16 + 6 * 410) * U) <= 1


# --- lookup: the queries and the weights are cut into parts, the codes are exact -------


def lookup_cases(dim):
    """(name, q, k, v, bar) of two events; keys and values are codes."""
    rows = 200
    q, k, v = torch.zeros((rows, dim)), torch.zeros((2, 1, dim)), torch.ones((2, 1, dim))
    q[:, 0], q[:, dim - 1] = 400 + draws(rows, 11), 400 + draws(rows, 12)
    k[0, 0, 0] = k[1, 0, dim - 1] = 1
    return [("weights", q, k, v, 16 * U), ("logits", q, k, v * torch.tensor([0.0, 1.0])[:, None, None],
                                           (16 + 6 * 402) * U)]


def lookup_exact(q, k, v, parts=(3, 3)):
    a = sum(split(q, parts[0], True)) if parts[0] < 3 else q.double().numpy()
    s = a @ k[:, 0].double().numpy().T
    w = np.exp(s - s.max(1, keepdims=True)).astype(np.float32)
    p = sum(split(torch.from_numpy(w), parts[1], True))
    return p @ v[:, 0].double().numpy() / w.astype(np.float64).sum(1, keepdims=True)


def test_lookup_bars_fail_for_a_lost_part():
    for name, q, k, v, bar in lookup_cases(32):
        want = lookup_exact(q, k, v)
        for parts in ((2, 3), (3, 2)):
            e = np.abs(lookup_exact(q, k, v, parts) - want).max() / bar
            print(f"{name} {parts}: {e:.2f}")
            assert (e > 2) == (parts == ((3, 2) if name == "weights" else (2, 3))), (name, parts)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("room", [2, 200])
def test_lookup_fp32_keeps_its_bits(dim, room):
    """In one launch (a table of 2 pages) and in two (room for 200)."""
    for name, q, k, v, bar in lookup_cases(dim):
        c = dl.HistoryCache(4, 1, room, 1, dim, 64)
        c.append(k.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int64, device="cuda"))
        got = c.lookup(q.view(1, -1, 1, dim).cuda(), scale=1.0)[0, :, 0].cpu().double().numpy()
        s = q.double().numpy() @ k[:, 0].double().numpy().T
        w = np.exp(s - s.max(1, keepdims=True))
        e = np.abs(got - w @ v[:, 0].double().numpy() / w.sum(1, keepdims=True)).max() / bar
        print(f"{name}: worst error / bar {e:.3f}", flush=True)
        assert e <= 1
