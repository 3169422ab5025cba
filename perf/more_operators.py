"""Cases of the calls that continue event histories with beams: the selection of a group's best continuations, the
reordering of its histories in the 8-bit paged cache, and the lookup of histories that share a prefix.

Each case has a plain form in elementary torch operations and the library's own calls (``own``).
"""
import math
import random

import numpy as np
import torch

own = False

PAGE_FLOOR = -100          # smallest exponent of a block's scale
ALL_EVENTS = 1 << 30
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# --- cases -------------------------------------------------------------------------


def listed():
    return [
        # one small request: a few users, a few beams each, over the items of the ranking example
        dict(name="select few f32", kind="select", dtype="float32", batch=4, beams=4, items=5000, keep=4,
             allowed="none", ended=False, fill=1),
        # a serving batch of beams over the rows of one embedding table
        dict(name="select beams bf16", kind="select", dtype="bfloat16", batch=64, beams=8, items=100000, keep=8,
             allowed="none", ended=False, fill=2),
        # wide beams over a catalogue of odd size, some beams ended, items that each beam may not take
        dict(name="select wide f16", kind="select", dtype="float16", batch=16, beams=64, items=20011, keep=64,
             allowed="each", ended=True, fill=3),
        # retrieval: the best hundred of a million items for each user, one beam, items out of stock left out
        dict(name="select retrieval f32", kind="select", dtype="float32", batch=128, beams=1, items=1000000, keep=100,
             allowed="all", ended=False, fill=4),
        # one step of the smallest request on the cache: beams reordered, an event behind each
        dict(name="step few f32", kind="step", dtype="float32", users=4, beams=4, max_len=100, kv_heads=2, dim=32,
             page=16, fill=5),
        # one step of a serving batch
        dict(name="step batch bf16", kind="step", dtype="bfloat16", users=64, beams=8, max_len=2000, kv_heads=8, dim=64,
             page=64, fill=6),
        # wide beams over long histories on small pages: long page lists
        dict(name="step wide f16", kind="step", dtype="float16", users=16, beams=64, max_len=8000, kv_heads=4, dim=64,
             page=16, fill=7),
        # the smallest request: beams of a few users with short histories
        dict(name="shared few f32", kind="shared", dtype="float32", users=4, members=4, ragged=False, max_len=200,
             tail=4, queries=1, heads=4, kv_heads=4, dim=32, page=16, window=ALL_EVENTS, sinks=0, fill=8),
        # a serving batch of beams, all of each history read
        dict(name="shared beams bf16", kind="shared", dtype="bfloat16", users=64, members=8, ragged=False, max_len=8000,
             tail=12, queries=1, heads=16, kv_heads=4, dim=64, page=32, window=ALL_EVENTS, sinks=0, fill=9),
        # sessions opened on stored histories, as many as came, each with events of its own; a window and the profile
        dict(name="shared sessions f16", kind="shared", dtype="float16", users=96, members=32, ragged=True, max_len=4000,
             tail=150, queries=1, heads=8, kv_heads=8, dim=64, page=16, window=1024, sinks=4, fill=10),
        # a slate of requests behind one common history
        dict(name="shared one bf16", kind="shared", dtype="bfloat16", users=1, members=256, ragged=False, max_len=8192,
             tail=60, queries=2, heads=16, kv_heads=4, dim=128, page=64, window=ALL_EVENTS, sinks=0, fill=11),
        # beams over lifelong histories of a batch of users
        dict(name="shared lifelong bf16", kind="shared", dtype="bfloat16", users=32, members=16, ragged=False,
             max_len=32000, tail=8, queries=1, heads=32, kv_heads=8, dim=128, page=64, window=ALL_EVENTS, sinks=0,
             fill=12),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["select", "select", "step", "shared", "shared"])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    kv = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([32, 64, 128])
    page = rng.choice([16, 32, 64])
    fill = rng.randrange(1 << 20)
    if kind == "select":
        beams = rng.choice([1, 2, 4, 5, 8, 16, 33, 64])
        items = log_int(rng, 60, 400000)
        most = max(1, min(300, 40000000 // (items * beams)))
        return dict(kind=kind, dtype=dtype, batch=log_int(rng, 1, most), beams=beams, items=items,
                    keep=min(items, rng.choice([beams, beams, 2 * beams, log_int(rng, 1, 128)]), 128),
                    allowed=rng.choice(["none", "none", "all", "each"]), ended=rng.random() < 0.3, fill=fill)
    if kind == "step":
        beams = rng.choice([1, 2, 4, 7, 8, 16, 30, 64])
        return dict(kind=kind, dtype=dtype, users=log_int(rng, 1, max(1, min(128, 1024 // beams))), beams=beams,
                    max_len=log_int(rng, 2, 5000), kv_heads=kv, dim=dim, page=page, fill=fill)
    max_len = log_int(rng, 4, 30000)
    group = rng.choice([1, 2, 4, 5])
    members = rng.choice([1, 2, 5, 8, 16, 40, 100])
    queries = rng.choice([1, 1, 1, 3])
    most = max(1, min(200, 2000000000 // (max_len * kv * members * dim * queries)))
    return dict(kind=kind, dtype=dtype, users=log_int(rng, 1, most), members=members, ragged=rng.random() < 0.5,
                max_len=max_len, tail=log_int(rng, 1, 200), queries=queries, heads=kv * group, kv_heads=kv, dim=dim,
                page=page, window=rng.choice([ALL_EVENTS, ALL_EVENTS, log_int(rng, 1, 5000)]),
                sinks=rng.choice([0, 4, 70]), fill=fill)


def ceil_div(a, b):
    return -(-a // b)


def groups_of(case):
    """(shared events, [own events of each member]) of every group, from the case's numbers alone."""
    r = random.Random(case["fill"] * 7 + 3)
    got = []
    for u in range(case["users"]):
        shared = case["max_len"] if u == 0 else r.randint(max(1, case["max_len"] // 4), case["max_len"])
        if case["kind"] == "step":
            got.append((shared, [r.randint(1, 20)] * case["beams"]))
        else:
            n = r.randint(1, case["members"]) if case["ragged"] and u else case["members"]
            got.append((shared, [r.randint(0, case["tail"]) for _ in range(n)]))
    return got


# --- inputs ------------------------------------------------------------------------


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def generator(seed):
    g = torch.Generator(device=device())
    g.manual_seed(int(seed))
    return g


def draw_values(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=device(), dtype=torch.float32) * scale).to(dtype)


def on_device(values, dtype=torch.int32):
    return torch.as_tensor(values, dtype=dtype, device=device())


def make_cache(g, groups, kv, dim, page, spare):
    """A cache whose slots hold the groups' members in order: full pages of the shared events once a group, the page
    that the shared events end in and the pages behind it for each member with events of its own."""
    dev = device()
    lists, need = [], 0
    for shared, own_events in groups:
        common = list(range(need, need + shared // page))
        need += len(common)
        part = None
        for n in own_events:
            if n == 0 and shared % page:
                if part is None:
                    part, need = need, need + 1
                lists.append(common + [part])
                continue
            more = ceil_div(shared + n, page) - len(common)
            lists.append(common + list(range(need, need + more)))
            need += more
    lens = [shared + n for shared, own_events in groups for n in own_events]
    n_pages = need + spare
    max_pages = max(ceil_div(n + 1, page) for n in lens)
    k = torch.empty((n_pages, kv, page, dim), dtype=torch.uint8, device=dev)
    v = torch.empty((n_pages, kv, dim, page), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 26) // (kv * page * dim))
    for a in range(0, n_pages, step):
        for t in (k, v):
            part = t[a:a + step]
            part.copy_((torch.randn(part.shape, generator=g, device=dev) * 100).clamp_(-448, 448)
                       .to(torch.float8_e4m3fn).view(torch.uint8))
    k_scale = torch.exp2(torch.randint(-8, -5, (n_pages, kv), generator=g, device=dev).float())
    v_scale = torch.exp2(torch.randint(-8, -5, (n_pages, kv), generator=g, device=dev).float())
    table = np.full((len(lists), max_pages), -1, dtype=np.int64)
    for i, row in enumerate(lists):
        table[i, :len(row)] = row
    order = torch.cat([torch.randperm(n_pages, generator=g, device=dev), on_device([-1], torch.int64)])
    table = order[on_device(table, torch.int64)]          # -1 takes the last entry, -1
    refs = torch.bincount(table[table >= 0], minlength=n_pages).to(torch.int32)
    c = dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table.to(torch.int32).contiguous(),
             lens=on_device(lens), refs=refs, free_pages=torch.full((n_pages,), -1, dtype=torch.int32, device=dev),
             counters=torch.zeros(4, dtype=torch.int32, device=dev))
    rebuild(c)
    return c


def units_of(rows):
    """The (row, page of the row's new part) pairs that an append of one event each touches."""
    rows = torch.arange(rows, device=device())
    return rows, torch.zeros_like(rows)


def prepare(case, seed):
    g = generator(seed)
    dtype = DTYPES[case["dtype"]]
    st = dict(case=case)
    if case["kind"] == "select":
        batch, beams, items = case["batch"], case["beams"], case["items"]
        logits = torch.empty((batch, beams, items), dtype=dtype, device=device())
        for b in range(0, batch, max(1, (1 << 26) // (beams * items))):
            part = logits[b:b + max(1, (1 << 26) // (beams * items))]
            part.copy_(torch.randn(part.shape, generator=g, device=device()) * 2.5)
        st["logits"] = logits
        st["scores"] = None
        if beams > 1:                                     # sums of log-probabilities; now and then a beam without one
            s = -3 - 2 * torch.rand((batch, beams), generator=g, device=device())
            dead = torch.rand((batch, beams), generator=g, device=device()) < 0.03
            dead[:, 0] = False
            st["scores"] = s.masked_fill(dead, float("-inf"))
        st["allowed"] = None
        if case["allowed"] != "none":
            shape = (items,) if case["allowed"] == "all" else (batch, beams, items)
            st["allowed"] = torch.rand(shape, generator=g, device=device()) < 0.9
        st["ended"] = None
        if case["ended"]:
            st["ended"] = torch.rand((batch, beams), generator=g, device=device()) < 0.15
        return st
    groups = groups_of(case)
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    rows = sum(len(m) for _, m in groups)
    if case["kind"] == "step":
        held = [shared + n for shared, m in groups for n in m]
        st["cache"] = make_cache(g, groups, kv, dim, page, 2 * rows + 5)
        # the parents of a step: the better beams have more successors
        parents = (torch.rand((case["users"], case["beams"]), generator=g, device=device()) ** 2 * case["beams"])
        st.update(parents=parents.to(torch.int32).clamp(max=case["beams"] - 1),
                  slots=torch.arange(rows, dtype=torch.int32, device=device()).reshape(case["users"], case["beams"]),
                  held=on_device(held), offsets=torch.arange(rows, dtype=torch.int64, device=device()),
                  k=draw_values((rows, kv, dim), g, dtype, 2.0), v=draw_values((rows, kv, dim), g, dtype, 0.5),
                  units=units_of(rows))
        return st
    st["cache"] = make_cache(g, groups, kv, dim, page, 3)
    st["q"] = draw_values((rows, case["queries"], case["heads"], dim), g, dtype)
    starts = np.cumsum([0] + [len(m) for _, m in groups])[:-1]
    st["groups"] = on_device(starts) if case["ragged"] else case["members"]
    return st


# --- plain forms -------------------------------------------------------------------


def plain_select(st):
    """Scores in 64 bits: the order is decided by them, and neighbours may lie closer than 32 bits tell apart."""
    case = st["case"]
    batch, beams, items, keep = case["batch"], case["beams"], case["items"], case["keep"]
    x = st["logits"].double()
    if st["allowed"] is not None:
        x = x.masked_fill(~st["allowed"], -math.inf)
    m = x.amax(-1, keepdim=True)
    usable = m.abs() < math.inf
    m = torch.where(usable, m, torch.zeros_like(m))
    x = x - m
    x = x - torch.log(torch.exp(x).sum(-1, keepdim=True))
    if st["scores"] is not None:
        x = x + st["scores"].double()[..., None]
    x = x.masked_fill(~usable, -math.inf)
    if st["ended"] is not None:
        x = x.masked_fill(st["ended"][..., None], -math.inf)
        x[..., 0] = torch.where(st["ended"], st["scores"].double() if st["scores"] is not None else
                                torch.zeros_like(x[..., 0]), x[..., 0])
    s, at = torch.sort(x.reshape(batch, beams * items), dim=1, descending=True, stable=True)
    s, at = s[:, :keep], at[:, :keep]
    none = s == -math.inf
    parent, item = at // items, at % items
    if st["ended"] is not None:
        item = item.masked_fill(st["ended"].gather(1, parent), -1)
    return dict(scores=s.float(), parents=parent.masked_fill(none, -1).to(torch.int32),
                items=item.masked_fill(none, -1).to(torch.int32))


def rebuild(c):
    """The free list: the pages without a holder, in descending order."""
    ids = torch.arange(c["refs"].numel(), dtype=torch.int32, device=c["refs"].device)
    free = c["refs"] == 0
    c["free_pages"].copy_(torch.sort(torch.where(free, ids, torch.full_like(ids, -1)), descending=True)[0])
    c["counters"][0] = free.sum()


def holders(c, rows, sign):
    """One holder more or less for every page that the table rows name."""
    c["refs"].scatter_add_(0, rows.clamp(min=0).long().reshape(-1), sign * (rows >= 0).to(torch.int32).reshape(-1))


def plain_truncate(c, slots, new_lens):
    page = c["k"].shape[2]
    rows = c["table"][slots]
    at = torch.arange(rows.shape[1], device=rows.device)
    drop = (at[None, :] >= ((new_lens.long() + page - 1) // page)[:, None]) & (rows >= 0)
    holders(c, torch.where(drop, rows, torch.full_like(rows, -1)), -1)
    c["table"][slots] = torch.where(drop, torch.full_like(rows, -1), rows)
    c["lens"][slots] = new_lens
    rebuild(c)


def plain_reorder(c, slots, parents):
    src = torch.gather(slots, 1, parents.long()).reshape(-1)
    slots = slots.reshape(-1)
    old, rows, lens = c["table"][slots], c["table"][src], c["lens"][src]
    holders(c, old, -1)
    holders(c, rows, 1)
    c["table"][slots] = rows
    c["lens"][slots] = lens
    rebuild(c)


def needed_scale(amax):
    """The smallest power of two 2^e, e >= PAGE_FLOOR, with amax / 2^e <= 448."""
    f, x = torch.frexp(amax)
    e = x - 9 + (f > 0.875).to(x.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, PAGE_FLOOR)).clamp(min=PAGE_FLOOR)
    return torch.ldexp(torch.ones_like(amax), e)


def to_codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def plain_append(c, slots, k, v, off, units):
    """Events behind the histories `slots`; the free list holds enough pages."""
    page = c["k"].shape[2]
    row, nth = units
    total = k.shape[0]
    ends = torch.cat([off[1:], off.new_full((1,), total)])
    count = ends - off
    old = c["lens"][slots].long()
    new = old + count
    first = old // page
    part = (old % page) > 0
    p_old = c["table"][slots, first.clamp(max=c["table"].shape[1] - 1)].clamp(min=0).long()
    shared = part & (c["refs"][p_old] > 1) & (count > 0)
    kept = part & ~shared
    need = (new + page - 1) // page - (old + page - 1) // page + shared.long()
    before = torch.cumsum(need, 0) - need
    taken = c["counters"][0].long() - 1 - (before[row] + nth - kept[row].long())
    keeps = kept[row] & (nth == 0)
    dst = torch.where(keeps, p_old[row], c["free_pages"][taken.clamp(min=0)].long())
    has_old = part[row] & (nth == 0)
    src = torch.where(has_old, p_old[row], dst)
    pos = ((first[row] + nth) * page)[:, None] + torch.arange(page, device=off.device)[None, :]
    is_new = (pos >= old[row][:, None]) & (pos < new[row][:, None])
    is_old = pos < old[row][:, None]
    event = (off[row] - old[row])[:, None] + pos
    event = torch.where(is_new, event, torch.zeros_like(event)).clamp(0, max(0, total - 1))
    for codes, scales, x, minor in ((c["k"], c["k_scale"], k, False), (c["v"], c["v_scale"], v, True)):
        val = x[event].float().transpose(1, 2)                       # (units, kv, page, dim)
        wn, wo = is_new[:, None, :, None], is_old[:, None, :, None]
        val = torch.where(wn, val, torch.zeros_like(val))
        was = torch.where(has_old[:, None], scales[src], torch.full_like(scales[src], 2.0 ** PAGE_FLOOR))
        s = torch.maximum(was, needed_scale(val.abs().amax((2, 3))))
        held = codes[src].transpose(2, 3) if minor else codes[src]
        stale = codes[dst].transpose(2, 3) if minor else codes[dst]
        moved = to_codes(held.view(torch.float8_e4m3fn).float() * (was / s)[:, :, None, None])
        out = torch.where(wn, to_codes(val / s[:, :, None, None]), torch.where(wo, moved, stale))
        codes[dst] = out.transpose(2, 3).contiguous() if minor else out
        scales[dst] = s
    c["refs"].scatter_add_(0, p_old, -shared.to(torch.int32))
    c["refs"].scatter_add_(0, dst, (~keeps).to(torch.int32))
    c["table"][slots[row], first[row] + nth] = dst.to(torch.int32)
    c["counters"][0] -= need.sum().to(torch.int32)
    c["lens"][slots] = new.to(torch.int32)


def soft(s, seen):
    """Softmax weights over the last axis where `seen`; rows without any are zero."""
    s = s.masked_fill(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def plain_shared(st):
    """Every row's whole history gathered and attended to, so many rows at a time as fit."""
    case, c, q = st["case"], st["cache"], st["q"]
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    batch, queries, heads, _ = q.shape
    out = torch.empty_like(q)
    span = c["table"].shape[1] * page
    some = max(1, (1 << 28) // (kv * span * dim))
    for b in range(0, batch, some):
        rows = c["table"][b:b + some].clamp(min=0).long()
        n = rows.shape[0]
        k = c["k"][rows].view(torch.float8_e4m3fn).float() * c["k_scale"][rows][..., None, None]
        k = k.transpose(1, 2).reshape(n, kv, span, dim)
        lens = c["lens"][b:b + some].long()[:, None]
        at = torch.arange(span, device=q.device)[None, :]
        seen = (at < lens) & ((at >= lens - case["window"]) | (at < case["sinks"]))
        qq = q[b:b + some].float().reshape(n, queries, kv, heads // kv, dim).transpose(1, 2).reshape(n, kv, -1, dim)
        p = soft(torch.matmul(k, qq.transpose(2, 3).contiguous()).transpose(2, 3).contiguous() * dim ** -0.5,
                 seen[:, None, None, :])
        del k
        v = c["v"][rows].view(torch.float8_e4m3fn).float() * c["v_scale"][rows][..., None, None]
        v = v.permute(0, 2, 1, 4, 3).reshape(n, kv, span, dim)
        o = torch.matmul(p, v).reshape(n, kv, queries, heads // kv, dim).transpose(1, 2)
        del v
        out[b:b + some] = o.reshape(n, queries, heads, dim).to(q.dtype)
    return out


# --- one pass ----------------------------------------------------------------------


def cache_outputs(c):
    n_free = c["counters"][0]
    at = torch.arange(c["free_pages"].numel(), device=n_free.device)
    return dict(k=c["k"].view(torch.float8_e4m3fn), v=c["v"].view(torch.float8_e4m3fn), k_scale=c["k_scale"],
                v_scale=c["v_scale"], table=c["table"], lens=c["lens"], refs=c["refs"],
                free=torch.where(at < n_free, c["free_pages"], torch.full_like(c["free_pages"], -1)))


def handle(st):
    """The cache object over the state's buffers, made on first use and kept as a server keeps it."""
    import dlrm_embedding_interaction_amd as dl
    if "handle" not in st:
        st["handle"] = dl.HistoryCache.wrap(**st["cache"])
    return st["handle"]


def run(st):
    case = st["case"]
    if case["kind"] == "select":
        if own:
            import dlrm_embedding_interaction_amd as dl
            scores, parents, items = dl.history_select(st["logits"], st["scores"], keep=case["keep"],
                                                       allowed=st["allowed"], ended=st["ended"])
            return dict(scores=scores, parents=parents, items=items)
        return plain_select(st)
    if case["kind"] == "shared":
        if own:
            return handle(st).lookup_shared(st["q"], st["groups"], window=case["window"], sinks=case["sinks"])
        return plain_shared(st)
    # each pass takes back the events of the last one, then reorders the beams and puts an event behind each
    c, slots = st["cache"], st["slots"].reshape(-1)
    if own:
        h = handle(st)
        h.truncate(slots, st["held"])
        h.reorder(st["parents"], slots=st["slots"])
        h.append(st["k"], st["v"], st["offsets"], slots=slots)
    else:
        plain_truncate(c, slots, st["held"])
        plain_reorder(c, st["slots"].long(), st["parents"])
        plain_append(c, slots, st["k"], st["v"], st["offsets"], st["units"])
    return cache_outputs(c)


# --- what a pass cannot do without -------------------------------------------------


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["kind"] == "select":
        rows, items = case["batch"] * case["beams"], case["items"]
        mask = dict(none=0, all=items, each=rows * items)[case["allowed"]]
        # an exponential, its argument and its sum, the comparison with the best so far, for each logit
        return dict(bytes=rows * items * size + mask + 8 * rows + 12 * case["batch"] * case["keep"],
                    flops=4 * rows * items)
    groups, kv, dim, page = groups_of(case), case["kv_heads"], case["dim"], case["page"]
    if case["kind"] == "step":
        # page lists read and written, the filled part of a last page that is shared copied (half of them, say), events
        rows = [shared + n for shared, m in groups for n in m]
        lists = sum(ceil_div(n, page) for n in rows)
        copied = 2 * 2 * kv * dim * sum(n % page for n in rows) // 2
        return dict(bytes=8 * lists + copied + 2 * len(rows) * kv * dim * (size + 1), flops=8 * len(rows) * kv * dim)
    total, flops, count = 0, 0, 0
    rows = case["queries"] * case["heads"]
    for shared, own_events in groups:
        lows = [max(0, shared + n - case["window"]) for n in own_events]
        seen = [shared + n - low + min(case["sinks"], low) for n, low in zip(own_events, lows)]
        low, lead = min(lows), min(case["sinks"], min(max(lows), shared))
        common = max(0, shared - low) + min(lead, low)
        alone = sum(min(n, case["window"]) for n in own_events)
        total += common + alone
        flops += 4 * dim * rows * sum(seen)
        count += len(own_events)
    return dict(bytes=2 * dim * kv * total + 8 * kv * ceil_div(total, page) + 2 * size * dim * rows * count, flops=flops)


# --- the definition, in 64 bits ----------------------------------------------------


def exact(case, seed):
    if case["kind"] == "select" and case["batch"] * case["beams"] * case["items"] > 3 * 10 ** 8:
        return None
    st = prepare(case, seed)
    if case["kind"] == "select":
        return exact_select(case, st)
    groups = groups_of(case)
    if case["kind"] == "shared":
        return exact_shared(case, st, groups)
    book = Book(st["cache"])
    k, v, parents = st["k"].double(), st["v"].double(), st["parents"].tolist()
    beams = case["beams"]
    for u in range(case["users"]):
        book.reorder(range(u * beams, (u + 1) * beams), parents[u])
    shared = {p for p, n in book.refs.items() if n > 1}
    book.free = sorted(p for p, n in book.refs.items() if not n)
    for i in range(case["users"] * beams):
        book.append(i, k[i], v[i], shared)
    return dict(k=book.k, v=book.v, k_scale=book.k_scale, v_scale=book.v_scale, table=None, lens=None, refs=None,
                free=None)


def exact_select(case, st):
    batch, beams, items, keep = case["batch"], case["beams"], case["items"], case["keep"]
    scores, parents, kept = [], [], []
    for b in range(batch):
        rows = []
        for w in range(beams):
            start = 0.0 if st["scores"] is None else st["scores"][b, w].double()
            if st["ended"] is not None and st["ended"][b, w]:
                row = torch.full((items,), -math.inf, dtype=torch.float64, device=st["logits"].device)
                row[0] = start
            else:
                row = st["logits"][b, w].double()
                if st["allowed"] is not None:
                    may = st["allowed"] if st["allowed"].dim() == 1 else st["allowed"][b, w]
                    row = torch.where(may, row, torch.full_like(row, -math.inf))
                row = torch.log_softmax(row, 0) + start
            rows.append(row)
        every = torch.cat(rows)
        worst = torch.topk(every, min(keep, every.numel()))[0][-1]
        at = torch.nonzero(every >= worst)[:, 0].cpu().numpy()       # rising: ties go to the lowest
        val = every[torch.as_tensor(at, device=every.device)].cpu().numpy()
        first = np.argsort(-val, kind="stable")[:keep]
        at, val = at[first], val[first]
        none = ~(val > -math.inf)
        over = np.zeros(len(at), bool) if st["ended"] is None else st["ended"][b].cpu().numpy()[at // items]
        scores.append(np.pad(val, (0, keep - len(at)), constant_values=-math.inf))
        parents.append(np.pad(np.where(none, -1, at // items), (0, keep - len(at)), constant_values=-1))
        kept.append(np.pad(np.where(none | over, -1, at % items), (0, keep - len(at)), constant_values=-1))
    return dict(scores=torch.from_numpy(np.stack(scores)), parents=torch.from_numpy(np.stack(parents)),
                items=torch.from_numpy(np.stack(kept)))


def exact_shared(case, st, groups):
    c, q = st["cache"], st["q"].double()
    out = torch.zeros_like(q)
    kv, page, dim = case["kv_heads"], case["page"], case["dim"]
    group = case["heads"] // kv
    lens = [shared + n for shared, m in groups for n in m]
    for b, n in enumerate(lens):
        pos = torch.arange(n, device=q.device)
        pos = pos[(pos >= n - case["window"]) | (pos < case["sinks"])]
        p, r = c["table"][b].long()[pos // page], pos % page
        k = c["k"][p, :, r].view(torch.float8_e4m3fn).double() * c["k_scale"][p].double()[..., None]      # (n, kv, dim)
        v = c["v"][p, :, :, r].view(torch.float8_e4m3fn).double() * c["v_scale"][p].double()[..., None]
        for h in range(kv):
            x = q[b, :, h * group:(h + 1) * group].reshape(-1, dim)
            w = torch.softmax(x @ k[:, h].T / math.sqrt(dim), 1)
            out[b, :, h * group:(h + 1) * group] = (w @ v[:, h]).reshape(case["queries"], group, dim)
    return out


def e4m3(x):
    """The nearest e4m3 value, ties to the even one; |x| <= 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40)))
    e = torch.where(torch.exp2(e) > x.abs(), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= x.abs(), e + 1, e).clamp(min=-6)
    return torch.round(x / torch.exp2(e - 3)) * torch.exp2(e - 3)


class Book:
    """A cache kept by hand, one history after the other: page lists on the host, values in 64 bits."""

    def __init__(self, c):
        self.page = c["k"].shape[2]
        self.k = c["k"].view(torch.float8_e4m3fn).double()
        self.v = c["v"].view(torch.float8_e4m3fn).double()
        self.k_scale, self.v_scale = c["k_scale"].double(), c["v_scale"].double()
        self.lists = [[p for p in row if p >= 0] for row in c["table"].tolist()]
        self.lens = c["lens"].tolist()
        self.refs = dict(enumerate([0] * self.k.shape[0]))
        for row in self.lists:
            for p in row:
                self.refs[p] += 1
        self.free = []

    def reorder(self, slots, parents):
        lists, lens = [list(self.lists[slots[p]]) for p in parents], [self.lens[slots[p]] for p in parents]
        for s, row, n in zip(slots, lists, lens):
            for p in self.lists[s]:
                self.refs[p] -= 1
            for p in row:
                self.refs[p] += 1
            self.lists[s], self.lens[s] = row, n

    def append(self, slot, k, v, shared):
        """One event (kv, dim)."""
        pages, (nth, a) = self.lists[slot], divmod(self.lens[slot], self.page)
        old = pages[nth] if a else None
        if a and old not in shared:
            p = old
        else:
            p = self.free.pop(0)
            self.refs[p] = 1
            if a:
                self.refs[old] -= 1
                pages[nth] = p
            else:
                pages.append(p)
        for codes, scales, x, minor in ((self.k, self.k_scale, k, False), (self.v, self.v_scale, v, True)):
            amax = x.abs().amax(1).clamp(min=2.0 ** -130)
            e = torch.ceil(torch.log2(amax / 448))
            e = torch.where(amax / 448 <= torch.exp2(e - 1), e - 1, e)
            e = torch.where(amax / 448 > torch.exp2(e), e + 1, e)
            s = torch.exp2(e.clamp(min=PAGE_FLOOR))
            part = codes[p].transpose(1, 2) if minor else codes[p]
            if a:
                s = torch.maximum(s, scales[old])
                was = codes[old].transpose(1, 2) if minor else codes[old]
                part[:, :a] = e4m3(was[:, :a] * (scales[old] / s)[:, None, None])
            part[:, a] = e4m3(x / s[:, None])
            scales[p] = s
        self.lens[slot] += 1
