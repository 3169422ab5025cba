"""Cases of the event-history operators: windowed attention over ragged histories, the 8-bit paged
history cache (append and lookup) and the management of its pages.

Each case has a plain form in elementary torch operations and the library's own calls (``own``).
"""
import math
import random

import torch

own = False

PAGE_FLOOR = -100          # smallest exponent of a block's scale
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# --- cases -------------------------------------------------------------------------


def listed():
    return [
        # the bag of 20 recent items of the multi-hot workload, attended to instead of summed: one small request
        dict(name="encode bag20 f32", kind="encode", dtype="float32", batch=64, max_len=20, heads=2, kv_heads=2,
             dim=32, window=20, sinks=0, padded=False, fill=1),
        # a ranking batch: a few hundred users' recent histories, a short window and the profile events in front
        dict(name="encode users bf16", kind="encode", dtype="bfloat16", batch=256, max_len=512, heads=4, kv_heads=4,
             dim=64, window=128, sinks=4, padded=False, fill=2),
        # longer histories with removed (padding) events, heads shared in groups of four
        dict(name="encode grouped f16", kind="encode", dtype="float16", batch=32, max_len=2048, heads=16, kv_heads=4,
             dim=128, window=512, sinks=5, padded=True, fill=3),
        # lifelong histories, encoded once when a user's cache is filled
        dict(name="encode lifelong bf16", kind="encode", dtype="bfloat16", batch=2, max_len=12001, heads=8,
             kv_heads=2, dim=128, window=4096, sinks=16, padded=False, fill=4),
        # one new event for each of the users of a batch
        dict(name="append events bf16", kind="append", dtype="bfloat16", batch=512, old_len=1000, new_len=1,
             kv_heads=4, dim=64, page=16, fill=5),
        # whole histories written behind the encoder
        dict(name="append histories bf16", kind="append", dtype="bfloat16", batch=128, old_len=0, new_len=1000,
             kv_heads=8, dim=128, page=64, fill=6),
        # the smallest request: a few users with short histories, fp32 like the Linear layers around it
        dict(name="lookup few f32", kind="lookup", dtype="float32", batch=4, max_len=200, queries=1, heads=4,
             kv_heads=4, dim=32, page=16, window=1 << 30, sinks=0, fill=7),
        # a batch of users, a window over long histories
        dict(name="lookup window bf16", kind="lookup", dtype="bfloat16", batch=256, max_len=8000, queries=1, heads=16,
             kv_heads=4, dim=64, page=32, window=1024, sinks=4, fill=8),
        # a slate of candidates for each user, every candidate a query of the same history
        dict(name="lookup candidates f16", kind="lookup", dtype="float16", batch=96, max_len=1500, queries=12,
             heads=4, kv_heads=4, dim=64, page=16, window=1 << 30, sinks=0, fill=9),
        # lifelong histories of a batch of users, all of them read
        dict(name="lookup lifelong bf16", kind="lookup", dtype="bfloat16", batch=128, max_len=32000, queries=1,
             heads=32, kv_heads=8, dim=128, page=64, window=1 << 30, sinks=0, fill=10),
        # a few sessions opened on stored histories, one event each, half of them closed, the pool compacted
        dict(name="pages few", kind="pages", dtype="float32", users=8, max_len=100, sessions=13, kv_heads=2, dim=32,
             page=16, fill=11),
        # the same for a large batch of sessions
        dict(name="pages batch", kind="pages", dtype="bfloat16", users=256, max_len=2000, sessions=1500, kv_heads=8,
             dim=64, page=64, fill=12),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["encode", "encode", "append", "lookup", "lookup", "pages"])
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([32, 64, 128])
    page = rng.choice([16, 32, 64])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    fill = rng.randrange(1 << 20)
    if kind == "encode":
        max_len = log_int(rng, 3, 10000)
        most = max(1, min(300, int(3.0e7 / max_len / max_len * 32 / (kv * group))))
        return dict(kind=kind, dtype=dtype, batch=log_int(rng, 1, most), max_len=max_len, heads=kv * group,
                    kv_heads=kv, dim=dim, window=log_int(rng, 1, 2 * max_len), sinks=rng.choice([0, 1, 4, 70]),
                    padded=rng.random() < 0.4, fill=fill)
    if kind == "append":
        new_len = log_int(rng, 1, 1000)
        return dict(kind=kind, dtype=dtype, batch=log_int(rng, 1, max(1, min(700, 60000 // new_len))),
                    old_len=rng.choice([0, log_int(rng, 1, 1500)]), new_len=new_len, kv_heads=kv, dim=dim, page=page,
                    fill=fill)
    if kind == "lookup":
        max_len = log_int(rng, 2, 30000)
        most = max(1, min(600, 4000000 * 8 // (max_len * kv)))
        return dict(kind=kind, dtype=dtype, batch=log_int(rng, 1, most), max_len=max_len,
                    queries=rng.choice([1, 1, 1, 3, 20]), heads=kv * group, kv_heads=kv, dim=dim, page=page,
                    window=rng.choice([1 << 30, log_int(rng, 1, 5000)]), sinks=rng.choice([0, 4, 33]), fill=fill)
    return dict(kind=kind, dtype=dtype, users=log_int(rng, 1, 256), max_len=log_int(rng, 1, 1500),
                sessions=log_int(rng, 2, 1000), kv_heads=kv, dim=dim, page=page, fill=fill)


def lengths(case, count, most, salt=0, empty=True):
    """Ragged lengths of a case: up to `most`, one of them `most`, about one in sixteen empty."""
    r = random.Random(case["fill"] * 7 + salt)
    got = [0 if empty and r.random() < 1 / 16 else r.randint(max(1, most // 4), most) for _ in range(count)]
    got[r.randrange(count)] = most
    return got


def ceil_div(a, b):
    return -(-a // b)


# --- inputs ------------------------------------------------------------------------


def device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def generator(seed):
    g = torch.Generator(device=device())
    g.manual_seed(int(seed))
    return g


def draw_values(shape, g, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=device(), dtype=torch.float32) * scale).to(dtype)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=device())


def offsets_of(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at[:-1], dtype=torch.int64, device=device()), at[-1]


def make_cache(g, held, kv, dim, page, n_pages, n_slots, max_pages, dense=False):
    """A cache whose slot i holds held[i] events on pages drawn at random: from all, or (dense) from the first ones."""
    dev = device()
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
    need = [ceil_div(n, page) for n in held]
    order = torch.randperm(sum(need) if dense else n_pages, generator=g, device=dev)[:sum(need)].to(torch.int32)
    table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=dev)
    rows = torch.tensor([i for i, c in enumerate(need) for _ in range(c)], dtype=torch.int64, device=dev)
    cols = torch.tensor([j for c in need for j in range(c)], dtype=torch.int64, device=dev)
    table[rows, cols] = order
    lens = torch.zeros(n_slots, dtype=torch.int32, device=dev)
    lens[:len(held)] = i32(held)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    refs[order.long()] = 1
    c = dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table, lens=lens, refs=refs,
             free_pages=torch.full((n_pages,), -1, dtype=torch.int32, device=dev),
             counters=torch.zeros(4, dtype=torch.int32, device=dev))
    rebuild(c)
    return c


def units_of(old, new, page):
    """The (row, page of the row's new part) pairs that an append touches."""
    rows, nth = [], []
    for b, (o, n) in enumerate(zip(old, new)):
        count = ceil_div(o + n, page) - o // page if n else 0
        rows += [b] * count
        nth += range(count)
    return (torch.tensor(rows, dtype=torch.int64, device=device()),
            torch.tensor(nth, dtype=torch.int64, device=device()))


def shape_of(case):
    """The sizes of a case that follow from its numbers alone."""
    kind = case["kind"]
    if kind == "encode":
        return dict(lens=lengths(case, case["batch"], case["max_len"]))
    if kind == "append":
        old = lengths(case, case["batch"], case["old_len"]) if case["old_len"] else [0] * case["batch"]
        new = [1] * case["batch"] if case["new_len"] == 1 else lengths(case, case["batch"], case["new_len"], 1)
        return dict(old=old, new=new)
    if kind == "lookup":
        return dict(lens=lengths(case, case["batch"], case["max_len"]))
    held = lengths(case, case["users"], case["max_len"], empty=False)
    r = random.Random(case["fill"] + 1)
    src = [r.randrange(case["users"]) for _ in range(case["sessions"])]
    return dict(held=held, src=src)


def prepare(case, seed):
    g = generator(seed)
    s = shape_of(case)
    dtype = DTYPES[case["dtype"]]
    kv, dim = case["kv_heads"], case["dim"]
    st = dict(case=case)
    if case["kind"] == "encode":
        off, n = offsets_of(s["lens"])
        st.update(q=draw_values((n, case["heads"], dim), g, dtype), k=draw_values((n, kv, dim), g, dtype),
                  v=draw_values((n, kv, dim), g, dtype), offsets=off,
                  padding=(torch.rand(n, generator=g, device=device()) < 0.1).to(torch.uint8)
                  if case["padded"] else None)
        return st
    page = case["page"]
    if case["kind"] == "append":
        width = max(ceil_div(o + n, page) for o, n in zip(s["old"], s["new"]))
        pages = sum(ceil_div(o + n, page) for o, n in zip(s["old"], s["new"])) + 7
        off, n = offsets_of(s["new"])
        st["cache"] = make_cache(g, s["old"], kv, dim, page, pages, case["batch"], width)
        st.update(k=draw_values((n, kv, dim), g, dtype, 2.0), v=draw_values((n, kv, dim), g, dtype, 0.5), offsets=off,
                  slots=torch.arange(case["batch"], dtype=torch.int32, device=device()),
                  held=i32(s["old"]), units=units_of(s["old"], s["new"], page))
        return st
    if case["kind"] == "lookup":
        width = ceil_div(max(s["lens"]), page)
        pages = sum(ceil_div(n, page) for n in s["lens"]) + 3
        st["cache"] = make_cache(g, s["lens"], kv, dim, page, pages, case["batch"], width)
        st["q"] = draw_values((case["batch"], case["queries"], case["heads"], dim), g, dtype)
        return st
    # pages: users' histories in slots [0, users), sessions behind them
    users, sessions = case["users"], case["sessions"]
    held = s["held"]
    width = ceil_div(max(held) + 1, page)
    pages = sum(ceil_div(n, page) for n in held) + 2 * sessions + 5
    c = make_cache(g, held, kv, dim, page, pages, users + sessions, width, dense=True)
    st["cache"] = c
    st.update(src=i32(s["src"]), dst=i32([users + i for i in range(sessions)]),
              closed=i32([users + i for i in range(0, sessions, 2)]),
              k=draw_values((sessions, kv, dim), g, dtype, 2.0), v=draw_values((sessions, kv, dim), g, dtype, 0.5),
              offsets=torch.arange(sessions, dtype=torch.int64, device=device()),
              units=units_of([held[i] for i in s["src"]], [1] * sessions, page))
    return st


# --- plain forms -------------------------------------------------------------------


def soft(s, seen):
    """Softmax weights over the last axis where `seen`; rows without any are zero."""
    s = s.masked_fill(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def plain_encode(st):
    case, off = st["case"], st["offsets"]
    n, heads, dim = st["q"].shape
    group = heads // case["kv_heads"]
    length = case["max_len"]
    ends = torch.cat([off[1:], off.new_full((1,), n)])
    lens = ends - off
    at = torch.arange(length, device=off.device)
    live = at[None, :] < lens[:, None]
    rows = torch.where(live, off[:, None] + at[None, :], torch.zeros_like(at)[None, :])

    def spread(x):
        return x[rows].float().transpose(1, 2)

    q, k, v = spread(st["q"]), spread(st["k"]), spread(st["v"])
    k, v = (x.repeat_interleave(group, dim=1) if group > 1 else x.contiguous() for x in (k, v))
    s = torch.matmul(q.contiguous(), k.transpose(2, 3)) * dim ** -0.5
    back = at[:, None] - at[None, :]
    seen = (back >= 0) & ((back < case["window"]) | (at[None, :] < case["sinks"]))
    seen = seen[None] & live[:, None, :]
    if st["padding"] is not None:
        seen = seen & (st["padding"][rows] == 0)[:, None, :]
    p = soft(s, seen[:, None])
    del s
    o = torch.matmul(p, v).transpose(1, 2).reshape(-1, heads, dim)
    token = torch.arange(n, device=off.device)
    b = torch.searchsorted(off, token, right=True) - 1   # the last of the histories that begin there: not an empty one
    return o[b * length + (token - off[b])].to(st["q"].dtype)


def rebuild(c):
    """The free list: the pages without a holder, in descending order."""
    ids = torch.arange(c["refs"].numel(), dtype=torch.int32, device=c["refs"].device)
    free = c["refs"] == 0
    c["free_pages"].copy_(torch.sort(torch.where(free, ids, torch.full_like(ids, -1)), descending=True)[0])
    c["counters"][0] = free.sum()


def plain_truncate(c, slots, new_lens):
    page = c["k"].shape[2]
    slots = slots.long()
    rows = c["table"][slots]
    at = torch.arange(rows.shape[1], device=rows.device)
    drop = (at[None, :] >= ((new_lens.long() + page - 1) // page)[:, None]) & (rows >= 0)
    c["refs"].scatter_add_(0, rows.clamp(min=0).long().reshape(-1), -drop.to(torch.int32).reshape(-1))
    c["table"][slots] = torch.where(drop, torch.full_like(rows, -1), rows)
    c["lens"][slots] = new_lens
    rebuild(c)


def plain_fork(c, src, dst):
    src, dst = src.long(), dst.long()
    old, rows = c["table"][dst], c["table"][src]
    c["refs"].scatter_add_(0, old.clamp(min=0).long().reshape(-1), -(old >= 0).to(torch.int32).reshape(-1))
    c["refs"].scatter_add_(0, rows.clamp(min=0).long().reshape(-1), (rows >= 0).to(torch.int32).reshape(-1))
    c["table"][dst] = rows
    c["lens"][dst] = c["lens"][src]
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
    slots = slots.long()
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


def plain_compact(c, most):
    """The used pages behind the first m move down into the free ones before; at most `most` move."""
    refs = c["refs"]
    n = refs.numel()
    ids = torch.arange(n, dtype=torch.int32, device=refs.device)
    used = refs > 0
    m = used.sum()
    mover, hole = used & (ids >= m), ~used & (ids < m)
    none = torch.full_like(ids, n)
    movers = torch.sort(torch.where(mover, ids, none))[0][:most].long()
    holes = torch.sort(torch.where(hole, ids, none))[0][:most].long()
    remap = torch.cat([ids, ids[:1]])
    remap[movers] = holes.to(torch.int32)
    remap = remap[:n]
    movers, holes = (x.clamp(max=n - 1) for x in (movers, holes))   # past the last: page n - 1, never a hole, to itself
    for t in (c["k"], c["v"], c["k_scale"], c["v_scale"]):
        t[holes] = t[movers]
    table = c["table"]
    c["table"].copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], table))
    counts = torch.zeros_like(refs)
    counts.scatter_add_(0, remap.long(), refs)
    refs.copy_(counts)
    rebuild(c)


def plain_lookup(st):
    case, c = st["case"], st["cache"]
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    q = st["q"]
    batch, queries, heads, _ = q.shape
    rows = c["table"][:batch].clamp(min=0).long()
    span = rows.shape[1] * page
    k = c["k"][rows].view(torch.float8_e4m3fn).float() * c["k_scale"][rows][..., None, None]
    k = k.transpose(1, 2).reshape(batch, kv, span, dim)
    lens = c["lens"][:batch].long()[:, None]
    at = torch.arange(span, device=q.device)[None, :]
    seen = (at < lens) & ((at >= lens - case["window"]) | (at < case["sinks"]))
    qq = q.float().reshape(batch, queries, kv, heads // kv, dim).transpose(1, 2).reshape(batch, kv, -1, dim)
    p = soft(torch.matmul(qq, k.transpose(2, 3)) * dim ** -0.5, seen[:, None, None, :])
    del k
    v = c["v"][rows].view(torch.float8_e4m3fn).float() * c["v_scale"][rows][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(batch, kv, span, dim)
    o = torch.matmul(p, v).reshape(batch, kv, queries, heads // kv, dim).transpose(1, 2)
    return o.reshape(batch, queries, heads, dim).to(q.dtype)


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
    if case["kind"] == "encode":
        if own:
            import dlrm_embedding_interaction_amd as dl
            return dl.history_attention(st["q"], st["k"], st["v"], st["offsets"], window=case["window"],
                                        sinks=case["sinks"], padding=st["padding"])
        return plain_encode(st)
    if case["kind"] == "lookup":
        if own:
            return handle(st).lookup(st["q"], window=case["window"], sinks=case["sinks"])
        return plain_lookup(st)
    c = st["cache"]
    if case["kind"] == "append":
        # each pass takes back what the last one added, then appends
        if own:
            h = handle(st)
            h.truncate(st["slots"], st["held"])
            h.append(st["k"], st["v"], st["offsets"], slots=st["slots"])
        else:
            plain_truncate(c, st["slots"], st["held"])
            plain_append(c, st["slots"], st["k"], st["v"], st["offsets"], st["units"])
        return cache_outputs(c)
    if own:
        h = handle(st)
        h.fork(st["src"], st["dst"])
        h.append(st["k"], st["v"], st["offsets"], slots=st["dst"])
        h.free(st["closed"])
        h.compact()
    else:
        plain_fork(c, st["src"], st["dst"])
        plain_append(c, st["dst"], st["k"], st["v"], st["offsets"], st["units"])
        plain_truncate(c, st["closed"], torch.zeros_like(st["closed"]))
        plain_compact(c, case["sessions"] + case["users"])
    return cache_outputs(c)


# --- what a pass cannot do without -------------------------------------------------


def pairs_of(n, window, sinks):
    """Visible (row, key) pairs of a history of n events."""
    total = 0
    full = min(n, window)
    total += full * (full + 1) // 2 + max(0, n - window) * window
    # sinks before the window: row i sees min(sinks, i - window + 1) more of them
    rest = max(0, n - window)
    lead = min(rest, sinks)
    return total + lead * (lead + 1) // 2 + max(0, rest - sinks) * sinks


def work(case):
    s = shape_of(case)
    size = 4 if case["dtype"] == "float32" else 2
    kv, dim = case["kv_heads"], case["dim"]
    if case["kind"] == "encode":
        n = sum(s["lens"])
        pairs = sum(pairs_of(x, case["window"], case["sinks"]) for x in s["lens"])
        return dict(bytes=size * dim * n * (2 * case["heads"] + 2 * kv) + 8 * len(s["lens"]),
                    flops=4 * dim * case["heads"] * pairs)
    if case["kind"] == "lookup":
        seen = [min(n, case["window"]) + min(case["sinks"], max(0, n - case["window"])) for n in s["lens"]]
        rows = case["queries"] * case["heads"]
        return dict(bytes=2 * dim * kv * sum(seen) + 8 * kv * sum(ceil_div(x, case["page"]) for x in seen) +
                    2 * size * dim * rows * len(seen), flops=4 * dim * rows * sum(seen))
    page = case["page"]
    if case["kind"] == "append":
        n = sum(s["new"])
        touched = sum(ceil_div(o + x, page) - o // page for o, x in zip(s["old"], s["new"]) if x)
        return dict(bytes=2 * n * kv * dim * (size + 1) + touched * (8 * kv + 8), flops=8 * n * kv * dim)
    # a new session reads its user's page list, copies the filled part of the last page and adds an event to it
    tails = [s["held"][u] % page for u in s["src"]]
    lists = sum(ceil_div(s["held"][u], page) for u in s["src"])
    n = case["sessions"]
    copied = 2 * 2 * kv * dim * sum(tails)
    moved = 2 * 2 * kv * dim * page * (n // 2)
    return dict(bytes=copied + moved + 2 * n * kv * dim * (size + 1) + 16 * lists, flops=8 * n * kv * dim)


# --- the definition, in 64 bits ----------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    s = shape_of(case)
    if case["kind"] == "encode":
        return exact_encode(case, st, s["lens"])
    if case["kind"] == "lookup":
        return exact_lookup(case, st, s["lens"])
    book = Book(st["cache"])
    k, v = st["k"].double(), st["v"].double()
    if case["kind"] == "append":
        at = 0
        for b, n in enumerate(s["new"]):
            book.append(b, k[at:at + n], v[at:at + n])
            at += n
    else:
        users = case["users"]
        for i, u in enumerate(s["src"]):
            book.fork(u, users + i)
        shared = {p for p, n in book.refs.items() if n > 1}
        for i in range(case["sessions"]):
            book.append(users + i, k[i:i + 1], v[i:i + 1], shared)
        for i in range(0, case["sessions"], 2):
            book.release(users + i)
        book.compact()
    return dict(k=book.k, v=book.v, k_scale=book.k_scale, v_scale=book.v_scale, table=None, lens=None, refs=None,
                free=None)


def exact_encode(case, st, lens):
    q, k, v = (st[x].double() for x in "qkv")
    out = torch.zeros_like(q)
    group = case["heads"] // case["kv_heads"]
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        if not n:
            continue
        pos = torch.arange(n, device=q.device)
        hide = (pos[None] > pos[:, None]) | ((pos[None] <= pos[:, None] - case["window"]) &
                                            (pos[None] >= case["sinks"]))
        if st["padding"] is not None:
            hide = hide | (st["padding"][rows] != 0)[None]
        empty = hide.all(1)
        bias = torch.zeros((n, n), dtype=torch.float64, device=q.device).masked_fill_(hide, -math.inf)
        bias[empty] = 0
        for h in range(case["kv_heads"]):
            for j in range(h * group, (h + 1) * group):
                w = torch.softmax(q[rows, j] @ k[rows, h].T / math.sqrt(case["dim"]) + bias, 1)
                w[empty] = 0
                out[rows, j] = w @ v[rows, h]
    return out


def exact_lookup(case, st, lens):
    c, q = st["cache"], st["q"].double()
    out = torch.zeros_like(q)
    group, page = case["heads"] // case["kv_heads"], case["page"]
    for b, n in enumerate(lens):
        pos = [j for j in range(n) if j >= n - case["window"] or j < case["sinks"]]
        if not pos:
            continue
        pos = torch.tensor(pos, device=q.device)
        p, r = c["table"][b].long()[pos // page], pos % page
        for h in range(case["kv_heads"]):
            k = c["k"][p, h, r].view(torch.float8_e4m3fn).double() * c["k_scale"][p, h, None].double()
            v = c["v"][p, h, :, r].view(torch.float8_e4m3fn).double() * c["v_scale"][p, h, None].double()
            x = q[b, :, h * group:(h + 1) * group].reshape(-1, case["dim"])
            w = torch.softmax(x @ k.T / math.sqrt(case["dim"]), 1)
            out[b, :, h * group:(h + 1) * group] = (w @ v).reshape(case["queries"], group, case["dim"])
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
        self.refs = {p: 0 for p in range(self.k.shape[0])}
        for row in self.lists:
            for p in row:
                self.refs[p] += 1
        self.free = sorted(p for p, n in self.refs.items() if not n)

    def release(self, slot):
        for p in self.lists[slot]:
            self.refs[p] -= 1
        self.lists[slot], self.lens[slot] = [], 0
        self.free = sorted(p for p, n in self.refs.items() if not n)

    def fork(self, src, dst):
        self.lists[dst], self.lens[dst] = list(self.lists[src]), self.lens[src]
        for p in self.lists[dst]:
            self.refs[p] += 1

    def append(self, slot, k, v, shared=()):
        page, pages = self.page, self.lists[slot]
        done = 0
        while done < k.shape[0]:
            nth, a = divmod(self.lens[slot], page)
            count = min(page - a, k.shape[0] - done)
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
                new = x[done:done + count].transpose(0, 1)          # (kv, count, dim)
                amax = new.abs().amax((1, 2)).clamp(min=2.0 ** -130)
                e = torch.ceil(torch.log2(amax / 448))
                e = torch.where(amax / 448 <= torch.exp2(e - 1), e - 1, e)
                e = torch.where(amax / 448 > torch.exp2(e), e + 1, e)
                s = torch.exp2(e.clamp(min=PAGE_FLOOR))
                part = codes[p].transpose(1, 2) if minor else codes[p]
                if a:
                    s = torch.maximum(s, scales[old])
                    was = codes[old].transpose(1, 2) if minor else codes[old]
                    part[:, :a] = e4m3(was[:, :a] * (scales[old] / s)[:, None, None])
                part[:, a:a + count] = e4m3(new / s[:, None, None])
                scales[p] = s
            self.lens[slot] += count
            done += count

    def compact(self):
        used = sorted(p for p, n in self.refs.items() if n)
        movers = [p for p in used if p >= len(used)]
        holes = [p for p in range(len(used)) if not self.refs[p]]
        for a, b in zip(movers, holes):
            for t in (self.k, self.v, self.k_scale, self.v_scale):
                t[b] = t[a]
