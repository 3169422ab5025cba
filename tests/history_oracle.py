"""The event-history operators written down plainly in 64 bits on the CPU, one history, event and page at a time.

Test-only.  Attention is a loop over histories and heads; the cache is a list of page numbers for each
history and float64 arrays of what the codes stand for.
"""
import numpy as np

FLOOR = -100


def e4m3(x):
    """Nearest e4m3 value, ties to even; not finite -> NaN.  |x| <= 448 where finite."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    a = np.where(fin, np.abs(x), 0.0)
    _, e = np.frexp(a)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.where(fin, np.round(np.where(fin, x, 0.0) / step) * step, np.nan)


def scale_for(block):
    """The smallest power of two >= 2^FLOOR under which the largest finite value is at most 448."""
    a = np.abs(block[np.isfinite(block)])
    top = a.max() if a.size else 0.0
    e = FLOOR
    while top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def sees(n, window, sinks):
    """(n, n) truth table: row i sees key j."""
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def weights(s, seen):
    s = np.where(seen, s, -np.inf)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(s - np.where(np.isinf(m), 0.0, m)), 0.0)
    t = p.sum(-1, keepdims=True)
    return p / np.where(t == 0, 1.0, t)


def attention(q, k, v, lens, window, sinks, scale, padding=None):
    """(out, sum of p |v|, largest sum of |scale q k| of the row): the last two for error bounds."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, mag, big = np.zeros_like(q), np.zeros_like(q), np.zeros((n, heads, 1))
    at = 0
    for c in lens:
        r = slice(at, at + c)
        at += c
        if c == 0:
            continue
        seen = sees(c, window, sinks)
        if padding is not None:
            seen = seen & (padding[r] == 0)[None, :]
        for h in range(heads):
            kk, vv = k[r, h // group], v[r, h // group]
            w = weights(scale * q[r, h] @ kk.T, seen)
            out[r, h] = w @ vv
            mag[r, h] = w @ np.abs(vv)
            big[r, h, 0] = np.where(seen, abs(scale) * np.abs(q[r, h]) @ np.abs(kk).T, 0).max(1)
    return out, mag, big


class Cache:
    """Histories on pages: lists[slot] of page numbers (None: trimmed), refs, and the values of the codes."""

    def __init__(self, n_pages, n_slots, max_pages, kv, dim, page):
        self.n_pages, self.max_pages, self.page = n_pages, max_pages, page
        self.k = np.zeros((n_pages, kv, page, dim))
        self.v = np.zeros((n_pages, kv, page, dim))
        self.ks, self.vs = np.ones((n_pages, kv)), np.ones((n_pages, kv))
        self.lists = [[] for _ in range(n_slots)]
        self.lens = [0] * n_slots
        self.refs = [0] * n_pages
        self.free = list(range(n_pages))
        self.refused = 0

    def _ok(self, slot):
        if 0 <= slot < len(self.lens):
            return True
        self.refused += 1
        return False

    def _rebuild(self):
        self.free = [p for p in range(self.n_pages) if self.refs[p] == 0]

    def append(self, slots, counts, k, v):
        """One call: decisions are taken for every history before anything changes."""
        at, plans, wanted, free = 0, [], 0, list(self.free)
        taken = 0
        for slot, n in zip(slots, counts):
            rows = slice(at, at + n)
            at += n
            if not self._ok(slot):
                continue
            old = self.lens[slot]
            part = old % self.page
            tail = self.lists[slot][old // self.page] if part and n else None
            if old + n > self.max_pages * self.page or (part and n and tail is None):
                self.refused += 1
                continue
            copy = bool(part and n and self.refs[tail] > 1)
            need = -(-(old + n) // self.page) - -(-old // self.page) + copy if n else 0
            if need and wanted + need > len(free):
                self.refused += 1
                wanted += need
                continue
            plans.append((slot, n, rows, old, tail, copy, free[wanted:wanted + need]))
            wanted += need
            taken = max(taken, wanted)
        self.free = free[taken:]
        for slot, n, rows, old, tail, copy, pages in plans:
            done = 0
            while done < n:
                nth, a = divmod(self.lens[slot], self.page)
                c = min(self.page - a, n - done)
                if a and not copy:
                    p = tail if nth == old // self.page else self.lists[slot][nth]
                else:
                    p = pages.pop(0)
                    self.refs[p] = 1
                    if a:
                        self.refs[tail] -= 1
                        self.lists[slot][nth] = p
                    else:
                        self.lists[slot].append(p)
                for val, sc, x in ((self.k, self.ks, k), (self.v, self.vs, v)):
                    new = x[rows][done:done + c]
                    for h in range(val.shape[1]):
                        s = scale_for(new[:, h])
                        if a:
                            was = sc[tail, h]
                            s = max(s, was)
                            val[p, h, :a] = e4m3(val[tail, h, :a] / s) * s
                        val[p, h, a:a + c] = e4m3(new[:, h] / s) * s
                        sc[p, h] = s
                copy = False
                self.lens[slot] += c
                done += c

    def _let_go(self, slot, keep):
        for i, p in enumerate(self.lists[slot]):
            if i >= keep and p is not None:
                self.refs[p] -= 1
        self.lists[slot] = self.lists[slot][:keep]

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            if not (0 <= s < len(self.lens) and 0 <= d < len(self.lens)):
                self.refused += 1
                continue
            self._let_go(d, 0)
            self.lists[d], self.lens[d] = list(self.lists[s]), self.lens[s]
            for p in self.lists[d]:
                if p is not None:
                    self.refs[p] += 1
        self._rebuild()

    def truncate(self, slots, lens):
        for s, n in zip(slots, lens):
            if not self._ok(s):
                continue
            if n < 0 or n > self.lens[s] or (n % self.page and self.lists[s][n // self.page] is None):
                self.refused += 1
                continue
            self._let_go(s, -(-n // self.page))
            self.lens[s] = n
        self._rebuild()

    def trim(self, slots, window, sinks):
        for s in slots:
            if not self._ok(s):
                continue
            for i, p in enumerate(self.lists[s]):
                events = range(i * self.page, (i + 1) * self.page)
                if p is not None and all(j >= sinks and j < self.lens[s] - window for j in events):
                    self.refs[p] -= 1
                    self.lists[s][i] = None
        self._rebuild()

    def compact(self):
        used = [p for p in range(self.n_pages) if self.refs[p]]
        m = len(used)
        move = dict(zip([p for p in used if p >= m], [p for p in range(m) if not self.refs[p]]))
        for a, b in move.items():
            for t in (self.k, self.v, self.ks, self.vs):
                t[b] = t[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.lists = [[move.get(p, p) for p in row] for row in self.lists]
        self._rebuild()

    def history(self, slot, h, window, sinks):
        """Visible keys and values of a slot's head, as a lookup sees them."""
        n = self.lens[slot]
        at = [j for j in range(n) if (j >= n - window or j < sinks)
              and j // self.page < len(self.lists[slot]) and self.lists[slot][j // self.page] is not None]
        p = [self.lists[slot][j // self.page] for j in at]
        r = [j % self.page for j in at]
        return self.k[p, h, r], self.v[p, h, r]

    def lookup(self, slots, q, window, sinks, scale):
        """q (batch, queries, heads, dim) -> (out, sum of p |v|, largest sum of |scale q k|)."""
        out, mag, big = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:3] + (1,))
        group = q.shape[2] // self.k.shape[1]
        for b, slot in enumerate(slots):
            if not 0 <= slot < len(self.lens):
                continue
            for h in range(q.shape[2]):
                k, v = self.history(slot, h // group, window, sinks)
                if not len(k):
                    continue
                x = q[b, :, h]
                w = weights(scale * x @ k.T, np.ones((len(x), len(k)), bool))
                out[b, :, h], mag[b, :, h] = w @ v, w @ np.abs(v)
                big[b, :, h, 0] = (abs(scale) * np.abs(x) @ np.abs(k).T).max(1)
        return out, mag, big
