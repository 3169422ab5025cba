"""Beams over event histories written down plainly in 64 bits on the CPU: the selection of continuations, and the
reordering of a cache kept by hand (history_oracle).  Test-only."""
import numpy as np

import history_oracle as ho


def select(logits, scores, keep, allowed=None, ended=None, end_item=-1):
    """logits (groups, beams, items) in float64 -> scores, parents, items of the keep best of each group."""
    groups, beams, items = logits.shape
    out = np.full((groups, keep), -np.inf), np.full((groups, keep), -1), np.full((groups, keep), -1)
    for g in range(groups):
        found = []
        for w in range(beams):
            s = 0.0 if scores is None else float(scores[g, w])
            if not np.isfinite(s):
                continue
            if ended is not None and ended[g, w]:
                found.append(([s], [0.0], [end_item], [w]))
                continue
            x = logits[g, w].copy()
            if allowed is not None:
                x[~(allowed if allowed.ndim == 1 else allowed[g, w])] = -np.inf
            if np.isnan(x).any() or not np.isfinite(x.max(initial=-np.inf)):
                continue
            at = np.nonzero(x > -np.inf)[0]
            m = x.max()
            lse = m + np.log(np.exp(x[at] - m).sum())
            found.append((s + (x[at] - lse), x[at], at, np.full(len(at), w)))
        if not found:
            continue
        s, x, at, w = (np.concatenate([np.asarray(f[i]) for f in found]) for i in range(4))
        order = np.lexsort((at, -x, w, -s))[:keep]         # score, then beam, then logit, then item
        n = len(order)
        out[0][g, :n], out[1][g, :n], out[2][g, :n] = s[order], w[order], at[order]
    return out


class Cache(ho.Cache):
    def reorder(self, slots, parents):
        """slots and parents: a list for each group."""
        for group, froms in zip(slots, parents):
            held = [(list(self.lists[s]), self.lens[s]) if 0 <= s < len(self.lens) else None for s in group]
            done = set()
            for s, p in zip(group, froms):
                bad = not 0 <= s < len(self.lens) or s in done
                if 0 <= s < len(self.lens):
                    done.add(s)
                if bad or not (p == -1 or (0 <= p < len(group) and held[p] is not None)):
                    self.refused += 1
                    continue
                self._let_go(s, 0)
                self.lists[s], self.lens[s] = ([], 0) if p == -1 else (list(held[p][0]), held[p][1])
                for page in self.lists[s]:
                    if page is not None:
                        self.refs[page] += 1
        self._rebuild()
