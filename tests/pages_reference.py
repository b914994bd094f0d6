"""Plain form of the page management, page by page on the host."""
import numpy as np

PAGE_ID, PLAN, PAGES = 1, 4, 8


class Pages:
    """refs and pools ([num_pages, ...] arrays) as the library keeps them on the device."""

    def __init__(self, pools, page_size, refs=None):
        self.pools, self.page_size, self.n = pools, page_size, len(pools[0])
        self.refs = [0] * self.n if refs is None else [int(x) for x in refs]
        self.err = 0

    def _inside(self, p):
        if 0 <= p < self.n:
            return True
        self.err |= PAGE_ID
        return False

    def alloc(self, n):
        ids = [p for p in range(self.n) if self.refs[p] == 0][:n]
        for p in ids:
            self.refs[p] = 1
        if len(ids) < n:
            self.err |= PAGES
        return ids + [-1] * (n - len(ids))

    def free(self, ids):
        for p in ids:
            if self._inside(p):
                if self.refs[p] > 0:
                    self.refs[p] -= 1
                else:
                    self.err |= PAGES

    def copy(self, src, dst):
        for s, d in zip(src, dst):
            if self._inside(s) and self._inside(d):
                for pool in self.pools:
                    pool[d] = pool[s]

    def fork(self, table, indptr, lens, parents, out_len):
        P, out, out_indptr = self.page_size, [], [0]
        sound = [0 <= b < len(lens) and 0 <= lens[b] and -(-lens[b] // P) <= indptr[b + 1] - indptr[b]
                 and indptr[b + 1] <= len(table) for b in parents]
        if not all(sound):
            self.err |= PLAN
        if sum(-(-lens[b] // P) for b, ok in zip(parents, sound) if ok) > out_len:
            self.err |= PLAN
            return None, [0] * (len(parents) + 1)
        fresh = iter(self.alloc(sum(lens[b] % P != 0 for b, ok in zip(parents, sound) if ok)))
        for b, ok in zip(parents, sound):
            n = lens[b] if ok else 0
            for j in range(-(-n // P)):
                p = table[indptr[b] + j]
                if (j + 1) * P > n:
                    new = next(fresh)
                    if new >= 0 and self._inside(p):
                        for pool in self.pools:
                            pool[new] = pool[p]
                    out.append(new)
                elif self._inside(p):
                    self.refs[p] += 1
                    out.append(p)
                else:
                    out.append(-1)
            out_indptr.append(len(out))
        return out, out_indptr

    def compact(self, table):
        remap = [p if n else -1 for p, n in enumerate(self.refs)]
        used = sum(n > 0 for n in self.refs)
        holes = [p for p in range(used) if not self.refs[p]]
        movers = [p for p in range(self.n - 1, used - 1, -1) if self.refs[p]]
        assert len(holes) == len(movers)
        for to, frm in zip(holes, movers):
            remap[frm] = to
            self.refs[to], self.refs[frm] = self.refs[frm], 0
            for pool in self.pools:
                pool[to] = pool[frm]
        out = []
        for p in table:
            if self._inside(p):
                self.err |= PAGES if remap[p] < 0 else 0
                p = remap[p]
            out.append(p)
        return out, remap


def random_state(rng, num_pages, used, batch, page_size):
    """Requests of random lengths on `used` random pages: table, indptr, lens, refs."""
    cuts = np.sort(rng.integers(0, used + 1, batch - 1)) if batch > 1 else np.zeros(0, int)
    indptr = np.concatenate([[0], cuts, [used]]).astype(np.int32)
    table = rng.permutation(num_pages)[:used].astype(np.int32)
    lens = [0 if n == 0 else int((n - 1) * page_size + rng.integers(1, page_size + 1)) for n in np.diff(indptr)]
    refs = np.zeros(num_pages, np.int32)
    refs[table] = 1
    return table, indptr, np.array(lens, np.int32), refs
