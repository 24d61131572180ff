"""The block table's operations, one page at a time, on Python lists; pools as numpy arrays [L][n_pages][Hkv][tiles][bytes]."""

SEQ, NOPAGE, PAGE = 32, 64, 2


class Pages:
    def __init__(self, max_seqs, per, page_size, n_pages, pools=()):
        self.table = [[-1] * per for _ in range(max_seqs)]
        self.len = [0] * max_seqs
        self.ref = [0] * n_pages
        self.ps, self.pools, self.status = page_size, list(pools), 0

    def _free(self):
        return [p for p, r in enumerate(self.ref) if r <= 0]

    def _known(self, i):
        return 0 <= i < len(self.len)

    def extend(self, ids, lens):
        free, full = self._free(), False
        for k, (i, n) in enumerate(zip(ids, lens)):
            if not self._known(i) or i in ids[:k]:
                self.status |= SEQ
                continue
            if n > self.ps * len(self.table[0]):
                self.status |= NOPAGE
                continue
            if n <= self.len[i]:
                continue
            have, need = -(-self.len[i] // self.ps), -(-n // self.ps)
            if full or need - have > len(free):
                self.status |= NOPAGE
                full = True
                continue
            for j in range(have, need):
                self.table[i][j] = free.pop(0)
                self.ref[self.table[i][j]] = 1
            self.len[i] = n

    def free(self, ids):
        for k, i in enumerate(ids):
            if not self._known(i) or i in ids[:k]:
                self.status |= SEQ
                continue
            for p in self.table[i]:
                if p >= 0:
                    self.ref[p] -= 1
            self.table[i] = [-1] * len(self.table[i])
            self.len[i] = 0

    def fork(self, parents, children):
        free, full = self._free(), False
        table, lens, ref = [list(r) for r in self.table], list(self.len), list(self.ref)
        for k, (p, c) in enumerate(zip(parents, children)):
            if not self._known(p) or not self._known(c) or p == c or self.len[c] or self.table[c][0] >= 0 or c in children[:k]:
                self.status |= SEQ
                continue
            n = self.len[p]
            if full or (n % self.ps and not free):
                self.status |= NOPAGE
                full = True
                continue
            row = [-1] * len(table[c])
            for j in range(n // self.ps):
                row[j] = self.table[p][j]
                ref[row[j]] += 1
            if n % self.ps:
                j = n // self.ps
                row[j] = free.pop(0)
                ref[row[j]] = 1
                tiles = -(-(n % self.ps) // 32)
                for pool in self.pools:
                    pool[:, row[j], :, :tiles] = pool[:, self.table[p][j], :, :tiles]
            table[c], lens[c] = row, n
        self.table, self.len, self.ref = table, lens, ref

    def compact(self):
        held = sum(r > 0 for r in self.ref)
        holes = [p for p in range(held) if self.ref[p] <= 0]
        movers = [p for p in range(held, len(self.ref)) if self.ref[p] > 0]
        to = dict(zip(movers, holes))
        if any(p >= len(self.ref) or (p >= 0 and self.ref[p] <= 0) for r in self.table for p in r):
            self.status |= PAGE  # entries of pages that nobody holds, which stay as they are
        for s, d in to.items():
            for pool in self.pools:
                pool[:, d] = pool[:, s]
            self.ref[d], self.ref[s] = self.ref[s], 0
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        return held

    def copy(self, src, dst):
        n = len(self.ref)
        for k, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < n and 0 <= d < n) or d in dst[:k] or d in src[:k] + src[k + 1:]:
                self.status |= PAGE
                continue
            for pool in self.pools:
                pool[:, d] = pool[:, s]
