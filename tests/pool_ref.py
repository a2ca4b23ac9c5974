"""The accounting of a cache's pages, entry by entry on lists, from the definitions alone."""


class Pool:
    """refs and table as lists; `bad` collects the records (where) that a call makes."""

    def __init__(self, refs, table, page):
        self.refs, self.table, self.page, self.bad = list(refs), [list(r) for r in table], page, set()
        self.cap = len(self.table[0]) * page

    def _free(self):
        return [p for p, c in enumerate(self.refs) if c == 0]

    def _given(self, needs):
        """For each asker the pages it gets, or None where the free ones do not last."""
        free, total, out = self._free(), 0, []
        for n in needs:
            total += n
            out.append([] if n == 0 else free[total - n:total] if total <= len(free) else None)
        return out

    def release(self, lo, hi):
        for r, row in enumerate(self.table):
            for i, p in enumerate(row):
                out = (i + 1) * self.page <= lo[r] or i * self.page >= hi[r] or hi[r] <= lo[r]
                if p < 0 or not out:
                    continue
                row[i] = -1
                if p >= len(self.refs):
                    self.bad.add(16)
                elif self.refs[p] <= 0:
                    self.bad.add(24)
                else:
                    self.refs[p] -= 1

    def reserve(self, lo, hi):
        missing = []
        for r, row in enumerate(self.table):
            if hi[r] > self.cap:
                self.bad.add(17)
            a, b = min(max(lo[r], 0), self.cap), min(max(hi[r], 0), self.cap)
            span = range(a // self.page, -(-b // self.page)) if hi[r] > lo[r] else ()
            missing.append([i for i in span if row[i] < 0])
        given = self._given([len(m) for m in missing])
        for row, m, pages in zip(self.table, missing, given):
            for i, p in zip(m, pages or ()):
                row[i] = p
                self.refs[p] = 1
        return [int(g is not None) for g in given]

    def fork(self, src, dst, tokens):
        rows, n = range(len(self.table)), len(src)
        can = []
        for k in range(n):
            ok = src[k] in rows and dst[k] in rows and src[k] != dst[k] and all(p < 0 for p in self.table[dst[k]])
            can.append(ok)
        first = {}
        for k in range(n):
            if can[k]:
                first.setdefault(dst[k], k)
        mine = [can[k] and first[dst[k]] == k for k in range(n)]
        can = [mine[k] and src[k] not in first for k in range(n)]
        length = []
        for t in tokens:
            if not 0 <= t <= self.cap:
                self.bad.add(17)
            length.append(min(max(t, 0), self.cap))
        given = self._given([int(can[k] and length[k] % self.page != 0) for k in range(n)])
        before = [list(r) for r in self.table]
        lists = [[-1] * n, [-1] * n, [0] * n, [0] * n]
        for k in range(n):
            if not can[k]:
                self.bad.add(25)
            if mine[k]:
                self.table[dst[k]][0] = -1
            if not can[k] or given[k] is None:
                continue
            lists[3][k] = 1
            full, part = divmod(length[k], self.page)
            parent, child = before[src[k]], self.table[dst[k]]
            for i in range(full):
                if 0 <= parent[i] < len(self.refs):
                    child[i] = parent[i]
                    self.refs[parent[i]] += 1
                else:
                    child[i] = -1
                    self.bad.add(16)
            if part:
                child[full] = given[k][0]
                self.refs[child[full]] = 1
                lists[1][k], lists[2][k] = child[full], part
                if 0 <= parent[full] < len(self.refs):
                    lists[0][k] = parent[full]
                else:
                    self.bad.add(16)
        return lists
