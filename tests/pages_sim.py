"""The books of a cache's pages, one step after the other on the host."""


class Sim:
    def __init__(self, requests, width, pages, page_size):
        self.R, self.W, self.P, self.ps = requests, width, pages, page_size
        self.table = [[-1] * width for _ in range(requests)]
        self.lengths = [0] * requests
        self.counts = [0] * pages
        self.data = list(range(pages))          # what each page holds: a label

    def need(self, r):
        return -(-self.lengths[r] // self.ps)

    def free_pages(self):
        return [p for p in range(self.P) if self.counts[p] <= 0]

    def extend(self, starts, tokens):
        slots = [-1] * tokens
        free, at = self.free_pages(), 0
        for r in range(self.R):
            start = min(max(starts[r], 0), tokens)
            n = min(max(starts[r + 1] - start, 0), tokens - start)
            new = self.lengths[r] + n
            if new > self.W * self.ps:
                continue
            more = -(-new // self.ps) - self.need(r)
            at += more
            if n == 0 or (more and at > len(free)):
                continue
            first = self.need(r)
            for e in range(more):
                page = free[at - more + e]
                self.table[r][first + e] = page
                self.counts[page] = 1
            for i in range(n):
                p = self.lengths[r] + i
                page = self.table[r][p // self.ps]
                slots[start + i] = page * self.ps + p % self.ps if 0 <= page < self.P else -1
            self.lengths[r] = new
        return slots

    def fork(self, parents, children):
        free, done, named = self.free_pages(), [], set()
        before = list(self.lengths)
        rows = [list(t) for t in self.table]
        for par, chi in zip(parents, children):
            inside = 0 <= par < self.R and 0 <= chi < self.R
            ok = inside and chi not in named and before[chi] == 0
            if inside:
                named.add(chi)
            if ok and before[par] % self.ps:
                ok = bool(free)
                if ok:
                    new = free.pop(0)
            done.append(int(ok))
            if not ok or before[par] == 0:
                continue
            n = -(-before[par] // self.ps)
            for e in range(n):
                page = rows[par][e]
                if e == n - 1 and before[par] % self.ps:
                    if page >= 0:
                        self.data[new] = self.data[page]
                    page = new
                    self.counts[new] = 0
                self.table[chi][e] = page
                if page >= 0:
                    self.counts[page] += 1
            self.lengths[chi] = before[par]
        return done

    def free(self, requests):
        for r in requests:
            if not 0 <= r < self.R:
                continue
            for e in range(self.need(r)):
                if self.table[r][e] >= 0:
                    self.counts[self.table[r][e]] -= 1
                self.table[r][e] = -1
            self.lengths[r] = 0

    def trim(self, window, sinks):
        for r in range(self.R):
            for e in range(self.need(r)):
                # every key of the page is behind the window of a token at position `length`, and no sink
                keys = range(e * self.ps, (e + 1) * self.ps)
                if all(j <= self.lengths[r] - window and j >= sinks for j in keys):
                    if self.table[r][e] >= 0:
                        self.counts[self.table[r][e]] -= 1
                    self.table[r][e] = -1

    def compact(self):
        used = [p for p in range(self.P) if self.counts[p] > 0]
        U = len(used)
        holes = [p for p in range(U) if self.counts[p] <= 0]
        to = [-1] * self.P
        for p in used:
            to[p] = p if p < U else holes.pop(0)
        data, counts = list(self.data), [0] * self.P
        for p in used:
            data[to[p]] = self.data[p]
            counts[to[p]] = self.counts[p]
        self.data, self.counts = data, counts
        for r in range(self.R):
            for e in range(self.need(r)):
                if self.table[r][e] >= 0:
                    self.table[r][e] = to[self.table[r][e]]
        return to
