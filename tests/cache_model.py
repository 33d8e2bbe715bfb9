"""The page operations on host lists, one step after another: what the cache
calls have to leave behind (tables, counts, lengths and, as token names, the
contents of the pages)."""


class Model:
    def __init__(self, n_pages, page_size, n, width):
        self.P, self.n_pages, self.width = page_size, n_pages, width
        self.ref = [0] * n_pages
        self.table = [[-1] * width for _ in range(n)]
        self.ctx = [0] * n
        self.data = [[None] * page_size for _ in range(n_pages)]  # a page's tokens, by name

    def pages(self, tokens):
        return -(-tokens // self.P)

    def held(self, b):
        return next((i for i, p in enumerate(self.table[b]) if p < 0), self.width)

    def free_words(self):
        return [sum(1 << i for i in range(32) if w * 32 + i < self.n_pages and not self.ref[w * 32 + i])
                for w in range(-(-self.n_pages // 32))]

    def lowest(self):
        p = self.ref.index(0)
        self.ref[p] = 1
        return p

    def fork(self, src, dst):
        bad = False
        for i, (s, d) in enumerate(zip(src, dst)):
            if s in dst or d in dst[:i] or not (0 <= s < len(self.ctx) and 0 <= d < len(self.ctx)) or self.ctx[d] or self.held(d):
                bad = True
                continue
            self.ctx[d] = self.ctx[s]
            for j in range(self.pages(self.ctx[s])):
                self.table[d][j] = self.table[s][j]
                self.ref[self.table[s][j]] += 1
        return bad

    def release(self, b, first):
        for i in range(first, self.held(b)):
            self.ref[self.table[b][i]] -= 1
            self.table[b][i] = -1

    def free(self, which):
        for b in which:
            if 0 <= b < len(self.ctx):
                self.release(b, 0)
                self.ctx[b] = 0

    def reserve(self, rows):
        """rows[b]: the window's rows. Returns (granted, short of pages, too wide for the table)."""
        granted, short, wide = [], False, False
        start = list(self.ref)
        for b, r in enumerate(rows):
            n, held = self.ctx[b], self.held(b)
            if r and n + r > self.width * self.P:
                wide = True
                granted.append(0)
                continue
            part = self.table[b][n // self.P] if r and n % self.P else -1
            copy = part >= 0 and self.ref[part] > 1
            need = max(0, self.pages(n + r) - held) + copy
            if (short and (need or (part >= 0 and start[part] > 1))) or need > self.ref.count(0):
                short = True
                granted.append(0)
                continue
            if copy:
                new = self.lowest()
                self.data[new][: n % self.P] = self.data[part][: n % self.P]
                self.ref[part] -= 1
                self.table[b][n // self.P] = new
            for i in range(held, held + need - copy):
                self.table[b][i] = self.lowest()
            granted.append(r)
        return granted, short, wide

    def append(self, windows, granted):
        """windows[b]: the names of the window's rows."""
        for b, names in enumerate(windows):
            if granted[b]:
                for w, x in enumerate(names):
                    t = self.ctx[b] + w
                    self.data[self.table[b][t // self.P]][t % self.P] = x

    def tokens(self, b, n=None):
        return [self.data[self.table[b][t // self.P]][t % self.P] for t in range(self.ctx[b] if n is None else n)]

    def commit(self, kept):
        """kept[b]: (place in the window, rows)."""
        for b, (begin, rows) in enumerate(kept):
            n = self.ctx[b]
            for j in range(rows if begin else 0):
                a, d = n + begin + j, n + j
                self.data[self.table[b][d // self.P]][d % self.P] = self.data[self.table[b][a // self.P]][a % self.P]
            self.ctx[b] = n + rows
            self.release(b, self.pages(self.ctx[b]))
