"""The pages of a cache on lists, one entry after the other: what the page calls mean."""
import random

import torch


class Model:
    def __init__(self, pages, page, rows, cols, H=2, d=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.pages, self.page, self.rows, self.cols, self.H, self.d = pages, page, rows, cols, H, d
        self.refs = [0] * pages
        self.table = [[-1] * cols for _ in range(rows)]
        self.kv = [0] * rows
        self.cache = {"K8": torch.randint(0, 0x7F, (pages, H, page, d), generator=g).to(torch.uint8), "sk": torch.rand((pages, H, page), generator=g),
                      "V8": torch.randint(0, 0x7F, (pages, H, page, d), generator=g).to(torch.uint8), "sv": torch.rand((pages, H, page), generator=g)}

    def bits(self):
        words = [sum(1 << i for i in range(32) if p + i < self.pages and not self.refs[p + i]) for p in range(0, self.pages, 32)]
        return [w - (1 << 32) if w >> 31 else w for w in words]

    @staticmethod
    def named(e):
        return -2 - e if e < -1 else e

    def written(self, n):
        """(row, column, first position) of the entries of a call of n tokens of each row, whose kv has them already."""
        out = []
        for b, m in enumerate(n):
            first = max(self.kv[b] - m, 0)
            if m and self.kv[b]:
                out += [(b, j, first) for j in range(first // self.page, (self.kv[b] - 1) // self.page + 1)]
        return out

    def reserve(self, n):
        """False: too few free pages."""
        at = self.written(n)
        refs, free, new = list(self.refs), [p for p in range(self.pages) if not self.refs[p]], []
        for b, j, first in at:
            p = self.named(self.table[b][j])
            if p >= 0 and refs[p] == 1:
                new.append(p)
                continue
            if not free:
                for b, j, _ in at:
                    p = self.named(self.table[b][j])
                    if p >= 0 and self.refs[p] > 1:
                        self.table[b][j] = -2 - p
                return False
            q = free.pop(0)
            if p >= 0:
                refs[p] -= 1
            refs[q] = 1
            new.append(q)
        for (b, j, first), q in zip(at, new):
            p = self.named(self.table[b][j])
            tokens = first - j * self.page
            if p >= 0 and p != q and tokens > 0:
                for x in self.cache.values():
                    x[q, :, :tokens] = x[p, :, :tokens]
            self.table[b][j] = q
        self.refs = refs
        return True

    def trim(self, lens):
        for b, m in enumerate(lens):
            if m < 0:
                continue
            for j in range(-(-m // self.page), self.cols):
                p = self.named(self.table[b][j])
                if p >= 0:
                    self.refs[p] -= 1
                self.table[b][j] = -1
            self.kv[b] = min(self.kv[b], m)

    def fork(self, parents, rows, lens=None):
        """Rows `rows` become forks of `parents`, both numbers of this table."""
        for i, (a, b) in enumerate(zip(parents, rows)):
            self.kv[b] = 0 if a < 0 else min(self.kv[a], lens[i]) if lens else self.kv[a]
            self.table[b] = [-1] * self.cols
            for j in range(-(-self.kv[b] // self.page)):
                self.table[b][j] = self.named(self.table[a][j])
                self.refs[self.table[b][j]] += 1

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        to = dict(zip([p for p in range(used, self.pages) if self.refs[p]], [p for p in range(used) if not self.refs[p]]))
        for a, b in to.items():
            for x in self.cache.values():
                x[b] = x[a]
            self.refs[a], self.refs[b] = 0, self.refs[a]
        self.table = [[e if e == -1 else (to.get(e, e) if e >= 0 else -2 - to.get(-2 - e, -2 - e)) for e in row] for row in self.table]
        return used

    def consistent(self):
        names = [0] * self.pages
        for row in self.table:
            for e in row:
                if e != -1:
                    names[self.named(e)] += 1
        return names == self.refs


def walk(model, rng, steps):
    """Random calls on a model with an even number of rows: yields (name, arguments) before the model makes each."""
    half = model.rows // 2
    for _ in range(steps):
        op = rng.choice(["grow", "grow", "grow", "take back", "fork", "fork", "end", "compact"])
        if op == "grow":
            n = [min(rng.choice([0, 0, 1, 1, 3, 20, 45]), model.cols * model.page - k) for k in model.kv]
            yield "reserve", n
        elif op == "take back":
            yield "trim", [rng.choice([-1, -1, max(0, k - rng.randint(0, 30)), k]) for k in model.kv]
        elif op == "end":
            yield "trim", [rng.choice([-1, -1, -1, 0]) for _ in model.kv]
        elif op == "compact":
            yield "compact", None
        else:
            first = rng.random() < 0.5
            rows = list(range(half)) if first else list(range(half, 2 * half))
            parents = [rng.choice([-1] + [r for r in range(2 * half) if r not in rows] * 3) for _ in rows]
            lens = [rng.randint(0, 60) for _ in rows] if rng.random() < 0.5 else None
            yield "fork", (parents, rows, lens)


def rng_of(seed):
    return random.Random(seed)
