"""Plain restatement of the operators on a cache's pages (numpy, row by row, no
code shared with the library)."""
import numpy as np


def up(tokens, page):
    return -(-max(int(tokens), 0) // page)


def fork(parent, child, length, cached, page, n_pages, table, shared, ring, counters):
    n, width = table.shape
    head, tail = int(counters[0]), int(counters[1])
    held = [max(int(c), 0) for c in cached]
    children = [int(c) for c in child]
    bad = need = 0
    for p, c, m in zip(parent, children, length):
        p, m = int(p), int(m)
        fine = 0 <= p < n and 0 <= c < n and p != c and 0 <= m
        fine = fine and m <= held[p] and held[c] == 0 and up(m, page) <= width and children.count(c) == 1
        bad += not fine
        need += m % page != 0
    short = bad + max(0, need - (tail - head))
    table, shared = table.copy(), shared.copy()
    src, dst = [-1] * len(children), [-1] * len(children)
    before = table.copy()
    if not short:
        for i, (p, c, m) in enumerate(zip(parent, children, length)):
            whole, rest = divmod(int(m), page)
            table[c] = -1
            for j in range(whole):
                table[c, j] = before[p, j]
                if 0 <= before[p, j] < n_pages:
                    shared[before[p, j]] += 1
            if rest:
                src[i], dst[i] = int(before[p, whole]), int(ring[head % n_pages])
                table[c, whole] = dst[i]
                head += 1
            held[c] = int(m)
    return dict(table=table, shared=shared, len=held, copy_src=src, copy_dst=dst, counters=[head, tail], short=short)


def release(cached, keep, page, n_pages, table, shared, ring, counters):
    n, width = table.shape
    head, tail = int(counters[0]), int(counters[1])
    out, shared, ring = np.full_like(table, -1), shared.copy(), ring.copy()
    left, free = [], set()
    for i in range(n):
        have = max(int(cached[i]), 0)
        stay = min(max(int(keep[i]), 0), have)
        left.append(stay)
        s, h = min(up(stay, page), width), min(up(have, page), width)
        out[i, :s] = table[i, :s]
        for p in table[i, s:h]:
            if 0 <= p < n_pages:
                if shared[p] > 0:
                    shared[p] -= 1
                else:
                    free.add(int(p))
    for p in sorted(free):
        ring[tail % n_pages] = p
        tail += 1
    return dict(table=out, shared=shared, ring=ring, len=left, counters=[head, tail])


def compact(cached, page, n_pages, table, shared, ring, counters, max_copies):
    n, width = table.shape
    live = [[j for j in range(min(up(cached[i], page), width)) if 0 <= table[i, j] < n_pages] for i in range(n)]
    used = sorted({int(table[i, j]) for i in range(n) for j in live[i]})
    m = len(used)
    src = [p for p in used if p >= m]
    dst = sorted(set(range(m)) - set(used))
    assert len(src) == len(dst)
    if len(src) > max_copies:
        return dict(table=table.copy(), shared=shared.copy(), ring=ring.copy(), counters=list(counters), copy_src=[-1] * max_copies,
                    copy_dst=[-1] * max_copies, short=len(src) - max_copies)
    to = {p: p for p in used}
    to.update(zip(src, dst))
    out, counts, ring = np.full_like(table, -1), np.zeros_like(shared), ring.copy()
    for i in range(n):
        for j in range(min(up(cached[i], page), width)):
            out[i, j] = to.get(int(table[i, j]), table[i, j])
    for p in used:
        counts[to[p]] = shared[p]
    ring[:n_pages - m] = np.arange(m, n_pages)
    pad = [-1] * (max_copies - len(src))
    return dict(table=out, shared=counts, ring=ring, counters=[0, n_pages - m], copy_src=src + pad, copy_dst=dst + pad, short=0)


class Rows:
    """Rows of given lengths over pages in a random order, some of them shared as
    forks leave them, and the ring of the free ones."""

    def __init__(self, seed, n, page, width, spare, share=0.3, empty=0.3, hole=0.0, lost=0):
        rng = np.random.default_rng(seed)
        self.rng, self.page, self.width = rng, page, width
        self.cached = np.where(rng.random(n) < empty, 0, rng.integers(0, width * page + 1, n)).astype(np.int32)
        self.table = np.full((n, width), -1, np.int32)
        need = sum(up(c, page) for c in self.cached)
        self.n_pages = max(1, need + spare + lost)
        perm, at = rng.permutation(self.n_pages).astype(np.int32), 0
        self.shared = np.zeros(self.n_pages, np.int32)
        for i in range(n):
            k = up(self.cached[i], page)
            s = 0
            if i and rng.random() < share:          # begins with the pages of an earlier row
                j = int(rng.integers(0, i))
                s = int(rng.integers(0, min(k, int(self.cached[j]) // page) + 1))
                self.table[i, :s] = self.table[j, :s]
                np.add.at(self.shared, self.table[j, :s], 1)
            self.table[i, s:k] = perm[at:at + k - s]
            at += k - s
        free = perm[at:self.n_pages - lost]
        head = int(rng.integers(0, 1 << 40))
        self.ring = np.full(self.n_pages, -1, np.int32)
        self.ring[(head + np.arange(len(free))) % self.n_pages] = free
        self.counters = [head, head + len(free)]
        if hole:
            self.table[rng.random(self.table.shape) < hole] = -1

    def forks(self, k, partial=True):
        """k forks into empty rows, as many as there are."""
        rng = self.rng
        kids = rng.permutation(np.flatnonzero(self.cached == 0))[:k]
        parents = np.flatnonzero(self.cached > 0)
        if not len(parents):
            parents = np.setdiff1d(np.arange(len(self.cached)), kids)[:1]
        p = rng.choice(parents, len(kids)).astype(np.int32)
        m = np.array([rng.integers(0, self.cached[x] + 1) if rng.random() < 0.6 else self.cached[x] for x in p], np.int32)
        if not partial:
            m = m // self.page * self.page
        return p, kids.astype(np.int32), m
