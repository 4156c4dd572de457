"""Oracle of the page tables: one request after the other, on Python lists.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np


class Pages:
    def __init__(self, table, lens, refs, bs):
        self.table = np.array(table, dtype=np.int32)
        self.lens = np.array(lens, dtype=np.int32)
        self.refs = np.array(refs, dtype=np.int32)
        self.bs = bs
        self.B, self.tb = self.table.shape
        self.n = len(self.refs)

    def ok(self, p):
        return 0 <= p < self.n

    def free_pages(self):
        return [p for p in range(self.n) if self.refs[p] <= 0]


def alloc(t: Pages, want):
    free, taken, full = t.free_pages(), 0, False
    status = []
    for b in range(t.B):
        w = int(want[b])
        if w < 0 or w > t.tb * t.bs:
            status.append(2)
            continue
        miss = [j for j in range(-(-w // t.bs)) if not t.ok(t.table[b, j])]
        if not miss:
            status.append(0)
            continue
        if full or taken + len(miss) > len(free):
            full = True
            status.append(1)
            continue
        for j in miss:
            t.table[b, j] = free[taken]
            t.refs[free[taken]] = 1
            taken += 1
        status.append(0)
    return np.array(status, np.int32)


def fork(t: Pages, src, dst):
    """Returns status and the (from, to) page copies."""
    free, taken, full = t.free_pages(), 0, False
    named = [int(z) for z in dst if 0 <= z < t.B]
    status, copies, seen = [], [], set()
    before = t.table.copy()
    for a, z in zip(map(int, src), map(int, dst)):
        in_range = 0 <= a < t.B and 0 <= z < t.B
        again = z in seen
        if 0 <= z < t.B:
            seen.add(z)
        if not in_range or again or a in named:
            status.append(2)
            continue
        L = min(max(int(t.lens[a]), 0), t.tb * t.bs)
        whole = L // t.bs
        row = [int(p) if t.ok(p) else -1 for p in before[a, :whole]]
        grow = [p for p in row if p >= 0]
        if L % t.bs and t.ok(before[a, whole]):
            if full or taken >= len(free):
                full = True
                status.append(1)
                continue
            page = free[taken]
            taken += 1
            copies.append((int(before[a, whole]), page))
            t.refs[page] = 1
            row.append(page)
        for p in grow:
            t.refs[p] += 1
        for p in t.table[z]:
            if t.ok(p):
                t.refs[p] -= 1
        t.table[z] = row + [-1] * (t.tb - len(row))
        t.lens[z] = L
        status.append(0)
    return np.array(status, np.int32), copies


def release(t: Pages, ids):
    for b in map(int, ids):
        if 0 <= b < t.B:
            for p in t.table[b]:
                if t.ok(p):
                    t.refs[p] -= 1
            t.table[b] = -1
            t.lens[b] = 0


def compact(t: Pages):
    """Returns table, refs, remap, n_live and the (from, to) page copies."""
    live = [p for p in range(t.n) if t.refs[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if t.refs[p] <= 0]
    movers = [p for p in live if p >= n]
    to = dict(zip(movers, holes))
    remap = np.array([to.get(p, p) if t.refs[p] > 0 else -1 for p in range(t.n)], np.int32)
    refs = np.zeros(t.n, np.int32)
    for p in live:
        refs[remap[p]] = t.refs[p]
    table = np.array([[remap[p] if t.ok(p) else -1 for p in row] for row in t.table], np.int32)
    return table.reshape(t.table.shape), refs, remap, n, [(m, to[m]) for m in movers]


def trim(t: Pages):
    for b in range(t.B):
        first = -(-max(int(t.lens[b]), 0) // t.bs)
        for j in range(first, t.tb):
            if t.ok(t.table[b, j]):
                t.refs[t.table[b, j]] -= 1
                t.table[b, j] = -1
