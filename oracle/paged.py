"""Oracle of the bf16 paged cache: rotation, append, attention, prompts, eviction.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

bf16 arrays are uint16 bits.  Rotations and attention are fp64; eviction sorts Python
tuples.  Everything loops over sequences, heads and tokens.
"""
from __future__ import annotations

import numpy as np


def widen(bits):
    with np.errstate(invalid="ignore"):                # signalling NaNs
        return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Cache:
    """k, v bits [n, H, bs, d], table [B, tb], lens [B], weight fp32 and pos [B * H, tb * bs]."""

    def __init__(self, k, v, table, lens, weight=None, pos=None, max_len=0):
        self.k, self.v = k.copy(), v.copy()
        self.table, self.lens = np.asarray(table), np.array(lens, np.int32)
        self.n, self.H, self.bs, self.d = k.shape
        self.B, tb = self.table.shape
        room = tb * self.bs
        self.cap = min(max_len, room) if max_len > 0 else room
        self.weight = None if weight is None else weight.copy()
        self.pos = None if pos is None else pos.copy()

    def length(self, b):
        return int(min(max(int(self.lens[b]), 0), self.cap))

    def at(self, b, t):
        """(page, row) of slot t, or None."""
        p = int(self.table[b, t // self.bs])
        return (p, t % self.bs) if 0 <= p < self.n else None


def chunks(starts, n_tokens, max_new=0):
    """[(first token, count)] of every sequence."""
    out = []
    for b in range(len(starts) - 1):
        a = min(max(int(starts[b]), 0), n_tokens)
        e = min(max(int(starts[b + 1]), a), n_tokens)
        out.append((a, min(e - a, max_new) if max_new else e - a))
    return out


def rope(x, positions, freq, mscale=1.0, interleaved=False, backward=False):
    """x fp64 [n, H, d].  Returns the rotated rows and, for an error bound, |x0| + |x1| of
    every rotated value (0 where values are copied)."""
    y, size = x.copy(), np.zeros_like(x)
    h = len(freq)
    for t, at in enumerate(positions):
        for i in range(h):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
            c, s = mscale * np.cos(int(at) * freq[i]), mscale * np.sin(int(at) * freq[i])
            s = -s if backward else s
            x0, x1 = x[t, :, a], x[t, :, b]
            y[t, :, a], y[t, :, b] = x0 * c - x1 * s, x1 * c + x0 * s
            size[t, :, a] = size[t, :, b] = np.abs(x0) + np.abs(x1)
    return y, size


def slots(c: Cache, starts, n_tokens):
    """(token, sequence, slot) of every token that is somebody's."""
    for b, (a, n) in enumerate(chunks(starts, n_tokens)):
        for i in range(n):
            yield a + i, b, c.length(b) - n + i


def append(c: Cache, k_bits, v_bits, starts, positions=None):
    """k_bits, v_bits [n, H, d], k rotated already."""
    for t, b, slot in slots(c, starts, len(k_bits)):
        where = c.at(b, slot) if slot >= 0 else None
        if where is None:
            continue
        c.k[where[0], :, where[1]], c.v[where[0], :, where[1]] = k_bits[t], v_bits[t]
        if c.weight is not None:
            c.weight[b * c.H: (b + 1) * c.H, slot] = 0
            c.pos[b * c.H: (b + 1) * c.H, slot] = slot if positions is None else positions[t]


def _row(q, k, v, scale):
    """Attention of one query over its keys: out, lse, weights, and for a bound the largest
    |scale| sum |q k| and sum p |v|."""
    if not len(k):
        return np.zeros(q.shape), -np.inf, np.zeros(0), 0.0, np.zeros(q.shape)
    s = scale * (k @ q)
    top = s.max()
    e = np.exp(s - top)
    p = e / e.sum()
    return p @ v, top + np.log(e.sum()), p, float((np.abs(scale) * (np.abs(k) @ np.abs(q))).max()), p @ np.abs(v)


def attend(c: Cache, q, starts, scale=0.0, max_new=0):
    """q fp64 [n, Hq, d].  Returns dict(out, lse, add, absdot, absout, mine): add [B * H, room] what the
    weights grow by, with add_err its relative error per unit of absdot, mine the tokens
    that are somebody's."""
    n, Hq, d = q.shape
    G = Hq // c.H
    scale = scale or 1.0 / np.sqrt(d)
    out, lse = np.zeros(q.shape), np.full((n, Hq), -np.inf)
    absdot, absout = np.zeros((n, Hq)), np.zeros(q.shape)
    room = c.table.shape[1] * c.bs
    add, add_dot = np.zeros((c.B * c.H, room)), np.zeros((c.B * c.H, room))
    mine = np.zeros(n, bool)
    for b, (a, m) in enumerate(chunks(starts, n, max_new)):
        L = c.length(b)
        t = np.array([x for x in range(L) if c.at(b, x)], np.int64)
        pg = c.table[b, t // c.bs].astype(np.int64)
        for h in range(c.H):
            k, v = widen(c.k[pg, h, t % c.bs]), widen(c.v[pg, h, t % c.bs])
            for i in range(m):
                see = t <= L - m + i
                for g in range(G):
                    row = (a + i, h * G + g)
                    out[row], lse[row], p, absdot[row], absout[row] = _row(q[row], k[see], v[see], scale)
                    add[b * c.H + h, t[see]] += p
                    add_dot[b * c.H + h, t[see]] += p * absdot[row]
        mine[a: a + m] = True
    return dict(out=out, lse=lse, add=add, add_dot=add_dot, absdot=absdot, absout=absout, mine=mine)


def prompt(q, k, v, starts, scale=0.0):
    """fp64 [n, Hq, d], [n, H, d].  As attend, without weights."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    out, lse = np.zeros(q.shape), np.full((n, Hq), -np.inf)
    absdot, absout, mine = np.zeros((n, Hq)), np.zeros(q.shape), np.zeros(n, bool)
    for a, m in chunks(starts, n):
        for i in range(m):
            for x in range(Hq):
                row = (a + i, x)
                out[row], lse[row], _, absdot[row], absout[row] = _row(q[row], k[a: a + i + 1, x // G], v[a: a + i + 1, x // G], scale)
        mine[a: a + m] = True
    return dict(out=out, lse=lse, absdot=absdot, absout=absout, mine=mine)


def evict(c: Cache, seen, budget, sinks, recent):
    used = [int(c.table[b, j]) for b in range(c.B) for j in range(-(-c.length(b) // c.bs))]
    for b in range(c.B):
        L = c.length(b)
        if L <= budget:
            continue
        below = [int(p) for p in c.table[b, : -(-budget // c.bs)] if 0 <= p < c.n]
        if any(used.count(p) > 1 for p in below):          # somebody else's too
            continue
        for h in range(c.H):
            n = b * c.H + h

            def order(t):
                p = int(c.pos[n, t])
                if p < sinks:
                    return (0, 0.0, p, t)
                if p >= int(seen[b]) - recent:
                    return (1, 0.0, -p, t)
                w = float(c.weight[n, t])
                return (2, np.inf if np.isnan(w) else -w, p, t)

            stay = set(sorted(range(L), key=order)[:budget])
            holes = [t for t in range(budget) if t not in stay]
            movers = sorted(t for t in stay if t >= budget)
            for src, dst in zip(movers, holes):
                x, y = c.at(b, src), c.at(b, dst)
                if x and y:
                    c.k[y[0], h, y[1]], c.v[y[0], h, y[1]] = c.k[x[0], h, x[1]], c.v[x[0], h, x[1]]
                c.weight[n, dst], c.pos[n, dst] = c.weight[n, src], c.pos[n, src]
        c.lens[b] = budget
