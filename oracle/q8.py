"""Oracle of the 8-bit paged cache: codes, scales, store, load, append, attention.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Codes are uint8 arrays (raw bits of e4m3 or int8).  Code and scale arithmetic
is the fp32 one that include/kvc.h states, one rounding per operation, so codes
and scales can be compared bit for bit; the attention is fp64.  Everything
loops over sequences, heads and pages.
"""
from __future__ import annotations

import numpy as np

E4M3, INT8 = 0, 1
f32 = np.float32


def _e4m3_table() -> np.ndarray:
    """Value of every e4m3 code (1 sign, 4 exponent bits with bias 7, 3 fraction
    bits; exponent 0 is subnormal; S.1111.111 is NaN, there is no infinity)."""
    out = np.empty(256, dtype=np.float64)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = np.nan if (e == 15 and m == 7) else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out[c] = -v if s else v
    return out


E4M3_VALUES = _e4m3_table()


def decode(codes: np.ndarray, fmt: int) -> np.ndarray:
    """fp64 values of codes (without scale)."""
    c = np.asarray(codes, dtype=np.uint8)
    return E4M3_VALUES[c] if fmt == E4M3 else c.view(np.int8).astype(np.float64)


def encode(y: np.ndarray, fmt: int) -> np.ndarray:
    """Codes of fp32 values already divided by the scale: nearest, ties to even.
    The sign of a zero follows y for e4m3."""
    y = np.asarray(y, dtype=f32)
    if fmt == INT8:
        return np.rint(y).astype(np.int8).view(np.uint8)
    pos = E4M3_VALUES[:127]                      # 0 .. 448, ascending
    a = np.abs(y.astype(np.float64))
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (pick | (np.signbit(y).astype(np.int64) << 7)).astype(np.uint8)


def page_scale(amax: float, fmt: int):
    """fp32 (scale, 1 / scale) of a page whose largest magnitude is amax."""
    amax = f32(amax)
    if fmt == E4M3:
        e = -126
        while float(amax) > 448.0 * 2.0 ** e:
            e += 1
        return f32(2.0 ** e), f32(2.0 ** -e)
    s = max(f32(amax / f32(127.0)), f32(2.0 ** -126))
    return s, f32(1.0) / s


def _bf16_f32(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(f32)


def _to_bf16(x: np.ndarray) -> np.ndarray:
    b = np.ascontiguousarray(x, dtype=f32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


class Cache:
    """codes [n, H, bs, d] uint8, scales [n, H] fp32, table [B, tb], lens [B]."""

    def __init__(self, k, v, ks, vs, table, lens, fmt, max_len=0):
        self.k, self.v, self.ks, self.vs = k.copy(), v.copy(), ks.copy(), vs.copy()
        self.table, self.lens, self.fmt = np.asarray(table), np.asarray(lens), fmt
        self.n, self.H, self.bs, self.d = k.shape
        self.B, tb = self.table.shape
        room = tb * self.bs
        self.cap = min(max_len, room) if max_len > 0 else room

    def length(self, b):
        return int(min(max(int(self.lens[b]), 0), self.cap))

    def page(self, b, j):
        p = int(self.table[b, j])
        return p if 0 <= p < self.n else -1

    def both(self):
        return ((self.k, self.ks), (self.v, self.vs))


def store(c: Cache, k, v, T, kept=None):
    """k, v: bf16 bits [B*H, t_stride, d]."""
    for b in range(c.B):
        top = T if kept is None else kept.shape[1]
        L = min(c.length(b), top)
        for h in range(c.H):
            n = b * c.H + h
            for s0 in range(0, L, c.bs):
                p = c.page(b, s0 // c.bs)
                if p < 0:
                    continue
                rows = min(c.bs, L - s0)
                src = [T - L + s0 + r if kept is None else int(kept[n, s0 + r]) for r in range(rows)]
                for rowsrc, (codes, scales) in zip((k, v), c.both()):
                    x = np.zeros((rows, c.d), f32)
                    for r, t in enumerate(src):
                        if 0 <= t < T:
                            x[r] = _bf16_f32(rowsrc[n, t])
                    s, inv = page_scale(np.abs(x).max(), c.fmt)
                    scales[p, h] = s
                    codes[p, h, :rows] = encode(x * inv, c.fmt)


def load(c: Cache, T):
    """bf16 bits [B*H, T, d] of K and V, left-padded."""
    out = []
    for codes, scales in c.both():
        y = np.zeros((c.B * c.H, T, c.d), np.uint16)
        for b in range(c.B):
            L = c.length(b)
            for t in range(max(0, L - T), L):
                p = c.page(b, t // c.bs)
                if p >= 0:
                    for h in range(c.H):
                        val = decode(codes[p, h, t % c.bs], c.fmt).astype(f32) * scales[p, h]
                        y[b * c.H + h, T - L + t] = _to_bf16(val)
        out.append(y)
    return out


def append(c: Cache, k_new, v_new, n_new=None):
    """k_new, v_new: bf16 bits [B*H, W, d]; the last n_new[b] rows of each."""
    W = k_new.shape[1]
    for b in range(c.B):
        L = c.length(b)
        mine = W if n_new is None else min(max(int(n_new[b]), 0), W)
        first = max(L - mine, 0)
        if first >= L:
            continue
        for j in range(first // c.bs, -(-L // c.bs)):
            p = c.page(b, j)
            if p < 0:
                continue
            s0 = j * c.bs
            a, e = max(first, s0) - s0, min(c.bs, L - s0)
            for h in range(c.H):
                for new, (codes, scales) in zip((k_new, v_new), c.both()):
                    x = _bf16_f32(new[b * c.H + h, s0 + a - (L - W): s0 + e - (L - W)])
                    s, inv = page_scale(np.abs(x).max(), c.fmt)
                    old = scales[p, h]
                    if a > 0:
                        if old >= s:
                            s, inv = old, f32(1.0) / old
                        else:
                            ratio = f32(old / s) if c.fmt == E4M3 else f32(old * inv)
                            was = decode(codes[p, h, :a], c.fmt).astype(f32)
                            codes[p, h, :a] = encode(was * ratio, c.fmt)
                    scales[p, h] = s
                    codes[p, h, a:e] = encode(x * inv, c.fmt)


def attend(c: Cache, q, scale=0.0):
    """fp64 attention.  q: fp64 [B*H, G, W, d].  Returns out, lse and for an error
    bound: the largest |scale * sum |q k|| of each row, sum p |v|, and
    max(p * vs) * sum |code_v|."""
    NH, G, W, d = q.shape
    scale = scale or 1.0 / np.sqrt(d)
    out = np.zeros(q.shape)
    lse = np.full((NH, G, W), -np.inf)
    absdot, absout, tail = np.zeros((NH, G, W)), np.zeros(q.shape), np.zeros((NH, G, W))
    for b in range(c.B):
        L = c.length(b)
        pos = np.arange(L)
        pages = np.array([c.page(b, j) for j in range(-(-L // c.bs))], dtype=np.int64)
        seen = pages[pos // c.bs] >= 0 if L else np.zeros(0, bool)
        pos = pos[seen]
        pg, sl = (pages[pos // c.bs], pos % c.bs) if L else (pos, pos)
        for h in range(c.H):
            n = b * c.H + h
            k = decode(c.k[pg, h, sl], c.fmt) * c.ks[pg, h].astype(np.float64)[:, None]
            vcode = decode(c.v[pg, h, sl], c.fmt)
            vs = c.vs[pg, h].astype(np.float64)
            v = vcode * vs[:, None]
            for w in range(W):
                m = pos <= L - W + w
                if not m.any():
                    continue
                s = scale * q[n, :, w] @ k[m].T                      # [G, T]
                top = s.max(1, keepdims=True)
                e = np.exp(s - top)
                p = e / e.sum(1, keepdims=True)
                out[n, :, w] = p @ v[m]
                lse[n, :, w] = top[:, 0] + np.log(e.sum(1))
                absdot[n, :, w] = (scale * np.abs(q[n, :, w]) @ np.abs(k[m]).T).max(1)
                absout[n, :, w] = p @ np.abs(v[m])
                tail[n, :, w] = (p * vs[m]).max(1) * np.abs(vcode[m]).sum(0).max()
    return out, lse, absdot, absout, tail
