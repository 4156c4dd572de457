"""Seeded bf16 paged caches for the tests, and error bounds of their operators."""
from __future__ import annotations

import numpy as np
import torch

from eviction_window_qk_amd import kvc, synth
from oracle import paged as og
from q8_utils import dev_bf16, random_rows, rng_of

NAN = np.uint16(0x7FC0)


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def random_cache(seed, B, H, d, bs, lens, tb=None, spare=3, holes=0.0, weights=False, max_len=0):
    """Oracle cache of random rows: pages in random order, rows that no slot below a
    length holds are NaN, and so are pages that no table names."""
    rng = rng_of(seed, B, H, d, bs)
    lens = np.asarray(lens, np.int32)
    tb = tb or max(1, -(-max(int(lens.max(initial=0)), 1) // bs))
    n = B * tb + spare
    table = rng.permutation(n)[: B * tb].reshape(B, tb).astype(np.int32)
    if holes:
        table = np.where(rng.random((B, tb)) < holes, rng.choice([-1, n, -2 ** 31], (B, tb)), table).astype(np.int32)
    used = np.zeros((n, bs), bool)
    for b in range(B):
        for t in range(min(int(lens[b]), tb * bs)):
            if 0 <= table[b, t // bs] < n:
                used[table[b, t // bs], t % bs] = True
    pools = [np.where(used[:, None, :, None], random_rows(seed + i, n, H, bs, d), NAN) for i in (1, 2)]
    w = p = None
    if weights:
        w = rng.random((B * H, tb * bs)).astype(np.float32)
        p = np.tile(np.arange(tb * bs, dtype=np.int32), (B * H, 1))
    return og.Cache(pools[0], pools[1], table, lens, w, p, max_len=max_len)


def to_gpu(c: og.Cache, max_len=0) -> kvc.PagedCache:
    return kvc.PagedCache(dev_bf16(c.k), dev_bf16(c.v), dev(c.table.astype(np.int32)), dev(c.lens),
                          weight=None if c.weight is None else dev(c.weight),
                          pos=None if c.pos is None else dev(c.pos), max_len=max_len)


def same_cache(g: kvc.PagedCache, c: og.Cache):
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(g.k_pool), c.k)
    np.testing.assert_array_equal(bits(g.v_pool), c.v)
    np.testing.assert_array_equal(g.seq_len.cpu().numpy(), c.lens)
    if c.weight is not None:
        np.testing.assert_array_equal(g.weight.cpu().numpy().view(np.uint32), c.weight.view(np.uint32))
        np.testing.assert_array_equal(g.pos.cpu().numpy(), c.pos)


def starts_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def check_rope(got_bits, ref, size, mscale):
    """Rotated rows against fp64.  A cosine or sine is off by 2^-20 of mscale at most (the
    turn, reduced in fp64, is rounded to 24 bits: 2^-23 radians; the function's own
    few last places; its product with mscale), two products and a sum in fp32 by 2^-22 of
    |x0| + |x1|, the result by half a bf16 step, 2^-8 of itself (or 2^-134)."""
    err = np.abs(og.widen(got_bits) - ref)
    m = abs(mscale)
    bound = size * m * (2.0 ** -20 + 2.0 ** -22) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + 2.0 ** -134
    bad = ~(err <= np.where(size > 0, bound, 0))
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, worst {np.nanmax(err[bad])}"


def check_attention(ref, out_bits, lse, T, untouched=None):
    """out (bits) and lse of the tokens that are somebody's against the fp64 oracle.

    Error sources, each at its largest:
      ds  a score: the fp32 sum of d exact products and the few roundings of its
          product with scale and of the reference's, (d + 8) * 2^-23 of sum |q k|
      p   a weight: 2 ds, exp2 at 2^-22; sums of T terms in fp32, T * 2^-24
      w   a weight in bf16: 2^-8 of itself
      out bf16, 2^-8 of itself
    """
    m = ref["mine"]
    d = ref["out"].shape[-1]
    got = og.widen(out_bits)
    ds = ref["absdot"] * (d + 8) * 2.0 ** -23
    rel = 2.0 ** -8 + 2 * ds + 2.0 ** -20 + T * 2.0 ** -24
    bound = rel[..., None] * ref["absout"] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref["out"]) + 1e-37
    err = np.abs(got - ref["out"])
    bad = ~(err <= bound) & m[:, None, None]
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} outputs off; worst {np.nanmax((err / bound)[bad]):.3g} of the "
                           f"bound, first at {np.argwhere(bad)[0]}")
    empty = np.isneginf(ref["lse"])
    np.testing.assert_array_equal(got[empty & m[:, None]], 0.0)
    lb = ds + 2.0 ** -20 + T * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(empty, 0, ref["lse"]))
    if lse is not None:
        gl = lse.cpu().numpy().astype(np.float64)
        np.testing.assert_array_equal(np.isneginf(gl)[m], empty[m])
        diff = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, ref["lse"]))
        assert (diff <= lb)[m].all(), f"lse off by {np.max((diff / lb)[m]):.3g} of the bound"
    if untouched is not None:
        np.testing.assert_array_equal(out_bits[~m], untouched)
    return lb


def check_weights(ref, before, after, d, rows):
    """What the slots' weights grew by: a softmax weight is off by its score's and its
    lse's error (2 * (d + 8) * 2^-23 of sum |q k| each way, see check_attention), exp2 and the product
    with log2(e) in fp32 of numbers up to |lse|, 2^-18 together; the sum over `rows` in fp32, and
    its own addition."""
    add = after.astype(np.float64) - before.astype(np.float64)
    L = np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0)).max(initial=0.0)
    T = ref["add"].shape[1]
    bound = (ref["add_dot"] * 3 * (d + 8) * 2.0 ** -23 + ref["add"] * (2.0 ** -18 + L * 2.0 ** -21 + (rows + T) * 2.0 ** -24)
             + 2.0 ** -23 * (np.abs(before) + ref["add"]) + 2.0 ** -120)
    err = np.abs(add - ref["add"])
    bad = ~(err <= np.where(ref["add"] > 0, bound, 2.0 ** -120))
    assert not bad.any(), f"{int(bad.sum())} weights off, worst {np.max((err / bound)[bad]):.3g} of the bound at {np.argwhere(bad)[0]}"
