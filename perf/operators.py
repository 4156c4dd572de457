"""The operators of the 8-bit paged cache, as they are measured.

A serving loop keeps the cache that the compression event leaves behind in pages
of 8-bit codes, one fp32 scale for each (page, KV head).  Five operators work on
it, and `run` makes one pass through one of them:

  attend   the new tokens' queries attend to the cache (decode, or a few drafted
           tokens at once)
  store    rows of a bf16 cache, all of them or the kept ones of an event, are
           written as 8-bit pages, and read back as bf16 rows
  append   the new tokens' rows go into each sequence's open page, whose scale
           grows where they do not fit, and the open end is read back
  fork     sequences are freed, forked again from others (whole pages shared, the
           open page copied) and given pages for what they decode next
  compact  the live pages move to the front of the pool, tables and counts follow

With `own` false the passes are plain torch operations in 32 bits, with `own`
true they are the calls of the library's binding.  Sizes are those of the
repository's Qwen-7B and Llama-8B shaped workloads and of its tiny one.

8-bit formats.  e4m3: scale = 2^e with the smallest e >= -126 that has
amax <= 448 * 2^e; code = x / scale rounded to nearest even.  int8:
scale = max(amax / 127, 2^-126); code = rint(x * (1 / scale)).  amax is taken
over the rows of one page and head.  A page that grows by an append keeps its
scale unless the new rows alone would need a larger one; then the rows that are
there are coded again: e4m3 rounds code * old / new, int8 rint(code * (old * (1 / new))).
"""
import math

import torch

own = False

E4M3, INT8 = "e4m3", "int8"
_TINY = 2.0 ** -126


def listed():
    return [
        # One short sequence of the tiny workload: nothing but latency.
        dict(name="attend_tiny", op="attend", fmt=E4M3, B=1, H=1, G=1, W=1, d=64, bs=16, lo=128, hi=128, holes=False),
        # One layer's decode step of the Qwen-shaped batch on its compressed cache (1024 kept, then decoded on).
        dict(name="attend_qwen_decode", op="attend", fmt=INT8, B=64, H=4, G=7, W=1, d=128, bs=16, lo=1024, hi=1152, holes=False),
        # One layer's decode step on the uncompressed 131072-token cache of one sequence.
        dict(name="attend_llama_128k", op="attend", fmt=E4M3, B=1, H=8, G=4, W=1, d=128, bs=64, lo=131072, hi=131072, holes=False),
        # Five drafted tokens of a ragged batch: empty and one-token sequences, pages of 24 rows, pages taken out.
        dict(name="attend_draft_ragged", op="attend", fmt=INT8, B=24, H=8, G=4, W=5, d=64, bs=24, lo=0, hi=16384, holes=True),
        # The Qwen-shaped event's kept rows become pages, all layers at once.
        dict(name="store_qwen_event", op="store", fmt=INT8, B=448, H=4, d=128, bs=16, T=768, K=256, lo=256, hi=256),
        # A prefilled 16K cache (four sequences of different lengths) becomes pages whole.
        dict(name="store_llama_16k", op="store", fmt=E4M3, B=4, H=8, d=128, bs=64, T=16384, K=0, lo=12001, hi=16384),
        # One token of one layer's batch.
        dict(name="append_qwen_layer", op="append", fmt=E4M3, B=16, H=4, W=1, d=128, bs=16, lo=256, hi=768),
        # Six tokens, odd pages, all layers of a batch.
        dict(name="append_drafts", op="append", fmt=INT8, B=1184, H=8, W=6, d=64, bs=24, lo=0, hi=400),
        # Two prompts sampled seven times each.
        dict(name="fork_samples", op="fork", fmt=E4M3, P=2, C=7, H=4, d=128, bs=16, lo=700, hi=768, spare=64),
        # A beam round of 64 prompts with eight beams each, on large pages.
        dict(name="fork_beams", op="fork", fmt=INT8, P=64, C=8, H=8, d=128, bs=128, lo=1, hi=4096, spare=700),
        # A small pool, half of its pages freed.
        dict(name="compact_small", op="compact", fmt=INT8, n=999, B=9, H=4, d=64, bs=24, live=0.5),
        # The pool of the Llama-shaped batch after half of its sequences have ended.
        dict(name="compact_large", op="compact", fmt=E4M3, n=32768, B=96, H=8, d=128, bs=16, live=0.6),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "store", "append", "fork", "compact"])
    c = dict(op=op, fmt=rng.choice([E4M3, INT8]), d=rng.choice([64, 128]), H=rng.randint(1, 9),
             bs=rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 100, 128, 256]))
    room = 1 << 23  # rows of one head, over all sequences and heads: 2 GB of codes at most
    if op == "attend":
        hi = _log(rng, 1, 131072)
        B = _log(rng, 1, max(1, min(256, (1 << 20) // hi // c["H"])))
        c.update(B=B, G=rng.randint(1, 12), W=rng.choice([1, 1, 1, 2, 5, 9]), hi=hi,
                 lo=rng.choice([0, hi, max(1, hi // 2)]), holes=rng.random() < 0.25)
    elif op == "store":
        T = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(448, (1 << 19) // T // c["H"])))
        K = rng.choice([0, max(1, T // 3), T])
        top = K or T
        c.update(B=B, T=T, K=K, hi=top, lo=rng.choice([0, top, top // 2]))
    elif op == "append":
        hi = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(1792, (room >> 2) // hi // c["H"])))
        c.update(B=B, W=rng.choice([1, 1, 2, 6, 17]), hi=hi, lo=rng.choice([0, hi // 2]))
    elif op == "fork":
        hi = _log(rng, 1, 4096)
        c.update(P=rng.randint(1, 32), C=rng.randint(1, 8), hi=hi, lo=rng.choice([1, hi]), spare=rng.choice([40, 600]))
        if c["bs"] < 16:
            c["hi"], c["lo"] = min(hi, 512), min(c["lo"], 512)
    else:
        n = _log(rng, 3, max(3, min(30000, (room >> 1) // (c["H"] * c["bs"]))))
        c.update(n=n, B=rng.randint(1, 100), live=rng.choice([0.0, 0.3, 0.6, 0.9, 1.0]))
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pow2(e):
    """2^e in fp32 for int32 e in -126..127, from its bits: exp2 and ldexp may be off by a step on the GPU."""
    return ((e + 127) << 23).view(torch.float32)


def _scale_of(amax, fmt):
    """fp32 scale of an fp32 amax."""
    if fmt == E4M3:
        m, e = torch.frexp(amax)                      # amax = m * 2^e, 0.5 <= m < 1
        e = torch.where(m > 0.875, e - 8, e - 9)      # 448 = 0.875 * 2^9
        e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
        return _pow2(e)
    return (amax / torch.full_like(amax, 127.0)).clamp(min=_TINY)   # a tensor: a division, not a product


def _code(x, scale, fmt):
    """Codes of x (fp32) under broadcast scales."""
    y = x * (1.0 / scale)
    if fmt == E4M3:
        return y.to(torch.float8_e4m3fn)
    return torch.round(y).to(torch.int8)


def _dtype(fmt):
    return torch.float8_e4m3fn if fmt == E4M3 else torch.int8


def _lens(c, g, B):
    lo, hi = c["lo"], c["hi"]
    n = torch.randint(lo, hi + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    if B > 2 and lo == 0:
        n[0], n[1], n[2] = 0, min(1, hi), hi
    return n


def _tables(c, g, lens, capacity, spare):
    """Tables of distinct pages in random order, -1 behind each sequence's last
    page.  Every sequence gets `capacity` rows of room at most."""
    bs, B = c["bs"], lens.numel()
    nb = max(1, -(-capacity // bs))
    n_blocks = B * nb + spare
    order = torch.randperm(n_blocks, generator=g, device="cuda", dtype=torch.int32)[: B * nb].reshape(B, nb)
    used = (lens + bs - 1) // bs
    table = torch.where(torch.arange(nb, device="cuda")[None] < used[:, None], order, torch.full_like(order, -1))
    return table.contiguous(), n_blocks


def _pools(c, g, n_blocks):
    """K and V pools of codes with the spread that coded normal values have, and
    scales that differ from page to page and head to head."""
    shape = (n_blocks, c["H"], c["bs"], c["d"])
    pools, scales = [], []
    for _ in range(2):
        if c["fmt"] == E4M3:
            raw = torch.randint(0, 0x7F, shape, generator=g, device="cuda", dtype=torch.uint8)      # finite
            sign = torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7
            # exponents of a normal sample: few codes are far below the largest
            raw = torch.maximum(raw, torch.randint(0, 0x7F, shape, generator=g, device="cuda", dtype=torch.uint8))
            pools.append((raw | sign).view(torch.float8_e4m3fn))
            e = torch.randint(-9, -6, shape[:2], generator=g, device="cuda", dtype=torch.int32)
            scales.append(_pow2(e))
        else:
            pools.append(torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8))
            scales.append(torch.rand(shape[:2], generator=g, device="cuda") * 0.02 + 0.01)
    return pools, scales


def _rows(g, *shape):
    """bf16 rows of normal values whose norms are log-normal, as keys' are."""
    x = torch.randn(shape, generator=g, device="cuda")
    r = torch.randn(shape[:-1], generator=g, device="cuda").mul_(0.5).exp_()
    return x.mul_(r[..., None]).to(torch.bfloat16)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"c": c}
    op, H, d, bs = c["op"], c["H"], c["d"], c["bs"]
    if op == "attend":
        s["len"] = _lens(c, g, c["B"])
        s["table"], n = _tables(c, g, s["len"], c["hi"], 8)
        if c["holes"]:   # pages taken out of the tables
            gone = torch.rand(s["table"].shape, generator=g, device="cuda") < 0.1
            s["table"] = torch.where(gone, torch.full_like(s["table"], -1), s["table"]).contiguous()
        (s["k"], s["v"]), (s["ks"], s["vs"]) = _pools(c, g, n)
        s["q"] = torch.randn((c["B"] * H, c["G"], c["W"], d), generator=g, device="cuda").to(torch.bfloat16)
    elif op == "store":
        s["len"] = _lens(c, g, c["B"])
        s["table"], n = _tables(c, g, s["len"], c["K"] or c["T"], 8)
        (s["k"], s["v"]), (s["ks"], s["vs"]) = _pools(c, g, n)
        s["k_rows"], s["v_rows"] = _rows(g, c["B"] * H, c["T"], d), _rows(g, c["B"] * H, c["T"], d)
        s["kept"] = None
        if c["K"]:       # K of T positions, ascending
            pick = torch.rand((c["B"] * H, c["T"]), generator=g, device="cuda").argsort(1)[:, : c["K"]]
            s["kept"] = pick.sort(1).values.to(torch.int32).contiguous()
    elif op == "append":
        old = _lens(c, g, c["B"])
        s["len"] = old + c["W"]
        s["table"], n = _tables(c, g, s["len"], c["hi"] + c["W"], 8)
        (s["k"], s["v"]), (s["ks"], s["vs"]) = _pools(c, g, n)
        s["k_new"], s["v_new"] = _rows(g, c["B"] * H, c["W"], d), _rows(g, c["B"] * H, c["W"], d)
    elif op == "fork":
        P, C = c["P"], c["C"]
        B = P * (C + 1)
        lens = _lens(c, g, P)
        s["src"] = torch.arange(P, device="cuda", dtype=torch.int32).repeat_interleave(C)
        s["dst"] = torch.arange(P, B, device="cuda", dtype=torch.int32)
        parents, n = _tables(c, g, lens, c["hi"], c["spare"])
        s["table"] = torch.full((B, parents.shape[1] + 1), -1, device="cuda", dtype=torch.int32)
        s["table"][:P, :-1] = parents
        s["len"] = torch.zeros(B, device="cuda", dtype=torch.int32)
        s["len"][:P] = lens
        s["refs"] = torch.zeros(n, device="cuda", dtype=torch.int32)
        s["refs"][parents[parents >= 0].long()] = 1
        s["want"] = torch.zeros(B, device="cuda", dtype=torch.int32)
        s["want"][P:] = lens.repeat_interleave(C) + 1      # one more token each
        (s["k"], s["v"]), (s["ks"], s["vs"]) = _pools(c, g, n)
    else:
        n, B = c["n"], c["B"]
        live = torch.rand(n, generator=g, device="cuda") < c["live"]
        ids = torch.nonzero(live)[:, 0].to(torch.int32)
        ids = ids[torch.randperm(ids.numel(), generator=g, device="cuda")]
        nb = -(-n // B) + 2
        s["table"] = torch.full((B, nb), -1, device="cuda", dtype=torch.int32)
        flat = torch.full((B * (nb - 2),), -1, device="cuda", dtype=torch.int32)
        flat[: ids.numel()] = ids
        s["table"][:, : nb - 2] = flat.reshape(B, nb - 2)
        s["refs"] = live.to(torch.int32)
        if ids.numel() and B > 1:                          # the first pages are shared with the last sequence
            share = s["table"][0, : nb - 2]
            got = share >= 0
            s["table"][B - 1, : nb - 2] = torch.where(got, share, s["table"][B - 1, : nb - 2])
            s["refs"] = torch.zeros(n + 1, device="cuda", dtype=torch.int32)
            at = torch.where(s["table"] >= 0, s["table"], torch.full_like(s["table"], n)).reshape(-1).long()
            s["refs"].scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
            s["refs"] = s["refs"][:n].contiguous()
        s["len"] = (s["table"] >= 0).sum(1).to(torch.int32) * bs
        (s["k"], s["v"]), (s["ks"], s["vs"]) = _pools(c, g, n)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _grab(pool, scale, table, dtype=torch.float32):
    """[B, H, nb * bs, d] values of the tables' pages; pages that are not there
    give zeros."""
    B, nb = table.shape
    n, H, bs, d = pool.shape
    there = (table >= 0) & (table < n)
    at = table.clamp(0, n - 1).long()
    x = pool.view(torch.uint8)[at].view(pool.dtype).to(dtype) * scale[at].to(dtype)[..., None, None]
    x = x.masked_fill(~there[..., None, None, None], 0)
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, nb * bs, d), there.repeat_interleave(bs, 1)


def _attend(s, c):
    B, H, G, W, d = c["B"], c["H"], c["G"], c["W"], c["d"]
    k, there = _grab(s["k"], s["ks"], s["table"])
    v, _ = _grab(s["v"], s["vs"], s["table"])
    q = s["q"].float().reshape(B, H, G * W, d)
    t = torch.arange(k.shape[2], device="cuda")
    end = s["len"][:, None].long() - W + torch.arange(W, device="cuda")[None]          # [B, W] last position seen
    mask = there[:, None, :] & (t[None, None] <= end[..., None])                       # [B, W, T]
    mask = mask[:, None, None].expand(B, H, G, W, -1).reshape(B, H, G * W, -1)
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = x.masked_fill(~mask, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    return out.to(torch.bfloat16).reshape(B * H, G, W, d), lse.reshape(B * H, G, W)


def _write(pool, scale, pages, ok, rows, amax_rows, fmt):
    """Codes `rows` [N, H, bs, d] into pages [N] at the slots where ok [N, bs] is
    set, under the scale of amax_rows [N, H]."""
    sc = _scale_of(amax_rows, fmt)
    codes = _code(rows, sc[..., None, None], fmt).view(torch.uint8)
    raw = pool.view(torch.uint8)
    raw[pages] = torch.where(ok[:, None, :, None], codes, raw[pages])
    scale[pages] = sc


def _store(s, c):
    B, H, d, bs, T = c["B"], c["H"], c["d"], c["bs"], c["T"]
    nb, n = s["table"].shape[1], s["k"].shape[0]
    j = torch.arange(nb * bs, device="cuda")
    if s["kept"] is None:
        length = s["len"].long()
        row = (T - length)[:, None, None] + j
        row = row.expand(B, H, -1)
    else:
        length = s["len"].long().clamp(max=c["K"])
        row = s["kept"].long().reshape(B, H, -1)[..., : nb * bs]
        row = torch.nn.functional.pad(row, (0, nb * bs - row.shape[-1]), value=-1)
    ok = (j[None] < length[:, None]).reshape(B, nb, bs)
    at = torch.nonzero(ok.any(-1) & (s["table"] >= 0) & (s["table"] < n))              # pages that get rows
    pages, ok = s["table"][at[:, 0], at[:, 1]].long(), ok[at[:, 0], at[:, 1]]
    live = ((row >= 0) & (row < T)).reshape(B, H, nb, bs)
    for rows, pool, scale in ((s["k_rows"], s["k"], s["ks"]), (s["v_rows"], s["v"], s["vs"])):
        x = rows.reshape(B, H, T, d).gather(2, row.clamp(0, T - 1)[..., None].expand(-1, -1, -1, d)).float()
        x = x.reshape(B, H, nb, bs, d).masked_fill(~live[..., None], 0).permute(0, 2, 1, 3, 4)
        x = x[at[:, 0], at[:, 1]].masked_fill(~ok[:, None, :, None], 0)
        _write(pool, scale, pages, ok, x, x.abs().amax((2, 3)), c["fmt"])
    return _load(s, c, c["K"] or T)


def _load(s, c, T):
    """The last T positions as bf16 rows, position t in row T - len + t."""
    B, H, d = c["B"], c["H"], c["d"]
    back = []
    t = torch.arange(T, device="cuda")[None] - T + s["len"].long()[:, None]            # position of each row
    for pool, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        x, _ = _grab(pool, scale, s["table"])
        at = t.clamp(0, x.shape[2] - 1)[:, None, :, None].expand(B, H, T, d)
        x = x.gather(2, at).masked_fill(((t < 0) | (t >= x.shape[2]))[:, None, :, None], 0)
        back.append(x.to(torch.bfloat16).reshape(B * H, T, d))
    return back


def _append(s, c):
    B, H, W, d, bs, fmt = c["B"], c["H"], c["W"], c["d"], c["bs"], c["fmt"]
    nb, n = s["table"].shape[1], s["k"].shape[0]
    first = (s["len"].long() - W).clamp(min=0)                                          # first new position
    j = torch.arange(nb * bs, device="cuda")[None]
    new = (j >= first[:, None]) & (j < s["len"][:, None])
    new, old = new.reshape(B, nb, bs), (j < first[:, None]).reshape(B, nb, bs)
    at = torch.nonzero(new.any(-1) & (s["table"] >= 0) & (s["table"] < n))
    b, p = at[:, 0], at[:, 1]
    pages, new, old = s["table"][b, p].long(), new[b, p], old[b, p]
    w = p[:, None] * bs + torch.arange(bs, device="cuda")[None] - s["len"].long()[b, None] + W
    w = w.clamp(0, W - 1)                                                                # new row of each slot
    for rows, pool, scale in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        x = rows.float().reshape(B, H, W, d)[b].gather(2, w[:, None, :, None].expand(-1, H, -1, d))
        x = x.masked_fill(~new[:, None, :, None], 0)
        need = _scale_of(x.abs().amax((2, 3)), fmt)
        had = scale[pages]
        grown = torch.where(old.any(1)[:, None] & (had >= need), had, need)
        raw = pool.view(torch.uint8)
        was = raw[pages]
        codes = was.view(pool.dtype).float()
        if fmt == E4M3:
            again = (codes * (had / grown)[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            again = torch.round(codes * (had * (1.0 / grown))[..., None, None]).clamp(-127, 127).to(torch.int8)
        keep = torch.where((grown != had)[..., None, None] & old[:, None, :, None], again.view(torch.uint8), was)
        raw[pages] = torch.where(new[:, None, :, None], _code(x, grown[..., None, None], fmt).view(torch.uint8), keep)
        scale[pages] = grown
    return _load(s, c, bs + W)


def _release(refs, entries):
    """Each entry (page id, or negative for none) gives up its page."""
    n = refs.numel()
    at = torch.where((entries >= 0) & (entries < n), entries, torch.full_like(entries, n)).reshape(-1).long()
    less = torch.zeros(n + 1, device="cuda", dtype=torch.int32).scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    refs -= less[:n]


def _fork(s, c):
    bs, table, lens, refs, src, dst = c["bs"], s["table"], s["len"], s["refs"], s["src"].long(), s["dst"].long()
    n, nb = refs.numel(), table.shape[1]
    # the old children give up their pages
    _release(refs, table[dst])
    table[dst], lens[dst] = -1, 0
    # forked again: whole pages shared, an open page copied to the lowest free one
    length = lens[src]
    whole, part = length // bs, length % bs > 0
    free = torch.nonzero(refs <= 0)[:, 0]
    rank = torch.cumsum(part.int(), 0) - part.int()
    fits = torch.cumsum(part.int(), 0) <= free.numel()
    done = fits | ~part
    own_page = free[rank.clamp(max=max(0, free.numel() - 1)).long()] if free.numel() else torch.zeros_like(src)
    j = torch.arange(nb, device="cuda")[None]
    row = torch.where(j < whole[:, None], table[src], torch.full_like(table[src], -1))
    more = torch.zeros(n + 1, device="cuda", dtype=torch.int32)
    at = torch.where((row >= 0) & done[:, None], row, torch.full_like(row, n)).reshape(-1).long()
    refs += more.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:n]
    copied = part & done
    open_page = table[src].gather(1, whole[:, None].clamp(max=nb - 1).long())[:, 0]
    row = torch.where((j == whole[:, None]) & copied[:, None], own_page[:, None].to(torch.int32), row)
    table[dst] = torch.where(done[:, None], row, table[dst])
    lens[dst] = torch.where(done, length, lens[dst])
    fork_status = torch.where(done, 0, 1).to(torch.int32)
    to, frm = own_page[copied], open_page[copied].long()
    refs[to] = 1
    for buf in (s["k"], s["v"], s["ks"], s["vs"]):
        x = buf.view(torch.uint8) if buf.dtype != torch.float32 else buf
        x[to] = x[frm]
    # pages for what they decode next
    need = (j < ((s["want"] + bs - 1) // bs)[:, None]) & (table < 0)
    count = need.sum(1)
    free = torch.nonzero(refs <= 0)[:, 0]
    served = torch.cumsum(count, 0) <= free.numel()
    need &= served[:, None]
    rank = torch.cumsum(need.reshape(-1).int(), 0) - 1
    if free.numel():
        page = free[rank.clamp(0, free.numel() - 1).long()].reshape(table.shape).to(torch.int32)
        table.copy_(torch.where(need, page, table))
        refs[page[need].long()] = 1
    return dict(table=table, refs=refs, len=lens, fork_status=fork_status,
                alloc_status=torch.where(served | (count == 0), 0, 1).to(torch.int32), **_bytes(s))


def _bytes(s):
    """The pages themselves, as bytes, and the scales."""
    return dict(k=s["k"].view(torch.uint8), v=s["v"].view(torch.uint8), ks=s["ks"], vs=s["vs"])


def _compact(s, c):
    refs, table = s["refs"], s["table"]
    n = refs.numel()
    live = refs > 0
    count = live.sum()
    ids = torch.arange(n, device="cuda")
    holes, movers = torch.nonzero(~live & (ids < count))[:, 0], torch.nonzero(live & (ids >= count))[:, 0]
    remap = torch.where(live, ids, torch.full_like(ids, -1))
    remap[movers] = holes
    new_refs = torch.where(live & (ids < count), refs, torch.zeros_like(refs))
    new_refs[holes] = refs[movers]
    there = (table >= 0) & (table < n)
    new_table = torch.where(there, remap[table.clamp(0, n - 1).long()].to(torch.int32), torch.full_like(table, -1))
    for buf in (s["k"], s["v"], s["ks"], s["vs"]):
        x = buf.view(torch.uint8) if buf.dtype != torch.float32 else buf
        x[holes] = x[movers]
    return dict(table=new_table, refs=new_refs, remap=remap.to(torch.int32),
                n_live=count.to(torch.int32).reshape(1), **_bytes(s))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _handles(s):
    """What a serving loop keeps beside its tensors: the cache, its page table and
    the list of its buffers."""
    from eviction_window_qk_amd import kvc
    if "kvc" not in s:
        s["kvc"] = kvc
        if s["c"]["op"] not in ("fork", "compact"):
            s["cache"] = kvc.Q8Cache(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["len"])
        else:
            s["pages"] = kvc.PageTable(s["table"], s["len"], s["refs"], s["c"]["bs"])
            s["bufs"] = kvc.PageBuffers([s["k"], s["v"], s["ks"], s["vs"]])
    return s["kvc"]


def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if not own:
        if op == "attend":
            out, lse = _attend(s, c)
            return dict(out=out, lse=lse)
        if op == "store":
            k, v = _store(s, c)
            return dict(k=k, v=v, ks=s["ks"], vs=s["vs"])
        if op == "append":
            k, v = _append(s, c)
            return dict(k=k, v=v, ks=s["ks"], vs=s["vs"])
        return _fork(s, c) if op == "fork" else _compact(s, c)
    kvc = _handles(s)
    if op == "attend":
        out, lse = kvc.q8_attend(s["cache"], s["q"], want_lse=True)
        return dict(out=out, lse=lse)
    if op == "store":
        kvc.q8_store(s["cache"], s["k_rows"], s["v_rows"], kept=s["kept"])
        k, v = kvc.q8_load(s["cache"], c["K"] or c["T"])
        return dict(k=k, v=v, ks=s["ks"], vs=s["vs"])
    if op == "append":
        kvc.q8_append(s["cache"], s["k_new"], s["v_new"])
        k, v = kvc.q8_load(s["cache"], c["bs"] + c["W"])
        return dict(k=k, v=v, ks=s["ks"], vs=s["vs"])
    if op == "fork":
        kvc.pages_free(s["pages"], s["dst"])
        st = kvc.pages_fork(s["pages"], s["src"], s["dst"], s["bufs"])
        al = kvc.pages_alloc(s["pages"], s["want"])
        return dict(table=s["table"], refs=s["refs"], len=s["len"], fork_status=st, alloc_status=al, **_bytes(s))
    got = kvc.pages_compact(s["pages"], s["bufs"])
    return dict(table=got["table"], refs=got["refs"], remap=got["remap"], n_live=got["n_live"], **_bytes(s))


def work(case):
    c = case
    H, d, bs = c["H"], c["d"], c["bs"]
    page = 2 * (H * bs * d + H * 4)                       # K and V codes of one page, with their scales
    if c["op"] == "attend":
        rows = c["B"] * H * (c["lo"] + c["hi"]) / 2 * (0.9 if c["holes"] else 1.0)
        q = c["B"] * H * c["G"] * c["W"]
        return {"bytes": rows * 2 * (d + 4 / bs) + q * (4 * d + 4), "flops": 4.0 * rows * c["G"] * c["W"] * d}
    if c["op"] == "store":
        rows = c["B"] * H * (c["lo"] + c["hi"]) / 2
        back = c["B"] * H * (c["K"] or c["T"])            # written, read, and the bf16 rows both ways
        return {"bytes": 2 * (rows * (2 * d + d + d) + back * 2 * d), "flops": 0}
    if c["op"] == "append":
        new = c["B"] * H * c["W"]
        back = c["B"] * H * (bs + c["W"])
        return {"bytes": 2 * (new * 3 * d + back * 3 * d), "flops": 0}
    if c["op"] == "fork":
        pairs, nb = c["P"] * c["C"], (c["lo"] + c["hi"]) / 2 / bs
        return {"bytes": pairs * (2 * page * (bs - 1) / bs + 4 * 4 * nb) + 64, "flops": 0}
    moved = c["n"] * c["live"] * (1 - c["live"])
    return {"bytes": 2 * moved * page + c["n"] * 12 + c["n"] * c["live"] * 8, "flops": 0}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(y):
    """y (fp64, |y| <= 448) to the nearest e4m3 value, ties to even: the step is
    2^(floor(log2 |y|) - 3), and 2^-9 below 2^-6."""
    e = torch.frexp(y).exponent - 1
    step = _pow2_64(e.clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _exact_scale(amax, fmt):
    if fmt == E4M3:
        return _pow2_64(torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448.0)).clamp(min=-126))
    return (amax / 127.0).clamp(min=_TINY)


def _exact_values(x, sc, fmt):
    return (_round_e4m3(x / sc) if fmt == E4M3 else torch.round(x / sc)) * sc


def exact(case, seed):
    c = dict(case)
    if c["op"] in ("fork", "compact"):
        return None                                       # whole numbers and copied bytes
    s = prepare(case, seed)
    B, H, d, bs = c["B"], c["H"], c["d"], c["bs"]
    lens, table = s["len"].tolist(), s["table"].long()
    if c["op"] == "attend":
        if B * H > 2048:
            return None
        G, W = c["G"], c["W"]
        out = torch.zeros((B, H, G, W, d), device="cuda", dtype=torch.float64)
        lse = torch.full((B, H, G, W), -math.inf, device="cuda", dtype=torch.float64)
        for b in range(B):
            L = lens[b]
            if L == 0:
                continue
            pos = torch.arange(L, device="cuda")
            page, slot = table[b][pos // bs], pos % bs
            seen = page >= 0
            pos, page, slot = pos[seen], page[seen], slot[seen]
            if not pos.numel():
                continue
            for h in range(H):
                k = s["k"].view(torch.uint8)[page, h, slot].view(s["k"].dtype).double() * s["ks"][page, h].double()[:, None]
                v = s["v"].view(torch.uint8)[page, h, slot].view(s["v"].dtype).double() * s["vs"][page, h].double()[:, None]
                q = s["q"][b * H + h].double()            # [G, W, d]
                x = torch.matmul(q.reshape(G * W, d), k.t().contiguous()).reshape(G, W, -1) / math.sqrt(d)
                for w in range(W):
                    m = pos <= L - W + w
                    if bool(m.any()):
                        y = x[:, w, m]
                        z = torch.logsumexp(y, -1)
                        lse[b, h, :, w] = z
                        out[b, h, :, w] = torch.exp(y - z[:, None]) @ v[m]
        return dict(out=out.reshape(B * H, G, W, d), lse=lse.reshape(B * H, G, W))
    T = (c["K"] or c["T"]) if c["op"] == "store" else bs + c["W"]   # rows that are read back
    got = []
    for name in ("k", "v"):
        y = torch.zeros((B * H, T, d), device="cuda", dtype=torch.float64)
        sc = s[name + "s"].double()
        codes = s[name].view(torch.uint8)
        for b in range(B):
            L, heads = lens[b], slice(b * H, (b + 1) * H)
            if c["op"] == "store":
                L = min(L, T)
                start, new = 0, s[name + "_rows"][heads, c["T"] - L:].double()
                if c["K"]:
                    at = s["kept"][heads, :L].long()[..., None].expand(-1, -1, d)
                    new = s[name + "_rows"][heads].double().gather(1, at)
            else:
                start, new = L - c["W"], s[name + "_new"][heads].double()
            if not L:
                continue
            first = max(0, L - T) // bs                   # pages that are read back
            pages = table[b, first: -(-L // bs)]
            now = sc[pages]                                # [pages, H]
            x = codes[pages].view(s[name].dtype).double() * now[..., None, None]
            x = x.transpose(0, 1).reshape(H, -1, d)        # [H, slots, d]
            pos = first * bs + torch.arange(x.shape[1], device="cuda")
            fresh, old = (pos >= start) & (pos < L), pos < start
            rows = torch.zeros_like(x)
            rows[:, fresh] = new[:, new.shape[1] - int(fresh.sum()):]
            by_page = lambda m: m.reshape(-1, bs).any(1)[:, None]  # noqa: E731
            need = _exact_scale(rows.reshape(H, -1, bs * d).abs().amax(2).t(), c["fmt"])
            then = torch.where(by_page(fresh), torch.where(by_page(old), torch.maximum(need, now), need), now)
            wide = then.t().repeat_interleave(bs, 1)[..., None]
            coded = _exact_values(torch.where(fresh[:, None], rows, x), wide, c["fmt"])
            moved = by_page(fresh).expand_as(then) & (then != now)
            x = torch.where(fresh[:, None] | (moved.t().repeat_interleave(bs, 1)[..., None]), coded, x)
            sc[pages] = then
            keep = pos[(pos < L) & (pos >= L - T)]
            y[heads, T - L + keep] = x[:, keep - first * bs]
        got.append((y, sc))
    return dict(k=got[0][0], v=got[1][0], ks=got[0][1], vs=got[1][1])
