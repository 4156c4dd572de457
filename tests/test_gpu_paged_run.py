"""The bf16 paged cache as a serving loop uses it: prompts, appends, attention, evictions and page
tables together, every step against the oracle run beside it; graphs, streams, threads; a head's
bits whatever else is in the call; offsets past 32 bits."""
import threading

import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import paged as og
from oracle import pages as op
import paged_utils as u
from q8_utils import dev_bf16, random_rows, rng_of, same_pages

pytestmark = pytest.mark.gpu


def freq_of(r, base=10000.0):
    return base ** (-2.0 * np.arange(r // 2) / r)


class Loop:
    """A serving loop's cache on both sides: the library's and the oracle's."""

    def __init__(self, B, H, G, d, bs, tb, n, r, inter):
        self.B, self.H, self.G, self.d, self.bs, self.r, self.inter = B, H, G, d, bs, r, inter
        z = np.zeros((n, H, bs, d), np.uint16)
        self.t = op.Pages(np.full((B, tb), -1), np.zeros(B), np.zeros(n), bs)
        self.c = og.Cache(z, z, self.t.table, self.t.lens, np.zeros((B * H, tb * bs), np.float32),
                          np.zeros((B * H, tb * bs), np.int32))
        self.c.table, self.c.lens = self.t.table, self.t.lens
        self.g = u.to_gpu(self.c)
        self.pages = kvc.PageTable(self.g.table, self.g.seq_len, torch.zeros(n, dtype=torch.int32, device="cuda"), bs)
        self.bufs = kvc.PageBuffers([self.g.k_pool, self.g.v_pool])
        self.seen = np.zeros(B, np.int32)
        self.plan = kvc.Rope(u.dev(freq_of(r)), interleaved=inter, mscale=1.05)

    def same(self):
        torch.cuda.synchronize()
        same_pages(self.pages, self.t)
        live = self.t.refs > 0
        np.testing.assert_array_equal(u.bits(self.g.k_pool)[live], self.c.k[live])
        np.testing.assert_array_equal(u.bits(self.g.v_pool)[live], self.c.v[live])
        np.testing.assert_array_equal(self.g.pos.cpu().numpy(), self.c.pos)
        np.testing.assert_array_equal(self.g.weight.cpu().numpy(), self.c.weight)

    def chunk(self, seed, new, pad=0, whole_prompts=False):
        """New tokens for every sequence: pages, append with the rotation, attention."""
        new = np.asarray(new)
        self.t.lens[:] = self.t.lens + new
        self.pages.seq_len.copy_(u.dev(self.t.lens))
        st = kvc.pages_alloc(self.pages, self.pages.seq_len)
        assert st.cpu().numpy().tolist() == op.alloc(self.t, self.t.lens).tolist()
        starts = u.starts_of(new)
        n = int(starts[-1]) + pad
        at = np.zeros(n, np.int32)
        for b in range(self.B):
            at[starts[b]: starts[b + 1]] = self.seen[b] + np.arange(new[b])
        self.seen += new.astype(np.int32)
        Hq, H = self.H * self.G, self.H
        qkv = random_rows(seed, n, Hq + 2 * H, self.d)
        dq = dev_bf16(qkv)
        q, k, v = dq[:, :Hq], dq[:, Hq: Hq + H], dq[:, Hq + H:]
        ds = u.dev(starts)
        q = kvc.paged_append(self.g, k, v, ds, positions=u.dev(at), rope=self.plan, q=q)
        turned = kvc.rope(self.plan, k, u.dev(at))
        m = int(starts[-1])
        ref, size = og.rope(og.widen(qkv[:m]), at[:m], freq_of(self.r), 1.05, self.inter)
        u.check_rope(u.bits(q)[:m], ref[:, :Hq], size[:, :Hq], 1.05)
        u.check_rope(u.bits(turned)[:m], ref[:, Hq: Hq + H], size[:, Hq: Hq + H], 1.05)
        og.append(self.c, u.bits(turned), qkv[:, Hq + H:], starts, at)
        out = torch.full((n, Hq, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        _, lse = kvc.paged_attend(self.g, q, ds, max_new=int(new.max()), out=out, want_lse=True)
        torch.cuda.synchronize()
        got = og.attend(self.c, og.widen(u.bits(q)), starts)
        T = int(self.t.lens.max())
        u.check_attention(got, u.bits(out), lse, T, untouched=0x40E0)
        u.check_weights(got, self.c.weight, self.g.weight.cpu().numpy(), self.d, self.G * int(new.max()))
        self.c.weight[:] = self.g.weight.cpu().numpy()
        if whole_prompts:        # the same attention without the cache, from the packed rows
            o, z = kvc.prompt_attend(q, turned, v, ds, want_lse=True)
            w = og.widen
            pr = og.prompt(w(u.bits(q)), w(u.bits(turned)), w(qkv[:, Hq + H:]), starts)
            u.check_attention(pr, u.bits(o), z, T)

    def evict(self, budget, sinks, recent):
        kvc.paged_evict(self.g, u.dev(self.seen), budget, sinks=sinks, recent=recent)
        og.evict(self.c, self.seen, budget, sinks, recent)
        kvc.pages_trim(self.pages)
        op.trim(self.t)


@pytest.mark.parametrize("d,bs,r,inter", [(128, 16, 128, False), (64, 12, 26, True)])
def test_prompts_decoding_evictions_and_forks(d, bs, r, inter):
    w = Loop(4, 2, 3, d, bs, 40, 120, r, inter)
    w.chunk(1, [150, 97, 16, 0], pad=3, whole_prompts=True)
    w.same()
    w.evict(64, 4, 16)
    w.same()
    for step in range(3):
        w.chunk(10 + step, [1, 1, 1, 0])
        w.evict(64, 4, 16)
        w.same()
    # a prompt goes on in a batch of decoding sequences
    w.chunk(20, [1, 60, 1, 33], pad=1)
    w.same()
    w.evict(70, 2, 8)
    w.same()
    # one forks: its full pages shared, the open one copied; the weights and positions follow
    src, dst = np.array([0], np.int32), np.array([3], np.int32)
    kvc.pages_fork(w.pages, u.dev(src), u.dev(dst), w.bufs)
    _, copies = op.fork(w.t, src, dst)
    for a, z in copies:
        w.c.k[z], w.c.v[z] = w.c.k[a], w.c.v[a]
    for x, y in ((w.g.weight, w.c.weight), (w.g.pos, w.c.pos)):
        x[3 * w.H: 4 * w.H] = x[: w.H]
        y[3 * w.H: 4 * w.H] = y[: w.H]
    w.seen[3] = w.seen[0]
    w.same()
    w.chunk(30, [1, 1, 0, 1])
    w.same()


def _step_inputs(B, H, G, d, i):
    qkv = random_rows(400 + i, B, (G + 2) * H, d)
    return dev_bf16(qkv)


@pytest.mark.parametrize("W", [1, 12])
def test_captured_step_replays(W):
    """Lengths raised, pages, append, attention with weights, eviction and trim in one graph: replays
    with new rows against eager calls on a copy, eager work in between."""
    B, H, G, d, bs, tb, K = 3, 2, 4, 128, 16, 20, 100
    c = u.random_cache(60, B, H, d, bs, [100, 100, 60], tb=tb, weights=True)
    for b, n in enumerate([7, 7, 4]):
        c.table[b, n:] = -1
    plan = kvc.Rope(u.dev(freq_of(d)))
    starts = u.dev(u.starts_of([W] * B))
    qkv = torch.zeros((B * W, (G + 2) * H, d), dtype=torch.bfloat16, device="cuda")
    side = []
    for _ in range(2):
        g = u.to_gpu(c)
        refs = torch.zeros(c.n, dtype=torch.int32, device="cuda")
        refs[torch.from_numpy(c.table[c.table >= 0]).long().cuda()] = 1
        side.append((g, kvc.PageTable(g.table, g.seq_len, refs, bs), torch.tensor([100, 100, 60], dtype=torch.int32, device="cuda")))

    def step(g, pages, seen):
        g.seq_len.add_(W)
        seen.add_(W)
        st = kvc.pages_alloc(pages, g.seq_len)
        at = (seen[:, None] + torch.arange(-W, 0, dtype=torch.int32, device="cuda")).reshape(-1)
        q = kvc.paged_append(g, qkv[:, G * H: (G + 1) * H], qkv[:, (G + 1) * H:], starts, positions=at, rope=plan,
                             q=qkv[:, : G * H])
        out, lse = kvc.paged_attend(g, q, starts, max_new=W, want_lse=True)
        kvc.paged_evict(g, seen, K, sinks=2, recent=8)
        kvc.pages_trim(pages)
        return st, out, lse

    warm = u.to_gpu(c)
    step(warm, kvc.PageTable(warm.table, warm.seq_len, torch.ones(c.n, dtype=torch.int32, device="cuda"), bs), side[0][2].clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*side[0])
    for i in range(5):
        qkv.copy_(dev_bf16(random_rows(70 + i, *qkv.shape)))
        graph.replay()
        ref = step(*side[1])
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a, b.view(torch.int16) if b.dtype == torch.bfloat16 else b)
        (ga, pa, _), (gb, pb, _) = side
        for name in ("table", "seq_len", "weight", "pos"):
            assert torch.equal(getattr(ga, name), getattr(gb, name)), name
        assert torch.equal(pa.refs, pb.refs)
        live = pa.refs > 0
        assert torch.equal(ga.k_pool[live].view(torch.int16), gb.k_pool[live].view(torch.int16))
        assert torch.equal(ga.v_pool[live].view(torch.int16), gb.v_pool[live].view(torch.int16))


def test_two_graphs_share_a_workspace():
    """Attention of few and of many rows captured with one workspace, replayed in turn on one stream."""
    H, G, d = 2, 4, 64
    c = u.random_cache(61, 2, H, d, 16, [1500, 1100], weights=True)
    g = u.to_gpu(c)
    work = []
    for new in ([1, 2], [40, 100]):
        q = dev_bf16(random_rows(62 + new[0], sum(new), G * H, d))
        work.append((q, u.dev(u.starts_of(new)), max(new)))
    ws = torch.empty(max(g.attend_workspace_bytes(G, q.shape[0], m) for q, _, m in work), dtype=torch.uint8, device="cuda")
    before = g.weight.clone()
    ref, grown = [], []
    for q, st, m in work:
        g.weight.copy_(before)
        ref.append(kvc.paged_attend(g, q, st, max_new=m))
        grown.append(g.weight.clone())
    graphs, outs = [], []
    for q, st, m in work:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        out = torch.empty_like(q)
        with torch.cuda.graph(graph):
            kvc.paged_attend(g, q, st, max_new=m, out=out, ws=ws)
        graphs.append(graph)
        outs.append(out)
    for _ in range(3):
        for i in (0, 1):
            g.weight.copy_(before)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i].view(torch.int16), ref[i].view(torch.int16))
            assert torch.equal(g.weight, grown[i])


def test_streams_and_threads():
    """Two caches at once, on two streams and from two host threads: the bits of each alone."""
    H, G, d = 2, 4, 128
    cases = []
    for i, new in enumerate(([1, 30, 2], [100, 1, 64])):
        c = u.random_cache(63 + i, 3, H, d, 16, [900, 300, 700], weights=True)
        q = dev_bf16(random_rows(65 + i, sum(new), G * H, d))
        k = dev_bf16(random_rows(67 + i, sum(new), H, d))
        cases.append((c, q, k, u.dev(u.starts_of(new)), u.dev(np.array([900, 300, 700], np.int32))))

    def work(g, q, k, st, seen):
        kvc.paged_append(g, k, k, st)
        out, lse = kvc.paged_attend(g, q, st, want_lse=True)
        kvc.paged_evict(g, seen, 200)
        return out, lse, g.weight.clone(), g.pos.clone(), g.seq_len.clone()

    ref = [work(u.to_gpu(c), q, k, st, s) for c, q, k, st, s in cases]
    torch.cuda.synchronize()
    fresh = [u.to_gpu(c) for c, *_ in cases]
    torch.cuda.synchronize()
    got, streams = [None, None], [torch.cuda.Stream(), torch.cuda.Stream()]

    def on(i, gs):
        with torch.cuda.stream(streams[i]):
            got[i] = work(gs[i], *cases[i][1:])

    for i in (0, 1):
        on(i, fresh)
    torch.cuda.synchronize()
    first = got[:]
    fresh = [u.to_gpu(c) for c, *_ in cases]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=on, args=(i, fresh)) for i in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for one in (first, got):
        for a, b in zip(one, ref):
            for x, y in zip(a, b):
                assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x, y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
    # a stream handed in
    s = torch.cuda.Stream()
    c, q, k, st, seen = cases[0]
    g = u.to_gpu(c)
    torch.cuda.synchronize()
    kvc.paged_append(g, k, k, st, stream=s)
    out = kvc.paged_attend(g, q, st, stream=s)
    kvc.paged_evict(g, seen, 200, stream=s)
    s.synchronize()
    assert torch.equal(out.view(torch.int16), ref[0][0].view(torch.int16)) and torch.equal(g.pos, ref[0][3])


@pytest.mark.parametrize("d", [64, 128])
def test_a_head_does_not_depend_on_its_call(d):
    """Every sequence alone, with a table of just its room, gives the bits it gets in the batch."""
    H, G = 3, 4
    lens, new = [5, 1300, 700, 0, 2100, 64, 5000], [5, 1, 8, 0, 90, 9, 2]
    c = u.random_cache(70, 7, H, d, 16, lens, weights=True)
    starts = u.starts_of(new)
    q = dev_bf16(random_rows(71, int(starts[-1]), G * H, d))
    g = u.to_gpu(c)
    out, lse = kvc.paged_attend(g, q, u.dev(starts), want_lse=True)
    kv = dev_bf16(random_rows(72, int(starts[-1]), 2 * H, d))
    po, pl = kvc.prompt_attend(q, kv[:, :H], kv[:, H:], u.dev(starts), want_lse=True)
    for b in range(7):
        if not new[b]:
            continue
        nb = -(-lens[b] // 16)
        rows = slice(int(starts[b]), int(starts[b + 1]))
        one = og.Cache(c.k, c.v, c.table[b: b + 1, :nb], c.lens[b: b + 1], c.weight[b * H: (b + 1) * H, : nb * 16],
                       c.pos[b * H: (b + 1) * H, : nb * 16])
        s = u.to_gpu(one)
        o, z = kvc.paged_attend(s, q[rows].contiguous(), u.dev(u.starts_of([new[b]])), want_lse=True)
        assert torch.equal(o.view(torch.int16), out[rows].view(torch.int16)) and torch.equal(z, lse[rows])
        assert torch.equal(s.weight, g.weight[b * H: (b + 1) * H, : nb * 16])
        # with a table of far more room
        far = np.full((1, 2600), -1, np.int32)
        far[0, :nb] = c.table[b, :nb]
        s2 = u.to_gpu(og.Cache(c.k, c.v, far, c.lens[b: b + 1]))
        o2 = kvc.paged_attend(s2, q[rows].contiguous(), u.dev(u.starts_of([new[b]])))
        assert torch.equal(o2.view(torch.int16), out[rows].view(torch.int16))
        # one KV head alone
        h = 1
        s1 = u.to_gpu(og.Cache(c.k[:, h: h + 1], c.v[:, h: h + 1], c.table[b: b + 1, :nb], c.lens[b: b + 1]))
        o1 = kvc.paged_attend(s1, q[rows, h * G: (h + 1) * G], u.dev(u.starts_of([new[b]])))
        assert torch.equal(o1.view(torch.int16), out[rows, h * G: (h + 1) * G].contiguous().view(torch.int16))
        o, z = kvc.prompt_attend(q[rows], kv[rows, :H], kv[rows, H:], u.dev(u.starts_of([new[b]])), want_lse=True)
        assert torch.equal(o.view(torch.int16), po[rows].view(torch.int16)) and torch.equal(z, pl[rows])


# (B, H, G, d, bs, longest, most new, holes, spare pages)
HEADS = [
    (14, 8, 3, 128, 16, 1536, 5, 0.0, 3),
    (14, 8, 3, 64, 24, 1500, 4, 0.2, 3),
    (32, 4, 7, 128, 5, 1030, 2, 0.2, 3),
    (33, 3, 1, 64, 7, 1100, 16, 0.0, 3),
    (58, 8, 2, 64, 16, 600, 3, 0.0, 3),                # more heads than CUs
    (26, 4, 16, 128, 64, 1300, 1, 0.1, 700),           # pools past the size that is read past the caches
    (26, 4, 16, 64, 64, 900, 1, 0.0, 1600),
    (3, 2, 5, 128, 16, 500, 3, 0.1, 3),                # one piece a head
    (5, 2, 4, 64, 7, 490, 4, 0.0, 3),
]


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("case", HEADS, ids=[str(i) for i in range(len(HEADS))])
def test_many_heads_of_few_pieces(case, weights):
    """Enough heads that a workgroup takes one whole: the oracle's results, and the bits that
    each sequence gets alone."""
    B, H, G, d, bs, longest, most, holes, spare = case
    print(f"[case] heads {case} {weights}", flush=True)
    rng = u.rng_of(80, *case[:6])
    lens = rng.integers(1, longest + 1, B)
    lens[:6] = [longest, 0, 1, min(512, longest), min(513, longest), longest - 1][: B]
    new = rng.integers(0, most + 1, B)
    new[:3] = [most, most, most]                       # the empty sequence has tokens too
    c = u.random_cache(81, B, H, d, bs, lens, holes=holes, spare=spare, weights=weights)
    starts = u.starts_of(new)
    n = int(starts[-1]) + 2
    q = dev_bf16(random_rows(82, n, G * H, d))
    g = u.to_gpu(c)
    out = torch.full((n, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = kvc.paged_attend(g, q, u.dev(starts), max_new=most, out=out, want_lse=True)
    torch.cuda.synchronize()
    ref = og.attend(c, og.widen(u.bits(q)), starts)
    u.check_attention(ref, u.bits(out), lse, longest, untouched=0x40E0)
    if weights:
        u.check_weights(ref, c.weight, g.weight.cpu().numpy(), d, G * most)
    for b in range(B):
        if not new[b]:
            continue
        rows, heads = slice(int(starts[b]), int(starts[b + 1])), slice(b * H, (b + 1) * H)
        one = kvc.PagedCache(g.k_pool, g.v_pool, g.table[b: b + 1], g.seq_len[b: b + 1],
                             weight=u.dev(c.weight[heads]) if weights else None,
                             pos=u.dev(c.pos[heads]) if weights else None)
        o, z = kvc.paged_attend(one, q[rows], u.dev(u.starts_of([new[b]])), want_lse=True)
        assert torch.equal(o.view(torch.int16), out[rows].view(torch.int16)) and torch.equal(z, lse[rows])
        if weights:
            assert torch.equal(one.weight, g.weight[heads])


@pytest.mark.parametrize("n", [40, 100, 300, 700])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_of_many_rows_alone_and_in_a_batch(d, n):
    """One sequence (few workgroups, of fewer keys and rows each) and twelve of them (many) give the
    same weights."""
    H, G, T = 4, 2, 4000
    c = u.random_cache(83, 1, H, d, 16, [T], weights=True)
    q = dev_bf16(random_rows(84, n, G * H, d))
    one = u.to_gpu(c)
    kvc.paged_attend(one, q, u.dev(u.starts_of([n])))
    u.check_weights(og.attend(c, og.widen(u.bits(q)), u.starts_of([n])), c.weight, one.weight.cpu().numpy(), d, G * n)
    B = 12
    many = kvc.PagedCache(one.k_pool, one.v_pool, one.table.repeat(B, 1), one.seq_len.repeat(B),
                          weight=u.dev(np.tile(c.weight, (B, 1))), pos=u.dev(np.tile(c.pos, (B, 1))))
    kvc.paged_attend(many, q.repeat(B, 1, 1), u.dev(u.starts_of([n] * B)))
    assert torch.equal(many.weight, one.weight.repeat(B, 1))


def test_workgroups_of_eight_waves_give_the_bits_of_four():
    """Long prompts and chunks of many heads (256 rows a workgroup), and each KV head of them alone (128)."""
    d, H, G = 128, 8, 8
    starts = u.dev(u.starts_of([2048, 37, 1100]))
    rows = dev_bf16(random_rows(85, 3190, (G + 2) * H, d))
    q, k, v = rows[:, : G * H], rows[:, G * H: (G + 1) * H], rows[:, (G + 1) * H:]
    out = torch.full((3190, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = kvc.prompt_attend(q, k, v, starts, out=out, want_lse=True)
    assert bool((out[3185:] == 7.0).all())
    for h in range(H):
        o, z = kvc.prompt_attend(q[:, h * G: (h + 1) * G], k[:, h: h + 1], v[:, h: h + 1], starts, want_lse=True)
        assert torch.equal(o[:3185].view(torch.int16), out[:3185, h * G: (h + 1) * G].contiguous().view(torch.int16))
        assert torch.equal(z[:3185], lse[:3185, h * G: (h + 1) * G])
    H, G = 4, 4
    c = u.random_cache(86, 2, H, d, 16, [8192, 7001])
    c.table[1, 200: 210] = -1
    starts = u.dev(u.starts_of([512, 401]))
    q = dev_bf16(random_rows(87, 915, G * H, d))
    out = torch.full((915, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = kvc.paged_attend(u.to_gpu(c), q, starts, out=out, want_lse=True)
    assert bool((out[913:] == 7.0).all())
    for h in range(H):
        one = u.to_gpu(og.Cache(c.k[:, h: h + 1], c.v[:, h: h + 1], c.table, c.lens))
        o, z = kvc.paged_attend(one, q[:, h * G: (h + 1) * G], starts, want_lse=True)
        assert torch.equal(o[:913].view(torch.int16), out[:913, h * G: (h + 1) * G].contiguous().view(torch.int16))
        assert torch.equal(z[:913], lse[:913, h * G: (h + 1) * G])


def test_max_len_bounds_the_lengths():
    c = u.random_cache(73, 2, 1, 64, 16, [300, 90], weights=True, max_len=200)
    c.lens[0] = 300
    q = random_rows(74, 42, 2, 64)
    starts = u.starts_of([40, 2])
    g = u.to_gpu(c, max_len=200)
    out, lse = kvc.paged_attend(g, dev_bf16(q), u.dev(starts), want_lse=True)
    u.check_attention(og.attend(c, og.widen(q), starts), u.bits(out), lse, 200)
    seen = np.array([300, 90], np.int32)
    kvc.paged_evict(g, u.dev(seen), 150, sinks=3, recent=5)
    c.weight = g.weight.cpu().numpy()
    before = c.weight.copy()
    og.evict(c, seen, 150, 3, 5)
    got = g.pos.cpu().numpy()
    assert g.seq_len.cpu().numpy().tolist() == [150, 90]
    assert (np.sort(got[0, :150]) < 200).all() and len(set(got[0, :150])) == 150
    assert (got[0, 150:] == np.arange(150, got.shape[1])).all() and (before[0, 200:] == c.weight[0, 200:]).all()


def _gpu_reference(q, k, v, limit, scale):
    """fp64 attention on the GPU: q [R, d], k, v [T, d], row r sees keys up to limit[r]."""
    x = (q.double() @ k.double().t().contiguous()) * scale
    x.masked_fill_(torch.arange(k.shape[0], device="cuda") > limit[:, None], -torch.inf)
    z = torch.logsumexp(x, -1)
    p = torch.exp(x - z[:, None])
    return p @ v.double(), z, p


@pytest.mark.parametrize("new", [1, 8, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_long_caches_and_offsets_past_32_bits(d, new):
    """140000 slots (pieces of the longest kind), in pages at the end of pools of more than 2^32 values."""
    H, G, bs, T = 1, 4, 256, 140000
    nb = -(-T // bs)
    n = (1 << 32) // (H * bs * d) + 4 * nb
    pools = [torch.empty((n, H, bs, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(80)
    rows = [torch.randn((nb, H, bs, d), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    ids = (n - 1 - torch.randperm(2 * nb, generator=gen, device="cuda")[:nb]).to(torch.int32)
    for p, r in zip(pools, rows):
        p[ids.long()] = r
    assert int(ids.min()) * H * bs * d > 1 << 32
    g = kvc.PagedCache(pools[0], pools[1], ids[None].contiguous(), torch.tensor([T], dtype=torch.int32, device="cuda"),
                       weight=torch.zeros((1, nb * bs), device="cuda"),
                       pos=torch.arange(nb * bs, device="cuda", dtype=torch.int32)[None].contiguous())
    q = torch.randn((new, G, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    starts = u.dev(u.starts_of([new]))
    knew = torch.randn((new, H, d), generator=gen, device="cuda", dtype=torch.bfloat16)
    kvc.paged_append(g, knew, knew, starts)
    k, v = (r.reshape(-1, d)[:T].clone() for r in rows)
    k[T - new:] = v[T - new:] = knew[:, 0]
    out, lse = kvc.paged_attend(g, q, starts, want_lse=True)
    limit = torch.arange(T - new, T, device="cuda").repeat_interleave(G)
    ref, z, p = _gpu_reference(q.reshape(-1, d), k, v, limit, d ** -0.5)
    # weights in bf16 and the result each by 2^-8 of what they are at most, scores as in check_attention
    ds = d ** -0.5 * float((q.double().abs().reshape(-1, d) @ k.double().abs().t().contiguous()).max()) * (d + 8) * 2.0 ** -23
    rel = 2.0 ** -8 + 2 * ds + 2.0 ** -20 + T * 2.0 ** -24
    bound = rel * (p @ v.double().abs()) * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    assert bool(((out.double().reshape(-1, d) - ref).abs() <= bound).all())
    assert float((lse.double().reshape(-1) - z).abs().max()) <= ds + 2.0 ** -20 + T * 2.0 ** -24 + 2.0 ** -18
    add = p.sum(0)
    err = (g.weight[0, :T].double() - add).abs()
    assert bool((err <= add * (3 * ds + 2.0 ** -17 + T * 2.0 ** -24) + 1e-30).all())
    kvc.paged_evict(g, torch.tensor([T], dtype=torch.int32, device="cuda"), 3000, sinks=4, recent=64)
    torch.cuda.synchronize()
    kept = g.pos[0, :3000].long()
    assert int(g.seq_len[0]) == 3000 and kept.unique().numel() == 3000
    slots = torch.arange(3000, device="cuda")
    got = pools[0][ids.long()[slots // bs], 0, slots % bs]
    assert torch.equal(got.view(torch.int16), k[kept].view(torch.int16))
