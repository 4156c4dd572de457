"""The 8-bit paged cache, its page table and the event together, as a serving loop
uses them: every step against the oracle run beside it."""
import threading

import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc, synth
from oracle import pages as op
from oracle import q8 as oq
import q8_utils as u

pytestmark = pytest.mark.gpu


class Loop:
    """A serving loop's cache on both sides: the library's and the oracle's."""

    def __init__(self, seed, B, H, d, bs, tb, n, fmt):
        self.B, self.H, self.d, self.bs, self.fmt = B, H, d, bs, fmt
        z = np.zeros((n, H, bs, d), np.uint8)
        one = np.ones((n, H), np.float32)
        self.t = op.Pages(np.full((B, tb), -1), np.zeros(B), np.zeros(n), bs)
        self.c = oq.Cache(z, z, one, one, self.t.table, self.t.lens, fmt)
        self.c.table, self.c.lens = self.t.table, self.t.lens        # one table for both
        g = u.to_gpu(self.c)
        self.pages = kvc.PageTable(g.table, g.seq_len, torch.zeros(n, dtype=torch.int32, device="cuda"), bs)
        self.g = g
        self.bufs = kvc.PageBuffers([g.k_pool, g.v_pool, g.k_scale, g.v_scale])

    def same(self):
        torch.cuda.synchronize()
        u.same_pages(self.pages, self.t)
        live = self.t.refs > 0
        for a, b in ((self.g.k_pool, self.c.k), (self.g.v_pool, self.c.v)):
            np.testing.assert_array_equal(u.bits8(a)[live], b[live])
        for a, b in ((self.g.k_scale, self.c.ks), (self.g.v_scale, self.c.vs)):
            np.testing.assert_array_equal(a.cpu().numpy()[live], b[live])

    def grow(self, want):
        want = np.asarray(want, np.int32)
        st = kvc.pages_alloc(self.pages, torch.from_numpy(want).cuda())
        assert st.cpu().numpy().tolist() == op.alloc(self.t, want).tolist()

    def set_len(self, lens):
        self.t.lens[:] = lens
        self.pages.seq_len.copy_(torch.from_numpy(self.t.lens))

    def store(self, k, v, T, kept=None):
        kvc.q8_store(self.g, u.dev_bf16(k), u.dev_bf16(v), T=T,
                     kept=None if kept is None else torch.from_numpy(kept).cuda())
        oq.store(self.c, k, v, T, kept)

    def decode(self, seed, W, G, active):
        """W more tokens for the sequences of `active`, then attention of all."""
        self.set_len(np.where(active, self.t.lens + W, self.t.lens))
        self.grow(self.t.lens)
        k, v = u.random_rows(seed, self.B * self.H, W, self.d), u.random_rows(seed + 1, self.B * self.H, W, self.d)
        n_new = None if active.all() else np.where(active, W, 0).astype(np.int32)
        kvc.q8_append(self.g, u.dev_bf16(k), u.dev_bf16(v),
                      n_new=None if n_new is None else torch.from_numpy(n_new).cuda())
        oq.append(self.c, k, v, n_new)
        q = u.random_rows(seed + 2, self.B * self.H, G, W, self.d)
        out, lse = kvc.q8_attend(self.g, u.dev_bf16(q), want_lse=True)
        torch.cuda.synchronize()
        u.check_attention(self.c, q, out, lse)

    def fork(self, src, dst):
        src, dst = np.array(src, np.int32), np.array(dst, np.int32)
        st = kvc.pages_fork(self.pages, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), self.bufs)
        ref, copies = op.fork(self.t, src, dst)
        assert st.cpu().numpy().tolist() == ref.tolist()
        for a, z in copies:
            for arr in (self.c.k, self.c.v, self.c.ks, self.c.vs):
                arr[z] = arr[a]

    def free(self, ids):
        kvc.pages_free(self.pages, torch.tensor(ids, dtype=torch.int32, device="cuda"))
        op.release(self.t, ids)

    def compact(self):
        got = kvc.pages_compact(self.pages, self.bufs)
        table, refs, remap, live, copies = op.compact(self.t)
        for a, z in copies:
            for arr in (self.c.k, self.c.v, self.c.ks, self.c.vs):
                arr[z] = arr[a]
        self.t.table[:], self.t.refs[:] = table, refs
        self.pages.table.copy_(got["table"])
        self.pages.refs.copy_(got["refs"])
        assert int(got["n_live"][0]) == live


@pytest.mark.parametrize("fmt", [oq.E4M3, oq.INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("bs,d", [(16, 128), (12, 64)])
def test_prompts_forks_decoding_an_event_and_compaction(fmt, bs, d):
    B, H, G, T = 6, 2, 4, 150
    w = Loop(1, B, H, d, bs, 30, 150, fmt)
    # three prompts
    w.set_len([150, 97, 16, 0, 0, 0])
    w.grow(w.t.lens)
    k, v = u.random_rows(2, B * H, T, d), u.random_rows(3, B * H, T, d)
    w.store(k, v, T)
    w.same()
    # two of them forked, decoding on apart
    w.fork([0, 1, 1], [3, 4, 5])
    w.same()
    for step in range(4):
        w.decode(100 + 10 * step, 1 if step % 2 else 3, G, np.ones(B, bool))
        w.same()
    # one ends, the pool is compacted, the others go on
    w.free([1, 1])
    w.compact()
    w.same()
    w.decode(200, 1, G, w.t.lens > 0)
    w.same()
    # an event on sequence 0: its rows back as bf16, compressed, stored again
    W, K = 8, 64
    L = int(w.t.lens[0])
    TT = 176
    gk, gv = kvc.q8_load(w.g, TT)
    rk, rv = oq.load(w.c, TT)
    np.testing.assert_array_equal(gk.view(torch.int16).cpu().numpy().view(np.uint16), rk)
    p = kvc.Params.from_dict(dict(synth.WORKLOADS["tiny"].params, window=W, group=G, head_dim=d, T=TT, budget=K),
                             n_heads=H)
    p.valid_len = torch.full((H,), L, dtype=torch.int32, device="cuda")
    q = u.dev_bf16(u.random_rows(300, H, G, W, d))
    ev = kvc.compress_event(p, q, gk[:H].contiguous(), gv[:H].contiguous())
    kept_one = ev["kept"].cpu().numpy()
    assert (kept_one >= TT - L).all() and (np.diff(kept_one, axis=1) > 0).all()
    kept = np.full((B * H, K), -1, np.int32)
    kept[:H] = kept_one
    w.free([0])
    lens = w.t.lens.copy()
    others = lens.copy()
    w.set_len(np.where(np.arange(B) == 0, K, 0))          # only sequence 0 is stored
    w.grow(w.t.lens)
    w.store(rk, rv, TT, kept)
    others[0] = K
    w.set_len(others)
    w.same()
    # the compacted rows, coded, are what the attention now reads
    w.decode(400, 1, G, w.t.lens > 0)
    w.same()


def test_a_fork_and_its_parent_do_not_touch_each_other():
    w = Loop(5, 4, 2, 64, 16, 6, 24, oq.E4M3)
    w.set_len([37, 0, 0, 0])
    w.grow(w.t.lens)
    k, v = u.random_rows(6, 8, 40, 64), u.random_rows(7, 8, 40, 64)
    w.store(k, v, 40)
    w.fork([0, 0], [2, 3])
    before = kvc.q8_load(w.g, 37)[0][:2].clone()
    w.decode(50, 1, 2, np.array([False, False, True, True]))
    after = kvc.q8_load(w.g, 37)[0][:2]
    assert torch.equal(before.view(torch.int16), after.view(torch.int16))
    w.same()


def _cache(seed, lens, H=2, d=128, bs=16, fmt=oq.INT8, tb=None):
    return u.random_cache(seed, len(lens), H, d, bs, lens, fmt, poison=False, tb=tb)


def test_captured_decode_step_replays():
    """alloc, append and attend in one graph, the lengths raised inside it: four
    replays with new rows against eager calls on a copy, eager work in between."""
    B, H, d, bs, G, tb = 5, 2, 128, 16, 4, 60
    lens = [1, 16, 40, 300, 700]
    c = _cache(1, lens, H, d, bs, tb=tb)
    used = [-(-n // bs) for n in lens]
    for b in range(B):
        c.table[b, used[b]:] = -1
    side = []
    for _ in range(2):
        g = u.to_gpu(c)
        refs = torch.zeros(c.n, dtype=torch.int32, device="cuda")
        refs[torch.from_numpy(c.table[c.table >= 0]).long().cuda()] = 1
        side.append((g, kvc.PageTable(g.table, g.seq_len, refs, bs)))
    k_in = torch.zeros((B * H, 1, d), dtype=torch.bfloat16, device="cuda")
    v_in, q_in = k_in.clone(), torch.zeros((B * H, G, 1, d), dtype=torch.bfloat16, device="cuda")

    def step(g, pages):
        g.seq_len.add_(1)
        st = kvc.pages_alloc(pages, g.seq_len)
        kvc.q8_append(g, k_in, v_in)
        return (st,) + tuple(kvc.q8_attend(g, q_in, want_lse=True))

    warm = u.to_gpu(c)
    kvc.q8_attend(warm, q_in)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*side[0])
    for i in range(4):
        for t, s in ((k_in, 10), (v_in, 20), (q_in, 30)):
            t.copy_(u.dev_bf16(u.random_rows(s + i, *t.shape)))
        graph.replay()
        ref = step(*side[1])
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and int(got[0].abs().sum()) == 0
        assert torch.equal(got[1].view(torch.int16), ref[1].view(torch.int16)) and torch.equal(got[2], ref[2])
        for a, b in zip((side[0][0].k_pool, side[0][0].v_pool), (side[1][0].k_pool, side[1][0].v_pool)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(side[0][1].table, side[1][1].table) and torch.equal(side[0][1].refs, side[1][1].refs)
        _ = (torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")).sum()
        torch.cuda.synchronize()


def test_captured_page_calls_replay():
    """fork and compact in a graph: the same inputs give the same tables and bytes."""
    t = u.random_pages(3, 12, 6, 16, 90)
    g = u.pages_to_gpu(t)
    pool = torch.randint(0, 256, (90, 500), dtype=torch.uint8, device="cuda")
    bufs = kvc.PageBuffers([pool])
    src = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    dst = torch.tensor([9, 10, 11], dtype=torch.int32, device="cuda")
    state = [x.clone() for x in (g.table, g.seq_len, g.refs, pool)]

    def call():
        st = kvc.pages_fork(g, src, dst, bufs)
        return dict(kvc.pages_compact(g, bufs), status=st)

    def restore():
        for x, y in zip((g.table, g.seq_len, g.refs, pool), state):
            x.copy_(y)

    want = {k: v.clone() for k, v in call().items()}
    after = [x.clone() for x in (g.table, g.seq_len, g.refs, pool)]
    restore()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), k
        for x, y in zip((g.table, g.seq_len, g.refs, pool), after):
            assert torch.equal(x, y)


def test_two_streams_and_two_threads():
    """Attention over two caches at once, on two streams and from two threads."""
    caches = [u.to_gpu(_cache(7, [900, 40, 3000])), u.to_gpu(_cache(8, [10, 2000], H=4, d=64, bs=24, fmt=oq.E4M3))]
    qs = [u.dev_bf16(u.random_rows(9, 6, 4, 1, 128)), u.dev_bf16(u.random_rows(10, 8, 7, 2, 64))]
    want = [kvc.q8_attend(c, q, want_lse=True) for c, q in zip(caches, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [kvc.q8_attend(c, q, want_lse=True, stream=s) for c, q, s in zip(caches, qs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
    out = [None, None]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(10):
                out[i] = kvc.q8_attend(caches[i], qs[i], want_lse=True)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("handle", [0, 1, 2], ids=["null", "legacy", "per_thread"])
def test_implicit_streams_of_the_c_entries(handle):
    """The runtime's implicit streams: their handles are numbers, not objects."""
    c = _cache(20, [700, 20])
    g = u.to_gpu(c)
    q = u.dev_bf16(u.random_rows(21, 4, 4, 1, 128))
    want = kvc.q8_attend(g, q)
    out, ws = torch.zeros_like(q), torch.empty(g.attend_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    refs = torch.zeros(c.n, dtype=torch.int32, device="cuda")
    pages = kvc.PageTable(torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), g.seq_len, refs, 16)
    lens = torch.tensor([33, 5], dtype=torch.int32, device="cuda")
    status, pws = torch.full_like(lens, 7), torch.empty(pages.workspace_bytes(), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    print(f"[case] stream handle {handle}", flush=True)
    L = kvc.lib()
    assert L.kvc_q8_attend(g._ref, 4, 1, 0.0, q.data_ptr(), out.data_ptr(), None, ws.data_ptr(), ws.numel(), handle) == 0
    assert L.kvc_pages_alloc(pages._ref, lens.data_ptr(), status.data_ptr(), pws.data_ptr(), pws.numel(), handle) == 0
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert status.tolist() == [0, 0] and pages.table.tolist() == [[0, 1, 2], [3, -1, -1]]


def test_two_graphs_replayed_at_once():
    """Two captured steps over one cache, each with workspaces of its own, on two
    streams."""
    g = u.to_gpu(_cache(18, [5000, 1200, 77]))
    qs = [u.dev_bf16(u.random_rows(19 + i, 6, 4, 1 + i, 128)) for i in range(2)]
    want = [kvc.q8_attend(g, q, want_lse=True) for q in qs]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in qs], []
    for graph, q in zip(graphs, qs):
        with torch.cuda.graph(graph):
            got.append(kvc.q8_attend(g, q, want_lse=True))
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(4):
        for a in got:
            a[0].zero_(), a[1].zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


def test_lengths_out_of_range_are_clamped():
    c = _cache(11, [20, 64, 5])
    c.lens = np.array([-7, 1000, 2 ** 31 - 1], np.int32)
    g = u.to_gpu(c)
    q = u.random_rows(12, 6, 3, 2, 128)
    out, lse = kvc.q8_attend(g, u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse)
    k, v = u.random_rows(13, 6, 2, 128), u.random_rows(14, 6, 2, 128)
    kvc.q8_append(g, u.dev_bf16(k), u.dev_bf16(v))
    oq.append(c, k, v)
    torch.cuda.synchronize()
    u.same_cache(g, c)


def test_given_outputs_and_workspace_are_used():
    g = u.to_gpu(_cache(15, [1500, 100]))
    q = u.dev_bf16(u.random_rows(16, 4, 4, 1, 128))
    out, lse = torch.empty_like(q), torch.empty((4, 4, 1), device="cuda")
    ws = torch.empty(g.attend_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    a = kvc.q8_attend(g, q, out=out, lse=lse, ws=ws)
    assert a[0] is out and a[1] is lse
    b = kvc.q8_attend(g, q)
    assert torch.equal(b.view(torch.int16), out.view(torch.int16))
    with pytest.raises(kvc.KvcError):
        kvc.q8_attend(g, q, ws=ws[:256])
    with pytest.raises(ValueError):
        kvc.q8_attend(g, q[:, :, :, :64])
    with pytest.raises(ValueError):
        kvc.q8_attend(g, q.transpose(0, 1))
    with pytest.raises(TypeError):
        kvc.q8_attend(g, q.float())
    with pytest.raises(kvc.KvcError):
        kvc.q8_attend(g, q, out=q)


def test_handles_keep_their_tensors():
    """Another table has to come with another handle: set on the old one, it would
    not be what the calls read."""
    c = _cache(17, [40, 3])
    g = u.to_gpu(c)
    pages = kvc.PageTable(g.table, g.seq_len, torch.ones(c.n, dtype=torch.int32, device="cuda"), 16)
    bufs = kvc.PageBuffers([g.k_pool, g.v_pool])
    out = kvc.pages_compact(pages, bufs)
    for handle, name in ((g, "table"), (g, "k_scale"), (pages, "table"), (pages, "refs"), (bufs, "tensors")):
        with pytest.raises(AttributeError, match="new one"):
            setattr(handle, name, out["table"])


def test_seeded_sweep():
    """Random shapes, lengths, holes and formats; every operator on each."""
    for i in range(40):
        rng = u.rng_of(1000 + i)
        fmt = int(rng.integers(0, 2))
        B, H = int(rng.integers(1, 5)), int(rng.integers(1, 4))
        d, bs = int(rng.choice([64, 128])), int(rng.choice([1, 3, 8, 16, 24, 33, 64, 130]))
        top = int(rng.choice([1, 5, 60, 400, 1500]))
        lens = rng.integers(0, top + 1, B)
        G, W = int(rng.integers(1, 10)), int(rng.choice([1, 1, 2, 7]))
        print(f"[case] sweep {i}: fmt={fmt} B={B} H={H} d={d} bs={bs} lens={lens.tolist()} G={G} W={W}", flush=True)
        c = u.random_cache(2000 + i, B, H, d, bs, lens, fmt, holes=float(rng.choice([0, 0, 0.2])))
        g = u.to_gpu(c)
        q = u.random_rows(3000 + i, B * H, G, W, d)
        out, lse = kvc.q8_attend(g, u.dev_bf16(q), want_lse=True)
        torch.cuda.synchronize()
        u.check_attention(c, q, out, lse)
        T = int(rng.integers(1, top + 20))
        k, v = u.random_rows(4000 + i, B * H, T, d), u.random_rows(5000 + i, B * H, T, d)
        kvc.q8_store(g, u.dev_bf16(k), u.dev_bf16(v))
        oq.store(c, k, v, T)
        kn, vn = u.random_rows(6000 + i, B * H, W, d), u.random_rows(7000 + i, B * H, W, d)
        c.ks, c.vs = np.nan_to_num(c.ks, nan=1.0), np.nan_to_num(c.vs, nan=1.0)
        g.k_scale.nan_to_num_(nan=1.0), g.v_scale.nan_to_num_(nan=1.0)
        kvc.q8_append(g, u.dev_bf16(kn), u.dev_bf16(vn))
        oq.append(c, kn, vn)
        torch.cuda.synchronize()
        u.same_cache(g, c)
