"""Forks and evictions of the bf16 paged cache: a page that two sequences share is never written."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import paged as og
from oracle import pages as op
import paged_utils as u
from q8_utils import rng_of
from test_gpu_paged_run import Loop

pytestmark = pytest.mark.gpu


def _fork(w, a, z):
    src, dst = np.array([a], np.int32), np.array([z], np.int32)
    kvc.pages_fork(w.pages, u.dev(src), u.dev(dst), w.bufs)
    _, copies = op.fork(w.t, src, dst)
    for x, y in copies:
        w.c.k[y], w.c.v[y] = w.c.k[x], w.c.v[x]
    _follow(w, a, z)


def _follow(w, a, z):
    """What belongs to a sequence and not to its pages."""
    for x, y in ((w.g.weight, w.c.weight), (w.g.pos, w.c.pos)):
        x[z * w.H: (z + 1) * w.H] = x[a * w.H: (a + 1) * w.H]
        y[z * w.H: (z + 1) * w.H] = y[a * w.H: (a + 1) * w.H]
    w.seen[z] = w.seen[a]


def _own_pages(w, a, z):
    """Gives sequence z, a fork of a, pages of its own."""
    kvc.pages_free(w.pages, u.dev(np.array([z], np.int32)))
    op.release(w.t, [z])
    w.t.lens[z] = w.t.lens[a]
    w.pages.seq_len[z] = w.pages.seq_len[a]
    st = kvc.pages_alloc(w.pages, w.pages.seq_len)
    assert st.cpu().numpy().tolist() == op.alloc(w.t, w.t.lens).tolist() == [0] * w.B
    kvc.pages_copy(w.g.table[a].clone(), w.g.table[z].clone(), w.bufs)
    for x, y in zip(w.t.table[a], w.t.table[z]):
        if x >= 0:
            w.c.k[y], w.c.v[y] = w.c.k[x], w.c.v[x]


@pytest.mark.parametrize("d,bs", [(128, 16), (64, 12)])
@pytest.mark.parametrize("length", [64, 70])
def test_forks_are_not_evicted_from_under_each_other(d, bs, length):
    """A fork at the budget, a step that appends to both, an eviction: both keep what they had, the other
    sequences are cut; with pages of their own both are cut."""
    w = Loop(4, 2, 3, d, bs, 40, 120, d, False)
    w.chunk(1, [length, 97, 5, 0])
    w.evict(64, 4, 16)
    _fork(w, 0, 3)
    w.same()
    for step in range(3):
        w.chunk(10 + step, [1, 1, 1, 2])
        w.evict(64, 4, 16)
        w.same()
        assert w.t.lens[0] == 64 + step + 1 and w.t.lens[3] == 64 + 2 * (step + 1) and w.t.lens[1] == 64
    # the fork's pages given up and taken anew: nothing is shared, both are cut
    _fork(w, 0, 3)
    _own_pages(w, 0, 3)
    w.same()
    w.chunk(20, [1, 1, 1, 1])
    w.evict(64, 4, 16)
    w.same()
    assert w.t.lens.tolist()[:2] == [64, 64] and w.t.lens[3] == 64
    w.chunk(21, [1, 0, 30, 1])
    w.same()


@pytest.mark.parametrize("seed", range(6))
def test_tables_that_share_pages_at_random(seed):
    """Pages named by other sequences, twice by one, behind lengths, or behind the budget only."""
    rng = rng_of(seed, 61)
    B, H, d, bs = 12, 2, 64, int(rng.choice([4, 7, 16]))
    lens = rng.integers(0, 90, B)
    c = u.random_cache(62 + seed, B, H, d, bs, lens, tb=90 // bs + 2, weights=True)
    for b in range(B):
        n = -(-int(lens[b]) // bs)
        if rng.random() < 0.4 and n:
            c.table[b, rng.integers(0, c.table.shape[1])] = c.table[rng.integers(0, B), rng.integers(0, n)]
        if rng.random() < 0.2:
            c.table[b, rng.integers(0, c.table.shape[1])] = rng.choice([-1, c.n, 10 ** 6])
    K = int(rng.integers(1, 60))
    g = u.to_gpu(c)
    before = c.lens.copy()
    kvc.paged_evict(g, u.dev(before.astype(np.int32)), K, sinks=2, recent=5)
    og.evict(c, before, K, 2, 5)
    u.same_cache(g, c)
    assert ((c.lens != before) <= (before > K)).all()


def test_replays_count_anew():
    """The counts start at zero in every replay of a captured eviction."""
    c = u.random_cache(70, 3, 2, 64, 16, [60, 60, 50], weights=True)
    c.table[2, 0] = c.table[1, 0]                            # 1 and 2 share a page
    g, seen = u.to_gpu(c), u.dev(np.array([60, 60, 50], np.int32))
    ws = torch.empty(g.evict_workspace_bytes(40), dtype=torch.uint8, device="cuda")
    keep = [x.clone() for x in (g.k_pool, g.v_pool, g.weight, g.pos, g.seq_len)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.paged_evict(g, seen, 40, ws=ws)
    og.evict(c, [60, 60, 50], 40, 4, 64)
    assert c.lens.tolist() == [40, 60, 50]
    for _ in range(3):
        for x, y in zip((g.k_pool, g.v_pool, g.weight, g.pos, g.seq_len), keep):
            x.copy_(y)
        graph.replay()
        u.same_cache(g, c)
