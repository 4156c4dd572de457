"""The 8-bit paged cache and the page tables without a GPU: struct layouts, what
the C entry points refuse (they return before anything is launched), and pins
of their oracle."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import pages as op
from oracle import q8 as oq

pytestmark = pytest.mark.skipif(not os.path.exists(kvc.LIB_PATH),
                                reason="libkvc.so not built (python -m eviction_window_qk_amd.build)")

INC = os.path.join(os.path.dirname(__file__), "..", "include")
FAKE = 1 << 40          # aligned, never dereferenced
GB = 1 << 32


@pytest.mark.parametrize("name,struct", [("kvc_q8_cache", kvc._CQ8Cache),
                                         ("kvc_page_table", kvc._CPageTable),
                                         ("kvc_page_buffer", kvc._CPageBuffer)])
def test_struct_layouts(tmp_path, name, struct):
    names = [f for f, _ in struct._fields_]
    body = "".join(f'  printf("%s %zu\\n", "{f}", offsetof({name}, {f}));\n' for f in names)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kvc.h"\nint main(void) {\n' + body +
                   f'  printf("sizeof %zu\\n", sizeof({name}));\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", INC, str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], check=True, capture_output=True,
                                                   text=True).stdout.splitlines())
    assert int(got.pop("sizeof")) == ctypes.sizeof(struct)
    assert {f: int(o) for f, o in got.items()} == {f: getattr(struct, f).offset for f in names}


def _cache(**kw):
    c = dict(n_seqs=3, kv_heads=4, head_dim=128, block_size=16, table_blocks=10, max_len=0, format=0,
             reserved=0, n_blocks=100, k_pool=FAKE, v_pool=FAKE + GB, k_scale=FAKE + 2 * GB,
             v_scale=FAKE + 3 * GB, table=FAKE + 4 * GB, seq_len=FAKE + 5 * GB)
    c.update(kw)
    return kvc._CQ8Cache(**c)


def _store(c, T=50, ts=50, kept=None, n_kept=0, k=FAKE + 6 * GB, v=FAKE + 7 * GB):
    return kvc.lib().kvc_q8_store(ctypes.addressof(c), T, ts, kept, n_kept, k, v, None)


def _load(c, T=50, ts=50, k=FAKE + 6 * GB, v=FAKE + 7 * GB):
    return kvc.lib().kvc_q8_load(ctypes.addressof(c), T, ts, k, v, None)


def _append(c, W=1, k=FAKE + 6 * GB, v=FAKE + 7 * GB, n_new=None):
    return kvc.lib().kvc_q8_append(ctypes.addressof(c), W, n_new, k, v, None)


def _attend(c, G=4, W=1, scale=0.0, q=FAKE + 6 * GB, out=FAKE + 7 * GB, lse=None, ws=FAKE + 8 * GB, n=1 << 20):
    return kvc.lib().kvc_q8_attend(ctypes.addressof(c), G, W, scale, q, out, lse, ws, n, None)


ALL = [_store, _load, _append, _attend]


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), -4), (dict(head_dim=0), -4), (dict(n_seqs=-1), -1), (dict(kv_heads=0), -1),
    (dict(block_size=0), -1), (dict(block_size=4097), -1), (dict(table_blocks=0), -1),
    (dict(max_len=-1), -1), (dict(format=2), -1), (dict(format=-1), -1), (dict(reserved=1), -1),
    (dict(n_blocks=0), -1), (dict(n_blocks=1 << 31), -1), (dict(n_blocks=1 << 26), -1),  # 2^32 rows
    (dict(n_seqs=1 << 22), -1),                                # 2^24 heads
    (dict(block_size=4096, table_blocks=(1 << 18) + 1), -1),   # past 2^30 positions
    (dict(k_pool=None), -1), (dict(v_pool=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
    (dict(table=None), -1), (dict(seq_len=None), -1), (dict(k_pool=FAKE + 8), -2),
    (dict(v_pool=FAKE + GB + 1), -2), (dict(table=FAKE + 4 * GB + 2), -2), (dict(v_scale=FAKE + 3 * GB + 1), -2),
])
def test_caches_refused(kw, code):
    for call in ALL:
        assert call(_cache(**kw)) == code, call.__name__


def test_null_cache_and_no_sequences():
    L = kvc.lib()
    assert L.kvc_q8_store(None, 1, 1, None, 0, FAKE, FAKE, None) == -1
    assert L.kvc_q8_attend_workspace_bytes(None, 1, 1) == ctypes.c_size_t(-1).value
    for call in ALL:
        assert call(_cache(n_seqs=0, k_pool=None, table=None)) == 0


def test_store_refusals():
    assert _store(_cache(), T=0, ts=0) == -1
    assert _store(_cache(), T=51) == -1                        # past the stride
    assert _store(_cache(), T=(1 << 27) + 1, ts=1 << 28) == -1
    assert _store(_cache(), kept=FAKE + 8 * GB, n_kept=0) == -1
    assert _store(_cache(), kept=None, n_kept=5) == -1
    assert _store(_cache(), k=None) == -1
    assert _store(_cache(), v=FAKE + 7 * GB + 8) == -2
    assert _store(_cache(), kept=FAKE + 8 * GB + 2, n_kept=5) == -2
    assert _store(_cache(), k=FAKE + 64) == -1                 # rows inside the pool
    assert _store(_cache(v_pool=FAKE)) == -1                   # both pools the same
    assert _store(_cache(k_scale=FAKE + GB + 64)) == -1        # scales inside a pool
    assert _store(_cache(table=FAKE + 2 * GB + 4)) == -1       # table inside the scales


def test_load_refusals():
    assert _load(_cache(), T=0) == -1
    assert _load(_cache(), T=60) == -1
    assert _load(_cache(), k=None, v=None) == -1
    assert _load(_cache(), v=FAKE + 7 * GB + 4) == -2
    assert _load(_cache(), k=FAKE) == -1
    assert _load(_cache(), v=FAKE + 6 * GB + 16) == -1         # the outputs overlap


def test_append_refusals():
    assert _append(_cache(), W=0) == -1
    assert _append(_cache(), k=None) == -1
    assert _append(_cache(), k=FAKE + 6 * GB + 4) == -2
    assert _append(_cache(), v=FAKE + 3 * GB) == -1
    assert _append(_cache(), n_new=FAKE + 8 * GB + 2) == -2
    assert _append(_cache(), n_new=FAKE + 64) == -1            # counts inside a pool


def test_attend_refusals():
    c = _cache(table_blocks=70)                                # 1120 positions: three pieces
    need = kvc.lib().kvc_q8_attend_workspace_bytes(ctypes.addressof(c), 4, 1)
    assert 3 * 4 * 4 * 3 * 128 * 4 < need < 1 << 20 and need % 256 == 0
    assert kvc.lib().kvc_q8_attend_workspace_bytes(ctypes.addressof(_cache()), 4, 1) == 0
    assert kvc.lib().kvc_q8_attend_workspace_bytes(ctypes.addressof(_cache()), 0, 1) == ctypes.c_size_t(-1).value
    assert _attend(c, G=0) == -1 and _attend(c, W=0) == -1
    assert _attend(c, G=65) == -4
    assert _attend(c, G=64, W=65) == -1                        # 4160 rows
    assert _attend(c, scale=-1.0) == -1
    assert _attend(c, scale=float("nan")) == -1 and _attend(c, scale=float("inf")) == -1
    assert _attend(c, scale=2.0 ** 127 * 1.5) == -1            # times log2(e) past fp32
    assert _attend(c, q=None) == -1 and _attend(c, out=None) == -1
    assert _attend(c, q=FAKE + 6 * GB + 2) == -2 and _attend(c, lse=FAKE + 9 * GB + 1) == -2
    assert _attend(c, ws=None) == -3 and _attend(c, n=need - 1) == -3
    assert _attend(c, ws=FAKE + 8 * GB + 64) == -2
    assert _attend(c, out=FAKE + 6 * GB) == -1 and _attend(c, out=FAKE) == -1
    assert _attend(c, lse=FAKE + 7 * GB + 16) == -1 and _attend(c, ws=FAKE + GB) == -1


def _table(**kw):
    t = dict(n_seqs=4, table_blocks=6, block_size=16, n_blocks=50, table=FAKE, seq_len=FAKE + GB, refs=FAKE + 2 * GB)
    t.update(kw)
    return kvc._CPageTable(**t)


def _bufs(*spans):
    b = (kvc._CPageBuffer * max(1, len(spans)))()
    for i, (base, size) in enumerate(spans):
        b[i].base, b[i].page_bytes = base, size
    return b


POOL = (FAKE + 10 * GB, 4096)


def _alloc(t, want=FAKE + 3 * GB, status=FAKE + 4 * GB, ws=FAKE + 5 * GB, n=1 << 20):
    return kvc.lib().kvc_pages_alloc(ctypes.addressof(t), want, status, ws, n, None)


def _fork(t, pairs=3, src=FAKE + 6 * GB, dst=FAKE + 7 * GB, bufs=(POOL,), n_bufs=None, status=FAKE + 4 * GB,
          ws=FAKE + 5 * GB, n=1 << 20):
    b = _bufs(*bufs)
    return kvc.lib().kvc_pages_fork(ctypes.addressof(t), pairs, src, dst, b, len(bufs) if n_bufs is None else n_bufs,
                                    status, ws, n, None)


def _free(t, n=2, ids=FAKE + 3 * GB):
    return kvc.lib().kvc_pages_free(ctypes.addressof(t), n, ids, None)


def _compact(t, bufs=(POOL,), to=FAKE + 6 * GB, refs=FAKE + 7 * GB, remap=FAKE + 8 * GB, live=FAKE + 9 * GB,
             ws=FAKE + 5 * GB, n=1 << 20):
    b = _bufs(*bufs)
    return kvc.lib().kvc_pages_compact(ctypes.addressof(t), b, len(bufs), to, refs, remap, live, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), -1), (dict(n_seqs=(1 << 20) + 1), -1), (dict(table_blocks=0), -1), (dict(block_size=0), -1),
    (dict(block_size=4097), -1), (dict(n_blocks=0), -1), (dict(n_blocks=(1 << 24) + 1), -1),
    (dict(block_size=4096, table_blocks=(1 << 18) + 1), -1),
    (dict(table=None), -1), (dict(seq_len=None), -1), (dict(refs=None), -1), (dict(refs=FAKE + 2 * GB + 2), -2),
])
def test_page_tables_refused(kw, code):
    for call in (_alloc, _fork, _free, _compact):
        assert call(_table(**kw)) == code, call.__name__


def test_page_calls_refused():
    assert _alloc(_table(), want=None) == -1 and _alloc(_table(), status=None) == -1
    assert _alloc(_table(), ws=None) == -3 and _alloc(_table(), n=16) == -3
    assert _alloc(_table(), ws=FAKE + 5 * GB + 4) == -2
    assert _alloc(_table(), want=FAKE) == -1                   # inside the table
    assert _alloc(_table(), status=FAKE + GB) == -1            # the lengths
    assert _alloc(_table(n_seqs=0, table=None), want=None) == 0
    assert _fork(_table(), pairs=-1) == -1 and _fork(_table(), src=None) == -1 and _fork(_table(), status=None) == -1
    assert _fork(_table(), pairs=0, src=None) == 0
    assert _fork(_table(n_seqs=0)) == -1
    assert _fork(_table(), ws=None) == -3 and _fork(_table(), dst=FAKE + 7 * GB + 1) == -2
    assert _fork(_table(), bufs=((None, 16),)) == -1 and _fork(_table(), bufs=((FAKE + 10 * GB, 0),)) == -1
    assert _fork(_table(), bufs=(POOL, (FAKE + 10 * GB + 4096, 16))) == -1       # overlapping buffers
    assert _fork(_table(), bufs=((FAKE + 64, 16),)) == -1      # over the table
    assert _fork(_table(), n_bufs=-1) == -1 and _fork(_table(), n_bufs=4097) == -1
    assert _free(_table(), n=-1) == -1 and _free(_table(), ids=None) == -1 and _free(_table(), n=0, ids=None) == 0
    assert _free(_table(), ids=FAKE + 2) == -2 and _free(_table(), ids=FAKE + 4) == -1
    assert _compact(_table(n_seqs=0)) == -1
    assert _compact(_table(), to=None) == -1 and _compact(_table(), to=FAKE) == -1 and _compact(_table(), ws=None) == -3
    assert _compact(_table(), refs=FAKE + 6 * GB) == -1 and _compact(_table(), live=FAKE + 9 * GB + 2) == -2
    L = kvc.lib()
    b = _bufs(POOL)
    assert L.kvc_pages_copy(0, 1, FAKE, FAKE + 64, b, 1, None) == -1
    assert L.kvc_pages_copy(9, -1, FAKE, FAKE + 64, b, 1, None) == -1
    assert L.kvc_pages_copy(9, 1, None, FAKE + 64, b, 1, None) == -1
    assert L.kvc_pages_copy(9, 1, FAKE + 10 * GB, FAKE, b, 1, None) == -1        # ids inside a buffer
    assert L.kvc_pages_copy(9, 1, FAKE + 2, FAKE, b, 1, None) == -2
    assert L.kvc_pages_copy(9, 0, None, None, b, 1, None) == 0
    assert L.kvc_pages_workspace_bytes(ctypes.addressof(_table(n_blocks=0)), 0) == 0
    assert L.kvc_pages_workspace_bytes(ctypes.addressof(_table()), -1) == 0
    assert L.kvc_pages_workspace_bytes(ctypes.addressof(_table()), 100) >= L.kvc_pages_workspace_bytes(
        ctypes.addressof(_table()), 0) > 0


def test_binding_refuses():
    f8 = torch.zeros((4, 2, 16, 64), dtype=torch.float8_e4m3fn)
    sc, tab, ln = torch.zeros((4, 2)), torch.zeros((1, 3), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        kvc.Q8Cache(f8, f8, sc, sc, tab, ln)                   # CPU tensors
    with pytest.raises(TypeError):
        kvc.Q8Cache(f8.view(torch.uint8), f8, sc, sc, tab, ln)
    with pytest.raises(ValueError):
        kvc.Q8Cache(f8[0], f8[0], sc, sc, tab, ln)
    with pytest.raises(ValueError):
        kvc.PageTable(tab, ln, torch.zeros(4, dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        kvc.PageTable(ln, ln, torch.zeros(4, dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        kvc.PageBuffers([f8])


# --- the oracle ---------------------------------------------------------------

def test_oracle_codes_against_an_independent_cast():
    y = np.random.default_rng(0).normal(size=100000).astype(np.float32) * 60
    y = np.clip(np.concatenate([y, y * 2.0 ** -10, [0, 2.0 ** -10, 3 * 2.0 ** -10, 448, -447.9]]), -448, 448).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(oq.encode(y, oq.E4M3), want.view(torch.uint8).numpy())
    np.testing.assert_array_equal(oq.decode(oq.encode(y, oq.E4M3), oq.E4M3), want.double().numpy())


def test_oracle_scales():
    assert oq.page_scale(448.0, oq.E4M3)[0] == 1.0 and oq.page_scale(450.0, oq.E4M3)[0] == 2.0
    assert oq.page_scale(1.75, oq.E4M3)[0] == 2.0 ** -8 and oq.page_scale(0.0, oq.E4M3)[0] == 2.0 ** -126
    assert oq.page_scale(127.0, oq.INT8)[0] == 1.0 and oq.page_scale(0.0, oq.INT8)[0] == np.float32(2.0 ** -126)


def test_oracle_attention_by_hand():
    """Two positions with equal scores average their values; one alone is returned."""
    k = np.zeros((1, 1, 2, 64), np.uint8)
    v = k.copy()
    v[0, 0, 0], v[0, 0, 1] = 4, 8
    one = np.ones((1, 1), np.float32)
    c = oq.Cache(k, v, one, one * 0.5, [[0]], [2], oq.INT8)
    out, lse, *_ = oq.attend(c, np.ones((1, 1, 2, 64)))
    np.testing.assert_allclose(out[0, 0, 0], 2.0)
    np.testing.assert_allclose(out[0, 0, 1], 3.0)
    np.testing.assert_allclose(lse[0, 0], [0.0, np.log(2.0)])


def test_oracle_pages_by_hand():
    t = op.Pages([[2, 0, -1], [-1, -1, -1]], [5, 0], [1, 0, 1, 0, 0], 4)
    st, copies = op.fork(t, [0], [1])
    assert st.tolist() == [0] and copies == [(0, 1)]
    assert t.table.tolist() == [[2, 0, -1], [2, 1, -1]] and t.refs.tolist() == [1, 1, 2, 0, 0]
    assert op.alloc(t, [9, 12]).tolist() == [0, 0]             # pages 3 and 4
    assert t.table.tolist() == [[2, 0, 3], [2, 1, 4]]
    op.release(t, [0, 0])
    assert t.refs.tolist() == [0, 1, 1, 0, 1] and t.lens.tolist() == [0, 5]
    table, refs, remap, n, moved = op.compact(t)
    assert n == 3 and moved == [(4, 0)] and table.tolist() == [[-1, -1, -1], [2, 1, 0]]
    assert refs.tolist() == [1, 1, 1, 0, 0] and remap.tolist() == [-1, 1, 2, -1, 0]
    assert op.alloc(t, [12, 0]).tolist() == [1, 0]             # two free, three wanted


# --- buffers of many layers -----------------------------------------------------

def _copy_of(spans, n_blocks=16, src=FAKE, dst=FAKE + GB):
    return kvc.lib().kvc_pages_copy(n_blocks, 1, src, dst, _bufs(*spans), len(spans), None)


def _layers(n, seed, n_blocks=16):
    """n buffers of different page sizes side by side, in random order."""
    rng = np.random.default_rng(seed)
    size = rng.integers(1, 5000, n)
    gap = rng.integers(0, 2, n) * rng.integers(1, 100, n)
    base = FAKE + 4 * GB + np.concatenate([[0], np.cumsum(size * n_blocks + gap)[:-1]])
    order = rng.permutation(n)
    return [(int(base[i]), int(size[i])) for i in order]


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")
@pytest.mark.parametrize("n", [2, 3, 17, 128, 4096])
def test_one_overlap_among_many_buffers(n):
    """One byte of two buffers, one inside another, or an id array inside one: refused
    wherever in the list they stand.  (Disjoint buffers would be launched: those
    calls are in the GPU tests.)"""
    for seed in range(6):
        rng = np.random.default_rng([n, seed])
        spans = _layers(n, seed)
        i, j = (int(x) for x in rng.choice(n, 2, replace=False))
        last = (spans[i][0] + spans[i][1] * 16 - 1, 1)         # 16 bytes from the last one of buffer i on
        inside = (spans[i][0] + spans[i][1] * 16 // 2, 1)
        same = spans[i]
        for other in (last, inside, same):
            bad = list(spans)
            bad[j] = other
            assert _copy_of(bad) == -1
        assert _copy_of(spans, src=(spans[i][0] + spans[i][1] * 16 - 1) & ~3) == -1
        assert _copy_of(spans, dst=spans[i][0] & ~3) == -1     # the word of its first byte


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can be launched")
def test_checking_many_buffers_is_quick():
    """The check of 4096 buffers sorts them: comparing all pairs took 9 ms and more."""
    import time
    spans = _layers(4096, 1)
    spans[-1] = (FAKE + 64, 16)                                # over the ids: refused by the last one
    b = _bufs(*spans)
    took = []
    for _ in range(7):
        t = time.perf_counter()
        assert kvc.lib().kvc_pages_copy(16, 100, FAKE, FAKE + GB, b, len(spans), None) == -1
        took.append(time.perf_counter() - t)
    assert min(took) < 3e-3, took


@pytest.mark.parametrize("n", [(1 << 32) + 16, 1 << 31, -(1 << 32) + 16, 16.5])
def test_binding_refuses_integers_that_c_would_wrap(n):
    i32 = dict(dtype=torch.int32)
    f8 = torch.zeros((4, 2, 16, 64), dtype=torch.float8_e4m3fn)
    sc, tab, ln = torch.zeros((4, 2)), torch.zeros((1, 3), **i32), torch.zeros(1, **i32)
    with pytest.raises(ValueError, match="block_size"):
        kvc.PageTable(tab, ln, torch.zeros(4, **i32), n)
    with pytest.raises(ValueError, match="max_len"):
        kvc.Q8Cache(f8, f8, sc, sc, tab, ln, max_len=n)
