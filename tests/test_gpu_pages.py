"""Page tables on the GPU against the oracle: tables, counts, lengths, statuses
and page bytes equal."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import pages as op
import q8_utils as u

pytestmark = pytest.mark.gpu

# B, table_blocks, block_size, n_blocks
SHAPES = [(1, 1, 1, 1), (3, 4, 16, 9), (20, 13, 24, 150), (64, 40, 16, 2000), (300, 20, 8, 4097),
          (50, 300, 1, 9000), (30, 40, 16, 40000),
          (20, 5000, 2, 90000),      # more pages than every workgroup counts for itself
          (5000, 3, 8, 12000)]       # more sequences than every workgroup sums


def _buffers(seed, n, widths=((4, 16), (3,), (2, 2, 2))):
    rng = u.rng_of(seed, n)
    bufs = [torch.from_numpy(rng.integers(0, 256, (n,) + w).astype(np.uint8)).cuda() for w in widths]
    bufs.append(torch.from_numpy(rng.standard_normal((n, 5)).astype(np.float32)).cuda())
    bufs.append(torch.from_numpy(rng.integers(0, 256, (n, 5000)).astype(np.uint8)).cuda())
    return bufs


def _host(bufs):
    return [b.cpu().numpy().copy() for b in bufs]


def _check_copies(bufs, before, copies):
    for b, was in zip(bufs, before):
        want = was.copy()
        for a, z in copies:
            want[z] = was[a]
        np.testing.assert_array_equal(b.cpu().numpy(), want)


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_alloc(shape):
    B, tb, bs, n = shape
    print(f"[case] alloc {shape}", flush=True)
    t = u.random_pages(1, B, tb, bs, n)
    g = u.pages_to_gpu(t)
    rng = u.rng_of(2, B)
    for step in range(4):
        want = np.minimum(t.lens + rng.integers(0, 2 * bs * (step + 1) + 1, B), tb * bs).astype(np.int32)
        if step == 1:
            want[:: 3] = 0
            want[1:: 7] = -5
            want[2:: 11] = tb * bs + 1
        if step == 3:
            want[:] = tb * bs
        st = kvc.pages_alloc(g, torch.from_numpy(want).cuda())
        ref = op.alloc(t, want)
        np.testing.assert_array_equal(st.cpu().numpy(), ref)
        u.same_pages(g, t)


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
def test_fork_and_free(shape):
    B, tb, bs, n = shape
    print(f"[case] fork {shape}", flush=True)
    t = u.random_pages(3, B, tb, bs, n)
    g = u.pages_to_gpu(t)
    tensors = _buffers(4, n)
    bufs = kvc.PageBuffers(tensors)
    rng = u.rng_of(5, B)
    for step in range(4):
        pairs = int(rng.integers(1, B + 3))
        src = rng.integers(-1, B + 1, pairs).astype(np.int32)
        dst = rng.integers(-1, B + 1, pairs).astype(np.int32)
        before = _host(tensors)
        st = kvc.pages_fork(g, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), bufs)
        ref, copies = op.fork(t, src, dst)
        np.testing.assert_array_equal(st.cpu().numpy(), ref)
        u.same_pages(g, t)
        _check_copies(tensors, before, copies)
        ids = rng.integers(-2, B + 2, max(1, B // 3)).astype(np.int32)
        ids[-1] = ids[0]                                   # named twice
        kvc.pages_free(g, torch.from_numpy(ids).cuda())
        op.release(t, ids)
        u.same_pages(g, t)


def test_many_children_of_one_prompt():
    """Every child shares the whole pages and owns its open one."""
    B, tb, bs, n = 40, 6, 16, 60
    t = op.Pages(np.full((B, tb), -1), np.zeros(B), np.zeros(n), bs)
    t.table[0, :4] = [50, 3, 7, 59]
    t.lens[0] = 50
    t.refs[[50, 3, 7, 59]] = 1
    g = u.pages_to_gpu(t)
    tensors = _buffers(6, n)
    before = _host(tensors)
    src = np.zeros(39, np.int32)
    dst = np.arange(1, 40, dtype=np.int32)
    st = kvc.pages_fork(g, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), kvc.PageBuffers(tensors))
    ref, copies = op.fork(t, src, dst)
    assert st.cpu().numpy().tolist() == ref.tolist() and (ref == 0).all()
    assert t.refs[50] == 40 and len(copies) == 39
    u.same_pages(g, t)
    _check_copies(tensors, before, copies)


def test_forks_past_the_free_pages():
    B, tb, bs, n = 12, 3, 8, 6
    t = op.Pages(np.full((B, tb), -1), np.zeros(B), np.zeros(n), bs)
    t.table[0, :2], t.lens[0] = [5, 2], 13                 # open page
    t.table[1, :1], t.lens[1] = [0], 8                     # whole page
    t.refs[[5, 2, 0]] = 1
    g = u.pages_to_gpu(t)
    tensors = _buffers(7, n)
    before = _host(tensors)
    src = np.array([0, 0, 1, 0, 0, 1], np.int32)
    dst = np.array([2, 3, 4, 5, 6, 7], np.int32)
    st = kvc.pages_fork(g, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), kvc.PageBuffers(tensors))
    ref, copies = op.fork(t, src, dst)
    assert ref.tolist() == [0, 0, 0, 0, 1, 0] and st.cpu().numpy().tolist() == ref.tolist()
    u.same_pages(g, t)
    _check_copies(tensors, before, copies)


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
@pytest.mark.parametrize("fill", [0.0, 0.5, 1.0])
def test_compact(shape, fill):
    B, tb, bs, n = shape
    print(f"[case] compact {shape} {fill}", flush=True)
    t = u.random_pages(8, B, tb, bs, n, fill=fill)
    t.table[0, -1] = n + 5                                  # names no page
    g = u.pages_to_gpu(t)
    tensors = _buffers(9, n)
    before = _host(tensors)
    got = kvc.pages_compact(g, kvc.PageBuffers(tensors))
    table, refs, remap, live, copies = op.compact(t)
    np.testing.assert_array_equal(got["table"].cpu().numpy(), table)
    np.testing.assert_array_equal(got["refs"].cpu().numpy(), refs)
    np.testing.assert_array_equal(got["remap"].cpu().numpy(), remap)
    assert int(got["n_live"][0]) == live
    u.same_pages(g, t)                                      # the old arrays stay
    _check_copies(tensors, before, copies)


def test_copy_pages_skips_bad_ids_and_takes_many_buffers():
    n = 30
    rng = u.rng_of(10)
    tensors = [torch.from_numpy(rng.integers(0, 256, (n, 7 + i % 40)).astype(np.uint8)).cuda() for i in range(130)]
    before = _host(tensors)
    src = np.array([3, -1, 5, 29, 31, 3], np.int32)
    dst = np.array([10, 11, 40, 12, 13, 14], np.int32)
    kvc.pages_copy(torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), kvc.PageBuffers(tensors))
    _check_copies(tensors, before, [(3, 10), (29, 12), (3, 14)])


def test_empty_requests():
    t = u.random_pages(11, 3, 2, 4, 5)
    g = u.pages_to_gpu(t)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    bufs = kvc.PageBuffers([])
    kvc.pages_free(g, none)
    assert kvc.pages_fork(g, none, none, bufs).numel() == 0
    kvc.pages_copy(none, none, bufs)
    one = torch.tensor([0], dtype=torch.int32, device="cuda")
    kvc.pages_copy(one, one, bufs)                          # no buffers: nothing to copy
    u.same_pages(g, t)


def test_tables_alone():
    """Forks and compactions of tables whose pages are kept elsewhere."""
    t = u.random_pages(12, 8, 5, 4, 30)
    g = u.pages_to_gpu(t)
    bufs = kvc.PageBuffers([])
    src, dst = np.array([0, 1], np.int32), np.array([6, 7], np.int32)
    st = kvc.pages_fork(g, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), bufs)
    assert st.cpu().numpy().tolist() == op.fork(t, src, dst)[0].tolist()
    u.same_pages(g, t)
    got = kvc.pages_compact(g, bufs)
    table, refs, remap, live, _ = op.compact(t)
    np.testing.assert_array_equal(got["table"].cpu().numpy(), table)
    np.testing.assert_array_equal(got["remap"].cpu().numpy(), remap)
    assert int(got["n_live"][0]) == live


def test_many_buffers_and_holes():
    """Forty buffers (several launches), entries of a source that name no page."""
    n = 40
    rng = u.rng_of(13)
    t = op.Pages(np.full((5, 4), -1), np.zeros(5), np.zeros(n), 8)
    t.table[0], t.lens[0] = [30, -1, 12, 39], 27            # open page 39, a hole before it
    t.table[1, :2], t.lens[1] = [5, 2 ** 31 - 1], 12        # the open entry names no page
    t.table[4, :1], t.lens[4] = [39 - 8], 8
    t.refs[[30, 12, 39, 5, 31]] = 1
    g = u.pages_to_gpu(t)
    tensors = [torch.from_numpy(rng.integers(0, 256, (n, 1 + 16 * i)).astype(np.uint8)).cuda() for i in range(40)]
    bufs = kvc.PageBuffers(tensors)
    before = _host(tensors)
    src, dst = np.array([0, 1], np.int32), np.array([2, 4], np.int32)
    st = kvc.pages_fork(g, torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda(), bufs)
    ref, copies = op.fork(t, src, dst)
    assert st.cpu().numpy().tolist() == ref.tolist() == [0, 0] and copies == [(39, 0)]
    u.same_pages(g, t)
    _check_copies(tensors, before, copies)
    before = _host(tensors)
    got = kvc.pages_compact(g, bufs)
    table, refs, remap, live, copies = op.compact(t)
    np.testing.assert_array_equal(got["table"].cpu().numpy(), table)
    np.testing.assert_array_equal(got["refs"].cpu().numpy(), refs)
    assert int(got["n_live"][0]) == live
    _check_copies(tensors, before, copies)


@pytest.mark.parametrize("n_bufs", [5, 64, 65, 300])
def test_buffers_side_by_side(n_bufs):
    """Buffers in any order without a byte between them, the ids and the page table among
    them: forked, copied and compacted like buffers of their own."""
    B, tb, bs, n = 6, 4, 8, 20
    t = u.random_pages(20, B, tb, bs, n, fill=1.0)
    rng = u.rng_of(21, n_bufs)
    widths = [int(w) * 4 for w in rng.integers(1, 40, n_bufs)]
    pieces = [n * w for w in widths] + [B * tb * 4, B * 4, n * 4, 4 * 4, 4 * 4]   # table, lengths, counts, src, dst
    slab = torch.from_numpy(rng.integers(0, 256, sum(pieces)).astype(np.uint8)).cuda()
    place, at = {}, 0
    for i in rng.permutation(len(pieces)):
        place[int(i)] = slab[at:at + pieces[i]]
        at += pieces[i]
    tensors = [place[i].view(n, widths[i]) for i in range(n_bufs)]
    table, lens, refs, src, dst = (place[n_bufs + i].view(torch.int32) for i in range(5))
    table = table.view(B, tb)
    for to, x in ((table, t.table), (lens, t.lens), (refs, t.refs), (src, [0, 1, 2, 3]), (dst, [4, 5, 4, 9])):
        to.copy_(torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)))
    g, bufs = kvc.PageTable(table, lens, refs, bs), kvc.PageBuffers(tensors)
    before = _host(tensors)
    st = kvc.pages_fork(g, src, dst, bufs)
    ref, copies = op.fork(t, [0, 1, 2, 3], [4, 5, 4, 9])
    assert st.cpu().numpy().tolist() == ref.tolist()
    u.same_pages(g, t)
    _check_copies(tensors, before, copies)
    src.copy_(torch.tensor([0, 5, 99, 2]))
    dst.copy_(torch.tensor([19, 18, 1, -1]))
    before = _host(tensors)
    kvc.pages_copy(src, dst, bufs)
    _check_copies(tensors, before, [(0, 19), (5, 18)])
    kvc.pages_free(g, torch.tensor([1], dtype=torch.int32, device="cuda"))
    op.release(t, [1])
    before = _host(tensors)
    out = kvc.pages_compact(g, bufs)
    new_table, new_refs, remap, live, moved = op.compact(t)
    assert int(out["n_live"]) == live
    np.testing.assert_array_equal(out["table"].cpu().numpy(), new_table)
    np.testing.assert_array_equal(out["remap"].cpu().numpy(), remap)
    _check_copies(tensors, before, moved)
