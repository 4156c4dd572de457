"""Host side of the bf16 paged cache, beside test_paged_host.py: what calls ask for, and pins of the
oracle for pages that are shared."""
import ctypes
import os

import numpy as np
import pytest

from eviction_window_qk_amd import kvc
from oracle import paged as og

pytestmark = pytest.mark.skipif(not os.path.exists(kvc.LIB_PATH),
                                reason="libkvc.so not built (python -m eviction_window_qk_amd.build)")

FAKE, GB = 1 << 40, 1 << 32   # aligned, never dereferenced


def _cache(**kw):
    c = dict(n_seqs=3, kv_heads=4, head_dim=128, block_size=16, table_blocks=10, max_len=0, n_blocks=100,
             k_pool=FAKE, v_pool=FAKE + GB, table=FAKE + 4 * GB, seq_len=FAKE + 5 * GB, weight=FAKE + 2 * GB,
             pos=FAKE + 3 * GB)
    c.update(kw)
    return kvc._CPagedCache(**c)


def test_evictions_ask_for_a_count_a_page():
    few, many = _cache(n_blocks=64), _cache(n_blocks=64 + 4096)
    a, b = (kvc.lib().kvc_paged_evict_workspace_bytes(ctypes.addressof(c), 50) for c in (few, many))
    assert b - a == 4 * 4096 and a >= 3 * 4 * (1 + 2 * 50) * 4 + 64 * 4


def test_oracle_leaves_sequences_that_share_pages():
    k = np.arange(6, dtype=np.uint16).repeat(128).reshape(6, 1, 2, 64)
    w = np.tile(np.float32([[1, 2, 3, 4]]), (3, 1))
    pos = np.tile(np.arange(4, dtype=np.int32), (3, 1))
    # 0 and 1 share page 0; 2 shares page 3, past its budget, with what lies behind 1's length
    c = og.Cache(k, k, [[0, 1], [0, 3], [2, 3]], [4, 2, 4], w, pos)
    og.evict(c, [4, 2, 4], 2, 0, 0)
    assert c.lens.tolist() == [4, 2, 2]
    assert c.pos[0].tolist() == [0, 1, 2, 3] and c.pos[2].tolist() == [2, 3, 2, 3]
    np.testing.assert_array_equal(c.k[[0, 1, 3]], k[[0, 1, 3]])
    np.testing.assert_array_equal(c.k[2], k[3])
    # a page twice in one sequence
    c = og.Cache(k, k, [[0, 0]], [4], w[:1], pos[:1])
    og.evict(c, [4], 3, 0, 0)
    assert c.lens.tolist() == [4]
