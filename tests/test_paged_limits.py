"""Host side of the bf16 paged cache, beside test_paged_host.py: what calls ask for, and pins of the
oracle for pages that are shared."""
import ctypes
import os
import subprocess

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


# ---------------------------------------------------------------------------
# workspace of the attention: every (row, piece) has a place, and few are spare
# ---------------------------------------------------------------------------

PLACES = r"""
#include <stdio.h>
#include <stdint.h>
#include <algorithm>
#include <vector>
#include "kvc_paged.h"
using namespace kvc;
static uint64_t s = 88172645463325252ull;
static uint64_t xr() { s ^= s << 13; s ^= s >> 7; s ^= s << 17; return s; }
static int spread(int most) { return int(xr() % (uint64_t(1) << (xr() % (64 - __builtin_clzll(uint64_t(most)) + 1)))) % (most + 1); }
int main() {
  long bad = 0, checked = 0;
  for (int it = 0; it < 20000; ++it) {
    const int B = 1 + spread(300), G = 1 + int(xr() % 64), cap = 1 + spread(it % 50 ? 300000 : (1 << 30));
    std::vector<int> starts{0}, len(B);
    int longest = 0;
    for (int b = 0; b < B; ++b) {
      const int n = spread(it % 3 ? 3 : 3000);
      longest = std::max(longest, n);
      starts.push_back(starts.back() + n);
      len[b] = xr() % 4 ? spread(cap) : cap;
    }
    const int n_tokens = starts.back() + int(xr() % 3), bound = xr() % 2 ? longest : 1 + spread(longest + 1);
    const int max_new = bound > 0 && bound < n_tokens ? bound : n_tokens;
    // as the library sizes a call
    const bool many = int64_t(G) * max_new > kFewRows;
    const int rows = int(std::min<int64_t>(int64_t(G) * max_new, kFewRows)), fp = few_max_pieces(cap), tp = tile_max_pieces(cap);
    Partials p{};
    p.most = many && tp > fp ? tp : fp;
    p.each = many && kTileWork * kTileRows > rows * fp ? kTileWork * kTileRows : rows * fp;
    for (int b = 0; b < B; ++b, ++checked) {
      const int a = starts[b], e = starts[b + 1], R = std::min(e - a, max_new) * G;
      const int64_t room = first_place(p, e, b + 1, G) - first_place(p, a, b, G);
      const int slots = first_slot(e, b + 1, G, tp) - first_slot(a, b, G, tp);
      if (R > kFewRows) {
        const int tiles = (R + kTileRows - 1) / kTileRows, pieces = tile_pieces(len[b], tiles);
        bad += pieces > tp || int64_t(R) * pieces > room || int64_t(tiles) * pieces > slots;
      } else {
        const int chunk = few_chunk(len[b]), pieces = std::max(1, (len[b] + chunk - 1) / chunk);
        bad += pieces > fp || int64_t(R) * pieces > room || slots < 0 || R > rows;
        bad += score_rows(e, b + 1, G, rows) - score_rows(a, b, G, rows) < R;
      }
      bad += room < 0;
    }
    bad += first_place(p, n_tokens, B, G) < first_place(p, starts[B], B, G) || first_slot(n_tokens, B, G, tp) < first_slot(starts[B], B, G, tp);
  }
  printf("%ld %ld\n", bad, checked);
  return 0;
}
"""


def test_every_row_and_piece_has_a_place(tmp_path):
    """The functions that number (row, piece) places and (tile, piece) workgroups, over random batches: what
    lies between a sequence's start and the next one's is enough for it."""
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("no hipcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "places.hip", tmp_path / "places"
    src.write_text(PLACES)
    subprocess.run([hipcc, "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-I", os.path.join(root, "include"), "-I",
                    os.path.join(root, "eviction_window_qk_amd", "csrc"), "-c", str(src), "-o", str(tmp_path / "places.o")], check=True)
    subprocess.run([hipcc, str(tmp_path / "places.o"), "-o", str(exe)], check=True)
    bad, checked = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert bad == 0 and checked > 100000


# (sequences, slots of a table, new tokens, most of a sequence, weights, bytes at most, as a share of the pools of a full table)
BYTES = [
    (64, 1024, 64 * 64, 64, False, 0.6), (255 + 1, 4096, 255 + 512, 512, False, 0.06), (255 + 1, 4096, 255 + 512, 512, True, 0.15),
    (63 + 1, 32768, 63 + 512, 512, False, 0.08), (255 + 1, 32768, 255 + 512, 512, True, 0.16), (63 + 1, 32768, 63 + 512, 512, True, 0.33),
    (1, 131072, 512, 512, False, 0.1), (64, 1152, 64, 1, True, 0.1), (64, 131072, 64, 1, True, 0.06),
]


@pytest.mark.parametrize("case", BYTES, ids=[str(i) for i in range(len(BYTES))])
def test_attention_asks_for_little_beside_the_pools(case):
    """8 KV heads of 128, 4 rows a token, pages of 16."""
    B, room, n, most, weights, share = case
    kw = {} if weights else dict(weight=None, pos=None)
    c = _cache(n_seqs=B, kv_heads=8, table_blocks=room // 16, n_blocks=B * room // 16, **kw)
    got = kvc.lib().kvc_paged_attend_workspace_bytes(ctypes.addressof(c), 4, n, most)
    pools = B * room * 8 * 128 * 4
    assert 0 < got < share * pools, f"{got / pools:.3f} of the pools"
