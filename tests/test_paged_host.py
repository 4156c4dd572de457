"""The bf16 paged cache without a GPU: struct layouts, what the C entry points refuse (they return
before anything is launched), the binding's refusals, frequencies, and pins of the oracle."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import paged as og
from oracle import pages as op

pytestmark = pytest.mark.skipif(not os.path.exists(kvc.LIB_PATH),
                                reason="libkvc.so not built (python -m eviction_window_qk_amd.build)")

INC = os.path.join(os.path.dirname(__file__), "..", "include")
FAKE = 1 << 40          # aligned, never dereferenced
GB = 1 << 32
BAD = ctypes.c_size_t(-1).value


@pytest.mark.parametrize("name,struct", [("kvc_paged_cache", kvc._CPagedCache), ("kvc_rows", kvc._CRows),
                                         ("kvc_rope_plan", kvc._CRopePlan)])
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
    c = dict(n_seqs=3, kv_heads=4, head_dim=128, block_size=16, table_blocks=10, max_len=0, n_blocks=100,
             k_pool=FAKE, v_pool=FAKE + GB, table=FAKE + 4 * GB, seq_len=FAKE + 5 * GB, weight=FAKE + 2 * GB,
             pos=FAKE + 3 * GB)
    c.update(kw)
    return kvc._CPagedCache(**c)


def _rows(at, ts=512, hs=128):
    return kvc._CRows(at, ts, hs)


def _plan(**kw):
    p = dict(freq=FAKE + 20 * GB, rot_dim=128, interleaved=0, mscale=1.0, reserved=0)
    p.update(kw)
    return kvc._CRopePlan(**p)


def _p(x):
    return None if x is None else ctypes.addressof(x)


def _append(c, n=5, starts=FAKE + 6 * GB, pos=FAKE + 7 * GB, plan=_plan(), G=2, q=_rows(FAKE + 8 * GB, 1024),
            qo=_rows(FAKE + 9 * GB, 1024), k=_rows(FAKE + 10 * GB), v=_rows(FAKE + 11 * GB)):
    return kvc.lib().kvc_paged_append(_p(c), n, starts, pos, _p(plan), G, _p(q), _p(qo), _p(k), _p(v), None)


def _attend(c, G=2, n=5, mx=0, starts=FAKE + 6 * GB, scale=0.0, q=_rows(FAKE + 8 * GB, 1024),
            out=_rows(FAKE + 9 * GB, 1024), lse=FAKE + 10 * GB, ws=FAKE + 12 * GB, nb=1 << 30):
    return kvc.lib().kvc_paged_attend(_p(c), G, n, mx, starts, scale, _p(q), _p(out), lse, ws, nb, None)


def _evict(c, seen=FAKE + 6 * GB, K=50, sinks=4, recent=8, ws=FAKE + 12 * GB, nb=1 << 30):
    return kvc.lib().kvc_paged_evict(_p(c), seen, K, sinks, recent, ws, nb, None)


def _rope(n=5, heads=4, d=128, plan=_plan(), back=0, pos=FAKE + 7 * GB, x=_rows(FAKE), y=_rows(FAKE + GB)):
    return kvc.lib().kvc_rope(n, heads, d, _p(plan), back, pos, _p(x), _p(y), None)


def _prompt(B=3, H=4, G=2, d=128, n=5, starts=FAKE + 6 * GB, scale=0.0, q=_rows(FAKE, 1024), k=_rows(FAKE + GB),
            v=_rows(FAKE + 2 * GB), out=_rows(FAKE + 3 * GB, 1024), lse=FAKE + 4 * GB):
    return kvc.lib().kvc_prompt_attend(B, H, G, d, n, starts, scale, _p(q), _p(k), _p(v), _p(out), lse, None)


CALLS = [_append, _attend, _evict]


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=96), -4), (dict(head_dim=0), -4), (dict(n_seqs=-1), -1), (dict(kv_heads=0), -1),
    (dict(block_size=0), -1), (dict(block_size=4097), -1), (dict(table_blocks=0), -1), (dict(max_len=-1), -1),
    (dict(n_blocks=0), -1), (dict(n_blocks=1 << 31), -1), (dict(n_blocks=1 << 26), -1), (dict(n_seqs=1 << 22), -1),
    (dict(block_size=4096, table_blocks=(1 << 18) + 1), -1), (dict(k_pool=None), -1), (dict(v_pool=None), -1),
    (dict(table=None), -1), (dict(seq_len=None), -1), (dict(weight=None), -1), (dict(pos=None), -1),
    (dict(k_pool=FAKE + 8), -2), (dict(v_pool=FAKE + GB + 2), -2), (dict(table=FAKE + 4 * GB + 2), -2),
    (dict(seq_len=FAKE + 5 * GB + 1), -2), (dict(weight=FAKE + 2 * GB + 2), -2), (dict(pos=FAKE + 3 * GB + 1), -2),
])
def test_caches_refused(kw, code):
    for call in CALLS:
        assert call(_cache(**kw)) == code, call.__name__


def test_null_caches_and_nothing_to_do():
    for call in CALLS:
        assert call(None) == -1
        assert call(_cache(n_seqs=0, k_pool=None, table=None)) == 0
    assert _append(_cache(k_pool=None), n=0) == 0 and _attend(_cache(k_pool=None), n=0) == 0
    assert _rope(n=0, x=None, pos=None) == 0
    assert _prompt(n=0, q=None) == 0 and _prompt(B=0, starts=None) == 0
    assert kvc.lib().kvc_paged_attend_workspace_bytes(None, 1, 1, 0) == BAD
    assert kvc.lib().kvc_paged_evict_workspace_bytes(None, 1) == 0


def test_append_refusals():
    c = _cache()
    assert _append(c, n=-1) == -1 and _append(c, n=(1 << 23) + 1) == -1
    assert _append(c, starts=None) == -1 and _append(c, k=None) == -1 and _append(c, v=_rows(None)) == -1
    assert _append(c, starts=FAKE + 6 * GB + 2) == -2 and _append(c, pos=FAKE + 7 * GB + 2) == -2
    assert _append(c, k=_rows(FAKE + 10 * GB + 8)) == -2 and _append(c, v=_rows(FAKE + 11 * GB, 513)) == -2
    assert _append(c, k=_rows(FAKE + 10 * GB, -512)) == -1
    assert _append(c, plan=None) == -1                           # q without a rotation
    assert _append(c, G=0) == -1 and _append(c, G=65) == -4
    assert _append(c, q=None) == -1 and _append(c, qo=None) == -1
    assert _append(c, qo=_rows(FAKE + 9 * GB, 1016)) == -1       # tokens run into each other
    assert _append(c, qo=_rows(FAKE + 9 * GB, 0, 0)) == -1
    assert _append(c, qo=_rows(FAKE + 8 * GB + 16, 1024)) == -1  # over q, shifted
    assert _append(c, k=_rows(FAKE + 64)) == -1                  # rows inside a pool
    assert _append(_cache(v_pool=FAKE)) == -1 and _append(_cache(pos=FAKE + 2 * GB)) == -1
    assert _append(_cache(weight=FAKE + 64)) == -1
    assert _append(c, pos=FAKE + 3 * GB) == -1                   # positions inside pos
    # q beside k and v in one tensor: apart, though their ranges are not
    w = 16 * 128
    q, k, v = _rows(FAKE + 8 * GB, w), _rows(FAKE + 8 * GB + 8 * 256, w), _rows(FAKE + 8 * GB + 12 * 256, w)
    assert _append(c, q=q, qo=q, k=_rows(FAKE + 8 * GB + 7 * 256, w), v=v) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), -1), (dict(rot_dim=3), -1), (dict(rot_dim=130), -1), (dict(rot_dim=-2), -1), (dict(interleaved=2), -1),
    (dict(reserved=1), -1), (dict(freq=None), -1), (dict(freq=FAKE + 20 * GB + 4), -2), (dict(mscale=float("nan")), -1),
    (dict(mscale=float("inf")), -1),
])
def test_plans_refused(kw, code):
    assert _rope(plan=_plan(**kw)) == code
    assert _append(_cache(), plan=_plan(**kw)) == code


def test_rope_refusals():
    assert _rope(d=96) == -4 and _rope(n=-1) == -1 and _rope(heads=0) == -1 and _rope(heads=65537) == -1
    assert _rope(n=1 << 20, heads=1 << 10) == -1 and _rope(back=2) == -1 and _rope(plan=None) == -1
    assert _rope(x=None) == -1 and _rope(y=None) == -1 and _rope(pos=None) == -1 and _rope(pos=FAKE + 7 * GB + 1) == -2
    assert _rope(y=_rows(FAKE + 256)) == -1                       # over x, shifted
    assert _rope(y=_rows(FAKE, 1024)) == -1                       # x with another stride
    assert _rope(y=_rows(FAKE + GB, 504)) == -1 and _rope(y=_rows(FAKE + GB, 128, 512)) == -1
    assert _rope(pos=FAKE + GB + 64) == -1                        # positions inside y
    assert _rope(y=_rows(FAKE + 20 * GB)) == -1                   # y over the frequencies


def test_attend_refusals():
    c = _cache(table_blocks=70)                                   # 1120 slots
    need = kvc.lib().kvc_paged_attend_workspace_bytes(_p(c), 2, 5, 0)
    assert 0 < need < 1 << 30 and need % 256 == 0
    assert kvc.lib().kvc_paged_attend_workspace_bytes(_p(c), 0, 5, 0) == BAD
    assert kvc.lib().kvc_paged_attend_workspace_bytes(_p(c), 65, 5, 0) == BAD
    assert kvc.lib().kvc_paged_attend_workspace_bytes(_p(_cache(weight=None, pos=None)), 2, 5, 0) == 0
    assert _attend(c, G=0) == -1 and _attend(c, G=65) == -4 and _attend(c, n=-1) == -1 and _attend(c, mx=-1) == -1
    assert _attend(c, n=1 << 23, G=64) == -1
    for s in (-1.0, float("nan"), float("inf"), 2.0 ** 127 * 1.5):
        assert _attend(c, scale=s) == -1
    assert _attend(c, q=None) == -1 and _attend(c, out=None) == -1 and _attend(c, starts=None) == -1
    assert _attend(c, starts=FAKE + 6 * GB + 1) == -2 and _attend(c, lse=FAKE + 10 * GB + 2) == -2
    assert _attend(c, ws=None) == -3 and _attend(c, nb=need - 1) == -3 and _attend(c, ws=FAKE + 12 * GB + 64) == -2
    assert _attend(c, out=_rows(FAKE + 8 * GB, 1024)) == -1       # out over q
    assert _attend(c, out=_rows(FAKE + GB + 64, 1024)) == -1 and _attend(c, lse=FAKE + 2 * GB) == -1
    assert _attend(c, ws=FAKE + 8 * GB) == -1                     # workspace over q
    assert _attend(c, starts=FAKE + 9 * GB + 64) == -1
    assert _attend(c, q=_rows(FAKE + 2 * GB, 1024)) == -1         # q inside the weights


def test_prompt_refusals():
    assert _prompt(d=96) == -4 and _prompt(G=65) == -4 and _prompt(G=0) == -1 and _prompt(H=0) == -1
    assert _prompt(H=65537) == -1 and _prompt(B=-1) == -1 and _prompt(n=-1) == -1 and _prompt(B=1 << 20) == -1
    assert _prompt(scale=-1.0) == -1 and _prompt(starts=None) == -1 and _prompt(starts=FAKE + 6 * GB + 2) == -2
    assert _prompt(q=None) == -1 and _prompt(k=None) == -1 and _prompt(v=_rows(FAKE + 2 * GB, 4)) == -2
    assert _prompt(out=_rows(FAKE + GB, 1024)) == -1 and _prompt(lse=FAKE + 64) == -1
    assert _prompt(out=_rows(FAKE + 3 * GB, 512)) == -1 and _prompt(lse=FAKE + 4 * GB + 2) == -2


def test_evict_refusals():
    c = _cache()
    need = kvc.lib().kvc_paged_evict_workspace_bytes(_p(c), 50)
    assert 3 * 4 * (1 + 2 * 50) * 4 <= need < 1 << 20
    assert kvc.lib().kvc_paged_evict_workspace_bytes(_p(c), 0) == 0
    assert _evict(c, K=0) == -1 and _evict(c, sinks=-1) == -1 and _evict(c, recent=-1) == -1
    assert _evict(_cache(weight=None, pos=None)) == -1 and _evict(c, seen=None) == -1 and _evict(c, seen=FAKE + 6 * GB + 1) == -2
    assert _evict(c, ws=None) == -3 and _evict(c, nb=need - 1) == -3 and _evict(c, ws=FAKE + 12 * GB + 4) == -2
    assert _evict(c, seen=FAKE + 5 * GB) == -1                    # seen is not the lengths, which change
    assert _evict(c, ws=FAKE) == -1 and _evict(_cache(seq_len=FAKE + 2 * GB)) == -1


def test_launches_past_the_grid_refused():
    """A workgroup counts a token's query heads in 31 bits; a launch has below 2^32 work-items."""
    L = kvc.lib()
    many = _cache(kv_heads=1 << 20)
    assert _append(many, n=1, G=17) == -1 and _attend(many, n=1, G=17) == -1
    assert L.kvc_paged_attend_workspace_bytes(_p(many), 17, 1, 0) == BAD
    assert L.kvc_paged_attend_workspace_bytes(_p(many), 16, 1, 0) != BAD
    wide = _cache(n_seqs=1 << 20, kv_heads=4)
    assert _evict(wide) == -1 and L.kvc_paged_evict_workspace_bytes(_p(wide), 50) == 0
    wide.n_seqs -= 1
    assert L.kvc_paged_evict_workspace_bytes(_p(wide), 50) >= 4 * ((1 << 20) - 1) * 101 * 4


def test_trim_refusals():
    t = kvc._CPageTable(n_seqs=3, table_blocks=10, block_size=16, n_blocks=100, table=FAKE, seq_len=FAKE + GB, refs=FAKE + 2 * GB)
    L = kvc.lib()
    assert L.kvc_pages_trim(None, None) == -1
    for name, value, code in (("n_blocks", 0, -1), ("table", None, -1), ("refs", FAKE + 2, -2), ("refs", FAKE, -1)):
        was = getattr(t, name)
        setattr(t, name, value)
        assert L.kvc_pages_trim(ctypes.addressof(t), None) == code
        setattr(t, name, was)
    t.n_seqs, t.table = 0, None
    assert L.kvc_pages_trim(ctypes.addressof(t), None) == 0


def test_binding_refuses_other_tensors():
    cpu = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        kvc.PagedCache(cpu, cpu, i32(1, 2), i32(1))                # on the CPU
    with pytest.raises(ValueError):
        kvc.PagedCache(cpu[0], cpu[0], i32(1, 2), i32(1))
    with pytest.raises(ValueError):
        kvc.PagedCache(cpu, cpu, i32(1, 2), i32(1), weight=torch.zeros(2, 32))
    with pytest.raises(ValueError):
        kvc.Rope(torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        kvc.prompt_attend(cpu[0], cpu[0], cpu[0], i32(2))


def test_frequencies():
    f, m = kvc.rope_frequencies(8)
    assert m == 1.0 and f.tolist() == [10000.0 ** (-2 * i / 8) for i in range(4)]
    f, m = kvc.rope_frequencies(8, scaling="linear", factor=4.0)
    assert m == 1.0 and torch.equal(f, kvc.rope_frequencies(8)[0] / 4)
    plain = kvc.rope_frequencies(128, base=500000.0)[0]
    f, _ = kvc.rope_frequencies(128, base=500000.0, scaling="ntk", factor=8.0)
    assert f[0] == plain[0] and abs(float(f[-1] * 8 / plain[-1]) - 1) < 1e-12
    f, m = kvc.rope_frequencies(128, base=500000.0, scaling="banded", factor=8.0, trained=8192)
    turns = 8192 * plain / (2 * math.pi)
    assert torch.equal(f[turns >= 4], plain[turns >= 4]) and torch.equal(f[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((f[mid] < plain[mid]) & (f[mid] > plain[mid] / 8)).all() and m == 1.0
    f, m = kvc.rope_frequencies(128, scaling="yarn", factor=16.0, trained=4096, slow=1, fast=32)
    plain = kvc.rope_frequencies(128)[0]
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(f[turns > 40], plain[turns > 40]) and torch.allclose(f[turns < 0.8], plain[turns < 0.8] / 16, rtol=1e-15)
    assert abs(m - (0.1 * math.log(16) + 1)) < 1e-15 and (f[1:] < f[:-1]).all()
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5), dict(scaling="other"),
               dict(scaling="banded"), dict(scaling="yarn", trained=10, slow=4.0, fast=4.0), dict(rot_dim=2, scaling="ntk")):
        with pytest.raises(ValueError):
            kvc.rope_frequencies(**{"rot_dim": 8, **kw})


def test_oracle_rope_pins():
    x = np.zeros((2, 1, 4))
    x[:, 0] = [1, 2, 3, 4]
    y, _ = og.rope(x, [0, 1], [math.pi / 2, math.pi], 1.0)
    np.testing.assert_allclose(y[0, 0], [1, 2, 3, 4])
    np.testing.assert_allclose(y[1, 0], [-3, -2, 1, -4], atol=1e-15)
    y, _ = og.rope(x, [0, 1], [math.pi / 2], 2.0, interleaved=True)
    np.testing.assert_allclose(y[1, 0], [-4, 2, 3, 4], atol=1e-15)
    z, _ = og.rope(y, [0, 1], [math.pi / 2], 0.5, interleaved=True, backward=True)
    np.testing.assert_allclose(z, x, atol=1e-15)


def test_oracle_attention_pins():
    """One key: its value.  Equal keys: the mean.  A cache of holes: nothing.  Weights sum to the rows."""
    one = np.uint16(0x3F80)
    k = np.full((3, 1, 2, 64), one)
    v = np.zeros((3, 1, 2, 64), np.uint16)
    v[2, 0, 0], v[0, 0, 0] = one, np.uint16(0x4040)               # 1 and 3
    c = og.Cache(k, v, [[2, 0], [-1, -1]], [3, 2], np.zeros((2, 4), np.float32), np.zeros((2, 4), np.int32))
    r = og.attend(c, np.ones((3, 2, 64)), [0, 2, 3])
    assert r["out"][0, 0, 0] == 0.5 and abs(r["out"][1, 1, 0] - 4 / 3) < 1e-15     # slots 0..1, then 0..2
    assert np.isneginf(r["lse"][2]).all() and (r["out"][2] == 0).all()
    np.testing.assert_allclose(r["add"][0], [2 * (1 / 2 + 1 / 3)] * 2 + [2 / 3, 0])
    assert (r["add"][1] == 0).all()
    p = og.prompt(np.ones((2, 1, 64)), np.ones((2, 1, 64)), np.stack([np.zeros((1, 64)), np.ones((1, 64))]), [0, 2])
    assert p["out"][0, 0, 0] == 0 and p["out"][1, 0, 0] == 0.5 and abs(p["lse"][1, 0] - (8 + math.log(2))) < 1e-14


def test_oracle_evict_pins():
    k = np.arange(6, dtype=np.uint16).repeat(64).reshape(1, 1, 6, 64)
    c = og.Cache(k, k, [[0]], [6], np.float32([[5, 1, 0, 9, 1, 3]]), np.array([[0, 1, 2, 3, 4, 5]], np.int32))
    og.evict(c, [6], 4, 1, 1)                                      # 0 a sink, 5 recent, 3 by weight, 1 before 4
    assert c.pos[0].tolist() == [0, 1, 5, 3, 4, 5] and c.lens[0] == 4
    assert c.k[0, 0, :, 0].tolist() == [0, 1, 5, 3, 4, 5] and c.weight[0, 2] == 3
    t = op.Pages([[1, 2, 0], [2, -1, -1]], [5, 0], [1, 1, 2], 4)
    op.trim(t)
    assert t.table.tolist() == [[1, 2, -1], [-1, -1, -1]] and t.refs.tolist() == [0, 1, 1]
