"""The 8-bit paged cache on the GPU against the oracle: codes, scales and loaded
rows bit for bit, the attention within a derived bound."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import q8 as oq
import q8_utils as u

pytestmark = pytest.mark.gpu

FMTS = [oq.E4M3, oq.INT8]

# (B, H, d, block_size, lengths, T)
STORE = [
    (1, 1, 64, 16, [1], 1),
    (3, 2, 128, 16, [0, 1, 37], 40),
    (2, 3, 128, 1, [5, 3], 7),
    (2, 2, 64, 24, [24, 49], 50),
    (2, 1, 128, 64, [64, 100], 130),
    (1, 2, 128, 100, [257], 300),
    (2, 1, 128, 128, [128, 129], 140),
    (1, 2, 64, 256, [300], 300),
    (1, 1, 128, 512, [700], 700),
    (2, 1, 64, 4096, [4100, 9], 4200),
]


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("case", STORE, ids=[f"{i}" for i in range(len(STORE))])
def test_store_and_load(case, fmt):
    B, H, d, bs, lens, T = case
    print(f"[case] store {case} {u.NAMES[fmt]}", flush=True)
    for kept_rows in (0, 1):
        c = u.random_cache(1, B, H, d, bs, lens, fmt, holes=0.0)
        k, v = u.random_rows(2, B * H, T + 3, d), u.random_rows(3, B * H, T + 3, d)
        k[0, T // 2] = 0
        kept = None
        if kept_rows:
            rng = u.rng_of(4, T)
            kept = np.sort(rng.integers(-1, T + 2, (B * H, max(1, T - 1))).astype(np.int32), axis=1)
        g = u.to_gpu(c)
        kvc.q8_store(g, u.dev_bf16(k), u.dev_bf16(v), T=T,
                     kept=None if kept is None else torch.from_numpy(kept).cuda())
        oq.store(c, k, v, T, kept)
        torch.cuda.synchronize()
        u.same_cache(g, c)
        for rows in (1, T, T + 5):
            gk, gv = kvc.q8_load(g, rows)
            if kept is not None and kept.shape[1] < max(lens):
                continue            # rows past the kept ones hold poison
            rk, rv = oq.load(c, rows)
            np.testing.assert_array_equal(gk.view(torch.int16).cpu().numpy().view(np.uint16), rk)
            np.testing.assert_array_equal(gv.view(torch.int16).cpu().numpy().view(np.uint16), rv)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
def test_store_extreme_values(fmt):
    """Zero pages, the smallest and largest bf16 magnitudes, exact scale borders."""
    B, H, d, bs, T = 6, 1, 64, 8, 8
    c = u.random_cache(5, B, H, d, bs, [8] * B, fmt)
    x = np.zeros((B, T, d), np.uint16)
    x[1, :, :] = 0x0001                       # smallest subnormal
    x[2, :, ::2] = 0x7F7F                     # largest finite
    x[2, :, 1::2] = 0x8080                    # -2^-126
    x[3] = u.synth.f32_to_bf16_bits(np.tile(np.float32([448.0, -447.0, 1.0, 0.0] * 16), (T, 1)))
    x[4] = u.synth.f32_to_bf16_bits(np.tile(np.float32([450.0, 3.5, 17.0, -2.0] * 16), (T, 1)))
    x[5] = u.random_rows(6, T, d)
    g = u.to_gpu(c)
    kvc.q8_store(g, u.dev_bf16(x), u.dev_bf16(x[::-1].copy()))
    oq.store(c, x, x[::-1].copy(), T)
    torch.cuda.synchronize()
    u.same_cache(g, c)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
def test_every_code_rounds_to_nearest_even(fmt):
    """All bf16 values of one binade range under a scale of one, ties among them."""
    d, bs = 64, 64
    vals = np.arange(0x3A00, 0x43E0, dtype=np.uint16)          # 2^-11 .. 448
    vals = vals[u.synth.bf16_bits_to_f32(vals) <= (448 if fmt == oq.E4M3 else 127)]
    x = np.zeros((1, bs, d), np.uint16)
    x.reshape(-1)[: vals.size] = vals
    x.reshape(-1)[-1] = u.synth.f32_to_bf16_bits(np.float32([448.0 if fmt == oq.E4M3 else 127.0]))[0]
    c = u.random_cache(7, 1, 1, d, bs, [bs], fmt)
    g = u.to_gpu(c)
    neg = np.where(x == 0, x, x | 0x8000)
    kvc.q8_store(g, u.dev_bf16(x), u.dev_bf16(neg))
    oq.store(c, x, neg, bs)
    torch.cuda.synchronize()
    assert float(g.k_scale[int(c.table[0, 0]), 0]) == 1.0
    u.same_cache(g, c)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
def test_load_every_code_at_the_ends_of_fp32(fmt):
    """Products that are subnormal, vanish, or lie next to the largest bf16."""
    scales = np.float32([0.0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -130, 2.0 ** -126, 1.37 * 2.0 ** -126,
                         2.0 ** -100, 1.0, 2.0 ** 118, 1.3 * 2.0 ** 118])
    B, d, bs = scales.size, 64, 8
    c = u.random_cache(44, B, 1, d, bs, [4] * B, fmt, poison=False)
    codes = np.array([x for x in range(256) if x & 0x7F != (0x7F if fmt == oq.E4M3 else -1)], np.uint8)
    for b in range(B):
        page = c.table[b, 0]
        c.k[page, 0, :4].reshape(-1)[: codes.size] = codes
        c.v[page] = c.k[page]
        c.ks[page] = c.vs[page] = scales[b]
    gk, gv = kvc.q8_load(u.to_gpu(c), 6)
    rk, rv = oq.load(c, 6)
    np.testing.assert_array_equal(gk.view(torch.int16).cpu().numpy().view(np.uint16), rk)
    np.testing.assert_array_equal(gv.view(torch.int16).cpu().numpy().view(np.uint16), rv)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
def test_append_to_pages_of_extreme_scales(fmt):
    """Earlier rows under scales from 0 over subnormal ones to 2^100, new rows from
    zero to the largest bf16: the earlier rows' codes and the scales."""
    scales = np.float32([0.0, 2.0 ** -149, 2.0 ** -126, 2.0 ** -30, 1.0, 0.7, 2.0 ** 60, 2.0 ** 100])
    tops = [0x0000, 0x0001, 0x0080, 0x3F80, 0x3F81, 0x7F7F]      # bf16 bits
    B, d, bs, W = scales.size * len(tops), 64, 16, 2
    lens = [9] * B
    c = u.random_cache(45, B, 1, d, bs, lens, fmt, poison=False)
    k = u.random_rows(46, B, W, d)
    f = u.synth.bf16_bits_to_f32(k)
    f /= np.abs(f).max((1, 2), keepdims=True)
    for b in range(B):
        c.ks[c.table[b, 0]] = c.vs[c.table[b, 0]] = scales[b // len(tops)]
        top = u.synth.bf16_bits_to_f32(np.array([tops[b % len(tops)]], np.uint16))[0]
        k[b] = u.synth.f32_to_bf16_bits((f[b] * top).astype(np.float32))
    v = k[:, ::-1].copy()
    g = u.to_gpu(c)
    for _ in range(2):
        kvc.q8_append(g, u.dev_bf16(k), u.dev_bf16(v))
    oq.append(c, k, v)
    torch.cuda.synchronize()
    u.same_cache(g, c)


APPEND = [
    # B, H, d, bs, lengths after, W
    (4, 2, 128, 16, [1, 16, 17, 40], 1),
    (3, 1, 64, 24, [2, 24, 50], 1),
    (4, 2, 128, 16, [0, 3, 18, 35], 5),
    (2, 1, 64, 1, [9, 3], 4),
    (2, 2, 128, 256, [300, 255], 40),
    (1, 1, 128, 64, [200], 150),
]


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("case", APPEND, ids=[f"{i}" for i in range(len(APPEND))])
@pytest.mark.parametrize("loud", [0.02, 1.0, 300.0])
def test_append(case, fmt, loud):
    """New rows smaller than the page's scale holds, about as large, and far larger."""
    B, H, d, bs, lens, W = case
    print(f"[case] append {case} {u.NAMES[fmt]} x{loud}", flush=True)
    c = u.random_cache(8, B, H, d, bs, lens, fmt)
    c.ks = np.where(np.isnan(c.ks), 1.0, c.ks).astype(np.float32)
    c.vs = np.where(np.isnan(c.vs), 1.0, c.vs).astype(np.float32)
    f = lambda s: u.synth.f32_to_bf16_bits((u.synth.bf16_bits_to_f32(u.random_rows(s, B * H, W, d)) * loud).astype(np.float32))
    k, v = f(9), f(10)
    g = u.to_gpu(c)
    kvc.q8_append(g, u.dev_bf16(k), u.dev_bf16(v))
    oq.append(c, k, v)
    torch.cuda.synchronize()
    u.same_cache(g, c)
    kvc.q8_append(g, u.dev_bf16(k), u.dev_bf16(v))      # again: nothing changes
    torch.cuda.synchronize()
    u.same_cache(g, c)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
def test_append_counts_per_sequence(fmt):
    B, H, d, bs, W = 6, 2, 64, 16, 5
    c = u.random_cache(27, B, H, d, bs, [20, 20, 33, 3, 40, 18], fmt, poison=False)
    n_new = np.array([0, 2, 5, 4, -3, 99], np.int32)
    k, v = u.random_rows(28, B * H, W, d), u.random_rows(29, B * H, W, d)
    g = u.to_gpu(c)
    kvc.q8_append(g, u.dev_bf16(k), u.dev_bf16(v), n_new=torch.from_numpy(n_new).cuda())
    oq.append(c, k, v, n_new)
    torch.cuda.synchronize()
    u.same_cache(g, c)


ATTEND = [
    # B, H, G, W, d, bs, lengths, holes
    (1, 1, 1, 1, 64, 16, [1], 0.0),
    (4, 2, 4, 1, 128, 16, [0, 1, 33, 300], 0.0),
    (3, 1, 7, 1, 128, 24, [31, 32, 257], 0.0),
    (2, 2, 16, 1, 64, 1, [100, 64], 0.0),
    (2, 1, 17, 1, 128, 64, [255, 513], 0.0),
    (3, 2, 4, 5, 64, 24, [0, 3, 700], 0.3),
    (2, 1, 9, 9, 128, 100, [90, 411], 0.0),
    (1, 1, 64, 1, 128, 16, [1000], 0.0),
    (2, 1, 1, 40, 64, 32, [39, 600], 0.5),
    (1, 2, 4, 1, 128, 4096, [5000], 0.0),
    (3, 1, 2, 2, 128, 16, [50, 60, 70], 1.0),
    (1, 1, 3, 1, 128, 128, [16500], 0.0),
    (1, 1, 2, 1, 64, 48, [140001], 0.02),
    (2, 2, 8, 5, 128, 16, [700, 41], 0.1),
    (2, 1, 11, 3, 64, 24, [1500, 3], 0.0),
    (1, 2, 6, 8, 64, 7, [900], 0.1),
    (1, 1, 16, 7, 128, 33, [1300], 0.0),
    (1, 2, 9, 8, 128, 16, [2000], 0.0),
]


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("case", ATTEND, ids=[f"{i}" for i in range(len(ATTEND))])
def test_attend(case, fmt):
    B, H, G, W, d, bs, lens, holes = case
    print(f"[case] attend {case} {u.NAMES[fmt]}", flush=True)
    c = u.random_cache(11, B, H, d, bs, lens, fmt, holes=holes)
    q = u.random_rows(12, B * H, G, W, d)
    g = u.to_gpu(c)
    out, lse = kvc.q8_attend(g, u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("spread", [6.0, 14.0])
def test_attend_scales_far_apart(fmt, spread):
    """Page scales over many powers of two, zero scales, large scores."""
    B, H, G, W, d, bs = 2, 2, 5, 1, 128, 8
    c = u.random_cache(13, B, H, d, bs, [400, 77], fmt, scale_spread=spread, poison=False)
    c.ks = np.minimum(c.ks, np.float32(0.05))
    c.vs[u.rng_of(14).random(c.vs.shape) < 0.2] = 0.0
    q = u.random_rows(15, B * H, G, W, d)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True, scale=0.25)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse, scale=0.25)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("where", ["all", "first", "middle"])
def test_attend_values_of_nothing(where, d, fmt):
    """Zero values over hundreds of keys weigh in the denominators like any others:
    in pages stored as zeros (scale 2^-126) and in pages of scale 0, next to values
    in the thousands."""
    B, H, G, W, bs, lens = 2, 2, 3, 2, 16, [1700, 40]
    c = u.random_cache(40, B, H, d, bs, lens, fmt, poison=False)
    c.vs = (c.vs * np.float32(2.0 ** 16)).astype(np.float32)
    at = {"all": [(0, 1700), (0, 40)], "first": [(0, 640), (0, 16)], "middle": [(512, 1264), (16, 32)]}[where]
    for b in range(B):
        pages = c.table[b, at[b][0] // bs:-(-at[b][1] // bs)]
        c.v[pages] = 0
        c.vs[pages, 0] = 2.0 ** -126
        c.vs[pages, 1] = 0.0
    q = u.random_rows(41, B * H, G, W, d)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse)
    if where == "all":
        assert not out.view(torch.int16).bitwise_and(0x7FFF).any()


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("power", [-90, 100])
def test_attend_values_at_the_ends_of_fp32(power, fmt):
    """Values of 2^-90 or 2^100 only: relative accuracy as at one.  In pages 2^60
    apart, hundreds of keys each, the small ones' outputs vanish beside the
    large, their weights do not."""
    B, H, G, W, d, bs = 1, 2, 3, 1, 128, 16
    c = u.random_cache(42, B, H, d, bs, [1500], fmt, poison=False)
    plain = c.vs.copy()
    q = u.random_rows(43, B * H, G, W, d)
    c.vs = (plain * np.float32(2.0 ** power)).astype(np.float32)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True)
    c.vs = plain
    u.check_attention(c, q, (out.double() * 2.0 ** -power).float(), lse)
    c.vs = (plain * np.float32(2.0 ** power)).astype(np.float32)
    c.vs[c.table[0, : 768 // bs]] *= np.float32(2.0 ** (60 if power < 0 else -60))
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("power", [-110, -60, 60, 110])
def test_attend_keys_at_the_ends_of_fp32(power, fmt):
    """Keys of 2^power under queries of 2^-power: the scores of keys of one."""
    B, H, G, W, d, bs = 1, 2, 5, 4, 64, 16
    c = u.random_cache(47, B, H, d, bs, [900], fmt, poison=False)
    q = u.random_rows(48, B * H, G, W, d)
    far = u.synth.f32_to_bf16_bits((u.synth.bf16_bits_to_f32(q) * np.float32(2.0 ** -power)).astype(np.float32))
    plain = c.ks.copy()
    c.ks = (plain * np.float32(2.0 ** power)).astype(np.float32)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(far), want_lse=True)
    torch.cuda.synchronize()
    c.ks = plain
    u.check_attention(c, q, out, lse)


def test_attend_query_range():
    """Queries from the smallest to large magnitudes, and a zero row."""
    B, H, G, W, d, bs = 1, 1, 6, 1, 128, 16
    c = u.random_cache(16, B, H, d, bs, [200], oq.E4M3)
    q = u.random_rows(17, 1, G, W, d)
    f = u.synth.bf16_bits_to_f32(q)
    for i, s in enumerate([0.0, 2.0 ** -130, 2.0 ** -40, 1.0, 2.0 ** 6, 2.0 ** -3]):
        f[0, i] *= np.float32(s)
    f[0, 3, 0, ::7] *= np.float32(2.0 ** -30)       # far below the row's largest
    q = u.synth.f32_to_bf16_bits(f)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("G,W,d", [(4, 1, 128), (5, 4, 64), (3, 8, 128), (8, 5, 128)])
def test_attend_rows_do_not_mix(G, W, d, fmt):
    """A query of NaN or infinity gives NaN in its own row; the other rows have the
    bits they have beside a query of zeros, and beside one of large scores."""
    c = u.random_cache(49, 2, 2, d, 16, [700, 19], fmt, holes=0.1)
    g = u.to_gpu(c)
    q = u.dev_bf16(u.random_rows(50, 4, G, W, d))
    row = (slice(None), G - 2, W - 1)
    got = []
    for fill in (0.0, 30.0, float("nan"), float("inf")):
        x = q.clone()
        x[row] = x[row] * fill if fill == 30.0 else fill
        got.append(kvc.q8_attend(g, x, want_lse=True))
    torch.cuda.synchronize()
    others = torch.ones((4, G, W), dtype=torch.bool, device="cuda")
    others[row] = False
    for out, lse in got[1:]:
        assert torch.equal(out[others].view(torch.int16), got[0][0][others].view(torch.int16))
        assert torch.equal(lse[others], got[0][1][others])
    assert torch.isfinite(got[1][0]).all()
    assert torch.isnan(got[2][0][row]).all() and torch.isnan(got[3][0][row]).all()


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("step", [0.004, 0.05, -0.05, 1.0])
def test_attend_scores_that_rise_and_fall(step, fmt):
    """Scores that grow or fall by `step` a key: maxima that move a little, a lot,
    and at every tile."""
    B, H, G, W, d, bs, L = 1, 1, 3, 2, 64, 16, 1300
    c = u.random_cache(51, B, H, d, bs, [L], fmt, poison=False)
    q = np.zeros((1, G, W, d), np.float32)
    q[..., 0] = 1.0                                     # the score is the key's first value
    q[..., 1:] = 0.01 * u.rng_of(52).normal(size=q[..., 1:].shape)
    pages = c.table[0]
    one = 0x38 if fmt == oq.E4M3 else 1                 # the code of 1
    c.k[pages] = 0
    c.k[pages, 0, :, 0] = one
    at = np.arange(pages.size) * bs * abs(step) * 8.0 / max(1.0, abs(step) * 8.0 * L / 2000.0)
    c.ks[pages, 0] = (at if step > 0 else at[::-1]).astype(np.float32)
    bits = u.synth.f32_to_bf16_bits(q)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(bits), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, bits, out, lse)


def test_max_len_bounds_the_length():
    c = u.random_cache(18, 2, 2, 64, 16, [300, 40], oq.INT8, poison=False)
    g = u.to_gpu(c, max_len=100)
    c2 = oq.Cache(c.k, c.v, c.ks, c.vs, c.table, c.lens, c.fmt, max_len=100)
    q = u.random_rows(19, 4, 3, 1, 64)
    out, lse = kvc.q8_attend(g, u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c2, q, out, lse)
    gk, _ = kvc.q8_load(g, 120)
    np.testing.assert_array_equal(gk.view(torch.int16).cpu().numpy().view(np.uint16), oq.load(c2, 120)[0])


def test_a_head_alone_gives_the_bits_it_has_in_a_batch():
    lens = [700, 33, 20000, 512]
    c = u.random_cache(20, 4, 2, 128, 16, lens, oq.E4M3)
    g = u.to_gpu(c)
    q = u.dev_bf16(u.random_rows(21, 8, 4, 2, 128))
    out, lse = kvc.q8_attend(g, q, want_lse=True)
    for b in range(4):
        tb = -(-lens[b] // 16)
        alone = kvc.Q8Cache(g.k_pool, g.v_pool, g.k_scale, g.v_scale,
                            g.table[b:b + 1, :tb].contiguous(), g.seq_len[b:b + 1].contiguous())
        o, l = kvc.q8_attend(alone, q[2 * b:2 * b + 2].contiguous(), want_lse=True)
        assert torch.equal(o.view(torch.int16), out[2 * b:2 * b + 2].view(torch.int16))
        assert torch.equal(l, lse[2 * b:2 * b + 2])


def test_untouched_rows_and_pages():
    """Rows past the length, pages of nobody and k/v rows >= T of a load stay."""
    c = u.random_cache(22, 2, 2, 64, 16, [20, 5], oq.INT8)
    g = u.to_gpu(c)
    out_k = torch.full((4, 30, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out_v = out_k.clone()
    kvc.q8_load(g, 24, k_out=out_k, v_out=out_v)
    assert bool((out_k[:, 24:] == 7.0).all()) and bool((out_v[:, 24:] == 7.0).all())
    u.same_cache(g, c)
    only_k, none = kvc.q8_load(g, 24, want_v=False)
    assert none is None and torch.equal(only_k.view(torch.int16), out_k[:, :24].contiguous().view(torch.int16))


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: the last pages hold the sequence."""
    H, bs, d = 8, 64, 128
    n = (1 << 32) // (H * bs * d) + 40                         # 4.3 GB of codes
    k = torch.zeros((n, H, bs, d), dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.ones((n, H), device="cuda")
    vs = torch.ones((n, H), device="cuda")
    table = torch.tensor([[n - 1, n - 7, n - 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    rows_k, rows_v = u.random_rows(23, H, 150, d), u.random_rows(24, H, 150, d)
    g = kvc.Q8Cache(k, v, ks, vs, table, lens)
    kvc.q8_store(g, u.dev_bf16(rows_k), u.dev_bf16(rows_v))
    ids = [n - 1, n - 7, n - 3]
    small = oq.Cache(np.zeros((3, H, bs, d), np.uint8), np.zeros((3, H, bs, d), np.uint8),
                     np.ones((3, H), np.float32), np.ones((3, H), np.float32), [[0, 1, 2]], [150], oq.INT8)
    oq.store(small, rows_k, rows_v, 150)
    np.testing.assert_array_equal(bits8_of(g.k_pool, ids), small.k)
    np.testing.assert_array_equal(bits8_of(g.v_pool, ids), small.v)
    q = u.random_rows(25, H, 4, 1, d)
    out, lse = kvc.q8_attend(g, u.dev_bf16(q), want_lse=True)
    u.check_attention(small, q, out, lse)
    new = u.random_rows(26, H, 1, d)
    lens += 1
    kvc.q8_append(g, u.dev_bf16(new), u.dev_bf16(new))
    small.lens = np.array([151])
    oq.append(small, new, new)
    np.testing.assert_array_equal(bits8_of(g.k_pool, ids), small.k)
    got, _ = kvc.q8_load(g, 151)
    np.testing.assert_array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), oq.load(small, 151)[0])


def bits8_of(pool, ids):
    return u.bits8(pool[torch.tensor(ids, device="cuda")].contiguous())
