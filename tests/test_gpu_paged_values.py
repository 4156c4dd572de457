"""Values of any finite size in the attention over bf16 pages and within prompts: a softmax's mean of
finite values is finite, however its scores climb."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc, synth
from oracle import paged as og
import paged_utils as u
from q8_utils import dev_bf16, random_rows, rng_of

pytestmark = pytest.mark.gpu

BIG = np.uint16(0x7F7F)     # the largest bf16


def loud(seed, shape, kind):
    """Values as bits: one column as large as bf16 holds, one of its negatives, one of both signs, the
    others of one size."""
    rng = rng_of(seed, *shape)
    x = rng.standard_normal(shape)
    x *= {"2^100": 2.0 ** 100, "2^126": 2.0 ** 124, "largest": 2.0 ** 124, "quiet": 2.0 ** -100}[kind]
    b = synth.f32_to_bf16_bits(x.astype(np.float32))
    if kind == "largest":
        b[..., 0], b[..., 1] = BIG, BIG | 0x8000
        b[..., 2] = np.where(rng.random(shape[:-1]) < 0.5, BIG, BIG | 0x8000)
    return b


def climbing(T, d, step):
    """Keys whose first value rises to `step` * T, and queries that read it: scores in nats, with scale 1."""
    k = np.zeros((T, d), np.float32)
    k[:, 0] = np.arange(T) * step
    k[:, 1] = np.sin(np.arange(T))
    return synth.f32_to_bf16_bits(k)


# (G, lens, new, bs): alone, in pieces, whole heads, more rows than 16, row tiles, pieces of them
CHUNKS = [
    (1, [1], [1], 16), (2, [300], [1], 16), (4, [2100], [1], 16), (4, [700], [6], 16), (1, [600], [3], 5),
    (4, [300], [60], 16), (2, [1500], [100], 24), (1, [1500], [70], 5), (2, [900, 40, 0, 700], [1, 40, 2, 90], 16),
]


@pytest.mark.parametrize("step", [0.0, 0.1, -0.1, 3.0])
@pytest.mark.parametrize("kind", ["2^100", "2^126", "largest", "quiet"])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_size_over_pages(d, kind, step):
    for i, (G, lens, new, bs) in enumerate(CHUNKS):
        print(f"[case] {i} d {d} {kind} {step}", flush=True)
        c = u.random_cache(90 + i, len(lens), 1, d, bs, lens, weights=i % 2 == 1)
        keys = climbing(max(lens), d, step)
        for b, L in enumerate(lens):
            for t in range(L):
                p, r = c.at(b, t)
                c.k[p, 0, r] = keys[t]
        c.v = np.where(c.v == u.NAN, c.v, loud(91 + i, c.v.shape, kind))
        starts = u.starts_of(new)
        q = random_rows(92 + i, int(starts[-1]), G, d)
        q[..., 0] = synth.f32_to_bf16_bits(np.float32([1.0]))[0]
        out, lse = kvc.paged_attend(u.to_gpu(c), dev_bf16(q), u.dev(starts), scale=1.0, want_lse=True)
        assert bool(torch.isfinite(out.float()).all())
        u.check_attention(og.attend(c, og.widen(q), starts, scale=1.0), u.bits(out), lse, max(lens))


@pytest.mark.parametrize("step", [0.0, 0.1, 3.0])
@pytest.mark.parametrize("kind", ["2^100", "2^126", "largest", "quiet"])
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_size_within_prompts(d, kind, step):
    lens, G = [300, 1, 129, 700], 2
    starts = u.starts_of(lens)
    n = int(starts[-1])
    k = np.concatenate([climbing(L, d, step) for L in lens])[:, None]
    v = loud(95, (n, 1, d), kind)
    q = random_rows(96, n, G, d)
    q[..., 0] = synth.f32_to_bf16_bits(np.float32([1.0]))[0]
    out, lse = kvc.prompt_attend(dev_bf16(q), dev_bf16(k), dev_bf16(v), u.dev(starts), scale=1.0, want_lse=True)
    assert bool(torch.isfinite(out.float()).all())
    u.check_attention(og.prompt(og.widen(q), og.widen(k), og.widen(v), starts, scale=1.0), u.bits(out), lse, max(lens))


def test_loud_heads_leave_the_others_their_bits():
    """Heads of one call with values of ordinary size get the bits that they get without loud ones beside them."""
    H, G, d, lens, new = 2, 4, 128, [1100, 900], [2, 70]
    c = u.random_cache(97, 2, H, d, 16, lens)
    starts = u.starts_of(new)
    q = dev_bf16(random_rows(98, int(starts[-1]), H * G, d))
    plain = kvc.paged_attend(u.to_gpu(c), q, u.dev(starts))
    c.v[:, 1] = np.where(c.v[:, 1] == u.NAN, c.v[:, 1], BIG)
    mixed = kvc.paged_attend(u.to_gpu(c), q, u.dev(starts))
    assert torch.equal(mixed[:, :G].contiguous().view(torch.int16), plain[:, :G].contiguous().view(torch.int16))
    # weights in bf16, off by 2^-8 of themselves, and the rounding of what they give
    big = float(og.widen(BIG))
    assert float(mixed[:, G:].double().min()) >= big * (1 - 2.0 ** -7) and float(mixed[:, G:].double().max()) <= big


def test_loud_workgroups_of_eight_waves_give_the_bits_of_four():
    """Long prompts and chunks (256 rows a workgroup) whose values are loud in one sequence, and for some keys only in the
    other, against each KV head alone (128 rows)."""
    d, H, G = 128, 8, 8
    lens = [2048, 37, 1100]
    starts = u.dev(u.starts_of(lens))
    n = sum(lens)
    bits = random_rows(100, n, (G + 2) * H, d)
    bits[:2048, (G + 1) * H:] = loud(101, (2048, H, d), "largest")
    bits[2900:2910, (G + 1) * H + 3] = loud(102, (10, d), "largest")
    rows = dev_bf16(bits)
    q, k, v = rows[:, : G * H], rows[:, G * H: (G + 1) * H], rows[:, (G + 1) * H:]
    out, lse = kvc.prompt_attend(q, k, v, starts, want_lse=True)
    assert bool(torch.isfinite(out.float()).all())
    for h in range(H):
        o, z = kvc.prompt_attend(q[:, h * G: (h + 1) * G], k[:, h: h + 1], v[:, h: h + 1], starts, want_lse=True)
        assert torch.equal(o.view(torch.int16), out[:, h * G: (h + 1) * G].contiguous().view(torch.int16))
        assert torch.equal(z, lse[:, h * G: (h + 1) * G])
    H, G = 4, 4
    c = u.random_cache(103, 2, H, d, 16, [8192, 7001])
    c.v[:, 1:3] = np.where(c.v[:, 1:3] == u.NAN, u.NAN, loud(104, c.v[:, 1:3].shape, "largest"))
    starts = u.dev(u.starts_of([512, 401]))
    q = dev_bf16(random_rows(105, 913, G * H, d))
    out, lse = kvc.paged_attend(u.to_gpu(c), q, starts, want_lse=True)
    assert bool(torch.isfinite(out.float()).all())
    for h in range(H):
        one = u.to_gpu(og.Cache(c.k[:, h: h + 1], c.v[:, h: h + 1], c.table, c.lens))
        o, z = kvc.paged_attend(one, q[:, h * G: (h + 1) * G], starts, want_lse=True)
        assert torch.equal(o.view(torch.int16), out[:, h * G: (h + 1) * G].contiguous().view(torch.int16))
        assert torch.equal(z, lse[:, h * G: (h + 1) * G])


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_loud_heads_taken_whole_give_the_bits_of_pieces(d, weights):
    """Enough heads that a workgroup takes one whole, loud ones among them, and each sequence alone."""
    B, H, G = 13, 8, 3
    lens = [1100, 1, 513, 0, 1024, 700, 1536, 20, 1100, 1100, 1300, 999, 512]
    c = u.random_cache(106, B, H, d, 16, lens, tb=96, weights=weights)
    v = loud(107, c.v.shape, "largest")
    v[:, ::3] = random_rows(108, *v[:, ::3].shape)
    c.v = np.where(c.v == u.NAN, c.v, v)
    starts = u.starts_of([2] * B)
    q = dev_bf16(random_rows(109, 2 * B, G * H, d))
    g = u.to_gpu(c)
    out, lse = kvc.paged_attend(g, q, u.dev(starts), max_new=2, want_lse=True)
    u.check_attention(og.attend(c, og.widen(u.bits(q)), starts), u.bits(out), lse, max(lens))
    for b in range(B):
        heads = slice(b * H, (b + 1) * H)
        one = kvc.PagedCache(g.k_pool, g.v_pool, g.table[b: b + 1], g.seq_len[b: b + 1],
                             weight=u.dev(c.weight[heads]) if weights else None, pos=u.dev(c.pos[heads]) if weights else None)
        o, z = kvc.paged_attend(one, q[2 * b: 2 * b + 2], u.dev(u.starts_of([2])), want_lse=True)
        assert torch.equal(o.view(torch.int16), out[2 * b: 2 * b + 2].view(torch.int16)) and torch.equal(z, lse[2 * b: 2 * b + 2])
        if weights:
            assert torch.equal(one.weight, g.weight[heads])


def test_loud_rows_go_by_their_own_wave():
    """One row a token: the first half of 256 rows sees fewer keys than the second, and its second pass does not go by these."""
    d, H, n = 128, 16, 8192
    starts = u.dev(u.starts_of([n]))
    bits = random_rows(110, n, 3 * H, d)
    bits[:, 2 * H:] = loud(111, (n, H, d), "largest")
    rows = dev_bf16(bits)
    q, k, v = rows[:, :H], rows[:, H: 2 * H], rows[:, 2 * H:]
    out, lse = kvc.prompt_attend(q, k, v, starts, want_lse=True)
    assert bool(torch.isfinite(out.float()).all())
    for h in range(0, H, 5):
        o, z = kvc.prompt_attend(q[:, h: h + 1], k[:, h: h + 1], v[:, h: h + 1], starts, want_lse=True)
        same = torch.equal(o.view(torch.int16), out[:, h: h + 1].contiguous().view(torch.int16))
        assert same and torch.equal(z, lse[:, h: h + 1])


@pytest.mark.parametrize("d", [64, 128])
def test_places_without_a_row_do_not_make_a_head_loud(d):
    """16 rows of a head, in a call of 16 rows a head and in one of 32: the places of the other 16 see all keys alike, and
    what their sums would be does not matter."""
    T, G = 1500, 16
    c = u.random_cache(112, 1, 1, d, 16, [T])
    v = np.abs(og.widen(random_rows(113, *c.v.shape)))
    c.v = np.where(c.v == u.NAN, c.v, synth.f32_to_bf16_bits((np.minimum(v, 1.9) * 2.0 ** 124).astype(np.float32)))
    # each wave's first keys hold one far above the others (pieces of 512, tiles of 32 keys): sums of rows stay finite
    rng = rng_of(114, d)
    k = rng.standard_normal((T, d)).astype(np.float32)
    q = rng.standard_normal((2, G, d)).astype(np.float32)
    q[..., 0] = 1.0
    t = np.arange(T)
    k[:, 0] = np.where((t % 512 < 128) & (t % 32 == 3), 100.0, 0.0)
    kb = synth.f32_to_bf16_bits(k)
    for t in range(T):
        p, r = c.at(0, t)
        c.k[p, 0, r] = kb[t]
    g = u.to_gpu(c)
    gq = dev_bf16(synth.f32_to_bf16_bits(q))
    one, z1 = kvc.paged_attend(g, gq[:1].contiguous(), u.dev(u.starts_of([1])), max_new=1, scale=1.0, want_lse=True)
    two, z2 = kvc.paged_attend(g, gq, u.dev(np.int32([0, 1])), max_new=2, scale=1.0, want_lse=True)
    assert bool(torch.isfinite(one.float()).all())
    same = torch.equal(one.view(torch.int16), two[:1].view(torch.int16)) and torch.equal(z1, z2[:1])
    assert same
