"""Attention over pages whose value scales lie far apart, on the GPU against the
fp64 oracle: rows that see quiet pages only, and quiet values beside loud keys of
the same score."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import q8 as oq
import q8_utils as u

pytestmark = pytest.mark.gpu

FMTS = [oq.E4M3, oq.INT8]


def check(c, q_bits, out, lse, weight_floor, spread):
    """out and lse against the fp64 oracle.  Per output, each at its largest:
      a weight in fp16      2^-11 of itself; weight_floor of the largest weight * vs
                            for each of its codes, where fp16 is subnormal
      an exponent           the score: (d + 8) * 2^-23 of sum |q k|; log2 of the value
                            scale (at most `spread` below the piece's largest) and
                            the running maximum around it, four roundings of at
                            most 2^-24 of spread + 16
      the sums              both, twice (weight and denominator), exp2 at 2^-22 and
                            T terms at 2^-24
      bf16                  2^-8
    """
    q = u.widen(q_bits)
    ref, ref_lse, absdot, absout, tail = oq.attend(c, q)
    T = max(c.length(b) for b in range(c.B))
    x = absdot * (c.d + 8) * 2.0 ** -23 + (spread + 16) * 2.0 ** -22
    rel = 2.0 ** -11 + 2 * x + 2.0 ** -20 + T * 2.0 ** -24
    bound = (rel[..., None] * absout + weight_floor * tail[..., None]) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outputs off, worst {np.max(err / np.maximum(bound, 1e-300)):.3g} of the bound"
    lb = x + 2.0 ** -20 + T * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref_lse)
    diff = np.abs(lse.cpu().numpy().astype(np.float64) - ref_lse)
    assert np.all(diff <= lb), f"lse off by {np.max(diff / lb):.3g} of the bound"


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 7)])
@pytest.mark.parametrize("apart", [30, 60, 78])
def test_drafts_before_a_loud_page(apart, d, bs, fmt):
    """The first drafted queries see pages 2^-apart as loud as those of the later
    drafts, which they do not attend to: their outputs are as exact as alone."""
    B, H, G, L = 1, 2, 2, 4 * bs
    W = 2 * bs + 4                                      # queries 0..3 end in the quiet pages
    c = u.random_cache(60, B, H, d, bs, [L], fmt, poison=False)
    c.vs[c.table[0, :2]] *= np.float32(2.0 ** -apart)
    q = u.random_rows(61, B * H, G, W, d)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    check(c, q, out, lse, 2.0 ** -25, apart + 8)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("score", [37.0, 100.0])
def test_weight_on_quiet_pages_only(score, fmt):
    """Keys of quiet pages (2^-60) score so much higher that the loud ones count for
    as little as they do, or for nothing."""
    H, G, W, d, bs = 2, 3, 1, 64, 8
    c = u.random_cache(62, 1, H, d, bs, [5 * bs], fmt, poison=False)
    quiet = c.table[0, 1:3]
    c.k[...] = 0
    c.k[quiet, :, :, 0] = 0x38 if fmt == oq.E4M3 else 1  # the code of 1
    c.ks[...] = np.float32(score * 8.0)                 # scale 1/8
    c.vs[quiet] *= np.float32(2.0 ** -60)
    q = np.zeros((H, G, W, d), np.float32)
    q[..., 0] = 1.0
    bits = u.synth.f32_to_bf16_bits(q)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(bits), want_lse=True)
    torch.cuda.synchronize()
    check(c, bits, out, lse, 2.0 ** -25, 68)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("loud_score", [0.0, -40.0, -100.0])
def test_a_loud_key_among_many_quiet_ones(loud_score, fmt):
    """35000 keys in pieces of 512 or more, 2^-90 as loud as one page in forty: the
    quiet ones carry the denominator, and where the loud ones score far lower the
    values too."""
    H, G, W, d, bs, L = 1, 2, 2, 64, 16, 35008
    c = u.random_cache(63, 1, H, d, bs, [L], fmt, poison=False)
    c.k[...] = 0
    c.vs *= np.float32(2.0 ** -90)
    loud = c.table[0, ::40]
    c.k[loud, :, :, 0] = 0xB8 if fmt == oq.E4M3 else 0xFF  # the code of -1
    c.ks[...] = np.float32(-loud_score * 8.0)              # scale 1/8
    c.vs[loud] *= np.float32(2.0 ** 90)
    q = np.zeros((H, G, W, d), np.float32)
    q[..., 0] = 1.0
    bits = u.synth.f32_to_bf16_bits(q)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(bits), want_lse=True)
    torch.cuda.synchronize()
    check(c, bits, out, lse, 2.0 ** -25, 98)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("bs", [1, 12])
@pytest.mark.parametrize("apart", [16, 26, 30])
def test_quiet_values_beside_loud_keys_of_the_same_score(apart, bs, fmt):
    """Two pages of equal scores, one 2^-apart as loud as the other, whose codes are zero
    in every other dimension: there the outputs are the quiet page's values, with
    11 bits down to 2^-23 of the loud ones and within 2^-34 of those below."""
    H, G, W, d = 2, 2, 1, 64
    c = u.random_cache(64, 1, H, d, bs, [2 * bs], fmt, poison=False)
    loud, quiet = c.table[0]
    c.v[loud, :, :, ::2] = 0
    c.vs[quiet] = np.float32(1.37)
    c.vs[loud] = np.float32(1.11 * 2.0 ** apart)
    bits = np.zeros((H, G, W, d), np.uint16)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(bits), want_lse=True)
    torch.cuda.synchronize()
    check(c, bits, out, lse, 2.0 ** -34, apart + 1)
