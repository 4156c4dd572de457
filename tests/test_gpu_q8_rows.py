"""The 8-bit attention's row counts past 112 (many query rows a KV head), scores
that climb at every key, and repeated calls, on the GPU."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import q8 as oq
import q8_utils as u

pytestmark = pytest.mark.gpu

FMTS = [oq.E4M3, oq.INT8]


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("bs", [16, 7])
@pytest.mark.parametrize("G,W,d", [(13, 5, 64), (10, 7, 64), (8, 10, 64),       # five blocks of 16 rows
                                   (43, 3, 128), (20, 7, 128), (16, 9, 128),    # nine
                                   (32, 5, 128), (40, 4, 64), (16, 32, 128), (64, 8, 64)])
def test_many_query_rows(G, W, d, bs, fmt):
    """65 to 512 rows: odd and even counts of 16-row blocks, the last one partly or
    wholly empty, pages that are a multiple of four rows and not, holes, a sequence
    shorter than the window."""
    print(f"[case] rows {G}x{W} d {d} bs {bs} {u.NAMES[fmt]}", flush=True)
    c = u.random_cache(70, 2, 1, d, bs, [900, 33], fmt, holes=0.1)
    q = u.random_rows(71, 2, G, W, d)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("d,bs", [(64, 64), (128, 24), (128, 5)])
def test_the_most_query_rows(d, bs, fmt):
    """4096 rows, every one of them against the oracle."""
    c = u.random_cache(72, 1, 1, d, bs, [700], fmt)
    q = u.random_rows(73, 1, 64, 64, d)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(q), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("step", [0.25, 1.0, -1.0, 5.0])
def test_scores_that_climb_at_every_key(step, fmt):
    """Pages of one row, each with its own key scale: key t scores step * t (or
    step * (L - 1 - t) downwards), so the running maximum moves inside every tile."""
    H, G, W, d, L = 1, 3, 2, 64, 300
    c = u.random_cache(74, 1, H, d, 1, [L], fmt, poison=False)
    c.k[...] = 0
    c.k[..., 0] = 0x38 if fmt == oq.E4M3 else 1         # the code of 1
    at = np.arange(L) if step > 0 else np.arange(L)[::-1]
    c.ks[c.table[0], 0] = (at * abs(step) * 8.0).astype(np.float32)   # scale 1/8
    q = np.zeros((H, G, W, d), np.float32)
    q[..., 0] = 1.0
    bits = u.synth.f32_to_bf16_bits(q)
    out, lse = kvc.q8_attend(u.to_gpu(c), u.dev_bf16(bits), want_lse=True)
    torch.cuda.synchronize()
    u.check_attention(c, bits, out, lse)


@pytest.mark.parametrize("fmt", FMTS, ids=["e4m3", "int8"])
@pytest.mark.parametrize("B,H,G,W,d,bs,lens", [
    (1, 1, 1, 1, 64, 16, [128]), (3, 4, 7, 1, 128, 16, [1090, 800, 1400]),
    (1, 8, 4, 1, 128, 16, [40000]), (4, 3, 5, 4, 64, 32, [0, 16384, 3000, 77]), (1, 2, 64, 20, 128, 9, [2500])])
def test_repeated_calls_repeat_their_bits(B, H, G, W, d, bs, lens, fmt):
    """The same call again, with outputs and workspace that hold NaN before: the same
    bits every time."""
    c = u.to_gpu(u.random_cache(75, B, H, d, bs, lens, fmt, holes=0.05))
    q = u.dev_bf16(u.random_rows(76, B * H, G, W, d))
    first = kvc.q8_attend(c, q, want_lse=True)
    for _ in range(4):
        ws = torch.full((c.attend_workspace_bytes(G, W),), 0xFF, dtype=torch.uint8, device="cuda")
        out, lse = torch.full_like(q, float("nan")), torch.full_like(first[1], float("nan"))
        kvc.q8_attend(c, q, out=out, lse=lse, ws=ws if ws.numel() else None)
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), first[1].view(torch.int32))
