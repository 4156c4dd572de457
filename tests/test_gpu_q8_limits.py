"""The 8-bit paged cache at sizes that take several launches, or offsets past 32
bits: a few heads of each against the oracle or against a small call."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import q8 as oq
import q8_utils as u

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_attention_over_tables_of_2_to_30_positions():
    """17 heads in tables with room for 2^30 positions each: the pieces of 16 heads
    fill a launch.  Same bits as with tables as long as the sequences."""
    B, bs, d, tb = 17, 4096, 64, 1 << 18
    lens = [1, 5, 100, 512, 513, 4096, 4097, 9000] + [300 + 40 * i for i in range(9)]
    small = u.random_cache(1, B, 1, d, bs, lens, oq.INT8, poison=False)
    g = u.to_gpu(small)
    table = torch.full((B, tb), -1, dtype=torch.int32, device="cuda")
    table[:, : small.table.shape[1]] = g.table
    wide = kvc.Q8Cache(g.k_pool, g.v_pool, g.k_scale, g.v_scale, table, g.seq_len)
    q = u.dev_bf16(u.random_rows(2, B, 1, 1, d))
    out, lse = kvc.q8_attend(wide, q, want_lse=True)
    ref, ref_lse = kvc.q8_attend(g, q, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16)) and torch.equal(lse, ref_lse)
    bounded = kvc.Q8Cache(g.k_pool, g.v_pool, g.k_scale, g.v_scale, table, g.seq_len, max_len=9000)
    assert bounded.attend_workspace_bytes(1) < wide.attend_workspace_bytes(1)
    out = kvc.q8_attend(bounded, q)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    u.check_attention(small, u.random_rows(2, B, 1, 1, d), ref, ref_lse)


def test_attention_of_the_most_rows_on_many_heads():
    """4096 query rows on 2100 heads: the pieces are joined in two launches.  The
    last heads have the bits they have alone."""
    B, H, G, W, d, bs, L = 300, 7, 64, 64, 64, 64, 700
    n = 40
    k = torch.randint(-127, 128, (n, H, bs, d), dtype=torch.int8, device="cuda")
    v = torch.randint(-127, 128, (n, H, bs, d), dtype=torch.int8, device="cuda")
    ks, vs = torch.rand((n, H), device="cuda") * 0.01, torch.rand((n, H), device="cuda")
    table = torch.randint(0, n, (B, -(-L // bs)), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    q = torch.randn((B * H, G, W, d), device="cuda", dtype=torch.bfloat16)
    c = kvc.Q8Cache(k, v, ks, vs, table, lens)
    out, lse = kvc.q8_attend(c, q, want_lse=True)
    for b in (0, 292, B - 1):                              # head 2048 is sequence 292's
        one = kvc.Q8Cache(k, v, ks, vs, table[b:b + 1].contiguous(), lens[:1].contiguous())
        o, s = kvc.q8_attend(one, q[b * H:(b + 1) * H].contiguous(), want_lse=True)
        assert torch.equal(o.view(torch.int16), out[b * H:(b + 1) * H].view(torch.int16))
        assert torch.equal(s, lse[b * H:(b + 1) * H])


@pytest.mark.parametrize("fmt", [oq.E4M3, oq.INT8])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_out_of_large_pools(fmt, d):
    """Keys out of pools of over 100 MB, read past the caches: the bits of the same
    call on pools that hold no other page, with dead pages and empty sequences."""
    B, H, G, W, bs = 5, 2, 4, 3, 16
    small = u.random_cache(3, B, H, d, bs, [0, 1, 77, 1100, 4097], fmt, holes=0.05, poison=True)
    g = u.to_gpu(small)
    held = g.k_pool.shape[0]
    n = -(-(101 << 20) // (2 * H * bs * d))
    at = torch.randperm(n, generator=torch.Generator().manual_seed(4))[:held].cuda()

    def spread(x):
        as_int = torch.int8 if x.element_size() == 1 else torch.int32
        y = torch.zeros((n, *x.shape[1:]), dtype=as_int, device="cuda")
        y[at] = x.view(as_int)
        return y.view(x.dtype)

    good = (g.table >= 0) & (g.table < held)
    table = torch.where(good, at[g.table.clamp(0, held - 1).long()].int(), torch.full_like(g.table, -1))
    big = kvc.Q8Cache(spread(g.k_pool), spread(g.v_pool), spread(g.k_scale), spread(g.v_scale), table, g.seq_len)
    bits = u.random_rows(5, B * H, G, W, d)
    q = u.dev_bf16(bits)
    out, lse = kvc.q8_attend(big, q, want_lse=True)
    ref, ref_lse = kvc.q8_attend(g, q, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16)) and torch.equal(lse, ref_lse)
    u.check_attention(small, bits, out, lse)


def test_store_in_two_launches():
    """33.6 million pages of one row: past 2^25 pages of K and V a second launch."""
    B, d, T = 260, 64, 65536
    n = B * T
    assert 2 * n > 1 << 25
    k = torch.randn((B, T, d), device="cuda", dtype=torch.bfloat16)
    v = torch.randn((B, T, d), device="cuda", dtype=torch.bfloat16)
    pool = lambda: torch.zeros((n, 1, 1, d), dtype=torch.float8_e4m3fn, device="cuda")
    c = kvc.Q8Cache(pool(), pool(), torch.zeros((n, 1), device="cuda"), torch.zeros((n, 1), device="cuda"),
                    torch.arange(n, dtype=torch.int32, device="cuda").reshape(B, T), _i32([T] * B))
    kvc.q8_store(c, k, v)
    torch.cuda.synchronize()
    for b in (0, 128, B - 1):
        for rows, codes, scale in ((k, c.k_pool, c.k_scale), (v, c.v_pool, c.v_scale)):
            at = torch.tensor([0, 1, T // 2, T - 1])
            x = rows[b, at].float().cpu().numpy()
            got = u.bits8(codes[b * T + at, 0, 0].contiguous())
            for i in range(4):
                s, inv = oq.page_scale(np.abs(x[i]).max(), oq.E4M3)
                assert float(scale[b * T + int(at[i]), 0]) == float(s)
                np.testing.assert_array_equal(got[i], oq.encode(x[i] * inv, oq.E4M3))
    back, _ = kvc.q8_load(c, 4, want_v=False)
    assert back.shape == (B, 4, d) and bool(torch.isfinite(back).all())


def test_page_copies_past_32_bits():
    """Pages of 16 MiB in a buffer of 5.4 GB, odd bytes beside it."""
    n, size = 320, 16 << 20
    big = torch.zeros((n, size), dtype=torch.uint8, device="cuda")
    odd = torch.zeros((n, 7), dtype=torch.uint8, device="cuda")
    for p in (317, 319):
        big[p] = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
        odd[p] = p % 256
    kvc.pages_copy(_i32([319, 317]), _i32([2, 300]), kvc.PageBuffers([big, odd]))
    torch.cuda.synchronize()
    assert torch.equal(big[2], big[319]) and torch.equal(big[300], big[317])
    assert torch.equal(odd[2], odd[319]) and torch.equal(odd[300], odd[317])
    assert int(big[:2].max()) == 0 and int(big[3:300].max()) == 0 and int(big[301:317].max()) == 0


@pytest.mark.parametrize("n", [(1 << 32) + 4, 1 << 31, -(1 << 32) + 4, 4.5])
def test_integers_that_c_would_wrap_are_refused(n):
    """2^32 + 4 rows are not 4 of them."""
    c = u.to_gpu(u.random_cache(6, 1, 1, 64, 16, [16], oq.INT8, poison=False))
    before = u.bits8(c.k_pool).copy()
    rows = torch.zeros((1, 16, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="T"):
        kvc.q8_store(c, rows, rows, T=n)
    with pytest.raises(ValueError, match="T"):
        kvc.q8_load(c, n, k_out=rows, want_v=False)
    for group, window in ((n, 1), (1, n)):
        with pytest.raises(ValueError, match="group|window"):
            c.attend_workspace_bytes(group, window)
    pages = kvc.PageTable(c.table, c.seq_len, _i32([1] * 8), 16)
    with pytest.raises(ValueError, match="n_pairs"):
        pages.workspace_bytes(n)
    np.testing.assert_array_equal(u.bits8(c.k_pool), before)


@pytest.mark.parametrize("scale", [1e-50, -1e-50, 2.0 ** -150])
def test_scales_that_fp32_takes_for_zero_are_refused(scale):
    """0 stands for 1 / sqrt(d); a scale that vanishes in fp32 does not."""
    c = u.to_gpu(u.random_cache(7, 1, 1, 64, 16, [16], oq.INT8, poison=False))
    q = u.dev_bf16(u.random_rows(8, 1, 2, 1, 64))
    with pytest.raises(ValueError, match="scale"):
        kvc.q8_attend(c, q, scale=scale)
    out = kvc.q8_attend(c, q, scale=2.0 ** -149)               # the smallest: every key weighs the same
    v = kvc.q8_load(c, 16)[1].float().mean(1)
    torch.testing.assert_close(out[0, :, 0].float(), v.expand(2, -1), rtol=2.0 ** -7, atol=2.0 ** -7)
