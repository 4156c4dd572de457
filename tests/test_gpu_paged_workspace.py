"""Workspaces of the bf16 paged cache: calls write nothing past what they ask for, and what an earlier call left
there does not matter."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
import paged_utils as u
from q8_utils import dev_bf16, random_rows, rng_of

pytestmark = pytest.mark.gpu


def _ws(need, fill):
    """need bytes of `fill`, and 64 KB behind them that stay as they are."""
    buf = torch.full((need + (1 << 16),), fill, dtype=torch.uint8, device="cuda")
    return buf, buf[:need]


# (B, H, G, d, bs, longest, shortest, most new, max_len)
CASES = [
    (5, 2, 4, 128, 16, 2100, 0, 60, 0), (9, 3, 7, 64, 24, 1500, 1, 1, 0), (3, 2, 16, 64, 5, 700, 0, 9, 600),
    (40, 1, 1, 128, 16, 513, 0, 40, 0), (2, 1, 33, 128, 64, 5000, 4000, 3, 0), (1, 4, 2, 64, 16, 3000, 3000, 900, 0),
    (64, 2, 4, 64, 16, 1024, 900, 12, 0), (7, 2, 3, 128, 256, 70000, 10, 30, 0), (100, 3, 1, 64, 16, 1100, 0, 33, 1100),
    (3, 1, 64, 128, 16, 33000, 1, 2, 0),
]


@pytest.mark.parametrize("weights", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_nothing_past_the_end(case, weights):
    B, H, G, d, bs, hi, lo, most, cap = case
    print(f"[case] {case} {weights}", flush=True)
    rng = rng_of(120, *case)
    lens = rng.integers(lo, hi + 1, B)
    lens[rng.integers(0, B)] = hi
    tb = -(-hi // bs) + 3
    n_blocks = B * tb + 3
    table = torch.from_numpy(rng.permutation(n_blocks)[: B * tb].reshape(B, tb).astype(np.int32)).cuda()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(121)
    pools = [torch.randn((n_blocks, H, bs, d), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    weight = torch.rand((B * H, tb * bs), generator=gen, device="cuda") if weights else None
    pos = torch.arange(tb * bs, dtype=torch.int32, device="cuda").repeat(B * H, 1) if weights else None
    seq = u.dev(lens.astype(np.int32))
    for most_now in (1, most):
        new = rng.integers(0, most_now + 1, B)
        new[0] = most_now
        q = dev_bf16(random_rows(122, int(new.sum()) + 2, G * H, d))
        starts = u.dev(u.starts_of(new))
        got = []
        for fill in (0, 0xff, 0x7f):               # bytes of zeros, NaN and large numbers
            w = weight.clone() if weights else None
            c = kvc.PagedCache(pools[0], pools[1], table, seq, weight=w, pos=pos, max_len=cap)
            buf, ws = _ws(c.attend_workspace_bytes(G, q.shape[0], most_now), fill)
            out = torch.zeros_like(q)
            _, lse = kvc.paged_attend(c, q, starts, max_new=most_now, out=out, want_lse=True, ws=ws if ws.numel() else None)
            torch.cuda.synchronize()
            assert bool((buf[ws.numel():] == fill).all())
            n = int(starts[-1])
            got.append((out.view(torch.int16), lse[:n]) + ((w,) if weights else ()))
        for other in got[1:]:
            for a, b in zip(got[0], other):
                assert torch.equal(a, b)
    if not weights:
        return
    for budget in (1, hi // 2, hi - 1, hi + 5):
        got = []
        for fill in (0, 0xff, 0x7f):
            k, v, w, p, s = (x.clone() for x in (pools[0], pools[1], weight, pos, seq))
            c = kvc.PagedCache(k, v, table, s, weight=w, pos=p, max_len=cap)
            buf, ws = _ws(c.evict_workspace_bytes(max(1, budget)), fill)
            kvc.paged_evict(c, seq, max(1, budget), sinks=2, recent=9, ws=ws)
            torch.cuda.synchronize()
            assert bool((buf[ws.numel():] == fill).all())
            got.append((k.view(torch.int16), v.view(torch.int16), w, p, s))
        for other in got[1:]:
            for a, b in zip(got[0], other):
                assert torch.equal(a, b)
