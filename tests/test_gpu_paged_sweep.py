"""Seeded random caches, chunks, prompts and evictions of the bf16 paged cache against the oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import paged as og
import paged_utils as u
from q8_utils import dev_bf16, random_rows

pytestmark = pytest.mark.gpu

WORK = 1_500_000                                       # rows times slots of a case at most, for the oracle


def _shape(rng):
    d, G, H = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3, 4, 7, 8, 16, 33, 64])), int(rng.integers(1, 7))
    B, hi, most = int(rng.choice([1, 2, 3, 5, 9, 20, 40])), int(np.exp(rng.uniform(0, np.log(2500)))), int(rng.choice([1, 1, 2, 4, 9, 40, 130]))
    while B * H * G * most * hi > WORK and max(B, most, G) > 1:
        if B == max(B, most, G):
            B //= 2
        elif most >= G:
            most //= 2
        else:
            G //= 2
    return d, G, H, B, hi, most


def _attend(rng, seed):
    d, G, H, B, hi, most = _shape(rng)
    bs = int(rng.choice([1, 3, 4, 5, 8, 16, 24, 64, 100, 256]))
    lens, new = rng.integers(0, hi + 1, B), rng.integers(0, most + 1, B)
    new[0] = max(1, new[0])
    weights, holes = bool(rng.integers(0, 2)), float(rng.choice([0, 0, 0.2]))
    cap = int(rng.choice([0, 0, max(1, hi // 2)]))
    print(f"[case {seed}] attend d {d} G {G} H {H} B {B} bs {bs} hi {hi} most {most} {weights} {holes} {cap}", flush=True)
    c = u.random_cache(seed, B, H, d, bs, lens, holes=holes, weights=weights, max_len=cap)
    starts = u.starts_of(new)
    n = int(starts[-1]) + int(rng.integers(0, 4))
    qkv = random_rows(seed + 1, n, (G + 2) * H, d)
    dq, at = dev_bf16(qkv), rng.integers(0, 1 << 20, n).astype(np.int32)
    g = u.to_gpu(c, max_len=cap)
    kvc.paged_append(g, dq[:, G * H: (G + 1) * H], dq[:, (G + 1) * H:], u.dev(starts), positions=u.dev(at))
    og.append(c, qkv[:, G * H: (G + 1) * H], qkv[:, (G + 1) * H:], starts, at)
    u.same_cache(g, c)
    out = torch.full((n, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = kvc.paged_attend(g, dq[:, : G * H], u.dev(starts), max_new=int(rng.choice([0, most])), out=out, want_lse=True)
    torch.cuda.synchronize()
    ref = og.attend(c, og.widen(qkv[:, : G * H]), starts)
    u.check_attention(ref, u.bits(out), lse, hi, untouched=0x40E0)
    if not weights:
        return u.same_cache(g, c)
    u.check_weights(ref, c.weight, g.weight.cpu().numpy(), d, G * int(new.max()))
    # an eviction of slots at other positions, distinct and in no order; some weights alike
    room = c.pos.shape[1]
    for r in range(B * H):
        c.pos[r] = rng.permutation(2 * room)[:room]
    c.weight[:] = g.weight.cpu().numpy()
    if rng.integers(0, 2):
        c.weight[:] = np.round(c.weight * 3)
    g = u.to_gpu(c, max_len=cap)
    budget, seen = int(rng.integers(1, hi + 1)), np.full(B, int(rng.choice([hi, 2 * hi])), np.int32)
    sinks, recent = int(rng.choice([0, 4])), int(rng.choice([0, 1, 64]))
    kvc.paged_evict(g, u.dev(seen), budget, sinks=sinks, recent=recent)
    og.evict(c, seen, budget, sinks, recent)
    u.same_cache(g, c)


def _prompt(rng, seed):
    d, G, H, B, hi, _ = _shape(rng)
    lens = rng.integers(0, max(1, min(hi, int((2 * WORK / (B * H * G)) ** 0.5) // 2)) + 1, B)
    pad = int(rng.integers(0, 4))
    n = max(1, int(lens.sum()) + pad)
    print(f"[case {seed}] prompt d {d} G {G} H {H} lens {lens.tolist()} n {n}", flush=True)
    starts = u.starts_of(lens)
    qkv = random_rows(seed, n, (G + 2) * H, d)
    qkv[int(starts[-1]):] = u.NAN
    dq = dev_bf16(qkv)
    out = torch.full((n, G * H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    _, lse = kvc.prompt_attend(dq[:, : G * H], dq[:, G * H: (G + 1) * H], dq[:, (G + 1) * H:], u.dev(starts), out=out, want_lse=True)
    w = og.widen(qkv)
    ref = og.prompt(w[:, : G * H], w[:, G * H: (G + 1) * H], w[:, (G + 1) * H:], starts)
    u.check_attention(ref, u.bits(out), lse, max(1, int(lens.max())), untouched=0x40E0)


@pytest.mark.parametrize("group", range(12))
def test_random_cases(group):
    for i in range(20):
        seed = 5000 + 20 * group + i
        rng = np.random.default_rng(seed)
        (_prompt if i % 5 == 4 else _attend)(rng, seed)
