"""A prompt, the same tokens as one chunk over pages, and as chunks of several sizes: every element and
every logarithm within its own bound of the oracle's, and so of each other."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
from oracle import paged as og
import paged_utils as u
from q8_utils import dev_bf16, random_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,H,G,n", [(128, 2, 4, 333), (64, 2, 4, 333), (128, 1, 1, 160)])
def test_prompts_and_chunks_against_the_same_oracle(d, H, G, n):
    Hq = H * G
    qkv = random_rows(41, n, Hq + 2 * H, d)
    dq = dev_bf16(qkv)
    q, k, v = dq[:, :Hq], dq[:, Hq: Hq + H], dq[:, Hq + H:]
    w = og.widen(qkv)
    ref = og.prompt(w[:, :Hq], w[:, Hq: Hq + H], w[:, Hq + H:], [0, n])
    starts = u.dev(u.starts_of([n]))
    out, lse = kvc.prompt_attend(q, k, v, starts, want_lse=True)
    u.check_attention(ref, u.bits(out), lse, n)
    g = u.to_gpu(u.random_cache(42, 1, H, d, 16, [n]))
    kvc.paged_append(g, k, v, starts)
    out, lse = kvc.paged_attend(g, q, starts, want_lse=True)
    u.check_attention(ref, u.bits(out), lse, n)
    # one after the other, as a long prompt comes: 100 tokens, then 1, 5 (few rows), 40, the rest
    g = u.to_gpu(u.random_cache(43, 1, H, d, 16, [n]))
    outs, logs, at = [], [], 0
    for m in (100, 1, 5, 40, n - 146):
        g.seq_len.fill_(at + m)
        part = slice(at, at + m)
        st = u.dev(u.starts_of([m]))
        kvc.paged_append(g, k[part], v[part], st)
        o, z = kvc.paged_attend(g, q[part], st, want_lse=True)
        outs.append(o)
        logs.append(z)
        at += m
    assert at == n
    u.check_attention(ref, u.bits(torch.cat(outs)), torch.cat(logs), n)
