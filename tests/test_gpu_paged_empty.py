"""Calls of the bf16 paged cache without tokens, whatever strides their empty tensors have."""
import numpy as np
import pytest
import torch

from eviction_window_qk_amd import kvc
import paged_utils as u

pytestmark = pytest.mark.gpu


def _empty(heads, d, strides):
    return torch.empty(0, dtype=torch.bfloat16, device="cuda").as_strided((0, heads, d), strides)


@pytest.mark.parametrize("strides", [(256, 64, 1), (0, 0, 0), (2, 2, 2)])
def test_no_tokens(strides):
    c = u.random_cache(1, 2, 1, 64, 16, [20, 3], weights=True)
    g = u.to_gpu(c)
    q, k = _empty(4, 64, strides), _empty(1, 64, strides)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    at = torch.zeros(0, dtype=torch.int32, device="cuda")
    plan = kvc.Rope(u.dev(10000.0 ** (-2.0 * np.arange(32) / 64)))
    assert kvc.rope(plan, q, at).shape == (0, 4, 64)
    assert kvc.paged_append(g, k, k, none, positions=at, rope=plan, q=q).shape == (0, 4, 64)
    out, lse = kvc.paged_attend(g, q, none, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = kvc.prompt_attend(q, k, k, none, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    u.same_cache(g, c)
