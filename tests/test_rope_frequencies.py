"""Frequencies of kvc.rope_frequencies where few positions were trained."""
import math

import pytest
import torch

from eviction_window_qk_amd import kvc


@pytest.mark.parametrize("scaling", ["banded", "yarn"])
@pytest.mark.parametrize("trained,slow,fast", [(1, 1, 32), (4, 1, 32), (500, 100, 200)])
def test_pairs_that_all_turn_too_seldom_are_all_divided(scaling, trained, slow, fast):
    plain = kvc.rope_frequencies(64)[0]
    assert (trained * plain / (2 * math.pi) < slow).all()
    f, _ = kvc.rope_frequencies(64, scaling=scaling, factor=8.0, trained=trained, slow=slow, fast=fast)
    assert torch.allclose(f, plain / 8, rtol=1e-15, atol=0)


@pytest.mark.parametrize("scaling", ["banded", "yarn"])
def test_pairs_that_all_turn_often_keep_their_frequency(scaling):
    plain = kvc.rope_frequencies(64, base=2.0)[0]
    f, _ = kvc.rope_frequencies(64, base=2.0, scaling=scaling, factor=8.0, trained=100000, slow=1, fast=32)
    assert torch.equal(f, plain)
