"""yarn's ramp where even the fastest pair does not turn once."""

import math

import pytest
import torch

import bit_w4a4_quantized_nvfp4_b200 as svdq


def test_pairs_that_turn_less_than_once_slow_by_the_factor():
    """However short the trained context: whole turns come at 2 pi positions."""
    for original in (1, 3, 6, 7, 20, 100, 1000):
        plain = svdq.rope_freqs(64, device="cpu").freq
        yarn = svdq.rope_freqs(64, scaling="yarn", factor=4.0, original_len=original, device="cpu").freq
        slow = plain * original / (2 * math.pi) < 1.0
        # (the ramp ends at the next whole pair index)
        first = int(math.ceil(64 * math.log(original / (2 * math.pi)) / (2 * math.log(10000.0))))
        for i in range(32):
            if slow[i] and i >= first:
                assert math.isclose(float(plain[i] / yarn[i]), 4.0, rel_tol=1e-12), (original, i)
        assert (plain / yarn >= 1.0 - 1e-12).all() and (plain / yarn <= 4.0 + 1e-12).all()
        assert (torch.diff(plain / yarn) >= -1e-12).all()
