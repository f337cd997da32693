"""Every variant of the 8-bit layer's kernels has sizes in the GPU tests that
reach it: a rule or a threshold that moves shows here. Host only."""

import math
import random

import pytest

import bit_w4a4_quantized_nvfp4_b200 as svdq
from bit_w4a4_quantized_nvfp4_b200 import build as svdq_build
from tests import _fp8_plans as plans


@pytest.fixture(scope="module", autouse=True)
def _lib():
    svdq_build.build()
    svdq.load()


def test_the_sizes_take_their_variants():
    for want, shapes in plans.LINEAR.items():
        for M, K, N in shapes:
            assert svdq.probe_fp8_linear_plan(M, K, N, plans.SMS) == want, (M, K, N)
    for (norm, residual, *want), shapes in plans.ACT.items():
        for M, K in shapes:
            assert svdq.probe_fp8_act_plan(M, K, norm, residual, plans.SMS) == tuple(want), (M, K, norm, residual)


def test_no_other_variant_is_reached():
    rng = random.Random(3)

    def log(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    for _ in range(60000):
        M, K, N = log(1, rng.choice([32, 3000, 100000])), 16 * log(1, 4000), 8 * log(1, 8000)
        assert svdq.probe_fp8_linear_plan(M, K, N, plans.SMS) in plans.LINEAR, (M, K, N)
        K = 16 * log(1, 2048)
        for norm, residual in ((0, 0), (1, 0), (1, 1)):
            assert (norm, residual, *svdq.probe_fp8_act_plan(M, K, norm, residual, plans.SMS)) in plans.ACT, (M, K)


def test_what_the_plans_refuse():
    for args in ((0, 16, 8, 148), (1, 0, 8, 148), (1, 16, 0, 148), (1, 16, 8, 1), (1, 24, 8, 148), (1, 16, 12, 148),
                 (1, 2 ** 31 - 16, 8, 148)):
        with pytest.raises(svdq.SvdqError):
            svdq.probe_fp8_linear_plan(*args)
    for args in ((0, 16, 1, 0, 148), (1, 24, 1, 0, 148), (1, 32784, 1, 0, 148), (1, 16, 0, 1, 148), (1, 16, 0, 0, 0)):
        with pytest.raises(svdq.SvdqError):
            svdq.probe_fp8_act_plan(*args)
