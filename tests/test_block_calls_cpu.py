"""Limits of the state space block's C calls, without a GPU (refusals come before any HIP call)."""
import os

import pytest

import gated_delta_rule_gdn2_amd as gdn2
from tests.test_abi_cpu import BF16, ERR_MISALIGNED, ERR_SHAPE, Fake


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn2.library_path()):
        pytest.skip("libgdn2.so not built")
    return gdn2._load()


def test_steps_take_any_stride_that_fits_32_bits(lib):
    """The last tokens of N long prompts lie a prompt apart.  (A state that is refused for its
    alignment alone: the strides have passed.)"""
    f = Fake()
    ssm = [f.p(i) for i in range(7)] + [f.p(7, 8), f.p(8)]
    scan = lambda xs, ts, bs, cs: lib.gdn2_ssm_step(*ssm, 3, 2, 1, 64, 64, xs, ts, bs, cs, BF16, 1, None)
    conv = lambda xs: lib.gdn2_short_conv_step(f.p(0), f.p(1), f.p(2), f.p(5, 8), f.p(4), 3, 64, xs, BF16, None)
    for far in (1 << 22, (1 << 31) - 8):
        assert scan(far, far, far, far) == ERR_MISALIGNED
        assert conv(far) == ERR_MISALIGNED
    far = 1 << 31
    for strides in ((far, 2, 64, 64), (128, far, 64, 64), (128, 2, far, 64), (128, 2, 64, far), (120, 2, 64, 64)):
        assert scan(*strides) == ERR_SHAPE, strides
    assert conv(far) == ERR_SHAPE and conv(56) == ERR_SHAPE
