"""CPU checks of what the optimizer step's C ABI refuses by its numbers (made-up
plans; nothing is launched)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def native():
    from lossless_bf16_weight_xor_amd import _native
    if not os.path.exists(_native.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return _native


def test_a_grad_scale_beyond_fp32_is_refused(native):
    """The step multiplies by the scale in fp32, whose largest number is 2^128 - 2^104;
    what rounds to more, from 2^128 - 2^103 on, is infinite there."""
    plan = native.StepPlan()
    plan.opaque[0] = int.from_bytes(b"F16DNORM", "little")
    for scale in (1e39, -1e39, 1e300, 2.0 ** 128 - 2.0 ** 103, 2.0 ** 103 - 2.0 ** 128):
        assert native.lib().bf16d_grad_norm(ctypes.byref(plan), 1.0, scale, None) == native.EINVAL
