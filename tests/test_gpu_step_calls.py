"""Calls of the optimizer step and the gradient norm on the GPU that go beside their
plain use: numbers at the border of fp32, a norm without a result, copies in
place, errors and steps left out around them."""
import math

import numpy as np
import pytest
import torch

from lossless_bf16_weight_xor_amd import AdamWBatch, GradNormBatch
from tests import step_reference as ref
from tests.gpu_util import log
from tests.test_gpu_step import DEV, Model

pytestmark = pytest.mark.gpu


def _same(a, b):
    return all(np.array_equal(x, y) for x, y in zip(a, b))


def test_grad_scale_up_to_the_largest_fp32_number():
    log("grad_scale at fp32's border")
    largest = 2.0 ** 128 - 2.0 ** 104
    border = 2.0 ** 128 - 2.0 ** 103      # what rounds to infinity
    grads = [torch.tensor([2.0 ** -130, -2.0 ** -140, 0.0], device=DEV)]
    norm = GradNormBatch(grads)
    for bad in (border, -border, 1e39, -1e300):
        with pytest.raises(ValueError, match="grad_scale"):
            norm.run(math.inf, bad)
    for good in (largest, -largest, math.nextafter(border, 0.0)):
        norm.run(math.inf, good)
        assert norm.scale.item() == math.copysign(largest, good)
        assert norm.nonfinite.item() == 0
        want = abs(good) * math.hypot(2.0 ** -130, 2.0 ** -140)
        assert norm.norm.item() == pytest.approx(want, rel=1e-14)
