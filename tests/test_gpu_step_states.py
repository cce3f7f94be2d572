"""The 8-bit states of the optimizer step on the GPU: every code under every scale
byte, and how much noise their rounding leaves beside 32-bit states."""
import math

import numpy as np
import pytest
import torch

from lossless_bf16_weight_xor_amd import AdamWBatch
from tests import step_reference as ref
from tests.gpu_util import log
from tests.test_gpu_step import DEV, Model, _gen, _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("moment", [0, 1], ids=["m", "v"])
def test_every_code_under_every_scale_byte(moment):
    """All codes, the signed ones in m alone, under the bytes 0 to 254, as far as fp32
    holds their values (from 2^-136, a denormal number, up): without a gradient
    and with betas of 1/2, a step halves them, moves weights that were 0 by them, and
    codes them anew."""
    log(f"every code and byte, moment {moment}")
    byte = np.arange(255)
    code = np.tile(np.arange(256), 255).astype(np.uint8)
    if moment == 1:
        code &= 0x7F
    value = ref.E4M3[code] * 2.0 ** (byte.repeat(256) - 127.0)
    code[~(np.abs(value) <= np.finfo(np.float32).max)] = 0     # and the NaN codes
    n = code.size
    m = Model([n], 3, 8, True, grads="fp32")
    m.grads[0].zero_()
    m.masters[0].zero_()
    codes = torch.from_numpy(code).to(DEV)
    scales = torch.from_numpy(byte.repeat(8).astype(np.uint8)).to(DEV)
    same = torch.full((n // 32,), 127, dtype=torch.uint8, device=DEV)
    # beside them v = 0, where d is eps, or m = 1
    other = torch.full((n,), 0x38 if moment else 0, dtype=torch.uint8, device=DEV)
    m.states = ([other], [codes], [same], [scales]) if moment else \
        ([codes], [other], [scales], [same])
    before = m.snapshot()
    kw = dict(lr=1.0, betas=(0.5, 0.5), eps=1e-10 if moment else 1.0, step=10 ** 6)
    m.batch(weight_decay=0.0).run(seed=4, **kw)
    torch.cuda.synchronize()
    m.check(before, decay=[0.0], seed=4, **kw)


@pytest.mark.parametrize("beta2,steps", [(0.95, 200), (0.99, 800), (0.999, 6000)])
def test_the_noise_of_8_bit_states(beta2, steps):
    """Gaussian gradients of sd s, the sds of a block's elements within a factor of 3 and
    those of the blocks over decades, into 32-bit and 8-bit states side by side.

    Bounds.  Both states see the same gradients, so their difference D follows
    D' = beta D + r, r the error of one rounding, whose mean is 0 whatever was
    before: E D^2 = E r^2 / (1 - beta^2) at most.  A step of the grid is at most 1/8 of
    the value, so with f its fraction E r^2 = f (1 - f) step^2 <= x^2 / 256, x the value
    that is rounded.  (Below the grid's normal range, 2^-13 of the block's largest, a
    step is 2^-16 of that: nothing beside the bounds.)
      m: E x^2 = s^2 (1 - beta1) / (1 + beta1) + E r^2 / (1 - beta1^2), beta1 = 0.9:
         rms(D) <= 0.146 of m's own rms.
      v, with k = 2 (1 - beta2) / (1 + beta2) its own variance and e^2 = E D^2, both in
         units of s^4: e^2 <= (1 + k + e^2) / (256 (1 - beta2^2)).  And as an
         old value is on the grid, its change is at least the distance to the grid:
         E r^2 <= E |change| x / 8 <= (1 - beta2) / 8 sqrt(E (g^2 - v)^2 E x^2), so
         e^2 <= sqrt((2 + k + e^2) (1 + k + e^2)) / (8 (1 + beta2)): e <= 0.33 at any of
         these beta2.
      m / sqrt(v), to the second order of v's relative error, and m's being
         apart from it (their random bits are): a bias of 3/8 e^2, and an rms error of
         at most sqrt(0.146^2 + e^2 / 4) + 3/8 e^2.
    The percentiles and the update's figures are printed beside their bounds."""
    n, beta1 = 1 << 18, 0.9
    gen = _gen(7)
    sd = (torch.rand(n, generator=gen, device=DEV) + 0.5) * 1e-3
    sd *= torch.exp(2 * _normal(n // 32, gen)).repeat_interleave(32)
    g = torch.zeros(n, device=DEV)
    wide, small = (AdamWBatch([torch.zeros(n, device=DEV).to(torch.bfloat16)], [g],
                              masters=[torch.zeros(n, device=DEV)], state_bits=bits,
                              weight_decay=0.0) for bits in (32, 8))
    for t in range(1, steps + 1):
        torch.mul(_normal(n, gen), sd, out=g)
        for batch in (wide, small):
            batch.run(lr=0.0, step=t, betas=(beta1, beta2), seed=3)
    torch.cuda.synchronize()
    s = sd.double().cpu().numpy()
    m8, v8 = (ref.decode(c[0].cpu().numpy(), b[0].cpu().numpy())
              for c, b in ((small.m, small.m_scale), (small.v, small.v_scale)))
    m, v = (x[0].double().cpu().numpy() for x in (wide.m, wide.v))
    rms = lambda x: math.sqrt(float(np.mean(x ** 2)))
    m_off = rms((m8 - m) / s) / rms(m / s)
    e = rms((v8 - v) / s ** 2)
    u8, u = m8 / np.sqrt(v8), m / np.sqrt(v)
    u_off, bias = rms(u8 - u) / rms(u), float(np.mean(u8 * u) / np.mean(u * u)) - 1
    log(f"beta2={beta2}: v8/v32 sd {np.std(v8 / v):.3f}, 1st to 99th percentile "
        f"{np.percentile(v8 / v, 1):.2f} to {np.percentile(v8 / v, 99):.2f}, v {e:.4f}, "
        f"m {m_off:.4f}, update {u_off:.4f}, bias {bias:.4f}")
    k = 2 * (1 - beta2) / (1 + beta2)
    e2 = 0.0
    for _ in range(60):      # both bounds' fixed points, from below: they only grow
        e2 = min((1 + k + e2) / (256 * (1 - beta2 ** 2)),
                 math.sqrt((2 + k + e2) * (1 + k + e2)) / (8 * (1 + beta2)))
    assert e <= math.sqrt(e2) <= 0.33
    assert m_off <= 0.146
    # (u8 - u) u has an sd below 0.25 sqrt(3) of u^2: 0.005 is 6 sds of 2^18 elements' mean
    assert abs(bias) <= 3 / 8 * e2 + 0.005
    assert u_off <= math.sqrt(0.146 ** 2 + e2 / 4) + 3 / 8 * e2
