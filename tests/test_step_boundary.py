"""CPU checks of the optimizer step's C ABI (bf16delta_step.h) and binding: exports,
struct sizes and every refusal that the host makes before any GPU work.  The
addresses are made up; nothing is launched."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from tests import step_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bf16delta_step.h")
BASE = 1 << 40      # 16-byte aligned addresses, far apart
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def native():
    from lossless_bf16_weight_xor_amd import _native
    if not os.path.exists(_native.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return _native


def _at(k):
    return BASE + (k << 28)


def test_every_declared_symbol_is_exported(native):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(bf16d_[a-z_]+)\s*\(", text))
    assert names == set(native.STEP_EXPORTED)
    lib = ctypes.CDLL(native.LIB_PATH)
    assert all(hasattr(lib, name) for name in names)


def test_struct_sizes_match_the_header(native):
    assert ctypes.sizeof(native.StepPlan) == 64
    assert ctypes.sizeof(native.Grad) == 24
    assert ctypes.sizeof(native.AdamWJob) == 88
    assert ctypes.sizeof(native.AdamWParams) == 64


def _norm_prepare(native, grads=None, count=None, table=_at(50), table_bytes=1 << 20,
                  result=_at(51), plan=True):
    grads = [(_at(0), 100, 0, 0)] if grads is None else grads
    arr = (native.Grad * max(1, len(grads)))(*[native.Grad(*g) for g in grads])
    p = ctypes.byref(native.StepPlan()) if plan else None
    return native.lib().bf16d_grad_norm_prepare(arr, len(grads) if count is None else count, table,
                                                table_bytes, result, None, p)


def test_norm_prepare_refusals(native):
    E = native.EINVAL
    call = lambda **kw: _norm_prepare(native, **kw)
    assert native.lib().bf16d_grad_norm_prepare(None, 1, _at(50), 1 << 20, _at(51), None,
                                                ctypes.byref(native.StepPlan())) == E
    assert call(count=0) == E
    assert call(table=None) == E and call(table=_at(50) + 8) == E
    assert call(result=None) == E and call(result=_at(51) + 4) == E
    assert call(plan=False) == E
    assert call(grads=[(None, 100, 0, 0)]) == E                   # no gradient
    assert call(grads=[(_at(0) + 2, 100, 0, 0)]) == E             # alignment
    assert call(grads=[(_at(0), 100, 2, 0)]) == E                 # unknown type
    assert call(grads=[(_at(0), 100, 0, 1)]) == E                 # reserved
    for n in ((1 << 62) + 1, 1 << 62, (1 << 64) - 1, 1 << 50):
        assert call(grads=[(_at(0), n, 0, 0)]) == E               # sizes
    assert call(result=_at(0) + 192) == E                         # in the gradients' last bytes
    assert call(grads=[(_at(0), 100, 1, 0)], result=_at(0) + 384) == E
    assert call(result=_at(50) + 16) == E                         # in the table
    assert call(table=_at(0)) == E                                # table over the gradients
    need = native.lib().bf16d_grad_norm_table_bytes(100, 1)
    assert call(table_bytes=need - 256 - 4) == E                  # a short table


JOB = dict(weights=_at(0), out=_at(1), master=_at(2), grad=_at(3), m=_at(4), v=_at(5),
           m_scale=0, v_scale=0, n=100, lr_scale=1.0, weight_decay=0.1, grad_dtype=0, reserved=0)


def _adam_prepare(native, jobs=None, count=None, bits=32, table=_at(50), table_bytes=1 << 20,
                  plan=True, **change):
    jobs = [{**JOB, **change}] if jobs is None else jobs
    arr = (native.AdamWJob * max(1, len(jobs)))(*[native.AdamWJob(*j.values()) for j in jobs])
    p = ctypes.byref(native.StepPlan()) if plan else None
    return native.lib().bf16d_adamw_prepare(arr, len(jobs) if count is None else count, bits,
                                            table, table_bytes, None, p)


def test_adamw_prepare_refusals(native):
    E = native.EINVAL
    call = lambda **kw: _adam_prepare(native, **kw)
    scales = dict(m_scale=_at(6), v_scale=_at(7), bits=8)
    assert native.lib().bf16d_adamw_prepare(None, 1, 32, _at(50), 1 << 20, None,
                                            ctypes.byref(native.StepPlan())) == E
    assert call(count=0) == E and call(bits=16) == E and call(bits=0) == E
    assert call(table=None) == E and call(table=_at(50) + 4) == E and call(plan=False) == E
    for name in ("out", "grad", "m", "v"):
        assert call(**{name: 0}) == E, name
        assert call(**scales, **{name: 0}) == E, name
    assert call(weights=0, master=0) == E
    for name in ("weights", "out", "master", "grad", "m", "v"):
        assert call(**{name: JOB[name] + 8}) == E, name
    for name in ("m_scale", "v_scale"):
        assert call(**{**scales, name: 0}) == E
        assert call(**{**scales, name: scales[name] + 4}) == E
        assert call(**{name: _at(6)}) == E        # scales with 32-bit states
    for name in ("lr_scale", "weight_decay"):
        for x in (NAN, INF, -1.0):
            assert call(**{name: x}) == E, (name, x)
    assert call(lr_scale=1e30, weight_decay=1e30) == E
    assert call(grad_dtype=2) == E and call(reserved=1) == E
    for n in ((1 << 62) + 1, 1 << 62, (1 << 64) - 1, 1 << 50):
        assert call(n=n) == E
    need = native.lib().bf16d_adamw_table_bytes(100, 1)
    assert call(table_bytes=need - 256) == E


def test_adamw_prepare_refuses_overlaps(native):
    E = native.EINVAL
    call = lambda **kw: _adam_prepare(native, **kw)
    n = JOB["n"]
    written = {"out": 2 * n, "master": 4 * n, "m": 4 * n, "v": 4 * n}
    for a, size in written.items():
        for b in ("grad", "out", "master", "m", "v"):
            if a != b:
                assert call(**{b: JOB[a] + size // 16 * 16 - 16}) == E, (a, b)
        assert call(table=JOB[a]) == E
    # the weights that are read, without a master copy: the same buffer or none of it
    assert call(master=0, weights=JOB["out"] + 16) == E
    assert call(master=0, weights=JOB["m"]) == E
    scales = dict(m_scale=_at(6), v_scale=_at(7), bits=8)
    assert call(**{**scales, "v_scale": _at(6)}) == E
    assert call(**{**scales, "m_scale": JOB["grad"]}) == E
    assert call(**{**scales, "v_scale": JOB["m"] + 96}) == E      # 100 codes
    # two jobs that share a written buffer
    other = {k: (x + (10 << 28) if k in ("weights", "out", "master", "grad", "m", "v") else x)
             for k, x in JOB.items()}
    for name in ("out", "master", "m", "v"):
        assert call(jobs=[JOB, {**other, name: JOB[name]}]) == E, name
    assert call(jobs=[JOB, {**other, "grad": JOB["m"]}]) == E


def _fake_plan(native, word):
    p = native.StepPlan()
    p.opaque[0] = word
    return p


def test_run_calls_refuse_foreign_plans_and_bad_numbers(native):
    lib, E = native.lib(), native.EINVAL
    norm_magic = int.from_bytes(b"F16DNORM", "little")
    adam_magic = int.from_bytes(b"F16DADAM", "little")
    for word in (0, adam_magic, norm_magic + 1):
        assert lib.bf16d_grad_norm(ctypes.byref(_fake_plan(native, word)), 1.0, 1.0, None) == E
    assert lib.bf16d_grad_norm(None, 1.0, 1.0, None) == E
    plan = _fake_plan(native, norm_magic)
    for max_norm in (0.0, -1.0, NAN):
        assert lib.bf16d_grad_norm(ctypes.byref(plan), max_norm, 1.0, None) == E
    for scale in (NAN, INF, -INF):
        assert lib.bf16d_grad_norm(ctypes.byref(plan), 1.0, scale, None) == E

    plan = _fake_plan(native, adam_magic)
    good = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, seed=0, lr_device=None,
                step_device=None)

    def call(plan=plan, norm=None, **kw):
        return lib.bf16d_adamw_step(ctypes.byref(plan),
                                    ctypes.byref(native.AdamWParams(*{**good, **kw}.values())),
                                    norm, None)

    assert lib.bf16d_adamw_step(None, ctypes.byref(native.AdamWParams()), None, None) == E
    assert lib.bf16d_adamw_step(ctypes.byref(plan), None, None, None) == E
    for word in (0, norm_magic):
        assert call(plan=_fake_plan(native, word)) == E
    for name in ("beta1", "beta2"):
        for x in (-0.1, 1.0, 1.5, NAN):
            assert call(**{name: x}) == E
    for eps in (0.0, -1e-8, 1e-39, 1e-30, 8.8e-16, NAN, INF, 1e39, 2.0 ** 101):
        assert call(eps=eps) == E
    for lr in (-1e-3, NAN, INF, 1e39):
        assert call(lr=lr) == E
    assert call(step=0) == E
    assert call(norm=BASE + 4) == E
    assert call(lr_device=BASE + 2) == E and call(step_device=BASE + 4) == E


def test_python_api_refuses_cpu_tensors_and_bad_lists(native):
    from lossless_bf16_weight_xor_amd import AdamWBatch, GradNormBatch
    w = [torch.zeros(16, dtype=torch.bfloat16)]
    g = [torch.zeros(16)]
    with pytest.raises(TypeError, match="HIP device"):
        GradNormBatch(g)
    with pytest.raises(TypeError, match="HIP device"):
        AdamWBatch(w, g)
    with pytest.raises(ValueError, match="empty"):
        GradNormBatch([])
    with pytest.raises(ValueError, match="empty"):
        AdamWBatch([], [])
    with pytest.raises(ValueError, match="state_bits"):
        AdamWBatch(w, g, state_bits=16)
    with pytest.raises(ValueError, match="one tensor per weight"):
        AdamWBatch(w, g + g)
    with pytest.raises(ValueError, match="one tensor per weight"):
        AdamWBatch(w, g, masters=[])


def test_table_sizes_grow_with_the_batch(native):
    lib = native.lib()
    for f in (lib.bf16d_grad_norm_table_bytes, lib.bf16d_adamw_table_bytes):
        assert 0 < f(0, 1) <= f(1, 1) <= f(10 ** 6, 1) < f(10 ** 9, 1) < f(10 ** 9, 300)


def test_random_bits_are_even_and_depend_on_everything():
    """The counter hash of bf16delta_step.h: each half of the bits, over numbers,
    steps and seeds, has the mean, spread and bit balance of independent
    uniform draws (6 sds), and neighbours and halves are not correlated."""
    n = 1 << 18
    a = ref.random_bits(0, n, 1, 1)
    for other in (ref.random_bits(0, n, 1, 2), ref.random_bits(0, n, 2, 1),
                  ref.random_bits(1 << 32, n, 1, 1), ref.random_bits(n, n, 1, 1)):
        assert abs(int((a == other).sum())) <= 6
        assert abs(np.corrcoef(a & 0xFFFF, other & 0xFFFF)[0, 1]) < 6 / math.sqrt(n)
        assert abs(np.corrcoef(a >> 16, other >> 16)[0, 1]) < 6 / math.sqrt(n)
    third = (a * np.uint32(0x9E3779B1)) >> 16
    for x in (a & 0xFFFF, a >> 16, third):
        u = x / 65536.0
        assert abs(u.mean() - 0.5) < 6 * math.sqrt(1 / 12 / n)
        assert abs(u.var() - 1 / 12) < 6 * math.sqrt(1 / 180 / n)
        assert abs(np.corrcoef(u[1:], u[:-1])[0, 1]) < 6 / math.sqrt(n)
        for bit in range(16):
            assert abs((x >> bit & 1).mean() - 0.5) < 6 * 0.5 / math.sqrt(n)
    for x, y in ((a & 0xFFFF, a >> 16), (a & 0xFFFF, third), (a >> 16, third)):
        assert abs(np.corrcoef(x, y)[0, 1]) < 6 / math.sqrt(n)


def test_the_reference_codes_are_those_of_the_type():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(codes, ref.E4M3, equal_nan=True)
    x = np.random.default_rng(0).standard_normal(4096) * np.logspace(-30, 30, 4096)
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.bfloat16).view(torch.int16).numpy()
    assert np.array_equal(ref.bf16_bits_nearest(x), want.view(np.uint16))
