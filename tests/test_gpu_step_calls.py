"""Calls of the optimizer step and the gradient norm on the GPU that go beside their
plain use: numbers at the border of fp32, a norm without a result, copies in
place, errors and steps left out around them."""
import ctypes
import math

import numpy as np
import pytest
import torch

from lossless_bf16_weight_xor_amd import AdamWBatch, GradNormBatch
from tests import step_reference as ref
from tests.gpu_util import log
from tests.test_gpu_step import DEV, Model, _gen, _normal

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


@pytest.mark.parametrize("bits,master", [(32, True), (8, True), (8, False)])
def test_a_norm_that_has_not_run_leaves_the_step_out(bits, master):
    """Its scale is no factor yet: a step with it may not take the gradients for zeros."""
    log(f"norm that has not run, bits={bits} master={master}")
    m = Model([5000, 33], 1, bits, master, apart=True)
    norm, batch = GradNormBatch(m.grads), m.batch(weight_decay=0.1)
    batch.run(lr=1e-3, step=1, norm=norm)
    torch.cuda.synchronize()
    now = m.snapshot()
    assert all(_same(a, b) for a, b in zip(now["s"], m.before["s"]))
    assert _same(now["p"], m.before["p"])
    assert _same(now["out"], [ref.bf16_bits_nearest(x.astype(np.float64)) for x in m.before["p"]]
                 if master else m.before["w"])
    # and once it has run, it is a step like any other
    kw = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8, step=1)
    norm.run()
    batch.run(norm=norm, **kw)
    torch.cuda.synchronize()
    m.check(m.before, decay=[0.1] * 2, **kw)


def _hip_runtime():
    """The HIP runtime that this process has loaded."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libamdhip64" in line}
    assert len(paths) == 1, paths
    return ctypes.CDLL(paths.pop())


def test_an_error_left_by_another_call_is_not_the_steps():
    """A refused runtime call leaves its error behind (here: a device that is not
    there); a norm and a step after it do their work and say so."""
    log("error of another call")
    m = Model([5000, 33], 1, 32, True)
    norm, batch = GradNormBatch(m.grads), m.batch(weight_decay=0.0)
    kw = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8, step=1)
    torch.cuda.synchronize()
    hip = _hip_runtime()
    try:
        assert hip.hipSetDevice(99) != 0
        norm.run()
        assert hip.hipSetDevice(99) != 0
        batch.run(norm=norm, **kw)
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert norm.nonfinite.item() == 0
    m.check(m.before, decay=[0.0] * 2, **kw)


def test_pairs_of_copies_that_share_memory_are_refused():
    """(old, new) means nothing where the step has written the old copy: the same
    tensors given twice, or one tensor's new copy in the place of another's old one."""
    log("pairs that share memory")
    m = Model([64, 40, 0], 7, 32, True)
    kw = dict(masters=m.masters, states=m.states)
    for out in (None, m.weights, [w.view(-1) for w in m.weights],
                [torch.empty_like(m.weights[0]), m.weights[0][:40], m.weights[2]],
                [torch.empty_like(m.weights[0]), m.weights[0][16:56], m.weights[2]]):
        with pytest.raises(ValueError, match="old copy"):
            AdamWBatch(m.weights, m.grads, out=out, **kw).pairs()
    both = torch.empty(2 * 64, dtype=torch.bfloat16, device=DEV)   # neighbours, but apart
    a, b = both[:64], both[64:]
    for w, out in (([a], [b]), ([b], [a])):
        (old, new), = AdamWBatch(w, m.grads[:1], out=out, masters=m.masters[:1]).pairs()
        assert old is w[0] and new is out[0]


@pytest.mark.parametrize("bits", [32, 8])
def test_a_left_out_step_in_a_graph_need_not_advance_the_number(bits):
    """step.add_(1 - norm.nonfinite) between the norm and the step: a replay whose
    gradients are not finite changes nothing, the number included, and the next
    one is what an eager loop that skips the batch does."""
    log(f"left out in a graph, bits={bits}")
    sizes = [20011, 333, 4096]
    a, b = (Model(sizes, 63, bits, True) for _ in range(2))
    norms = [GradNormBatch(x.grads) for x in (a, b)]
    batches = [x.batch() for x in (a, b)]
    step = torch.tensor(0, dtype=torch.int64, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norms[0].run(max_norm=0.5)
        step.add_(1 - norms[0].nonfinite)
        batches[0].run(lr=1e-3, step=step, seed=4, norm=norms[0])
    gen = _gen(6)
    t = 0
    for poison in (False, True, False, True, True, False):
        for x, y in zip(a.grads, b.grads):
            x.copy_(_normal(x.numel(), gen, 1e-2))
            y.copy_(x)
        if poison:
            a.grads[1][7] = math.nan
        graph.replay()
        if not poison:
            t += 1
            norms[1].run(max_norm=0.5)
            batches[1].run(lr=1e-3, step=t, seed=4, norm=norms[1])
        torch.cuda.synchronize()
        assert step.item() == t
        x, y = a.snapshot(), b.snapshot()
        assert _same(x["w"], y["w"]) and _same(x["p"], y["p"])
        assert all(_same(i, j) for i, j in zip(x["s"], y["s"]))


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_moved_are_prepared_anew(bits):
    """Parameters whose gradients were set to None and made again: batches prepared
    over the new ones, with the old batch's states, go on where it stopped."""
    log(f"moved gradients, bits={bits}")
    sizes = [5000, 33]
    moved, fixed = (Model(sizes, 64, bits, True) for _ in range(2))
    kept = fixed.batch()
    names = ("m", "v", "m_scale", "v_scale")[:2 if bits == 32 else 4]
    last = moved.batch()
    gen = _gen(8)
    for t in range(1, 4):
        for j, g in enumerate(fixed.grads):
            g.copy_(_normal(sizes[j], gen, 1e-2))
            moved.grads[j] = g.clone()
        norm = GradNormBatch(moved.grads)
        last = AdamWBatch(moved.weights, moved.grads, masters=moved.masters, state_bits=bits,
                          states=[getattr(last, x) for x in names])
        norm.run(max_norm=0.1)
        last.run(lr=1e-3, step=t, seed=2, norm=norm)
        kept.run(lr=1e-3, step=t, seed=2, norm=norm)      # of equal gradients
    torch.cuda.synchronize()
    x, y = moved.snapshot(), fixed.snapshot()
    assert _same(x["w"], y["w"]) and _same(x["p"], y["p"])
    assert all(_same(i, j) for i, j in zip(x["s"], y["s"]))
