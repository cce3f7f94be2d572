"""CPU checks of what the optimizer step's binding tells torch's allocator when a call
runs on another stream than the one its buffers were allocated on.  The library, the
streams and record_stream are stand-ins; nothing is launched."""
import contextlib
import types

import pytest
import torch

from lossless_bf16_weight_xor_amd import _native
from lossless_bf16_weight_xor_amd import step as step_module

HOME, SIDE, THIRD = 0, 7, 9      # stream handles


class World:
    """The current device, its current stream, which devices capture, and which
    storages were recorded on which streams."""

    def __init__(self):
        self.device = self.batch_device = None   # the batches' one, as torch names the CPU
        self.stream = HOME
        self.capturing = set()
        self.recorded = set()

    def has(self, tensor, stream):
        return (tensor.untyped_storage().data_ptr(), stream) in self.recorded


@pytest.fixture
def world(monkeypatch):
    w = World()

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 256 if name.endswith("table_bytes") else _native.OK

    @contextlib.contextmanager
    def use(device):
        old, w.device = w.device, getattr(device, "index", device)
        yield
        w.device = old

    def record(tensor, stream):
        w.recorded.add((tensor.untyped_storage().data_ptr(), stream.cuda_stream))

    monkeypatch.setattr(_native, "lib", Lib)
    monkeypatch.setattr(step_module, "_device_ptr", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(step_module, "_raw_stream", lambda index: w.stream)
    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: w.device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=w.stream))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                        lambda: w.device in w.capturing)
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    return w


def _batch(bits, **kw):
    sizes = [600, 33, 0]
    return step_module.AdamWBatch([torch.zeros(n, dtype=torch.bfloat16) for n in sizes],
                                  [torch.zeros(n) for n in sizes], state_bits=bits, **kw)


@pytest.mark.parametrize("bits", [32, 8])
def test_own_states_are_held_for_the_stream_that_works_on_them(world, bits):
    b = _batch(bits)
    own = [b.table, b.m[0], b.v[0]] + ([b.m_scale[0], b.v_scale[0]] if bits == 8 else [])
    b.run(lr=1e-3, step=1)
    assert not world.recorded          # on the stream they come from
    world.stream = SIDE
    b.run(lr=1e-3, step=2)
    assert all(world.has(t, SIDE) for t in own)
    # every tensor's states are views of the arenas that are held
    for part in (b.m, b.v) + ((b.m_scale, b.v_scale) if bits == 8 else ()):
        assert all(world.has(t, SIDE) for t in part)


def test_given_states_are_left_to_their_owner(world):
    m, v = ([torch.zeros(n) for n in (600, 33, 0)] for _ in range(2))
    b = _batch(32, states=(m, v))
    world.stream = SIDE
    b.run(lr=1e-3, step=1)
    assert world.recorded == {(b.table.untyped_storage().data_ptr(), SIDE)}


def test_the_norms_result_is_held_for_the_step_that_reads_it(world):
    norm = step_module.GradNormBatch([torch.zeros(600)])
    world.stream = SIDE
    b = _batch(32)                     # at home on the other stream
    b.run(lr=1e-3, step=1)
    assert not world.recorded
    b.run(lr=1e-3, step=1, norm=norm)
    assert world.has(norm.result, SIDE)
    world.stream = HOME
    world.recorded.clear()
    b.run(lr=1e-3, step=2, norm=norm)  # the norm's own stream
    assert not world.has(norm.result, HOME) and world.has(b.table, HOME)
    world.stream = THIRD
    norm.run()
    assert world.has(norm.result, THIRD) and world.has(norm.table, THIRD)


@pytest.mark.parametrize("capturing", [False, True])
def test_a_capture_is_looked_for_on_the_batchs_device(world, capturing):
    """Another device is current: whether its stream is captured says nothing."""
    b = _batch(32)
    world.device = 1
    world.capturing = {b._index if capturing else 1}
    world.stream = SIDE
    b.run(lr=1e-3, step=1)
    assert world.has(b.table, SIDE) != capturing
    assert world.device == 1
