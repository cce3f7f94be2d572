"""The trainer's side of a weight update (bf16delta_step.h): the AdamW step that
makes a checkpoint's new BF16 weights, and the global gradient norm that
clips it.  Argument marshalling only; the pair (old, new) goes on to
CompressBatch.

    norm = GradNormBatch(grads)
    step = AdamWBatch(weights, grads, masters=masters, out=spare)
    for t in range(1, steps + 1):
        ...                                   # zero grads in place, backward into them
        norm.run(max_norm=1.0)
        step.run(lr=1e-5, step=t, norm=norm)  # spare holds the new weights
"""
from __future__ import annotations

import bisect
import ctypes
import math
from typing import Sequence

import torch

from . import _native
from . import _check_rc

_GRAD_TYPES = {torch.bfloat16: _native.GRAD_BF16, torch.float32: _native.GRAD_F32}
_SPAN = 512          # elements: an arena's tensors start on multiples of this
_SCALE_BLOCK = 32    # elements that share a scale byte
_F32_END = 2.0 ** 128 - 2.0 ** 103   # the least number that is infinite in fp32


def _device_ptr(t, what: str, dtypes, numel: int, device) -> int:
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == device.index
            and t.dtype in dtypes and t.numel() == numel and t.is_contiguous()):
        p = t.data_ptr()
        if p % 16 == 0 or not numel:
            return p if numel else 0
    _refuse(t, what, dtypes, numel, device)


def _refuse(t, what: str, dtypes, numel: int, device) -> None:
    """Says what is wrong with a tensor that _device_ptr did not take."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{what} must be a tensor on a HIP device (got "
                        f"{getattr(t, 'device', type(t))}); there is no CPU path")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be of type {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.device != device:
        raise ValueError("all tensors of a batch must be on one device")
    if t.numel() != numel:
        raise ValueError(f"{what} has {t.numel()} elements, {numel} are needed")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    raise ValueError(f"{what} must be 16-byte aligned")


def _list(tensors, count: int, what: str) -> list:
    tensors = list(tensors)
    if len(tensors) != count:
        raise ValueError(f"{what}: one tensor per weight tensor ({count}), got {len(tensors)}")
    return tensors


def _per_tensor(value, count: int, what: str) -> list:
    values = [float(value)] * count if isinstance(value, (int, float)) else \
        [float(x) for x in value]
    if len(values) != count or not all(math.isfinite(x) and x >= 0.0 for x in values):
        raise ValueError(f"{what} must be a finite number of at least 0, or one per tensor")
    return values


def _scalar_ptr(t: torch.Tensor, what: str, dtypes, device) -> int:
    if t.dtype not in dtypes or t.device != device or t.numel() != 1:
        raise TypeError(f"{what} must be a number or one {' or '.join(map(str, dtypes))} on the "
                        f"batch's device")
    return t.data_ptr()


def _slow_raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle by device index: 0.1 us, where the public form
# takes 1.9 of a call's 6.5 (a torch built without GPU support lacks the first).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _slow_raw_stream)


class _Prepared:
    """A table uploaded once and a plan; calls on the current stream of its device."""

    def _prepare(self, device: torch.device, table_bytes: int, call, what: str) -> None:
        """call(table pointer, its bytes, stream, plan) -> status"""
        self.device = device
        self._index = device.index
        with torch.cuda.device(device):
            self.table = torch.empty(table_bytes, dtype=torch.uint8, device=device)
            self.plan = _native.StepPlan()
            self._stream0 = _raw_stream(device.index)
            _check_rc(call(self.table.data_ptr(), table_bytes, self._stream0,
                           ctypes.byref(self.plan)), what)
        self._plan_ref = ctypes.byref(self.plan)

    def _owned(self) -> list:
        """The buffers this object allocated."""
        return [self.table]

    def _hold(self, stream: int) -> None:
        """Tells the allocator that `stream`, the device's current one, works on the own
        buffers (not in a capture: a graph needs the object alive anyway)."""
        if stream == self._stream0:
            return
        with torch.cuda.device(self.device):   # the capture asked for is the current device's
            if not torch.cuda.is_current_stream_capturing():
                s = torch.cuda.current_stream()
                for t in self._owned():
                    t.record_stream(s)

    def _call(self, fn, what: str, *args) -> None:
        """fn(plan, *args, stream) on the current stream of the batch's device."""
        stream = _raw_stream(self._index)
        self._hold(stream)
        if torch.cuda.current_device() == self._index:
            rc = fn(self._plan_ref, *args, stream)
        else:
            with torch.cuda.device(self.device):
                rc = fn(self._plan_ref, *args, stream)
        _check_rc(rc, what)


class GradNormBatch(_Prepared):
    """The global L2 norm of a fixed list of gradient tensors (bf16 or fp32,
    mixed as they come), prepared once (bf16d_grad_norm).

    run() enqueues one kernel on the current stream; it may be captured into
    a graph (keep this object and the gradients alive as long as the graph).
    The outcome stays on the device, as 0-dim views of one small buffer:
      norm      : float64, |grad_scale| * sqrt(sum of squares)
      scale     : float32, grad_scale * min(1, max_norm / norm), what
                  AdamWBatch multiplies the gradients by
      nonfinite : int32, 1 if a gradient is infinite or NaN (AdamWBatch then
                  leaves the step out), and before the first run
    The gradients' addresses are fixed: zero them in place between steps
    (zero_grad(set_to_none=False); torch's default drops the tensors, this object
    would go on reading the old ones, and it cannot tell).  Gradients that have
    moved want a new object.  Calls of one object must not overlap in time.

    Where each rank holds a part of the gradients, run without clipping,
    all-reduce norm.square() (sum) and nonfinite (max), and write the whole
    model's norm, scale and flag back into the views: AdamWBatch reads them
    there."""

    def __init__(self, grads: Sequence[torch.Tensor]):
        self.grads = list(grads)   # keep the tensors alive
        if not self.grads:
            raise ValueError("empty batch")
        count = len(self.grads)
        device = getattr(self.grads[0], "device", None)
        jobs = (_native.Grad * count)()
        for j, g in enumerate(self.grads):
            n = g.numel() if isinstance(g, torch.Tensor) else 0
            p = _device_ptr(g, "gradient", tuple(_GRAD_TYPES), n, device)
            jobs[j] = _native.Grad(p, n, _GRAD_TYPES[g.dtype], 0)
        self.result = torch.zeros(2, dtype=torch.float64, device=device)
        self.norm = self.result[0]
        words = self.result.view(torch.int32)
        self.scale = words[2:3].view(torch.float32)[0]
        self.nonfinite = words[3]
        self.nonfinite.fill_(1)   # nothing to scale by before the first run
        lib = _native.lib()
        self._fn = lib.bf16d_grad_norm
        total = sum(g.numel() for g in self.grads)
        self._prepare(device, int(lib.bf16d_grad_norm_table_bytes(total, count)),
                      lambda table, size, stream, plan: lib.bf16d_grad_norm_prepare(
                          jobs, count, table, size, self.result.data_ptr(), stream, plan),
                      "bf16d_grad_norm_prepare")

    def _owned(self) -> list:
        return [self.table, self.result]

    def run(self, max_norm: float = math.inf, grad_scale: float = 1.0) -> None:
        """max_norm: above 0, infinity for no clipping.  grad_scale: what the
        stored gradients are multiplied by (finite in fp32)."""
        if not max_norm > 0 or not abs(grad_scale) < _F32_END:
            raise ValueError("max_norm must be above 0 and grad_scale finite in fp32")
        self._call(self._fn, "bf16d_grad_norm", max_norm, grad_scale)


class AdamWBatch(_Prepared):
    """One AdamW step over a fixed list of tensors, prepared once
    (bf16d_adamw_step; the formulas, the rounding and the 8-bit states are
    described in bf16delta_step.h).

    weights : bf16 tensors, the working weights before the step
    grads   : bf16 or fp32, one per weight tensor
    masters : fp32 master copies, updated in place; without them the bf16
              weights are what is trained, and are rounded stochastically
    out     : bf16 tensors that receive the new weights; None for in place.
              With two working copies, the batch (a -> b) and another one
              (b -> a) over the same states take turns, and pairs() is what
              CompressBatch takes.
    states  : (m, v) lists of fp32 tensors, or for state_bits=8 (m, v,
              m_scale, v_scale): uint8 (or float8_e4m3fn) codes, and uint8 (or
              float8_e8m0fnu) scale bytes, one per 32 elements.  They are
              updated in place.  None: zeros, allocated here (the attributes
              m, v, m_scale, v_scale are the lists in either case).  States
              allocated here are held for whatever stream a step runs on; tensors
              that are passed in stay their owner's, as in any torch call.
    weight_decay, lr_scale : a number, or one per tensor
    A tensor that several names share is listed once.  All buffers keep their
    addresses: zero the gradients in place (zero_grad(set_to_none=False)), or, after
    torch's default has dropped them, prepare a new batch over the new ones with
    this one's lists as its states: nothing here can tell that a gradient moved.
    Calls of one object must not overlap in time, nor replays of graphs that
    hold them (keep it alive as long as those)."""

    def __init__(self, weights: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 masters: Sequence[torch.Tensor] | None = None,
                 out: Sequence[torch.Tensor] | None = None, states=None, state_bits: int = 32,
                 weight_decay=0.01, lr_scale=1.0):
        self.weights = list(weights)
        if not self.weights:
            raise ValueError("empty batch")
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        count = len(self.weights)
        self.state_bits = state_bits
        self.grads = _list(grads, count, "grads")
        self.masters = None if masters is None else _list(masters, count, "masters")
        self.out = self.weights if out is None else _list(out, count, "out")
        device = getattr(self.weights[0], "device", None)
        sizes = [w.numel() if isinstance(w, torch.Tensor) else 0 for w in self.weights]
        places = [_device_ptr(w, "weights", (torch.bfloat16,), n, device)
                  for w, n in zip(self.weights, sizes)]
        parts = 2 if state_bits == 32 else 4
        self._arenas = []
        if states is None:
            states = self._new_states(sizes, device)
        elif len(states) != parts:
            raise ValueError(f"states must be {parts} lists of tensors for {state_bits}-bit states")
        names = ("m", "v", "m_scale", "v_scale")[:parts]
        lists = [_list(s, count, name) for s, name in zip(states, names)]
        self.m, self.v = lists[:2]
        self.m_scale, self.v_scale = lists[2:] if parts == 4 else (None, None)
        decay = _per_tensor(weight_decay, count, "weight_decay")
        rate = _per_tensor(lr_scale, count, "lr_scale")
        code = (torch.float32,) if state_bits == 32 else (torch.uint8, torch.float8_e4m3fn)
        byte = (torch.uint8, torch.float8_e8m0fnu)
        jobs = (_native.AdamWJob * count)()
        for j, n in enumerate(sizes):
            blocks = -(-n // _SCALE_BLOCK)
            g = self.grads[j]
            jobs[j] = _native.AdamWJob(
                places[j],
                places[j] if self.out is self.weights else
                _device_ptr(self.out[j], "out", (torch.bfloat16,), n, device),
                0 if masters is None else
                _device_ptr(self.masters[j], "master", (torch.float32,), n, device),
                _device_ptr(g, "gradient", tuple(_GRAD_TYPES), n, device),
                _device_ptr(self.m[j], "m", code, n, device),
                _device_ptr(self.v[j], "v", code, n, device),
                0 if parts == 2 else _device_ptr(self.m_scale[j], "m_scale", byte, blocks, device),
                0 if parts == 2 else _device_ptr(self.v_scale[j], "v_scale", byte, blocks, device),
                n, rate[j], decay[j], _GRAD_TYPES[g.dtype], 0)
        lib = _native.lib()
        self._fn = lib.bf16d_adamw_step
        self._params = _native.AdamWParams()
        self._params_ref = ctypes.byref(self._params)
        self._prepare(device, int(lib.bf16d_adamw_table_bytes(sum(sizes), count)),
                      lambda table, size, stream, plan: lib.bf16d_adamw_prepare(
                          jobs, count, state_bits, table, size, stream, plan),
                      "bf16d_adamw_prepare")

    def _new_states(self, sizes, device):
        """Zero states of every tensor, as views of one arena per kind."""
        starts, at = [], 0
        for n in sizes:
            starts.append(at)
            at += -(-n // _SPAN) * _SPAN

        def arena(dtype, per):
            flat = torch.zeros(max(at, _SPAN) // per, dtype=dtype, device=device)
            self._arenas.append(flat)
            return [flat[a // per:a // per + -(-n // per)] for a, n in zip(starts, sizes)]

        if self.state_bits == 32:
            return arena(torch.float32, 1), arena(torch.float32, 1)
        return (arena(torch.uint8, 1), arena(torch.uint8, 1), arena(torch.uint8, _SCALE_BLOCK),
                arena(torch.uint8, _SCALE_BLOCK))

    def _owned(self) -> list:
        return [self.table, *self._arenas]

    def pairs(self) -> list[tuple[torch.Tensor, torch.Tensor]]:
        """(weights, out) per tensor, for CompressBatch; needs an `out` of its own."""
        ends = lambda t: (t.data_ptr(), t.data_ptr() + 2 * t.numel())
        # the new copies are apart from each other: by their starts, and so by their ends
        new = sorted(ends(t) for t in self.out if t.numel())

        def written(t):
            lo, hi = ends(t)
            k = bisect.bisect_left(new, (hi,))   # the new copies before it begin below hi
            return t.numel() and k and new[k - 1][1] > lo

        if self.out is self.weights or any(map(written, self.weights)):
            raise ValueError("the step writes over the weights: there is no old copy to "
                             "compare with")
        return list(zip(self.weights, self.out))

    def run(self, lr, step, betas: tuple[float, float] = (0.9, 0.95), eps: float = 1e-8,
            seed: int = 0, norm: GradNormBatch | None = None) -> None:
        """Enqueue one step on the current stream; it may be captured into a graph.

        lr   : a number, or a float32 device tensor that the kernel reads
        step : the step's number from 1, or an int64 device tensor that the
               kernel reads (for graphs: advance it in the graph, and keep
               both tensors alive as long as it).  A step that is left out is no
               step: step.add_(1 - norm.nonfinite) between the norm and this
               call counts only those that are made.  Device tensors cost 1 to 3 %
               of a step's time, but a third with 8-bit states and no masters
        seed : of the stochastic rounding, with the step's number
        norm : a GradNormBatch that has run on these gradients: its scale
               multiplies them, and the step is left out if it found them not finite"""
        p = self._params
        p.lr_device = p.step_device = None
        if isinstance(lr, torch.Tensor):
            p.lr, p.lr_device = 0.0, _scalar_ptr(lr, "lr", (torch.float32,), self.device)
        else:
            p.lr = lr
        if isinstance(step, torch.Tensor):
            p.step, p.step_device = 1, _scalar_ptr(step, "step", (torch.int64,), self.device)
        else:
            p.step = step if step > 0 else 0
        p.beta1, p.beta2 = betas
        p.eps = eps
        p.seed = seed & 0xFFFFFFFFFFFFFFFF
        where = None
        if norm is not None:
            if norm.device != self.device:
                raise ValueError("the norm and the step must be on one device")
            norm._hold(_raw_stream(self._index))   # it may be at home on another stream
            where = norm.result.data_ptr()
        self._call(self._fn, "bf16d_adamw_step", self._params_ref, where)
