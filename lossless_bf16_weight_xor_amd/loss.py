"""The losses of a policy update (bf16delta_loss.h): log probabilities of given
tokens with entropy and top alternatives, the clipped policy loss, the gradient
of the logits, and a router's balance loss.  Argument marshalling only; the
gradients go on through the model to GradNormBatch and AdamWBatch.

    probs = TokenLogProbs(rows, vocab, entropy=True)
    loss = PolicyLoss(rows)
    probs.run(logits, tokens)
    loss.run(probs.logp, old_logp, advantages, weights=weights, entropy=probs.entropy,
             entropy_coef=1e-3, scale=1 / tokens_of_the_batch)
    probs.backward(logits, tokens, loss.grad_logp, out=logits, grad_entropy=loss.grad_entropy)
    ...                                   # logits hold their gradient

Every call enqueues one kernel on the current stream and nothing else, and may be
captured into a graph (keep the object and the tensors alive as long as it).  Results
stay on the device, in buffers of the object that its next run overwrites.  Calls
of one object must not overlap in time, nor replays of graphs that hold them.
Tensors that are passed in stay their owner's, as in any torch call.  A backward call
records nothing in an autograd graph; it counts as an in-place write of `out`, so that a
graph which has saved those logits for its own backward refuses to use their gradient.
"""
from __future__ import annotations

import ctypes
import itertools
import math
import struct

import torch
from torch.autograd.graph import increment_version

from . import _native
from . import _check_rc
from .step import _raw_stream

_LOGITS = {torch.bfloat16: _native.LOGITS_BF16, torch.float32: _native.LOGITS_F32}
_IDS = {torch.int64: _native.IDS_I64, torch.int32: _native.IDS_I32}
_F32 = (torch.float32,)
_BYTES = (torch.bool, torch.uint8)
_MAX_ROWS = (1 << 24) - 1
# The parts of the jobs that a call fills in, packed at once: 0.5 us, where a field
# at a time takes 1 of a call's 6.
_LOGPROB = struct.Struct("8Q4Id").pack_into
_LOGPROB_GRAD = struct.Struct("11Q4I3Q").pack_into
_POLICY = struct.Struct("9Q5d").pack_into
_BALANCE = struct.Struct("6Q4I").pack_into
_BALANCE_GRAD = struct.Struct("6Q2I3d").pack_into


def _refuse(t, what: str, dtypes, shape, device) -> None:
    """Says what is wrong with a tensor that a call did not take."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{what} must be a tensor on a HIP device (got "
                        f"{getattr(t, 'device', type(t))}); there is no CPU path")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be of type {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    if len(t.shape) != len(shape) or any(a is not None and a != b
                                         for a, b in zip(shape, t.shape)):
        wanted = ", ".join("any" if a is None else str(a) for a in shape)
        raise ValueError(f"{what} must have the shape ({wanted}), got {tuple(t.shape)}")
    raise ValueError(f"{what}: the elements of a row must be adjacent, got strides {t.stride()}")


def _row(t, what: str, dtypes, n: int, device) -> int:
    """The address of n adjacent elements of any shape."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == device.index
            and t.dtype in dtypes):
        _refuse(t, what, dtypes, (None,), device)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must hold {n} elements, contiguous; got {tuple(t.shape)} with "
                         f"strides {t.stride()}")
    return t.data_ptr()


class _Op:
    """Buffers on one device, and calls on its current stream."""

    def __init__(self, rows: int, device):
        if not 0 <= int(rows) <= _MAX_ROWS:
            raise ValueError(f"rows must be from 0 to {_MAX_ROWS}, got {rows}")
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise TypeError(f"a HIP device is needed, got {device}; there is no CPU path")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.rows = int(rows)
        self.device = device
        self._index = device.index
        self._lib = _native.lib()
        with torch.cuda.device(device):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("prepare the operator before the capture: its workspace has "
                                   "to be cleared once")
            self._stream0 = _raw_stream(device.index)

    def _buffers(self, *parts) -> list:
        """Zeros of each (shape, dtype), None for None, in one allocation that is
        cleared for any stream when this returns."""
        sizes = [0 if p is None else math.prod(p[0]) * p[1].itemsize for p in parts]
        starts = list(itertools.accumulate((-(-n // 256) * 256 for n in sizes), initial=0))
        self._arena = torch.zeros(max(starts[-1], 1), dtype=torch.uint8, device=self.device)
        with torch.cuda.device(self.device):
            torch.cuda.current_stream().synchronize()
        return [None if p is None else self._arena[at:at + n].view(p[1]).view(p[0])
                for p, at, n in zip(parts, starts, sizes)]

    def _count(self, n: int) -> int:
        if n > self.rows:
            raise ValueError(f"{n} rows, but the operator was prepared for {self.rows}")
        return n

    def _hold(self, stream: int) -> None:
        """Tells the allocator that another stream than the buffers' own works on them
        (not in a capture: a graph needs the object alive anyway)."""
        with torch.cuda.device(self.device):
            if not torch.cuda.is_current_stream_capturing():
                self._arena.record_stream(torch.cuda.current_stream())

    def _call(self, fn, what: str, args) -> None:
        """fn(*args, stream) on the current stream of the operator's device."""
        stream = _raw_stream(self._index)
        if stream != self._stream0:
            self._hold(stream)
        if torch.cuda.current_device() == self._index:
            rc = fn(*args, stream)
        else:
            with torch.cuda.device(self.device):
                rc = fn(*args, stream)
        if rc:
            _check_rc(rc, what)


class TokenLogProbs(_Op):
    """Log probabilities of given tokens, with the distributions' entropy and the top
    alternatives, and the gradient of the logits (bf16d_logprob,
    bf16d_logprob_backward; special rows are described in bf16delta_loss.h).

    rows    : the most rows (tokens) of a call
    vocab   : logits of a row
    entropy : whether the entropy is computed, too
    top     : how many alternatives, at most 64

    After a run over n rows, the first n entries of
      logp     : float32, ln p of the given token; 0 where it is negative (a row
                 that is left out)
      entropy  : float32 (None without)
      top_ids  : int64 (rows, top), the largest logits' ids, largest first, equal
                 ones by their id; -1 where there are no more
      top_logp : float32 (rows, top)
    are its results, flat in the order of the rows; what is behind them is left as it
    was."""

    def __init__(self, rows: int, vocab: int, device=None, entropy: bool = False, top: int = 0):
        if not 1 <= vocab <= _native.MAX_VOCAB:
            raise ValueError(f"vocab must be from 1 to {_native.MAX_VOCAB}, got {vocab}")
        if not 0 <= top <= _native.MAX_TOP:
            raise ValueError(f"top must be from 0 to {_native.MAX_TOP}, got {top}")
        if top and not rows < 1 << 22:
            raise ValueError(f"rows must be below 2^22 with alternatives, got {rows}")
        super().__init__(rows, device)
        self.vocab, self.top = int(vocab), int(top)
        size = int(self._lib.bf16d_logprob_workspace_bytes(self.rows, self.vocab, self.top))
        each, alternatives = (self.rows,), (self.rows, self.top)
        (self.logp, self.entropy, self.stats, self.top_ids, self.top_logp,
         self._workspace) = self._buffers(
            (each, torch.float32), (each, torch.float32) if entropy else None,
            ((self.rows, 4), torch.float32), (alternatives, torch.int64) if top else None,
            (alternatives, torch.float32) if top else None, ((size,), torch.uint8))
        self._ran = None    # rows of the last run
        at = lambda t: t.data_ptr() if t is not None else None
        self._job = _native.LogprobJob(logp=at(self.logp), entropy=at(self.entropy),
                                       stats=at(self.stats), top_ids=at(self.top_ids),
                                       top_logp=at(self.top_logp))
        self._fn = self._lib.bf16d_logprob
        self._args = (ctypes.byref(self._job), self._workspace.data_ptr(), size)
        self._stats = self.stats.data_ptr()
        self._grad_job = _native.LogprobGradJob()
        self._grad_fn = self._lib.bf16d_logprob_backward
        self._grad_args = (ctypes.byref(self._grad_job),)

    def _rows_of(self, logits, tokens) -> tuple:
        """(rows, shape of the logits, their type and the tokens'; address and strides of
        the logits, of the tokens, outer, inner).  Each question to a tensor takes 0.1 us."""
        if not (isinstance(logits, torch.Tensor) and logits.get_device() == self._index
                and (kind := _LOGITS.get(logits.dtype)) is not None):
            _refuse(logits, "logits", _LOGITS, (None, self.vocab), self.device)
        shape, strides = logits.shape, logits.stride()
        if not (isinstance(tokens, torch.Tensor) and tokens.get_device() == self._index
                and (ids := _IDS.get(tokens.dtype)) is not None):
            _refuse(tokens, "tokens", _IDS, shape[:-1], self.device)
        places, steps = tokens.shape, tokens.stride()
        dims = len(shape)
        if dims == 2:
            (inner, vocab), outer = shape, 1
            l_outer = t_outer = 0
        elif dims == 3:
            outer, inner, vocab = shape
            l_outer, t_outer = strides[0], steps[0] if len(steps) == 2 else 0
        else:
            raise ValueError(f"logits must be (rows, vocab) or (batch, length, vocab), got "
                             f"{tuple(shape)}")
        n = outer * inner
        if vocab != self.vocab or (strides[-1] != 1 and vocab > 1 and n):
            _refuse(logits, "logits", _LOGITS, (*shape[:-1], self.vocab), self.device)
        if len(places) != dims - 1 or places[-1] != inner or (dims == 3 and places[0] != outer):
            _refuse(tokens, "tokens", _IDS, shape[:-1], self.device)
        if n > self.rows:
            self._count(n)
        return (n, shape, kind, ids, logits.data_ptr(), l_outer, strides[-2], tokens.data_ptr(),
                t_outer, steps[-1], outer, inner)

    def run(self, logits: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0) -> None:
        """logits: bf16 or fp32, (rows, vocab) or (batch, length, vocab), a row's
        elements adjacent, any strides else.  tokens: int64 or int32, one id a row (a
        negative one leaves the row out).  temperature: what the logits are divided
        by, from 2^-20 to 2^20."""
        if not 2.0 ** -20 <= temperature <= 2.0 ** 20:
            raise ValueError(f"temperature must be from 2^-20 to 2^20, got {temperature}")
        n, _, kind, ids, *rows = self._rows_of(logits, tokens)
        _LOGPROB(self._job, 0, *rows, self.vocab, kind, ids, self.top, temperature)
        self._call(self._fn, "bf16d_logprob", self._args)
        self._ran = n

    def backward(self, logits: torch.Tensor, tokens: torch.Tensor, grad_logp: torch.Tensor,
                 out: torch.Tensor, grad_entropy: torch.Tensor | None = None) -> None:
        """The gradient of sum(grad_logp * logp + grad_entropy * entropy) by the logits, into
        `out` (their type and shape; the logits themselves are fine).  logits and
        tokens: those of the last run; grad_logp, grad_entropy: float32, one a row."""
        n, shape, kind, ids, x, x_outer, x_inner, y, y_outer, y_inner, outer, inner = \
            self._rows_of(logits, tokens)
        if n != self._ran:
            raise ValueError(f"{n} rows, but the last run had {self._ran}: backward needs its "
                             f"softmax sums")
        if not (isinstance(out, torch.Tensor) and out.get_device() == self._index
                and out.dtype == logits.dtype and out.shape == shape):
            _refuse(out, "out", (logits.dtype,), shape, self.device)
        strides = out.stride()
        if strides[-1] != 1 and self.vocab > 1 and n:
            _refuse(out, "out", (logits.dtype,), shape, self.device)
        a = _row(grad_logp, "grad_logp", _F32, n, self.device)
        h = 0
        if grad_entropy is not None:
            if self.entropy is None:
                raise ValueError("grad_entropy needs an operator prepared with entropy=True")
            h = _row(grad_entropy, "grad_entropy", _F32, n, self.device)
        _LOGPROB_GRAD(self._grad_job, 0, x, x_outer, x_inner, y, y_outer, y_inner,
                      out.data_ptr(), strides[0] if len(strides) == 3 else 0, strides[-2], outer,
                      inner, self.vocab, kind, ids, 0, self._stats, a, h)
        self._call(self._grad_fn, "bf16d_logprob_backward", self._grad_args)
        increment_version(out)


class PolicyLoss(_Op):
    """The clipped policy loss of up to `rows` tokens and its gradients
    (bf16d_policy_loss; the formulas are in bf16delta_loss.h).

    After a run over n tokens, on the device:
      grad_logp, grad_entropy : float32, their first n entries (the second one's are 0
                where entropy_coef is, as in a run without entropies)
      loss    : scale * the weighted sum of the tokens' losses
      weight  : the sum of the weights
      kl, clipped, entropy : weighted means, of r - 1 - ln r, of the tokens whose
                ratio was clipped, and of the entropies
    the last five as 0-dim float32 views of one small buffer."""

    def __init__(self, rows: int, device=None):
        super().__init__(rows, device)
        size = int(self._lib.bf16d_policy_loss_workspace_bytes())
        each = ((self.rows,), torch.float32)
        self.grad_logp, self.grad_entropy, self.result, self._workspace = self._buffers(
            each, each, ((8,), torch.float32), ((size,), torch.uint8))
        self.loss, self.weight, self.kl, self.clipped, self.entropy = self.result[:5].unbind()
        self._job = _native.PolicyJob()
        self._fn = self._lib.bf16d_policy_loss
        self._args = (ctypes.byref(self._job), self.result.data_ptr(),
                      self._workspace.data_ptr(), size)
        self._grads = self.grad_logp.data_ptr(), self.grad_entropy.data_ptr()

    def run(self, logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor,
            weights: torch.Tensor | None = None, ref_logp: torch.Tensor | None = None,
            entropy: torch.Tensor | None = None, clip: tuple[float, float] = (0.2, 0.2),
            kl_coef: float = 0.0, entropy_coef: float = 0.0, scale: float = 1.0) -> None:
        """All tensors: float32, contiguous, one number a token.

        logp, old_logp : under the policy, and under the one that drew the tokens
        weights  : of the tokens (0: left out, whatever its numbers are); None: all 1
        ref_logp : under the reference policy, for kl_coef
        entropy  : of the policy, for entropy_coef and the mean
        clip     : how far a ratio counts below and above 1 (infinity above: no bound)
        scale    : of the loss and the gradients, 1 / the batch's tokens for example"""
        if not isinstance(logp, torch.Tensor):
            _refuse(logp, "logp", _F32, (None,), self.device)
        n, device = self._count(logp.numel()), self.device
        if (kl_coef != 0.0 and ref_logp is None) or (entropy_coef != 0.0 and entropy is None):
            raise ValueError("kl_coef needs ref_logp, and entropy_coef needs entropy")
        low, high = clip
        grad_logp, grad_entropy = self._grads
        _POLICY(self._job, 0, _row(logp, "logp", _F32, n, device),
                _row(old_logp, "old_logp", _F32, n, device),
                _row(advantages, "advantages", _F32, n, device),
                0 if weights is None else _row(weights, "weights", _F32, n, device),
                0 if ref_logp is None else _row(ref_logp, "ref_logp", _F32, n, device),
                0 if entropy is None else _row(entropy, "entropy", _F32, n, device),
                grad_logp, grad_entropy, n, low, high, kl_coef, entropy_coef, scale)
        self._call(self._fn, "bf16d_policy_loss", self._args)


class RouterBalance(_Op):
    """The balance loss of a router over `experts`, how often each was chosen, and the
    gradient of the router's logits (bf16d_balance, bf16d_balance_backward; the
    formulas are in bf16delta_loss.h), for up to `rows` tokens a call.

    After a run, on the device:
      counts  : int64, one number an expert
      tokens  : int64, the tokens that count
      loss    : balance_coef * balance + z_coef * z, NaN where an id is out of range
      balance : 1 where the choices or the probabilities are even
      z       : the mean square of ln sum e^x
    the last four as 0-dim views of one small buffer.

    Where several ranks hold a part of the batch each, all-reduce counts and tokens
    (sum) between run and backward: the gradients are then those of the whole
    batch's loss."""

    def __init__(self, rows: int, experts: int, device=None, balance_coef: float = 0.01,
                 z_coef: float = 0.0):
        if not 1 <= experts <= _native.MAX_EXPERTS:
            raise ValueError(f"experts must be from 1 to {_native.MAX_EXPERTS}, got {experts}")
        super().__init__(rows, device)
        self.experts = int(experts)
        size = int(self._lib.bf16d_balance_workspace_bytes(self.experts))
        self.counts, self.result, self._workspace = self._buffers(
            ((self.experts,), torch.int64), ((4,), torch.int64), ((size,), torch.uint8))
        self.loss, self.balance, self.z = self.result.view(torch.float32)[:3].unbind()
        self.tokens = self.result[2]
        self._ran = None    # rows of the last run
        self._coefs = float(balance_coef), float(z_coef)
        self._job = _native.BalanceJob(balance_coef=balance_coef, z_coef=z_coef,
                                       counts=self.counts.data_ptr())
        self._fn = self._lib.bf16d_balance
        self._args = (ctypes.byref(self._job), self.result.data_ptr(),
                      self._workspace.data_ptr(), size)
        self._grad_job = _native.BalanceGradJob(counts=self.counts.data_ptr(),
                                                tokens=self.tokens.data_ptr(),
                                                result=self.result.data_ptr())
        self._grad_fn = self._lib.bf16d_balance_backward
        self._grad_args = (ctypes.byref(self._grad_job),)

    def _rows_of(self, logits, mask) -> tuple:
        """(rows, shape of the logits, their type, address, row stride, the mask's address)"""
        if not (isinstance(logits, torch.Tensor) and logits.get_device() == self._index
                and (kind := _LOGITS.get(logits.dtype)) is not None
                and len(shape := logits.shape) == 2):
            _refuse(logits, "logits", _LOGITS, (None, self.experts), self.device)
        n, experts = shape
        stride, step = logits.stride()
        if experts != self.experts or (step != 1 and experts > 1 and n):
            _refuse(logits, "logits", _LOGITS, (None, self.experts), self.device)
        if n > self.rows:
            self._count(n)
        return (n, shape, kind, logits.data_ptr(), stride,
                0 if mask is None else _row(mask, "mask", _BYTES, n, self.device))

    def run(self, logits: torch.Tensor, chosen: torch.Tensor,
            mask: torch.Tensor | None = None) -> None:
        """logits: bf16 or fp32, (tokens, experts).  chosen: int64 or int32, (tokens,
        choices), the ids of each token's experts (a negative one is no choice).
        mask: bool or uint8, which tokens count; None: all."""
        n, _, kind, x, stride, seen = self._rows_of(logits, mask)
        if not (isinstance(chosen, torch.Tensor) and chosen.get_device() == self._index
                and (ids := _IDS.get(chosen.dtype)) is not None
                and len(shape := chosen.shape) == 2 and shape[0] == n):
            _refuse(chosen, "chosen", _IDS, (n, None), self.device)
        choices = shape[1]
        if not 1 <= choices <= self.experts:
            raise ValueError(f"chosen must name from 1 to {self.experts} experts a token, got "
                             f"{choices}")
        chosen_stride, step = chosen.stride()
        if step != 1 and choices > 1 and n:
            _refuse(chosen, "chosen", _IDS, (n, None), self.device)
        _BALANCE(self._job, 0, x, chosen.data_ptr(), seen, n, stride, chosen_stride,
                 self.experts, choices, kind, ids)
        self._call(self._fn, "bf16d_balance", self._args)
        self._ran = n

    def backward(self, logits: torch.Tensor, out: torch.Tensor, mask: torch.Tensor | None = None,
                 scale: float = 1.0) -> None:
        """scale * the gradient of the loss by the logits, into `out` (their type and shape;
        the logits themselves are fine).  logits, mask: those of the last run."""
        n, shape, kind, x, stride, seen = self._rows_of(logits, mask)
        if n != self._ran:
            raise ValueError(f"{n} rows, but the last run had {self._ran}: backward needs its counts")
        if not (isinstance(out, torch.Tensor) and out.get_device() == self._index
                and out.dtype == logits.dtype and out.shape == shape):
            _refuse(out, "out", (logits.dtype,), shape, self.device)
        out_stride, step = out.stride()
        if step != 1 and self.experts > 1 and n:
            _refuse(out, "out", (logits.dtype,), shape, self.device)
        _BALANCE_GRAD(self._grad_job, 0, x, out.data_ptr(), seen, n, stride, out_stride,
                      self.experts, kind, *self._coefs, scale)
        self._call(self._grad_fn, "bf16d_balance_backward", self._grad_args)
        increment_version(out)
