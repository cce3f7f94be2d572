"""Results of the losses' objects over calls of different kinds: a run without entropies
after one with them, ratios far from 1, another number of rows, and gradients over
tensors that an autograd graph has saved."""
import math

import pytest
import torch

from lossless_bf16_weight_xor_amd import PolicyLoss, RouterBalance, TokenLogProbs
from tests import loss_reference as ref
from tests.gpu_util import log
from tests.test_gpu_loss import DEV, _policy, _policy_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 300, 70000])
def test_the_entropies_gradient_after_a_run_without_them(n):
    """It is that of the last run, 0, and not what an earlier run has left."""
    log(f"no entropies {n}")
    op = PolicyLoss(n + 2, DEV)
    s = _policy_inputs(n, n)
    for weights in (s["weights"], None):
        _policy(op, s, "with", entropy_coef=0.5)
        assert n < 10 or (op.grad_entropy[:n] != 0).any()
        op.grad_entropy[n:] = 5.0
        _policy(op, s | {"entropy": None, "weights": weights}, "without")
        assert (op.grad_entropy[:n] == 0).all() and (op.grad_entropy[n:] == 5.0).all()
    # what a trainer whose bonus has been switched off makes of it
    x, y = torch.randn(n, 40, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV)
    probs = TokenLogProbs(n, 40, DEV, entropy=True)
    probs.run(x, y)
    got, want = torch.empty_like(x), torch.empty_like(x)
    probs.backward(x, y, op.grad_logp[:n], got, grad_entropy=op.grad_entropy[:n])
    probs.backward(x, y, op.grad_logp[:n], want, grad_entropy=torch.zeros(n, device=DEV))
    assert torch.equal(got, want)


def test_ratios_far_below_one():
    """An unclipped ratio keeps its digits down to the smallest that fp32 holds."""
    log("far ratios")
    u = torch.cat([-torch.arange(0, 104, 0.25), -1.0 + torch.linspace(-0.01, 0.01, 99)])
    n = u.numel()
    for old in (-0.5, 0.0, -37.125):
        s = dict(logp=u + old, old=torch.full((n,), old), adv=torch.full((n,), 1.7))
        op = PolicyLoss(n, DEV)
        want = _policy(op, s, f"old {old}")          # to one rounding
        assert (op.grad_logp[:n].cpu()[want["grad_logp"] < -2.0 ** -149] < 0).all()
        # with a factor that lifts them into the range of fp32's normal numbers
        _policy(op, s, f"old {old} scaled", scale=1e30)


def test_ratios_over_the_whole_range():
    """Ratios, and distances from a reference, between and around the halves of ln 2, next
    to 1, far above, and beyond the range of 64 bits."""
    log("whole range")
    half = math.log(2.0) / 2
    steps = torch.cat([torch.arange(-600, 241) * half, torch.arange(-400, 400) * 1e-9,
                       10.0 ** torch.arange(-30, -1, dtype=torch.float32)])
    u = torch.cat([steps, torch.nextafter(steps, steps + 1), torch.nextafter(steps, steps - 1)])
    n, zero = u.numel(), torch.zeros(u.numel())
    op = PolicyLoss(n, DEV)
    s = dict(logp=u, old=zero, adv=torch.where(u > 0, -1.0, 1.0))        # none is clipped
    want = _policy(op, s, "ratios", scale=1e-30)
    assert want["clipped"] == 0
    _policy(op, dict(logp=zero, old=zero, adv=zero, ref=u), "reference", kl_coef=0.7, scale=1e-30)
    for far in (750.0, 1e5, 3e38, math.inf):
        for sign in (1.0, -1.0):
            one = torch.tensor([far * sign])
            _policy(op, dict(logp=one, old=zero[:1], adv=torch.tensor([-sign])), f"{one}")
            _policy(op, dict(logp=zero[:1], old=zero[:1], adv=zero[:1], ref=one), f"ref {one}",
                    kl_coef=1.0)


def test_a_routers_gradient_of_other_rows_is_refused():
    log("other rows")
    x = torch.randn(6, 8, device=DEV)
    ids = torch.zeros(6, 2, dtype=torch.int64, device=DEV)
    op = RouterBalance(6, 8, DEV)
    op.run(x, ids)
    for rows in (5, 0):
        with pytest.raises(ValueError, match="last run had 6"):
            op.backward(x[:rows], torch.empty_like(x[:rows]))
    op.run(x[:5], ids[:5])
    with pytest.raises(ValueError, match="last run had 5"):
        op.backward(x, torch.empty_like(x))
    out = torch.full_like(x, 7.0)
    op.backward(x[:5], out[:5])
    want = ref.balance(x[:5].cpu(), ids[:5].cpu())
    ref.check(out[:5], want["grad"], want["grad_off"], "grad")
    assert (out[5] == 7.0).all()


def test_a_graph_that_saved_the_logits_sees_their_gradient_over_them():
    """backward() counts as a write of `out`: autograd refuses to use what it has saved of
    it, instead of taking the gradient for the logits."""
    log("saved logits")
    weight = torch.randn(16, 40, device=DEV, requires_grad=True)
    states = torch.randn(6, 16, device=DEV)
    y = torch.arange(6, device=DEV)
    a = torch.ones(6, device=DEV)
    probs, router = TokenLogProbs(6, 40, DEV), RouterBalance(6, 40, DEV)

    def calls():
        yield lambda x: (probs.run(x, y), probs.backward(x, y, a, out=x))
        yield lambda x: (router.run(x, y[:, None]), router.backward(x, x))

    for call in calls():
        logits = states @ weight
        saved = logits.square().sum()        # keeps the logits for its backward
        call(logits.detach())                # the same memory
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            saved.backward()
        # beside the logits nothing is in the way, nor in a graph that has not saved them
        logits = states @ weight
        saved, linear = logits.square().sum(), logits.sum()
        out = torch.empty_like(logits)
        before = out._version, logits._version
        call_out = (lambda x: (probs.run(x, y), probs.backward(x, y, a, out=out)))
        call_out(logits.detach())
        assert out._version > before[0] and logits._version == before[1]
        (saved + linear).backward()
    # tensors without a counter are fine
    with torch.inference_mode():
        x = states @ weight
        for call in calls():
            call(x.clone())
    torch.cuda.synchronize()
