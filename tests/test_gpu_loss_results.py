"""Results of the losses' objects over calls of different kinds: a run without entropies
after one with them, ratios far from 1, another number of rows, and gradients over
tensors that an autograd graph has saved."""
import pytest
import torch

from lossless_bf16_weight_xor_amd import PolicyLoss, TokenLogProbs
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
