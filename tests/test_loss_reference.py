"""The reference of the losses against differences and torch's own functions, on the CPU."""
import math

import pytest
import torch

from tests import loss_reference as ref


def _rows(seed, n=5, vocab=37, t=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, vocab, generator=g, dtype=ref.F64) * 2
    x[1, 5:9] = -math.inf
    y = torch.tensor([3, 0, 36, 10, 1])
    return x, y, ref.Rows(x, y, t, top=7)


@pytest.mark.parametrize("t", [1.0, 0.7, 3.0])
def test_log_probabilities_are_torchs(t):
    x, y, r = _rows(0, t=t)
    lp = torch.log_softmax(x / t, 1)
    assert torch.allclose(r.lp, lp, rtol=1e-13, atol=1e-13)
    assert torch.allclose(r.entropy[:, 0], torch.special.entr(lp.exp()).sum(1), rtol=1e-12)
    best = x.topk(7, dim=1)
    assert torch.equal(r.top_ids, best.indices)


@pytest.mark.parametrize("t", [1.0, 0.7])
def test_the_logits_gradient_is_that_of_differences(t):
    x, y, r = _rows(1, t=t)
    a, h = torch.randn(5, dtype=torch.float32), torch.randn(5, dtype=torch.float32)
    g, _ = r.grad(a, h, torch.float32)

    def value(x):
        r = ref.Rows(x, y, t)
        return (a * r.logp + h * r.entropy[:, 0]).sum()

    step = 1e-6
    for i, j in ((0, 3), (0, 4), (1, 0), (1, 6), (2, 36), (3, 11), (4, 1), (4, 30)):
        if x[i, j] == -math.inf:
            assert g[i, j] == 0
            continue
        lo, hi = x.clone(), x.clone()
        lo[i, j] -= step
        hi[i, j] += step
        assert (value(hi) - value(lo)) / (2 * step) == pytest.approx(g[i, j].item(), abs=1e-7)


def test_the_policy_gradients_are_those_of_differences():
    g = torch.Generator().manual_seed(3)
    n = 40
    old = -torch.rand(n, generator=g, dtype=ref.F64) * 5
    lp = old + 0.3 * torch.randn(n, generator=g, dtype=ref.F64)
    adv, w = torch.randn(n, generator=g, dtype=ref.F64), torch.rand(n, generator=g, dtype=ref.F64)
    kw = dict(weights=w, ref=lp + 0.2, clip=(0.2, 0.3), kl_coef=0.3, entropy_coef=0.1, scale=0.7)
    h = torch.rand(n, generator=g, dtype=ref.F64)
    kw["ref"] = kw["ref"].clone()
    found = ref.policy(lp, old, adv, entropy=h, **kw)
    assert 0 < found["clipped"] < 1
    for i in range(n):
        step = torch.zeros(n, dtype=ref.F64)
        step[i] = 1e-6
        for name, lo, hi in (
                ("grad_logp", ref.policy(lp - step, old, adv, entropy=h, **kw),
                 ref.policy(lp + step, old, adv, entropy=h, **kw)),
                ("grad_entropy", ref.policy(lp, old, adv, entropy=h - step, **kw),
                 ref.policy(lp, old, adv, entropy=h + step, **kw))):
            slope = (hi["loss"] - lo["loss"]) / 2e-6
            assert slope.item() == pytest.approx(found[name][i].item(), abs=1e-7), (name, i)


def test_the_balance_gradient_is_that_of_differences():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(9, 6, generator=g, dtype=ref.F64)
    x[4, 2] = -math.inf
    x[7] = -math.inf
    chosen = x.topk(2, dim=1).indices
    chosen[0, 1] = -1
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1, 1, 1], dtype=torch.bool)
    kw = dict(mask=mask, balance_coef=0.3, z_coef=0.2)
    found = ref.balance(x, chosen, **kw)
    assert int(found["counts"].sum()) == 15 and int(found["tokens"]) == 8
    for i in range(9):
        for j in range(6):
            if x[i, j] == -math.inf:
                assert found["grad"][i, j] == 0
                continue
            lo, hi = x.clone(), x.clone()
            lo[i, j] -= 1e-6
            hi[i, j] += 1e-6
            slope = (ref.balance(hi, chosen, **kw)["loss"] - ref.balance(lo, chosen, **kw)["loss"])
            assert slope.item() / 2e-6 == pytest.approx(found["grad"][i, j].item(), abs=1e-8)
    even = ref.balance(torch.zeros(8, 4), torch.arange(8)[:, None] % 4)
    assert even["balance"].item() == pytest.approx(1.0)
