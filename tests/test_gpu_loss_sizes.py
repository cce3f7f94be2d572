"""The losses on the GPU at the sizes where their work is cut differently: whole
rows and parts, one workgroup and many, turns that begin in the middle of a vector,
lists of alternatives that are long, and many equal values."""
import math

import pytest
import torch

from lossless_bf16_weight_xor_amd import PolicyLoss, RouterBalance, TokenLogProbs
from tests import loss_reference as ref
from tests.gpu_util import log
from tests.test_gpu_loss import (DEV, TYPES, _check_forward, _check_router, _coefs, _gen, _logits,
                                 _one, _policy, _policy_inputs, _router, _tokens, both_types)

pytestmark = pytest.mark.gpu
INF = math.inf


@both_types
@pytest.mark.parametrize("vocab", [4093, 16379, 16384, 16389, 32761, 32768, 32775, 65537])
@pytest.mark.parametrize("top", [0, 7])
def test_rows_around_a_workgroups_turn(kind, vocab, top):
    """Contiguous rows of odd lengths begin at every place within 16 bytes."""
    _one(kind, 9, vocab, vocab + top, top=top, grad=top == 0)


@both_types
@pytest.mark.parametrize("n,vocab,top", [(65, 70001, 20), (86, 66000, 3), (128, 34001, 9),
                                         (129, 34001, 9), (200, 49999, 64)])
def test_alternatives_of_rows_in_parts(kind, n, vocab, top):
    """As many parts as there are workgroups for, and rows that are not cut."""
    _one(kind, n, vocab, vocab + n, top=top, grad=False)


@both_types
@pytest.mark.parametrize("n,vocab,top", [(256, 16500, 5), (257, 33003, 20), (300, 40003, 64),
                                         (280, 70001, 1), (255, 33000, 33)])
def test_alternatives_of_many_rows(kind, n, vocab, top):
    """Several turns of one workgroup, and rows in a few parts."""
    log(f"{kind} {n}x{vocab} top {top}")
    x, y = _logits(n, vocab, n, kind), _tokens(n, vocab, n)
    op = TokenLogProbs(n, vocab, DEV, entropy=True, top=top)
    op.run(x.to(DEV), y.to(DEV))
    for first in (0, n - 20):
        some = slice(first, first + 20)
        want = ref.Rows(x[some], y[some], top=top)
        ref.check(op.logp[some], want.logp, want.logp_off, "logp")
        assert torch.equal(op.top_ids[some].cpu(), want.top_ids), first
        ref.check(op.top_logp[some], want.top_logp, want.top_off, "top_logp")
    # the rest against torch's own order of the same values
    best = x.float().sort(dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(op.top_ids.cpu(), best)


@both_types
@pytest.mark.parametrize("values", [1, 2, 30, 300])
@pytest.mark.parametrize("vocab", [900, 5000, 33000, 70000])
def test_alternatives_among_few_values(kind, values, vocab):
    """From a handful of candidates to more than a workgroup collects."""
    log(f"{kind} {values} values of {vocab}")
    g = _gen(values)
    x = torch.randint(0, values, (3, vocab), generator=g).float().div(8).to(TYPES[kind])
    y = _tokens(3, vocab, 1)
    for top in (1, 20, 64):
        op = TokenLogProbs(3, vocab, DEV, top=top)
        op.run(x.to(DEV), y.to(DEV))
        _check_forward(op, ref.Rows(x, y, top=top), 3, f"top {top}", top)


@both_types
@pytest.mark.parametrize("n", [1, 3, 300])
def test_negative_tokens_of_either_type(kind, n):
    log(f"{kind} {n}")
    vocab = 9001
    x = _logits(n, vocab, n, kind).to(DEV)
    for dtype in (torch.int32, torch.int64):
        for value in (-1, -100, torch.iinfo(dtype).min):
            y = torch.full((n,), value, dtype=dtype, device=DEV)
            op = TokenLogProbs(n, vocab, DEV, entropy=True, top=2)
            op.logp.fill_(7.0)
            op.run(x, y)
            assert (op.logp == 0).all() and (op.entropy == 0).all()
            assert (op.top_ids == -1).all() and (op.top_logp == -INF).all()
            out = torch.full_like(x, 7.0)
            op.backward(x, y, torch.ones(n, device=DEV), out)
            assert (out == 0).all()
        y = torch.full((n,), torch.iinfo(dtype).max, dtype=dtype, device=DEV)
        op.run(x, y)
        assert op.logp.isnan().all()
        op.backward(x, y, torch.ones(n, device=DEV), out)
        assert out.isnan().all()


def test_more_rows_than_a_grid_holds_turns():
    """1e6 rows, of one vector or two each."""
    log("1e6 rows")
    n, vocab = 1000003, 11
    g = torch.Generator(DEV)
    g.manual_seed(0)
    x = torch.randn(n, vocab, generator=g, device=DEV)
    y = torch.randint(0, vocab, (n,), generator=g, device=DEV)
    a = torch.randn(n, generator=g, device=DEV)
    op = TokenLogProbs(n, vocab, DEV, entropy=True)
    op.run(x, y)
    out = torch.empty_like(x)
    op.backward(x, y, a, out)
    some = torch.cat([torch.arange(500), torch.arange(n - 500, n)])
    want = ref.Rows(x.cpu()[some], y.cpu()[some])
    ref.check(op.logp.cpu()[some], want.logp, want.logp_off, "logp")
    ref.check(out.cpu()[some], *want.grad(a.cpu()[some], None, torch.float32), "grad")
    lp = torch.log_softmax(x.double(), 1).gather(1, y[:, None])[:, 0]
    assert (op.logp - lp).abs().max() < 1e-5


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2048, 2049, 16384, 16385, 17409, 262143, 262145,
                               600011])
def test_policy_loss_by_its_workgroups(n):
    log(f"policy {n}")
    op = PolicyLoss(n, DEV)
    s = _policy_inputs(n, n)
    for _ in range(2):
        _policy(op, s, f"n={n}", clip=(0.2, 0.3), kl_coef=0.1, entropy_coef=0.01, scale=1 / n)
    # and a shorter one through the same workspace
    s = {k: v[:n // 2] for k, v in s.items()}
    _policy(op, s, f"half of {n}", clip=(0.2, 0.2))


@pytest.mark.parametrize("kind,rows,experts,choices", [
    # rows of many tokens on few lanes, of several pieces each ...
    ("fp32", 16500, 37, 2), ("bf16", 16500, 71, 9), ("bf16", 8300, 137, 3), ("bf16", 8300, 260, 8),
    ("fp32", 8300, 140, 17), ("fp32", 8300, 253, 4), ("bf16", 4200, 391, 33), ("bf16", 4200, 766, 2),
    ("fp32", 4200, 500, 6), ("fp32", 300, 1021, 65), ("fp32", 4200, 300, 5), ("bf16", 600, 1020, 3),
    # ... and the same ones with more
    ("fp32", 9000, 37, 2), ("bf16", 1100, 71, 9), ("bf16", 4000, 137, 3), ("bf16", 4096, 260, 8),
    ("fp32", 8192, 253, 4), ("bf16", 4096, 391, 33), ("fp32", 30, 253, 4), ("bf16", 3, 391, 33)])
def test_balance_by_its_lanes(kind, rows, experts, choices):
    log(f"balance {kind} {rows}x{experts}")
    x, chosen, mask = _router(rows, experts, choices, rows, kind)
    x[rows // 2] = -math.inf
    op = RouterBalance(rows, experts, DEV, z_coef=0.01)
    want = ref.balance(x, chosen, mask, 0.01, 0.01)
    big = torch.full((rows + 2, experts + 3), 7.0, dtype=x.dtype, device=DEV)
    view = big[1:-1, 2:-1]
    view.copy_(x)
    for _ in range(2):
        op.run(view, chosen.to(DEV), mask=mask.to(DEV))
        _check_router(op, want, f"{rows}x{experts}")
    op.backward(view, view, mask=mask.to(DEV))    # in place
    ref.check(view, want["grad"], want["grad_off"], "grad")
    view.fill_(7.0)
    assert (big == 7.0).all()


@pytest.mark.parametrize("kind,rows,experts,choices", [
    ("fp32", 255, 64, 8), ("fp32", 257, 64, 8), ("fp32", 1025, 64, 2), ("fp32", 40009, 64, 4),
    ("bf16", 4099, 8, 2), ("bf16", 70001, 8, 1), ("bf16", 130, 520, 9), ("bf16", 5000, 264, 3),
    ("fp32", 66, 1000, 2), ("bf16", 4500, 1024, 2), ("fp32", 5001, 260, 6)])
def test_balance_by_its_workgroups(kind, rows, experts, choices):
    log(f"balance {kind} {rows}x{experts}")
    x, chosen, mask = _router(rows, experts, choices, rows, kind)
    op = RouterBalance(rows, experts, DEV, z_coef=0.01)
    want = ref.balance(x, chosen, mask, 0.01, 0.01)
    dx = x.to(DEV)
    out = torch.empty_like(dx)
    for _ in range(2):
        op.run(dx, chosen.to(DEV), mask=mask.to(DEV))
        _check_router(op, want, f"{rows}x{experts}")
        op.backward(dx, out, mask=mask.to(DEV))
        ref.check(out, want["grad"], want["grad_off"], "grad")


@pytest.mark.parametrize("rows", [40, 30000])
def test_balance_of_one_expert_and_of_none(rows):
    log(f"one expert {rows}")
    x, _, _ = _router(rows, 16, 1, 2, "fp32")
    op = RouterBalance(rows, 16, DEV)
    one = torch.full((rows, 3), 11, dtype=torch.int32, device=DEV)
    op.run(x.to(DEV), one)
    _check_router(op, ref.balance(x, one.cpu()), "one")
    for value in (-1, torch.iinfo(torch.int32).min):
        none = torch.full((rows, 3), value, dtype=torch.int32, device=DEV)
        op.run(x.to(DEV), none)
        assert (op.counts == 0).all() and op.balance == 0 and op.tokens == rows


def test_operators_for_no_rows():
    log("prepared for no rows")
    empty = torch.empty(0, device=DEV)
    for top, entropy in ((0, False), (3, True)):
        op = TokenLogProbs(0, 50, DEV, entropy=entropy, top=top)
        x, y = torch.empty(0, 50, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
        op.run(x, y)
        op.backward(x, y, empty, x)
        with pytest.raises(ValueError, match="prepared for 0"):
            op.run(torch.empty(1, 50, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV))
    loss = PolicyLoss(0, DEV)
    loss.result.fill_(7.0)
    loss.run(empty, empty, empty, entropy=empty)
    assert (loss.result[:5] == 0).all()
    router = RouterBalance(0, 50, DEV)
    router.counts.fill_(7)
    router.run(x, torch.empty(0, 2, dtype=torch.int32, device=DEV))
    router.backward(x, x)
    assert router.tokens == 0 and router.loss == 0 and (router.counts == 0).all()


def test_buffers_are_held_for_another_stream(monkeypatch):
    """A run on another stream than the buffers' own tells torch's allocator."""
    log("held")
    held = []
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: held.append((t.untyped_storage().data_ptr(), s.cuda_stream)))
    x, y = torch.randn(4, 50, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV)
    a = torch.zeros(4, device=DEV)
    probs, loss, router = TokenLogProbs(4, 50, DEV, top=1), PolicyLoss(4, DEV), \
        RouterBalance(4, 50, DEV)
    calls = [lambda: probs.run(x, y), lambda: probs.backward(x, y, a, torch.empty_like(x)),
             lambda: loss.run(a, a.clone(), a.clone()), lambda: router.run(x, y[:, None]),
             lambda: router.backward(x, torch.empty_like(x))]
    for call in calls:
        call()
    assert not held
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for call, op in zip(calls, (probs, probs, loss, router, router)):
            held.clear()
            call()
            assert held == [(op.result.untyped_storage().data_ptr() if op is not probs else
                             op.logp.untyped_storage().data_ptr(), side.cuda_stream)]
    torch.cuda.synchronize()
