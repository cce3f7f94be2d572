"""CPU checks of the losses' C ABI (bf16delta_loss.h) and binding: exports, struct
sizes and every refusal that the host makes before any GPU work.  The addresses are
made up; nothing is launched."""
import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bf16delta_loss.h")
BASE = 1 << 40      # 16-byte aligned addresses, far apart
NAN, INF = math.nan, math.inf
BAD_COEFS = (NAN, INF, -INF)


@pytest.fixture(scope="module")
def native():
    from lossless_bf16_weight_xor_amd import _native
    if not os.path.exists(_native.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return _native


def _at(k):
    return BASE + (k << 36)


def test_every_declared_symbol_is_exported(native):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(bf16d_[a-z_]+)\s*\(", text))
    assert names == set(native.LOSS_EXPORTED)
    lib = ctypes.CDLL(native.LIB_PATH)
    assert all(hasattr(lib, name) for name in names)


def test_struct_sizes_match_the_header(native):
    assert ctypes.sizeof(native.LogprobJob) == 2 * 24 + 2 * 8 + 4 * 4 + 8 + 5 * 8
    assert ctypes.sizeof(native.LogprobGradJob) == 3 * 24 + 2 * 8 + 4 * 4 + 3 * 8
    assert ctypes.sizeof(native.PolicyJob) == 9 * 8 + 5 * 8
    assert ctypes.sizeof(native.BalanceJob) == 6 * 8 + 4 * 4 + 3 * 8
    assert ctypes.sizeof(native.BalanceGradJob) == 6 * 8 + 2 * 4 + 6 * 8


def test_the_limits_match_the_header(native):
    text = open(HEADER).read()
    assert "BF16D_MAX_VOCAB   (1u << 28)" in text and native.MAX_VOCAB == 1 << 28
    assert "BF16D_MAX_TOP     64u" in text and native.MAX_TOP == 64
    assert "BF16D_MAX_EXPERTS 1024u" in text and native.MAX_EXPERTS == 1024


LOGPROB = dict(logits=_at(0), logits_outer=0, logits_inner=1000, tokens=_at(1), tokens_outer=0,
               tokens_inner=1, outer=1, inner=4, vocab=1000, logits_dtype=0, token_dtype=0, top=3,
               temperature=1.0, logp=_at(2), entropy=_at(3), stats=_at(4), top_ids=_at(5),
               top_logp=_at(6))


def _logprob(native, workspace=_at(9), size=1 << 20, **change):
    job = native.LogprobJob(**{**LOGPROB, **change})
    return native.lib().bf16d_logprob(ctypes.byref(job), workspace, size, None)


def test_logprob_refusals(native):
    E = native.EINVAL
    call = lambda **kw: _logprob(native, **kw)
    assert native.lib().bf16d_logprob(None, _at(9), 1 << 20, None) == E
    for name in ("logits", "tokens", "logp", "top_ids", "top_logp"):
        assert call(**{name: 0}) == E, name
    assert call(top=0) == E                              # arrays of alternatives without any
    assert call(logits=_at(0) + 1) == E and call(logits=_at(0) + 2, logits_dtype=1) == E
    assert call(tokens=_at(1) + 4) == E and call(tokens=_at(1) + 2, token_dtype=1) == E
    for name in ("logp", "entropy", "stats", "top_ids", "top_logp"):
        assert call(**{name: LOGPROB[name] + 8}) == E, name
    assert call(vocab=0) == E and call(vocab=(1 << 28) + 1) == E
    assert call(top=65) == E
    for name in ("logits_dtype", "token_dtype"):
        assert call(**{name: 2}) == E
    for t in (0.0, -1.0, NAN, INF, 2.0 ** -21, 2.0 ** 21):
        assert call(temperature=t) == E
    # rows: too many, and strides whose bytes pass 2^62
    for outer, inner in ((1, 1 << 24), (1 << 24, 1), (1 << 13, 1 << 13), (1 << 40, 1 << 40),
                         (0, 1 << 24)):
        assert call(outer=outer, inner=inner) == E
    assert call(inner=1 << 22) == E          # alternatives of as many rows
    for name in ("logits_inner", "tokens_inner"):
        for stride in (1 << 61, (1 << 64) - 1):
            assert call(**{name: stride}) == E
            assert call(**{name.replace("inner", "outer"): stride}, outer=4, inner=1) == E


def test_logprob_refuses_a_short_workspace(native):
    E = native.EINVAL
    # 4 rows of 5 turns each
    wide = dict(vocab=40000, logits_inner=40000)
    need = native.lib().bf16d_logprob_workspace_bytes(4, 40000, 3)
    assert need >= 4 * 256 + 4 * 5 * 5 * 8
    assert _logprob(native, size=4 * 256 + 4 * 5 * 5 * 8 - 8, **wide) == E
    assert _logprob(native, workspace=None, **wide) == E
    assert _logprob(native, workspace=_at(9) + 8, **wide) == E
    assert _logprob(native, workspace=_at(2), **wide) == E        # over an output


def test_logprob_refuses_overlaps(native):
    E = native.EINVAL
    written = {"logp": 16, "entropy": 16, "stats": 64, "top_ids": 96, "top_logp": 48}
    for a, size in written.items():
        for b in ("logits", "tokens", *written):
            if a != b:
                assert _logprob(native, **{b: LOGPROB[a] + size - 16}) == E, (a, b)
    # in the last row's last bytes, of both levels
    end = _at(0) + 2 * (3 * 1000 + 1000)
    assert _logprob(native, logp=end - 16) == E
    two = dict(outer=2, inner=2, logits_outer=5000, logits_inner=1000)
    assert _logprob(native, logp=_at(0) + 2 * (5000 + 2000) - 16, **two) == E


GRAD = dict(logits=_at(0), logits_outer=0, logits_inner=1000, tokens=_at(1), tokens_outer=0,
            tokens_inner=1, out=_at(2), out_outer=0, out_inner=1000, outer=1, inner=4,
            vocab=1000, logits_dtype=0, token_dtype=0, reserved=0, stats=_at(3), grad_logp=_at(4),
            grad_entropy=_at(5))


def _grad(native, **change):
    return native.lib().bf16d_logprob_backward(
        ctypes.byref(native.LogprobGradJob(**{**GRAD, **change})), None)


def test_logprob_backward_refusals(native):
    E = native.EINVAL
    assert native.lib().bf16d_logprob_backward(None, None) == E
    for name in ("logits", "tokens", "out", "stats", "grad_logp"):
        assert _grad(native, **{name: 0}) == E, name
    assert _grad(native, out=_at(2) + 1) == E and _grad(native, out=_at(2) + 2, logits_dtype=1) == E
    assert _grad(native, stats=_at(3) + 8) == E
    assert _grad(native, grad_logp=_at(4) + 2) == E and _grad(native, grad_entropy=_at(5) + 1) == E
    assert _grad(native, vocab=0) == E and _grad(native, vocab=(1 << 28) + 1) == E
    assert _grad(native, reserved=1) == E
    for name in ("logits_dtype", "token_dtype"):
        assert _grad(native, **{name: 2}) == E
    assert _grad(native, inner=1 << 24) == E
    # rows of the output that share elements
    for change in (dict(out_inner=999), dict(out_inner=0),
                   dict(outer=2, inner=2, out_outer=1999, out_inner=1000),
                   dict(outer=2, inner=2, out_outer=1000, out_inner=1000),
                   dict(outer=2, inner=2, out_outer=1000, out_inner=1999),
                   dict(outer=2, inner=2, out_outer=0, out_inner=1000)):
        assert _grad(native, **change) == E, change
    # partly over the logits, over what is read, in place with other strides
    assert _grad(native, out=_at(0) + 16) == E
    assert _grad(native, out=_at(0), out_inner=1008) == E
    assert _grad(native, out=_at(0) + 2 * 1000, logits_inner=2000, out_inner=2000) == E
    for name in ("tokens", "stats", "grad_logp", "grad_entropy"):
        assert _grad(native, out=GRAD[name]) == E, name


POLICY = dict(logp=_at(0), old=_at(1), advantages=_at(2), weights=_at(3), ref=_at(4),
              entropy=_at(5), grad_logp=_at(6), grad_entropy=_at(7), n=100, clip_low=0.2,
              clip_high=0.2, kl_coef=0.1, entropy_coef=0.1, scale=1.0)


def _policy(native, result=_at(8), workspace=_at(9), size=1 << 20, **change):
    return native.lib().bf16d_policy_loss(ctypes.byref(native.PolicyJob(**{**POLICY, **change})),
                                          result, workspace, size, None)


def test_policy_refusals(native):
    E = native.EINVAL
    need = native.lib().bf16d_policy_loss_workspace_bytes()
    assert native.lib().bf16d_policy_loss(None, _at(8), _at(9), need, None) == E
    assert _policy(native, size=need - 1) == E
    assert _policy(native, workspace=None) == E and _policy(native, workspace=_at(9) + 8) == E
    assert _policy(native, result=None) == E and _policy(native, result=_at(8) + 8) == E
    for name in ("logp", "old", "advantages", "grad_logp", "ref", "entropy"):
        assert _policy(native, **{name: 0}) == E, name
    for name in ("logp", "old", "advantages", "weights", "ref", "entropy"):
        assert _policy(native, **{name: POLICY[name] + 2}) == E, name
    for name in ("grad_logp", "grad_entropy"):
        assert _policy(native, **{name: POLICY[name] + 8}) == E, name
    for x in (-0.1, 1.0, NAN, INF):
        assert _policy(native, clip_low=x) == E
    for x in (-0.1, NAN, -INF):
        assert _policy(native, clip_high=x) == E
    for name in ("kl_coef", "entropy_coef", "scale"):
        for x in BAD_COEFS:
            assert _policy(native, **{name: x}) == E, name
    assert _policy(native, n=1 << 40) == E
    for name in ("logp", "old", "advantages", "weights", "ref", "entropy"):
        for out in ("grad_logp", "grad_entropy"):
            assert _policy(native, **{out: POLICY[name] + 384}) == E, (name, out)
        assert _policy(native, result=POLICY[name]) == E
        assert _policy(native, workspace=POLICY[name]) == E
    assert _policy(native, grad_entropy=_at(6)) == E
    assert _policy(native, workspace=_at(8)) == E


BALANCE = dict(logits=_at(0), chosen=_at(1), mask=_at(2), rows=10, logits_stride=8,
               chosen_stride=2, experts=8, choices=2, logits_dtype=0, chosen_dtype=0,
               balance_coef=0.01, z_coef=0.0, counts=_at(3))


def _balance(native, result=_at(8), workspace=_at(9), size=1 << 20, **change):
    return native.lib().bf16d_balance(ctypes.byref(native.BalanceJob(**{**BALANCE, **change})),
                                      result, workspace, size, None)


def test_balance_refusals(native):
    E = native.EINVAL
    need = native.lib().bf16d_balance_workspace_bytes(8)
    assert native.lib().bf16d_balance(None, _at(8), _at(9), need, None) == E
    assert _balance(native, size=need - 1) == E
    assert _balance(native, workspace=None) == E and _balance(native, workspace=_at(9) + 8) == E
    assert _balance(native, result=None) == E and _balance(native, result=_at(8) + 8) == E
    for name in ("logits", "chosen", "counts"):
        assert _balance(native, **{name: 0}) == E, name
    assert _balance(native, logits=_at(0) + 1) == E
    assert _balance(native, logits=_at(0) + 2, logits_dtype=1) == E
    assert _balance(native, chosen=_at(1) + 4) == E and _balance(native, counts=_at(3) + 8) == E
    assert _balance(native, experts=0) == E and _balance(native, experts=1025) == E
    assert _balance(native, choices=0) == E and _balance(native, choices=9) == E
    assert _balance(native, logits_dtype=2) == E and _balance(native, chosen_dtype=2) == E
    assert _balance(native, rows=1 << 24) == E
    for name in ("logits_stride", "chosen_stride"):
        for x in (1 << 60, (1 << 64) - 1):
            assert _balance(native, **{name: x}) == E
    for name in ("balance_coef", "z_coef"):
        for x in BAD_COEFS:
            assert _balance(native, **{name: x}) == E
    for other in ("logits", "chosen", "mask"):
        assert _balance(native, counts=BALANCE[other]) == E
        assert _balance(native, result=BALANCE[other]) == E
        assert _balance(native, workspace=BALANCE[other]) == E
    assert _balance(native, result=_at(3) + 48) == E


BALANCE_GRAD = dict(logits=_at(0), out=_at(1), mask=_at(2), rows=10, logits_stride=8,
                    out_stride=8, experts=8, logits_dtype=0, balance_coef=0.01, z_coef=0.1,
                    scale=1.0, counts=_at(3), tokens=_at(4), result=_at(5))


def _balance_grad(native, **change):
    return native.lib().bf16d_balance_backward(
        ctypes.byref(native.BalanceGradJob(**{**BALANCE_GRAD, **change})), None)


def test_balance_backward_refusals(native):
    E = native.EINVAL
    call = lambda **kw: _balance_grad(native, **kw)
    assert native.lib().bf16d_balance_backward(None, None) == E
    for name in ("logits", "out", "counts", "tokens"):
        assert call(**{name: 0}) == E, name
    assert call(out=_at(1) + 1) == E and call(counts=_at(3) + 4) == E
    assert call(tokens=_at(4) + 4) == E and call(result=_at(5) + 4) == E
    assert call(experts=0) == E and call(experts=1025) == E and call(logits_dtype=2) == E
    assert call(rows=1 << 24) == E and call(out_stride=7) == E and call(out_stride=1 << 61) == E
    for name in ("balance_coef", "z_coef", "scale"):
        for x in BAD_COEFS:
            assert call(**{name: x}) == E
    assert call(balance_coef=1e30, scale=1e30) == E and call(z_coef=1e30, scale=1e30) == E
    assert call(out=_at(0) + 2) == E and call(out=_at(0), out_stride=9) == E
    for name in ("mask", "counts", "tokens", "result"):
        assert call(out=BALANCE_GRAD[name]) == E, name


def test_workspaces_grow_with_the_call(native):
    f = native.lib().bf16d_logprob_workspace_bytes
    assert f(0, 100000, 5) == 0 and f(100, 0, 0) == 0
    assert f(100, 4093, 5) == 0             # one turn at any alignment: nothing to join
    assert 0 < f(1, 100000, 0) < f(1, 100000, 5) <= f(2, 100000, 5) <= f(10 ** 6, 100000, 5)
    assert f(10 ** 6, 1 << 28, 64) < 2 << 20
    # what a call of fewer rows needs is never more: rows * parts, for every number of rows
    for turns in (2, 3, 7, 33, 5000):
        vocab = turns * 4096
        for rows in (1, 2, 3, 5, 31, 100, 500, 1000, 1023, 1024, 5000):
            words = (f(rows, vocab, 3) - 1024) // 8
            for fewer in {k for k in (1, 2, rows // 2, rows - 1, rows) if 0 < k <= rows}:
                parts = min(-(-256 // fewer), turns)
                if parts > 1:
                    assert words >= fewer * parts * 5, (turns, rows, fewer)
    g = native.lib().bf16d_balance_workspace_bytes
    assert 0 < g(1) < g(64) < g(1024) == g(5000)


def test_python_api_refuses_cpu_tensors_and_bad_sizes(native):
    from lossless_bf16_weight_xor_amd import PolicyLoss, RouterBalance, TokenLogProbs
    for make in (lambda d: TokenLogProbs(4, 100, d), lambda d: PolicyLoss(4, d),
                 lambda d: RouterBalance(4, 8, d)):
        with pytest.raises(TypeError, match="HIP device"):
            make("cpu")
    for vocab in (0, -1, (1 << 28) + 1):
        with pytest.raises(ValueError, match="vocab"):
            TokenLogProbs(4, vocab)
    for top in (-1, 65):
        with pytest.raises(ValueError, match="top"):
            TokenLogProbs(4, 100, top=top)
    for experts in (0, 1025):
        with pytest.raises(ValueError, match="experts"):
            RouterBalance(4, experts)
    with pytest.raises(ValueError, match="below 2\\^22"):
        TokenLogProbs(1 << 22, 100, top=1)
    for rows in (-1, 1 << 24):
        for make in (lambda: TokenLogProbs(rows, 100, "cuda:0"), lambda: PolicyLoss(rows, "cuda:0"),
                     lambda: RouterBalance(rows, 8, "cuda:0")):
            with pytest.raises(ValueError, match="rows"):
                make()
