"""The losses on the GPU (bf16delta_loss.h), each against its definition in 64 bits
(tests/loss_reference.py, which derives the bounds), and a whole update: logits,
losses, gradients, norm, step, compress, decompress, logits again."""
import math

import pytest
import torch

import lossless_bf16_weight_xor_amd as bd
from lossless_bf16_weight_xor_amd import PolicyLoss, RouterBalance, TokenLogProbs
from tests import loss_reference as ref
from tests.gpu_util import log

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
INF, NAN = math.inf, math.nan
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
both_types = pytest.mark.parametrize("kind", ["bf16", "fp32"])


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _logits(n, vocab, seed, kind, spread=2.5):
    """Flat and peaked rows (CPU), some entries of -infinity."""
    g = _gen(seed)
    x = torch.randn(n, vocab, generator=g) * (0.3 + spread * torch.rand(n, 1, generator=g))
    if vocab > 8:
        x[torch.rand(n, vocab, generator=g) < 0.01] = -INF
        x[:, vocab // 2] = 4.0
    return x.to(TYPES[kind])


def _tokens(n, vocab, seed):
    return torch.randint(0, vocab, (n,), generator=_gen(seed + 1))


def _coefs(n, seed):
    g = _gen(seed + 2)
    return torch.randn(n, generator=g), 0.3 * torch.randn(n, generator=g)


def _check_forward(op, want, n, what, top=0):
    ref.check(op.logp[:n], want.logp, want.logp_off, what + " logp")
    if op.entropy is not None:
        ref.check(op.entropy[:n], want.entropy[:, 0], want.h_off[:, 0], what + " entropy")
    if top:
        assert torch.equal(op.top_ids[:n].cpu(), want.top_ids), what + " top_ids"
        ref.check(op.top_logp[:n], want.top_logp, want.top_off, what + " top_logp")


def _one(kind, n, vocab, seed, entropy=True, top=0, temperature=1.0, grad=True):
    x, y = _logits(n, vocab, seed, kind), _tokens(n, vocab, seed)
    what = f"{kind} {n}x{vocab} entropy={entropy} top={top} T={temperature}"
    log(what)
    op = TokenLogProbs(n, vocab, DEV, entropy=entropy, top=top)
    dx, dy = x.to(DEV), y.to(DEV)
    op.run(dx, dy, temperature=temperature)
    want = ref.Rows(x, y, temperature, top=min(top, vocab))
    if top > vocab:
        assert (op.top_ids[:, vocab:] == -1).all() and (op.top_logp[:, vocab:] == -INF).all()
        op.top_ids, op.top_logp = op.top_ids[:, :vocab], op.top_logp[:, :vocab]
    _check_forward(op, want, n, what, top)
    if grad:
        a, h = _coefs(n, seed)
        out = torch.full_like(dx, 7.0)
        op.backward(dx, dy, a.to(DEV), out, grad_entropy=h.to(DEV) if entropy else None)
        ref.check(out, *want.grad(a, h if entropy else None, x.dtype), what + " grad")
    return op, want


# every edge of a vector, a wave, a workgroup's turn, and rows of many turns
VOCABS = [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 63, 65, 255, 1003, 2048, 4095, 4096, 4097, 8191,
          8192, 8193, 12289, 40003]


@both_types
@pytest.mark.parametrize("vocab", VOCABS)
def test_every_edge_of_a_row(kind, vocab):
    _one(kind, 3, vocab, vocab, top=min(5, vocab))
    _one(kind, 2, vocab, vocab + 7, entropy=False, temperature=0.7)


@both_types
@pytest.mark.parametrize("n,vocab", [(1, 131077), (2, 70001), (31, 30011), (600, 9001),
                                     (1023, 9000), (1025, 8200), (1500, 40)])
def test_rows_in_parts_and_whole(kind, n, vocab):
    _one(kind, n, vocab, n, top=3 if n < 100 else 0)


@both_types
@pytest.mark.parametrize("top", [1, 2, 20, 63, 64])
def test_every_number_of_alternatives(kind, top):
    _one(kind, 4, 33000, top, entropy=top % 2 == 0, top=top, grad=False)
    _one(kind, 3, 50, top, top=top, grad=False)


@both_types
@pytest.mark.parametrize("temperature", [2.0 ** -20, 0.01, 0.3, 1.7, 50.0, 2.0 ** 20])
def test_temperatures(kind, temperature):
    _one(kind, 5, 3001, 11, top=4, temperature=temperature)


@both_types
def test_alternatives_of_rows_in_order(kind):
    """Rows that rise, fall, or hold few values: every element may be among the
    largest when it is read, and equal ones go by their ids."""
    vocab, top = 20000, 40
    rise = torch.arange(vocab, dtype=torch.float32) / 64
    rows = [rise, rise.flip(0), torch.zeros(vocab), -rise.abs() % 3, (rise * 64) % 2,
            torch.where(torch.arange(vocab) % 1000 == 999, 1.0, 0.0),
            torch.where(torch.arange(vocab) % 2 == 0, -0.0, 0.0),
            torch.where(torch.arange(vocab) >= vocab - 10, 0.0, -INF),
            torch.where(torch.arange(vocab) % 512 < 8, rise, rise - 500)]
    x = torch.stack(rows).to(TYPES[kind])
    y = torch.full((len(rows),), vocab - 1)
    for n in (len(rows), 1):
        op = TokenLogProbs(n, vocab, DEV, top=top)
        for first in range(0, len(rows), n):
            log(f"{kind} rows from {first}")
            op.run(x[first:first + n].to(DEV), y[first:first + n].to(DEV))
            _check_forward(op, ref.Rows(x[first:first + n], y[first:first + n], top=top), n,
                           f"row {first}", top)


@both_types
@pytest.mark.parametrize("vocab", [50, 40000])
def test_rows_that_are_special(kind, vocab):
    """Left out, empty, masked with the lowest value, of one value, with NaN or infinity."""
    log(f"{kind} {vocab}")
    low = torch.finfo(TYPES[kind]).min
    x = _logits(12, vocab, 5, kind)
    y = _tokens(12, vocab, 5)
    x[:, vocab // 2] = 4.0
    x[torch.arange(12), y] = 2.0
    x[0] = NAN                 # left out
    y[0] = -1
    x[1] = -INF                # empty
    x[2] = low                 # masked whole: even
    x[3] = low
    x[3, 7], y[3] = 1.5, 7     # one is left
    x[4] = -INF
    x[4, 9], y[4] = -2.0, 9    # the same by -infinity
    x[5, y[5]] = -INF          # a token that cannot occur
    x[6, 3] = NAN
    x[7, 3] = INF
    x[8] = -low                # the largest value, even
    y[9] = vocab               # no token
    x[10] = 0.0
    x[10, 1::2] = -low
    y[10] = 1
    top = 5
    op = TokenLogProbs(12, vocab, DEV, entropy=True, top=top)
    dx, dy = x.to(DEV), y.to(DEV)
    op.run(dx, dy)
    lp, h, ids, alt = (t.cpu() for t in (op.logp, op.entropy, op.top_ids, op.top_logp))
    fine = torch.tensor([2, 3, 4, 5, 8, 10, 11])
    want = ref.Rows(x[fine], y[fine], top=top)
    ref.check(lp[fine], want.logp, want.logp_off, "logp")
    ref.check(h[fine], want.entropy[:, 0], want.h_off[:, 0], "entropy")
    assert torch.equal(ids[fine], want.top_ids)
    ref.check(alt[fine], want.top_logp, want.top_off, "top_logp")
    assert lp[0] == 0 and h[0] == 0 and lp[1] == -INF and h[1] == 0
    assert (ids[:2] == -1).all() and (alt[:2] == -INF).all()
    assert lp[5] == -INF and lp[4] == 0 and h[4] == 0 and ids[4].tolist() == [9, -1, -1, -1, -1]
    assert ids[3].tolist() == [7, 0, 1, 2, 3]
    for row in (6, 7):
        assert lp[row].isnan() and h[row].isnan() and alt[row].isnan().all()
        assert 3 not in ids[6]
    assert lp[9].isnan() and h[9].isfinite() and alt[9].isfinite().all()

    a, g = _coefs(12, 9)
    a[11] = g[11] = 0.0        # nothing to pass on
    x[11, 4] = NAN
    dx = x.to(DEV)
    out = torch.full_like(dx, 7.0)
    op.backward(dx, dy, a.to(DEV), out, grad_entropy=g.to(DEV))
    got = out.cpu()
    assert (got[[0, 1, 11]] == 0).all()
    assert got[[6, 7, 9]].isnan().all()
    grad, off = want.grad(a[fine], g[fine], x.dtype)
    ref.check(got[fine[:-1]], grad[:-1], off[:-1], "grad")
    # in place over the logits, without the entropy
    op.backward(dx, dy, a.to(DEV), dx)
    got = dx.cpu()
    assert (got[[0, 1, 11]] == 0).all() and got[[6, 7, 9]].isnan().all()
    grad, off = want.grad(a[fine], None, x.dtype)
    ref.check(got[fine[:-1]], grad[:-1], off[:-1], "grad in place")


@both_types
@pytest.mark.parametrize("vocab", [50, 40000])
def test_log_probabilities_below_the_range_of_fp32(kind, vocab):
    """The lowest value over a small temperature: -infinity as a number, finite in a gradient."""
    log(f"{kind} {vocab}")
    low = torch.finfo(TYPES[kind]).min
    x = _logits(4, vocab, 31, kind)
    y = _tokens(4, vocab, 31)
    x[0, 1:] = low             # one of weight, the given token another
    y[0] = 3
    x[1] = low                 # even: nothing is below the range
    x[2, ::2] = low
    x[2, y[2]] = 1.0
    x[3, y[3]] = low
    top = 5
    op = TokenLogProbs(4, vocab, DEV, entropy=True, top=top)
    dx, dy = x.to(DEV), y.to(DEV)
    op.run(dx, dy, temperature=0.05)
    want = ref.Rows(x, y, 0.05, top=top)
    # what lies below -max rounds to -infinity in fp32
    below = lambda t: t < -torch.finfo(torch.float32).max
    for got, value, off in ((op.logp.cpu(), want.logp, want.logp_off),
                            (op.top_logp.cpu(), want.top_logp, want.top_off)):
        assert (got[below(value)] == -INF).all()
        ref.check(got[~below(value)], value[~below(value)], off[~below(value)], "logp")
    assert below(want.logp).tolist() == [True, False, False, True]
    assert torch.equal(op.top_ids.cpu(), want.top_ids)
    ref.check(op.entropy.cpu(), want.entropy[:, 0], want.h_off[:, 0], "entropy")
    a, g = _coefs(4, 9)
    out = torch.full_like(dx, 7.0)
    op.backward(dx, dy, a.to(DEV), out, grad_entropy=g.to(DEV))
    grad, off = want.grad(a, g, x.dtype)
    ref.check(out.cpu(), grad, off, "grad")


def _strided(kind, vocab, seed):
    """Views of wider buffers: (name, logits, tokens, out) factories over (3, 5) rows."""
    dt = TYPES[kind]
    x, y = _logits(15, vocab, seed, kind).view(3, 5, vocab), _tokens(15, vocab, seed).view(3, 5)
    fill = lambda *s: torch.full(s, 7.0, dtype=dt, device=DEV)
    big, ids = fill(3, 6, vocab), torch.zeros(3, 6, dtype=torch.int64, device=DEV)
    big[:, :-1], ids[:, 1:] = x.to(DEV), y.to(DEV)
    yield "shifted", x, y, big[:, :-1], ids[:, 1:], fill(3, 6, vocab)[:, :-1]
    wide = fill(3, 5, vocab + 11)
    wide[..., 3:vocab + 3] = x.to(DEV)
    yield "inside", x, y, wide[..., 3:vocab + 3], y.to(DEV).int(), fill(3, 5, vocab + 5)[..., 1:-4]
    turned = x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    yield "turned", x, y, turned, y.t().contiguous().to(DEV).t(), \
        fill(5, 3, vocab).transpose(0, 1)
    yield "same row", x[:1, :1].expand(3, 5, vocab), y[:1, :1].expand(3, 5), \
        x[:1, :1].to(DEV).expand(3, 5, vocab), y[:1, :1].to(DEV).expand(3, 5), fill(3, 5, vocab)
    every = fill(30, vocab)
    every[::2] = x.view(15, vocab).to(DEV)
    yield "every second", x.view(15, vocab), y.view(15), every[::2], \
        y.view(15).to(DEV).int().repeat_interleave(3)[::3], fill(45, vocab)[::3]


@both_types
@pytest.mark.parametrize("vocab", [13, 1000, 9001])
def test_strides_and_alignments(kind, vocab):
    a, h = _coefs(15, 3)
    for name, x, y, dx, dy, out in _strided(kind, vocab, vocab):
        log(f"{kind} {vocab} {name}")
        op = TokenLogProbs(20, vocab, DEV, entropy=True, top=2)
        op.logp.fill_(5.0)
        op.top_ids.fill_(-7)
        op.run(dx, dy)
        want = ref.Rows(x.reshape(15, vocab), y.reshape(15), top=2)
        _check_forward(op, want, 15, name, 2)
        assert (op.logp[15:] == 5.0).all() and (op.top_ids[15:] == -7).all()   # as they were
        before = out._base.clone() if out._base is not None else None
        op.backward(dx, dy, a.to(DEV), out, grad_entropy=h.to(DEV))
        g, off = want.grad(a, h, x.dtype)
        ref.check(out.reshape(15, vocab), g, off, name + " grad")
        if before is not None:      # and nothing beside it is written
            out.fill_(7.0)
            assert torch.equal(out._base, before), name
        if name in ("shifted", "inside", "turned"):      # in place
            base = dx._base if dx._base is not None else dx
            kept = base.clone()
            view = kept.as_strided(dx.shape, dx.stride(), dx.storage_offset())
            op.backward(dx, dy, a.to(DEV), dx, grad_entropy=h.to(DEV))
            ref.check(dx.reshape(15, vocab), g, off, name + " grad in place")
            view.copy_(dx)
            assert torch.equal(base, kept), name


def test_the_logits_gradient_is_that_of_differences():
    """Of the kernel's own values, in fp32: the loss moves by the gradient times a step."""
    log("differences")
    n, vocab = 6, 600
    x, y = _logits(n, vocab, 21, "fp32"), _tokens(n, vocab, 21)
    x[x == -INF] = -3.0
    a, h = _coefs(n, 21)
    op = TokenLogProbs(n, vocab, DEV, entropy=True)
    dx, dy = x.to(DEV), y.to(DEV)
    op.run(dx, dy, temperature=1.3)
    out = torch.empty_like(dx)
    op.backward(dx, dy, a.to(DEV), out, grad_entropy=h.to(DEV))
    for k in range(4):
        way = torch.randn(n, vocab, generator=_gen(k))
        way /= way.norm()
        step = 0.03
        value = []
        for s in (step, -step):
            op.run((x + s * way).to(DEV), dy, temperature=1.3)
            value.append((a.double() * op.logp.cpu().double()
                          + h.double() * op.entropy.cpu().double()).sum())
        slope = (value[0] - value[1]) / (2 * step)
        want = (out.cpu().double() * way.double()).sum()
        # third derivatives of a unit direction stay below 10 (|a| + |h| ln V) / T^3;
        # the values are good to 1e-5
        size = (a.abs() + 7 * h.abs()).sum()
        assert abs(slope - want) < step ** 2 * 10 / 6 * size + 2e-5 * size / step


@both_types
def test_no_rows_and_too_many(kind):
    log("no rows")
    op = TokenLogProbs(4, 100, DEV, entropy=True, top=2)
    empty = torch.empty(0, 100, dtype=TYPES[kind], device=DEV)
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    op.run(empty, ids)
    op.backward(empty, ids, torch.empty(0, device=DEV), empty)
    op.run(torch.empty(0, 3, 100, dtype=TYPES[kind], device=DEV), ids.view(0, 3))
    x = torch.zeros(5, 100, dtype=TYPES[kind], device=DEV)
    with pytest.raises(ValueError, match="prepared for 4"):
        op.run(x, torch.zeros(5, dtype=torch.int64, device=DEV))


def test_refusals_of_the_binding():
    log("refusals")
    op = TokenLogProbs(4, 100, DEV)
    x = torch.zeros(4, 100, device=DEV)
    y = torch.zeros(4, dtype=torch.int64, device=DEV)
    a = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError, match="last run"):
        op.backward(x, y, a, x)
    op.run(x, y)
    for bad in (x.half(), x.double(), x.cpu(), None):
        with pytest.raises(TypeError):
            op.run(bad, y)
    for bad in (x[:, :99], x[:3], x.t().contiguous().t(), x[0], x.view(4, 1, 1, 100)):
        with pytest.raises(ValueError):
            op.run(bad, y)
    for bad in (y.float(), y.cpu(), y.short()):
        with pytest.raises(TypeError):
            op.run(x, bad)
    with pytest.raises(ValueError):
        op.run(x, y[:3])
    for t in (0.0, -1.0, NAN, INF):
        with pytest.raises(ValueError, match="temperature"):
            op.run(x, y, temperature=t)
    with pytest.raises(ValueError, match="last run had 4"):
        op.backward(x[:3], y[:3], a[:3], x[:3])
    with pytest.raises(ValueError, match="entropy=True"):
        op.backward(x, y, a, x, grad_entropy=a)
    with pytest.raises(TypeError):
        op.backward(x, y, a, x.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        op.backward(x, y, a, torch.zeros(5, 100, device=DEV))
    for bad in (a[:3], torch.zeros(8, device=DEV)[::2]):
        with pytest.raises(ValueError):
            op.backward(x, y, bad, x)
    # rows of the output that are one, or that lie over the logits
    with pytest.raises(RuntimeError, match="EINVAL"):
        op.backward(x, y, a, torch.zeros(1, 100, device=DEV).expand(4, 100))
    both = torch.zeros(5, 100, device=DEV)
    with pytest.raises(RuntimeError, match="EINVAL"):
        op.backward(both[:4], y, a, both[1:])
    loss = PolicyLoss(4, DEV)
    with pytest.raises(ValueError, match="ref_logp"):
        loss.run(a, a.clone(), a.clone(), kl_coef=0.1)
    with pytest.raises(ValueError, match="entropy"):
        loss.run(a, a.clone(), a.clone(), entropy_coef=0.1)
    for clip in ((1.0, 0.2), (-0.1, 0.2), (0.2, -0.1), (NAN, 0.2)):
        with pytest.raises(RuntimeError, match="EINVAL"):
            loss.run(a, a, a, clip=clip)
    with pytest.raises(ValueError):
        loss.run(a, a[:3], a)
    with pytest.raises(TypeError):
        loss.run(a.double(), a, a)
    with pytest.raises(ValueError, match="prepared for 4"):
        loss.run(torch.zeros(5, device=DEV), a, a)
    router = RouterBalance(4, 100, DEV)
    with pytest.raises(ValueError, match="run"):
        router.backward(x, x)
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    for bad in (ids[:3], ids[0], torch.zeros(4, 101, dtype=torch.int64, device=DEV)):
        with pytest.raises(ValueError):
            router.run(x, bad)
    with pytest.raises(TypeError):
        router.run(x, ids.float())
    with pytest.raises(ValueError):
        router.run(x[:, :99], ids)
    with pytest.raises(TypeError):
        router.run(x, ids, mask=torch.ones(4, device=DEV))
    with pytest.raises(ValueError):
        router.run(x, ids, mask=torch.ones(3, dtype=torch.bool, device=DEV))


# ------------------------------------------------------------- policy loss ---

def _policy_inputs(n, seed):
    g = _gen(seed)
    old = -3 * torch.rand(n, generator=g)
    lp = old + 0.25 * torch.randn(n, generator=g)
    adv = torch.randn(n, generator=g)
    w = torch.rand(n, generator=g) * (torch.rand(n, generator=g) > 0.2)
    return dict(logp=lp, old=old, adv=adv, weights=w, ref=lp + 0.2 * torch.randn(n, generator=g),
                entropy=2 * torch.rand(n, generator=g))


def _policy(op, s, what, **kw):
    to = lambda k: None if s.get(k) is None else s[k].to(DEV)
    n = s["logp"].numel()
    op.run(to("logp"), to("old"), to("adv"), weights=to("weights"), ref_logp=to("ref"),
           entropy=to("entropy"), **kw)
    want = ref.policy(**s, **kw)
    for name in ("loss", "weight", "kl", "clipped", "entropy"):
        ref.check(getattr(op, name), want[name], want["off"][name], f"{what} {name}")
    for name in ("grad_logp",) + ("grad_entropy",) * (s.get("entropy") is not None):
        off = ref.U * 1.01 * want[name].abs() + 2.0 ** -149
        ref.check(getattr(op, name)[:n], want[name], off, f"{what} {name}")
    return want


@pytest.mark.parametrize("n", [0, 1, 2, 63, 64, 65, 255, 256, 257, 4096, 65535, 65536, 65537,
                               200001])
def test_policy_loss(n):
    log(f"policy {n}")
    op = PolicyLoss(n + 3, DEV)
    op.grad_logp.fill_(5.0)
    s = _policy_inputs(n, n)
    want = _policy(op, s, f"n={n}", clip=(0.2, 0.3), kl_coef=0.1, entropy_coef=0.01, scale=0.3)
    assert n < 100 or 0.05 < want["clipped"] < 0.95
    assert (op.grad_logp[n:] == 5.0).all()
    # and without the terms that may be left out
    s = s | {"weights": None, "ref": None, "entropy": None}
    _policy(op, s, f"n={n} plain", clip=(0.1, INF))


def test_policy_loss_of_special_tokens():
    """Weights of 0 hide anything; ratios at the ends; advantages of 0; no weight at all."""
    log("special tokens")
    lp = torch.tensor([NAN, -INF, -INF, -1.0, -200.0, -0.5, -INF, -1.0, -1.0, 0.0, -2.0])
    old = torch.tensor([0.0, NAN, -1.0, -200.0, -1.0, -0.5, -2.0, -1.0, -3.0, -0.0, -1.0])
    adv = torch.tensor([1.0, INF, 1.0, 2.0, -2.0, 0.0, -1.0, 0.0, 0.0, -0.0, 1e30])
    w = torch.tensor([0.0, 0.0, 1.0, 1.0, 1.0, 1.0, 1.0, 0.5, 0.5, 1.0, 1e-3])
    op = PolicyLoss(11, DEV)
    _policy(op, dict(logp=lp, old=old, adv=adv, weights=w), "special", clip=(0.2, 0.2))
    assert (op.grad_logp[:2] == 0).all()
    s = _policy_inputs(300, 5) | {"weights": torch.zeros(300)}
    s["logp"][7] = NAN
    _policy(op_all := PolicyLoss(300, DEV), s, "no weight", kl_coef=1.0, entropy_coef=1.0)
    assert all(getattr(op_all, k) == 0 for k in ("loss", "weight", "kl", "clipped", "entropy"))
    # NaN where it counts is seen
    s["weights"][7] = 1.0
    op_all.run(*(s[k].to(DEV) for k in ("logp", "old", "adv")), weights=s["weights"].to(DEV))
    assert op_all.loss.isnan() and op_all.grad_logp[7].isnan()
    assert op_all.grad_logp[:7].isfinite().all()
    # a large advantage against an unbounded ratio
    big = dict(logp=torch.tensor([0.0]), old=torch.tensor([-800.0]), adv=torch.tensor([-1.0]))
    op.run(*(t.to(DEV) for t in big.values()))
    assert op.loss == INF and op.grad_logp[0] == INF


def test_a_ratio_on_the_border_is_not_clipped():
    log("border")
    # clip bounds whose logarithms are exact: the ratio is 1 + clip as far as 64 bits go
    old = torch.zeros(4)
    lp = torch.tensor([0.25, -0.25, 0.25, -0.25])
    adv = torch.tensor([1.0, -1.0, -1.0, 1.0])
    high, low = math.expm1(0.25), -math.expm1(-0.25)
    op = PolicyLoss(4, DEV)
    for way, cut in ((1e-12, 0.0), (-1e-12, 0.5)):
        op.run(lp.to(DEV), old.to(DEV), adv.to(DEV), clip=(low + way, high + way))
        assert op.clipped.item() == cut


@pytest.mark.parametrize("n", [5, 70000])
def test_policy_loss_is_repeatable(n):
    log(f"repeatable {n}")
    s = {k: v.to(DEV) for k, v in _policy_inputs(n, 8).items()}
    op = PolicyLoss(n, DEV)
    seen = set()
    for _ in range(5):
        op.run(s["logp"], s["old"], s["adv"], weights=s["weights"])
        seen.add((op.loss.item(), op.kl.item(), op.clipped.item()))
    assert len(seen) == 1


# ---------------------------------------------------------------- balance ---

def _router(rows, experts, choices, seed, kind):
    g = _gen(seed)
    x = (torch.randn(rows, experts, generator=g) * (0.5 + torch.rand(rows, 1, generator=g))
         + torch.randn(experts, generator=g)).to(TYPES[kind])
    chosen = x.float().topk(choices, dim=1).indices if rows else \
        torch.empty(0, choices, dtype=torch.int64)
    return x, chosen, torch.rand(rows, generator=g) > 0.1


def _check_router(op, want, what):
    assert torch.equal(op.counts.cpu(), want["counts"]), what
    assert op.tokens.item() == want["tokens"].item(), what
    for name in ("balance", "z", "loss"):
        ref.check(getattr(op, name), want[name], want["off"][name], f"{what} {name}")


@both_types
@pytest.mark.parametrize("rows,experts,choices", [
    (0, 8, 2), (1, 1, 1), (1, 8, 2), (3, 2, 1), (5, 3, 3), (64, 8, 2), (100, 31, 4), (100, 32, 4),
    (100, 33, 4), (777, 63, 8), (777, 64, 8), (777, 65, 8), (500, 127, 2), (500, 129, 7),
    (300, 256, 8), (300, 257, 8), (200, 511, 9), (200, 513, 6), (90, 1023, 3), (90, 1024, 70),
    (5000, 16, 2), (3001, 6, 6)])
def test_balance(kind, rows, experts, choices):
    what = f"{kind} {rows}x{experts} {choices} chosen"
    log(what)
    x, chosen, mask = _router(rows, experts, choices, rows + experts, kind)
    op = RouterBalance(rows, experts, DEV, balance_coef=0.02, z_coef=0.003)
    dx, dm = x.to(DEV), mask.to(DEV)
    for m, ids in ((dm, chosen.to(DEV)), (None, chosen.to(DEV).int())):
        want = ref.balance(x, chosen, None if m is None else mask, 0.02, 0.003, scale=3.0)
        op.run(dx, ids, mask=m)
        _check_router(op, want, what)
        out = torch.full_like(dx, 7.0)
        op.backward(dx, out, mask=m, scale=3.0)
        ref.check(out, want["grad"], want["grad_off"], what + " grad")
    if rows:
        op.backward(dx, dx, scale=3.0)      # in place
        ref.check(dx, want["grad"], want["grad_off"], what + " grad in place")


@both_types
@pytest.mark.parametrize("experts", [5, 70])
def test_balance_strides_and_guards(kind, experts):
    log(f"{kind} {experts}")
    rows, choices = 41, 3
    x, chosen, mask = _router(rows, experts, choices, 3, kind)
    wide = torch.full((rows, experts + 5), 7.0, dtype=TYPES[kind], device=DEV)
    wide[:, 3:experts + 3] = x.to(DEV)
    ids = torch.full((rows, choices + 4), 1 << 40, dtype=torch.int64, device=DEV)
    ids[:, 2:choices + 2] = chosen.to(DEV)
    op = RouterBalance(rows, experts, DEV, z_coef=0.1)
    want = ref.balance(x, chosen, mask, 0.01, 0.1)
    op.run(wide[:, 3:experts + 3], ids[:, 2:choices + 2], mask=mask.to(DEV).to(torch.uint8) * 255)
    _check_router(op, want, "strided")
    out = torch.full((rows + 2, experts + 9), 7.0, dtype=TYPES[kind], device=DEV)
    view = out[1:-1, 1:experts + 1]
    op.backward(wide[:, 3:experts + 3], view, mask=mask.to(DEV))
    ref.check(view, want["grad"], want["grad_off"], "strided grad")
    view.fill_(7.0)
    assert (out == 7.0).all()
    # the same row for every token, and one choice for all
    one = x[:1].to(DEV).expand(rows, experts)
    op.run(one, chosen[:1].to(DEV).expand(rows, choices))
    _check_router(op, ref.balance(x[:1].expand(rows, experts), chosen[:1].expand(rows, choices),
                                  None, 0.01, 0.1), "expanded")


@both_types
def test_balance_of_special_rows(kind):
    log(f"{kind} special rows")
    low = torch.finfo(TYPES[kind]).min
    x, chosen, mask = _router(60, 20, 3, 4, kind)
    x[0, 3:9] = -INF
    x[1] = -INF
    x[2] = low
    x[3] = low
    x[3, 5] = 0.0
    mask[:8] = True
    mask[8] = False
    x[8] = NAN                # hidden
    chosen[8] = 1000
    chosen[4] = -1            # no choices
    chosen[5, 1:] = -5
    chosen[6] = 7             # one expert three times
    op = RouterBalance(60, 20, DEV, z_coef=0.0)
    out = torch.empty(60, 20, dtype=TYPES[kind], device=DEV)
    for _ in range(2):
        op.run(x.to(DEV), chosen.to(DEV), mask=mask.to(DEV))
        want = ref.balance(x, chosen, mask, 0.01, 0.0)
        assert torch.equal(op.counts.cpu(), want["counts"])
        ref.check(op.balance, want["balance"], want["off"]["balance"], "balance")
        op.backward(x.to(DEV), out, mask=mask.to(DEV))
        ref.check(out, want["grad"], want["grad_off"], "grad")
        # an id out of range: no loss, and no gradient
        bad = chosen.clone()
        bad[7, 2] = 20
        op.run(x.to(DEV), bad.to(DEV), mask=mask.to(DEV))
        assert op.loss.isnan() and op.balance.isnan() and not op.z.isnan()
        op.backward(x.to(DEV), out, mask=mask.to(DEV))
        assert out[mask.to(DEV)].isnan().all() and (out[~mask.to(DEV)] == 0).all()
        # NaN and infinity where they count
        for value in (NAN, INF):
            spoilt = x.clone()
            spoilt[9, 2], seen = value, mask.clone()
            seen[9] = True
            op.run(spoilt.to(DEV), chosen.to(DEV), mask=seen.to(DEV))
            assert op.loss.isnan() and op.balance.isnan() and op.z.isnan()
            assert torch.equal(op.counts.cpu(), ref.balance(x, chosen, seen)["counts"])
    # nothing that counts
    none = torch.zeros(60, dtype=torch.bool, device=DEV)
    op.run(x.to(DEV), chosen.to(DEV), mask=none)
    assert op.tokens == 0 and op.loss == 0 and op.balance == 0 and op.z == 0
    assert (op.counts == 0).all()
    op.backward(x.to(DEV), out, mask=none)
    assert (out == 0).all()
    # no choices at all
    op.run(x[10:].to(DEV), torch.full((50, 3), -1, device=DEV))
    assert op.tokens == 50 and op.balance == 0


def test_balance_over_ranks():
    """Counts and tokens summed over two halves: the gradients of the whole batch."""
    log("two halves")
    x, chosen, mask = _router(400, 24, 2, 6, "fp32")
    whole = RouterBalance(400, 24, DEV, z_coef=0.01)
    whole.run(x.to(DEV), chosen.to(DEV), mask=mask.to(DEV))
    want = torch.empty(400, 24, device=DEV)
    whole.backward(x.to(DEV), want, mask=mask.to(DEV))
    parts = [slice(0, 150), slice(150, 400)]
    ops = [RouterBalance(400, 24, DEV, z_coef=0.01) for _ in parts]
    for op, p in zip(ops, parts):
        op.run(x[p].to(DEV), chosen[p].to(DEV), mask=mask[p].to(DEV))
    counts, tokens = sum(op.counts for op in ops), sum(op.tokens for op in ops)
    for op, p in zip(ops, parts):
        op.counts.copy_(counts)
        op.tokens.copy_(tokens)
        out = torch.empty_like(want[p])
        op.backward(x[p].to(DEV), out, mask=mask[p].to(DEV))
        assert torch.equal(out, want[p])


# -------------------------------------------------- streams, graphs, updates ---

class Chain:
    """Logits, their losses and gradients, as one update makes them."""

    def __init__(self, n, vocab, kind, seed):
        self.n, self.vocab, self.kind = n, vocab, kind
        self.x = torch.empty(n, vocab, dtype=TYPES[kind], device=DEV)
        self.y = torch.empty(n, dtype=torch.int64, device=DEV)
        self.old, self.adv = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        self.out = torch.empty_like(self.x)
        self.router_x = torch.empty(n, 24, device=DEV)
        self.ids = torch.empty(n, 2, dtype=torch.int64, device=DEV)
        self.router_out = torch.empty_like(self.router_x)
        self.probs = TokenLogProbs(n, vocab, DEV, entropy=True, top=4)
        self.loss = PolicyLoss(n, DEV)
        self.router = RouterBalance(n, 24, DEV, z_coef=0.01)
        self.fill(seed)

    def fill(self, seed):
        x, y = _logits(self.n, self.vocab, seed, self.kind), _tokens(self.n, self.vocab, seed)
        x[torch.arange(self.n), y] = 3.0
        y[self.n // 2] = -1
        s = _policy_inputs(self.n, seed)
        self.x.copy_(x)
        self.y.copy_(y)
        self.old.copy_(s["old"])
        self.adv.copy_(s["adv"])
        r, ids, _ = _router(self.n, 24, 2, seed, "fp32")
        self.router_x.copy_(r)
        self.ids.copy_(ids)

    def step(self):
        self.probs.run(self.x, self.y, temperature=0.9)
        self.loss.run(self.probs.logp, self.old, self.adv, entropy=self.probs.entropy,
                      entropy_coef=0.01, scale=1 / self.n)
        self.probs.backward(self.x, self.y, self.loss.grad_logp, self.out,
                            grad_entropy=self.loss.grad_entropy)
        self.router.run(self.router_x, self.ids)
        self.router.backward(self.router_x, self.router_out)

    def outputs(self):
        p, l, r = self.probs, self.loss, self.router
        return [t.clone() for t in (p.logp, p.entropy, p.stats, p.top_ids, p.top_logp, l.result,
                                    l.grad_logp, l.grad_entropy, self.out, r.counts, r.result,
                                    self.router_out)]


def _bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.itemsize])


def _same(a, b):
    return all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))


@both_types
@pytest.mark.parametrize("n,vocab", [(3, 40000), (1100, 3000)])
def test_captured_updates_repeat_the_eager_ones(kind, n, vocab):
    log(f"graph {kind} {n}x{vocab}")
    c = Chain(n, vocab, kind, 0)
    eager = {}
    for seed in range(3):
        c.fill(seed)
        c.step()
        eager[seed] = c.outputs()
    assert not _same(eager[0], eager[1])
    c.fill(0)
    c.step()
    assert _same(c.outputs(), eager[0])        # and the same bits again
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step()
    for seed in (1, 2, 0, 0, 2):
        c.fill(seed)
        graph.replay()
        got = c.outputs()
        assert _same(got, eager[seed]), seed
        c.fill((seed + 1) % 3)                  # eager work between the replays
        c.step()
        assert _same(c.outputs(), eager[(seed + 1) % 3])


def test_two_chains_on_two_streams():
    log("two streams")
    chains = [Chain(5, 30000, "bf16", 1), Chain(700, 2500, "fp32", 2)]
    alone = []
    for c in chains:
        c.step()
        alone.append(c.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.step()
    torch.cuda.synchronize()
    for c, want in zip(chains, alone):
        assert _same(c.outputs(), want)


def test_one_object_over_calls_of_many_sizes():
    """Its workspace serves every number of rows, in turn, whole rows and rows in parts."""
    log("many sizes")
    op = TokenLogProbs(1100, 20000, DEV, entropy=True, top=6)
    for k, n in enumerate((1100, 1, 37, 2, 1100, 400, 1)):
        kind = ("bf16", "fp32")[k % 2]
        x, y = _logits(n, 20000, k, kind), _tokens(n, 20000, k)
        op.run(x.to(DEV), y.to(DEV))
        some = slice(0, min(n, 40))
        want = ref.Rows(x[some], y[some], top=6)
        _check_forward(op, want, min(n, 40), f"{n} rows", 6)


def test_preparing_inside_a_capture_is_refused():
    log("capture")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        try:
            with pytest.raises(RuntimeError, match="before the capture"):
                TokenLogProbs(4, 100, DEV)
        finally:
            graph.capture_end()
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits():
    """Rows that begin past 2^32 elements of one buffer."""
    log("far rows")
    n, vocab, step = 3, 5000, (1 << 31) + 9
    far = torch.empty(2 * step + vocab, dtype=torch.bfloat16, device=DEV)
    rows = far.as_strided((n, vocab), (step, 1))
    x, y = _logits(n, vocab, 4, "bf16"), _tokens(n, vocab, 4)
    rows.copy_(x)
    op = TokenLogProbs(n, vocab, DEV, entropy=True, top=3)
    op.run(rows, y.to(DEV))
    want = ref.Rows(x, y, top=3)
    _check_forward(op, want, n, "far", 3)
    a, h = _coefs(n, 4)
    op.backward(rows, y.to(DEV), a.to(DEV), rows, grad_entropy=h.to(DEV))
    ref.check(rows, *want.grad(a, h, x.dtype), "far grad")


def test_a_whole_update():
    """A trainer's update of a tiny policy: its logits, the losses, the gradients by the
    chain rule, the norm, the step, and the delta; the sampler that applies it gives
    the tokens the very probabilities that the trainer gives them."""
    log("update")
    n, hidden, vocab = 96, 64, 512
    g = torch.Generator(DEV)
    g.manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    master = 0.1 * rand(vocab, hidden)
    w = [master.to(torch.bfloat16), torch.empty(vocab, hidden, dtype=torch.bfloat16, device=DEV)]
    sampler = w[0].clone()
    states = rand(n, hidden).to(torch.bfloat16)
    tokens = torch.randint(0, vocab, (n,), generator=g, device=DEV)
    adv = rand(n)
    weights = (torch.arange(n, device=DEV) % 8 != 0).float()
    tokens[weights == 0] = -1
    probs, seen = (TokenLogProbs(n, vocab, DEV, entropy=True) for _ in range(2))
    loss = PolicyLoss(n, DEV)
    grad = torch.zeros(vocab, hidden, device=DEV)
    norm = bd.GradNormBatch([grad])
    moments = ([torch.zeros_like(master)], [torch.zeros_like(master)])
    steps = [bd.AdamWBatch([a], [grad], masters=[master], out=[b], states=moments,
                           weight_decay=0.0) for a, b in (w, w[::-1])]
    forward = lambda weight: (states.float() @ weight.float().t()).to(torch.bfloat16)
    seen.run(forward(sampler), tokens)
    old = seen.logp.clone()
    for t in range(1, 4):
        a, b = (w, w[::-1])[t % 2 == 0]
        logits = forward(a)
        x = logits.cpu()
        probs.run(logits, tokens)
        loss.run(probs.logp, old, adv, weights=weights, entropy=probs.entropy, entropy_coef=0.01,
                 scale=1 / n)
        if t == 1:      # the same policy drew the tokens
            assert loss.kl == 0 and loss.clipped == 0 and torch.equal(probs.logp, old)
        probs.backward(logits, tokens, loss.grad_logp, out=logits, grad_entropy=loss.grad_entropy)
        live = tokens.cpu() >= 0
        want, off = ref.Rows(x[live], tokens.cpu()[live]).grad(
            loss.grad_logp.cpu()[live], loss.grad_entropy.cpu()[live], torch.bfloat16)
        ref.check(logits.cpu()[live], want, off, f"gradient {t}")
        assert (logits.cpu()[~live] == 0).all()
        grad.copy_(logits.float().t().contiguous() @ states.float())
        norm.run(max_norm=1.0)
        steps[t % 2 == 0].run(lr=1e-2, step=t, norm=norm)
        assert norm.nonfinite == 0 and not torch.equal(a, b)
        payload, checksum = bd.delta_compress(a, b)
        bd.delta_decompress(sampler, payload, checksum)
        assert torch.equal(sampler.view(torch.int16), b.view(torch.int16))
        probs.run(forward(b), tokens)
        seen.run(forward(sampler), tokens)
        assert _same([probs.logp, probs.entropy], [seen.logp, seen.entropy])
    # an id that is no token reaches the step's flag
    tokens[1] = vocab
    probs.run(forward(w[0]), tokens)
    loss.run(probs.logp, old, adv, weights=weights)
    logits = forward(w[0])
    probs.backward(logits, tokens, loss.grad_logp, out=logits)
    flag = bd.GradNormBatch([logits.view(-1)])
    flag.run()
    assert flag.nonfinite == 1
