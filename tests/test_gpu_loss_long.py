"""The losses over the longest axes that they take: rows of up to 2^28 logits, whose sums
have to keep their digits, routers of up to 2^24 tokens, and a gradient of more
turns than a grid has workgroups.

The bounds are those of tests/loss_reference.py with a number of sums, N, that does not
grow with a row."""
import math

import pytest
import torch

from lossless_bf16_weight_xor_amd import RouterBalance, TokenLogProbs
from tests import loss_reference as ref
from tests.gpu_util import log
from tests.test_gpu_loss import DEV, TYPES, both_types

pytestmark = pytest.mark.gpu
U = ref.U

# Sums that a term of a row passes, each adding u: its vector's (7 in bf16) and its turn's (3),
# those of 32 turns, then 64 bits; to 32 bits (1); the lanes, the waves and the parts, as
# often again for rows in parts (2 x 10 + 1), with five shifts of 3u there; 6 for the term's own
# exponential and the results.
N = 7 + 3 + 32 + 1 + 21 + 15 + 6
# A shift of the sums in 64 bits has an error in proportion to its distance (the product and
# its coefficient 3u, the series 4u), and the distances add up to |d|.
SHIFT = 8


def _zeros(vocab):
    """Where the maximum is: 8192 elements of every 2^19, so that a sum begins there and
    the terms that follow are not 1."""
    return (torch.arange(vocab) // 8192) % 64 == 0


def _two_values(value, zeros, others, temperature):
    """(ln S, H, and the bounds of both) of a row of so many logits 0 and others of `value`,
    in 64 bits; s, q as in tests/loss_reference.py."""
    d = value / temperature
    s = zeros + others * math.exp(d)
    p = others * math.exp(d) / s
    q, ln_s = p * -d, math.log(s)
    s_off = U * (SHIFT * q + N + 3)
    ln_off = s_off + 2 * U * ln_s
    h_off = 1.01 * (ln_off + SHIFT * U * p * d * d + q * (2 * s_off + U * (N + 8))
                    + 2 * U * (ln_s + q))
    return ln_s, ln_s + q, 1.01 * ln_off, h_off


# 32000 and 131072: ordinary ones; 2^20 + 5 and 2^24 whole and in parts; and, in one row whose
# memory all tokens share, the longest that a call takes
@both_types
@pytest.mark.parametrize("vocab,inner", [(32000, 64), (131072, 64), ((1 << 20) + 5, 64),
                                         ((1 << 20) + 5, 4), (1 << 24, 33), (1 << 24, 5),
                                         (1 << 28, 33)])
def test_sums_of_equal_logits(kind, vocab, inner):
    """Terms that are all alike are rounded alike: a sum that takes them one by one drifts."""
    log(f"{kind} {vocab} x {inner}")
    rows = 1 if vocab == 1 << 28 else 8
    values = torch.tensor([-0.3, -0.7, -1.1, -1.3, -1.7, -2.1, -2.7, -3.3])[-rows:].to(TYPES[kind])
    inner = inner * 8 // rows
    zero = _zeros(vocab)
    zeros = int(zero.sum())
    x = values.to(DEV)[:, None].repeat(1, vocab)
    x[:, zero.to(DEV)] = 0.0
    y = torch.tensor([0, 8200, vocab // 2, vocab - 1]).repeat(inner)[:inner]
    op = TokenLogProbs(rows * inner, vocab, DEV, entropy=True)
    for temperature in (1.0, 0.7):
        op.run(x[:, None, :].expand(rows, inner, vocab), y.to(DEV).expand(rows, inner),
               temperature)
        logp, entropy = op.logp.view(rows, inner).cpu(), op.entropy.view(rows, inner).cpu()
        for row, value in enumerate(values.tolist()):
            ln_s, h, ln_off, h_off = _two_values(value, zeros, vocab - zeros, temperature)
            d = torch.zeros(inner, dtype=ref.F64).masked_fill(~zero[y], value / temperature)
            want = d - ln_s
            ref.check(logp[row], want, ln_off + 1.01 * U * (3 * d.abs() + want.abs()),
                      f"logp of {value}")
            ref.check(entropy[row], torch.full((inner,), h, dtype=ref.F64), h_off,
                      f"entropy of {value}")


@both_types
def test_the_gradient_of_equal_logits(kind):
    """The sums' error is that of every element of a gradient."""
    log(f"{kind} gradient")
    vocab, inner = (1 << 20) + 5, 300
    value = torch.tensor(-1.3).to(TYPES[kind]).item()
    zero = _zeros(vocab)
    zeros = int(zero.sum())
    x = torch.full((1, vocab), value, dtype=TYPES[kind], device=DEV)
    x[:, zero.to(DEV)] = 0.0
    y = torch.full((inner,), 9, device=DEV)
    op = TokenLogProbs(inner, vocab, DEV, entropy=True)
    op.run(x.expand(inner, vocab), y)
    out = torch.empty(inner, vocab, dtype=x.dtype, device=DEV)
    a = torch.linspace(-1.0, 1.0, inner, device=DEV)
    op.backward(x.expand(inner, vocab), y, a, out)
    ln_s, _, ln_off, _ = _two_values(value, zeros, vocab - zeros, 1.0)
    half = ref.BF16 if kind == "bf16" else U
    for j in (0, 8, 10, 8200, vocab // 2 - 1, vocab - 1):
        d = 0.0 if zero[j] else value
        off = ln_off + U * (3 * abs(d) + 8 + abs(d - ln_s)) + half
        want = -a.cpu().double() * math.exp(d - ln_s)
        ref.check(out[:, j], want, want.abs() * off * 1.01 + ref.TINY, f"element {j}")


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("rise", [0.25, 1.0, 30.0, 3000.0])
def test_sums_of_a_row_that_rises(whole, rise):
    """Every turn has a new maximum, by which all sums before are shifted."""
    vocab, n = (1 << 23) + 3, 260 if whole else 5
    log(f"rises by {rise}, {n} rows")
    x = torch.linspace(0.0, rise, vocab)
    y = torch.tensor([vocab - 1])
    op = TokenLogProbs(n, vocab, DEV, entropy=True)
    op.run(x.to(DEV).expand(n, vocab), y.to(DEV).expand(n))
    d = x.double() - x[-1].double()
    p = d.exp()
    s = p.sum()
    p /= s
    q, ln_s = (p * -d).sum(), s.log()
    s_off = U * (SHIFT * q + N + 3)
    # the shifts within 32 turns, and those of more than 1/32 in the logarithm to 2 of
    # what is left of the sums in 64 bits: 3u each
    s_off += 3 * U * (32 + 1 / (1 - 2 ** -(1 / 32)))
    ln_off = 1.01 * (s_off + 2 * U * ln_s)
    ref.check(op.logp, -ln_s.expand(n), ln_off, "logp")
    h_off = 1.01 * (ln_off + SHIFT * U * (p * d * d).sum() + q * (2 * s_off + U * (N + 8))
                    + 2 * U * (ln_s + q))
    ref.check(op.entropy, (ln_s + q).expand(n), h_off, "entropy")


@both_types
def test_sums_of_equal_logits_with_alternatives(kind):
    log(f"{kind} alternatives")
    vocab, n, value = (1 << 21) + 5, 130, -0.75
    zero = _zeros(vocab)
    zeros = int(zero.sum())
    x = torch.full((1, vocab), value, dtype=TYPES[kind], device=DEV)
    x[:, zero.to(DEV)] = 0.0
    y = torch.full((n,), vocab - 1, device=DEV)      # a zero, too
    op = TokenLogProbs(n, vocab, DEV, entropy=True, top=60)
    op.run(x.expand(n, vocab), y)
    ln_s, h, ln_off, h_off = _two_values(value, zeros, vocab - zeros, 1.0)
    want = torch.full((n,), -ln_s, dtype=ref.F64)
    ref.check(op.logp, want, ln_off + 1.01 * U * ln_s, "logp")
    ref.check(op.entropy, torch.full((n,), h, dtype=ref.F64), h_off, "entropy")
    assert torch.equal(op.top_ids.cpu(), torch.arange(60).expand(n, 60))
    ref.check(op.top_logp, torch.full((n, 60), -ln_s, dtype=ref.F64), ln_off + U * ln_s, "top")


@both_types
@pytest.mark.parametrize("vocab,top", [((1 << 19) + 3, 0), ((1 << 21) + 3, 2)])
def test_long_rows_that_are_special(kind, vocab, top):
    """Nothing but -infinity, in all turns or in the first ones; NaN and infinity early and
    late; the lowest value; rows that are left out."""
    log(f"{kind} {vocab}")
    low, inf = torch.finfo(TYPES[kind]).min, math.inf
    x = torch.full((9, vocab), -0.75, dtype=TYPES[kind])
    x[0] = -inf
    x[1, :-1] = -inf            # all weight on the last element
    x[2, : vocab // 2] = -inf
    x[3, vocab // 2:] = -inf
    x[4, 5] = math.nan
    x[5, -1] = math.nan
    x[6, -1] = inf
    x[7] = low
    y = torch.full((9,), vocab - 1)
    y[8] = -1
    inner = 29
    op = TokenLogProbs(9 * inner, vocab, DEV, entropy=True, top=top)
    op.run(x.to(DEV)[:, None, :].expand(9, inner, vocab), y.to(DEV)[:, None].expand(9, inner))
    logp, entropy = op.logp.view(9, inner).cpu(), op.entropy.view(9, inner).cpu()
    assert (logp[0] == -inf).all() and (entropy[0] == 0).all()
    assert (logp[1] == 0).all() and (entropy[1] == 0).all()
    for row, count in ((2, vocab - vocab // 2), (3, vocab // 2), (7, vocab)):
        ln_s, h, ln_off, h_off = _two_values(-1.0, count, 0, 1.0)
        off = torch.full((inner,), h_off, dtype=ref.F64)
        ref.check(entropy[row], torch.full((inner,), h, dtype=ref.F64), off, f"entropy {row}")
        want = torch.full((inner,), -inf if row == 3 else -ln_s, dtype=ref.F64)
        ref.check(logp[row], want, ln_off + 1.01 * U * ln_s, f"logp {row}")
    assert logp[4:7].isnan().all() and entropy[4:7].isnan().all()
    assert (logp[8] == 0).all() and (entropy[8] == 0).all()
    if top:
        ids = op.top_ids.view(9, inner, top)[:, 0].tolist()
        assert ids[0] == ids[8] == [-1, -1] and ids[1] == [vocab - 1, -1]
        assert ids[2] == [vocab // 2, vocab // 2 + 1] and ids[3] == ids[7] == [0, 1]


@pytest.mark.parametrize("kind,experts", [("bf16", 1024), ("fp32", 1021), ("fp32", 513),
                                          ("bf16", 40)])
def test_sums_of_very_many_tokens(kind, experts):
    """2^24 - 1 tokens that share a row: each expert's probabilities, all alike, add up."""
    rows = (1 << 24) - 1
    log(f"{kind} {rows}x{experts}")
    x = torch.zeros(1, experts, dtype=TYPES[kind])
    x[0, ::3] = -0.7
    x[0, 5] = 1.3
    d = x[0].double() - x[0].double().max()
    s = d.exp().sum()
    lse = x[0].double().max() + s.log()
    p = d.exp() / s
    op = RouterBalance(rows, experts, DEV, z_coef=0.01)
    for e in (0, 1, 5, experts - 1):
        chosen = torch.tensor([[e]], device=DEV)
        op.run(x.to(DEV).expand(rows, experts), chosen.expand(rows, 1))
        assert op.tokens == rows and op.counts[e] == rows and op.counts.sum() == rows
        # p: tests/loss_reference.py; 64 sums of a lane before it hands them over, two
        # joins of lanes; a step of 2^-37 for each time, a row at least; the result
        p_off = U * (3 * d[e].abs() + 3 * (p * d.abs()).sum() + 9 + math.log2(experts))
        off = p[e] * (p_off + U * (64 + 2 + 1)) + 2.0 ** -37
        ref.check(op.balance, experts * p[e], 1.01 * experts * off, f"balance of {e}")
        lse_off = U * (3 * (p * d.abs()).sum() + 4 + math.log2(experts) + 3 * s.log() + lse.abs())
        ref.check(op.z, lse ** 2, 1.01 * 2 * lse * lse_off + 2 * U * lse ** 2, "z")


@both_types
@pytest.mark.parametrize("rows,experts", [(600000, 520), (2200001, 40)])
def test_tokens_of_more_turns_than_a_lane_adds_up(kind, rows, experts):
    """Different rows, the last turns short; a wave that ends within its second 64 turns."""
    log(f"{kind} {rows}x{experts}")
    g = torch.Generator(DEV)
    g.manual_seed(rows)
    x = torch.randn(rows, experts, generator=g, device=DEV).to(TYPES[kind])
    chosen = torch.randint(0, experts, (rows, 2), generator=g, device=DEV)
    mask = torch.rand(rows, generator=g, device=DEV) > 0.1
    op = RouterBalance(rows, experts, DEV, z_coef=0.01)
    op.run(x, chosen, mask=mask)
    p = torch.zeros(experts, dtype=ref.F64, device=DEV)
    z = 0.0
    for a in range(0, rows, 1 << 17):
        live = mask[a:a + (1 << 17)]
        y = x[a:a + (1 << 17)][live].double()
        p += y.softmax(1).sum(0)
        z += y.logsumexp(1).square().sum().item()
    counts = torch.bincount(chosen[mask].flatten(), minlength=experts)
    n = int(mask.sum())
    assert torch.equal(op.counts, counts) and op.tokens == n
    want = (experts * (counts.double() / counts.sum() * p).sum() / n).cpu()
    # |d| of normal numbers stays below 12, its mean by p below 6
    off = U * (3 * 12 + 3 * 6 + 9 + math.log2(experts) + 64 + 2 + 1)
    ref.check(op.balance, want, 1.01 * (off * want + experts * 2.0 ** -37), "balance")
    lse = 12.0                     # and ln of the sum of e^x
    lse_off = U * (3 * 6 + 4 + math.log2(experts) + 3 * lse + lse)
    want = torch.tensor(z / n, dtype=ref.F64)
    ref.check(op.z, want, 1.01 * 2 * want.sqrt() * lse_off + 2 * U * want, "z")


def test_a_gradient_of_more_turns_than_a_grid_has_workgroups():
    """2^24 / 3 rows of three turns: a workgroup takes two of them, the last one of a
    row one.  183 GB are written; the logits and their stats are of a few rows each."""
    rows, vocab, kinds = ((1 << 24) // 3) // 7 * 7 + 7, 16385, 7
    size = 2 * rows * vocab
    assert 3 * rows > (1 << 24)
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    if free < size + (8 << 30):
        pytest.skip(f"needs {size >> 30} GiB, {free >> 30} are free")
    log(f"{rows} rows of {vocab}, {size >> 30} GiB")
    g = torch.Generator().manual_seed(0)
    x = (2 * torch.randn(1, vocab, generator=g)).to(torch.bfloat16)
    y = torch.tensor([0, 8191, 8192, 16383, 16384, -1, 77])
    a = torch.randn(kinds, generator=g)
    op = TokenLogProbs(rows, vocab, DEV)
    logits, tokens = x.to(DEV).expand(rows, vocab), y.to(DEV).repeat(rows // kinds)
    op.run(logits, tokens)
    live = y >= 0
    want = ref.Rows(x.expand(int(live.sum()), vocab), y[live])
    ref.check(op.logp[:kinds][live.to(DEV)], want.logp, want.logp_off, "logp")
    assert (op.logp.view(-1, kinds) == op.logp[:kinds]).all()
    log("gradient")
    out = torch.empty(rows, vocab, dtype=torch.bfloat16, device=DEV)
    op.backward(logits, tokens, a.to(DEV).repeat(rows // kinds), out)
    grad, off = want.grad(a[live], None, torch.bfloat16)
    ref.check(out[:kinds][live.to(DEV)], grad, off, "grad")
    assert (out[5] == 0).all()
    # rows of the same kind have the same bits
    bits = out.view(torch.int16).view(-1, kinds, vocab)
    step = 1 << 15
    for first in range(0, rows // kinds, step):
        assert (bits[first:first + step] == bits[0]).all(), first
    del bits, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,top", [((1 << 24) - 1, 0), ((1 << 22) - 1, 2)])
def test_the_most_rows_of_a_call(rows, top):
    """As many workgroups as a grid's 2^32 threads allow, of 4 waves and of 16."""
    log(f"{rows} rows, top {top}")
    vocab, kinds = 5, 1 << 20
    g = torch.Generator().manual_seed(top)
    x, y = torch.randn(kinds, vocab, generator=g), torch.randint(0, vocab, (kinds,), generator=g)
    times = -(-rows // kinds)
    logits, tokens = (t.to(DEV).repeat(times, *[1] * (t.dim() - 1))[:rows] for t in (x, y))
    op = TokenLogProbs(rows, vocab, DEV, entropy=True, top=top)
    op.run(logits, tokens)
    want = ref.Rows(x, y, top=top)
    ref.check(op.logp[:kinds], want.logp, want.logp_off, "logp")
    ref.check(op.entropy[:kinds], want.entropy[:, 0], want.h_off[:, 0], "entropy")
    a = torch.linspace(-1.0, 1.0, kinds)
    op.backward(logits, tokens, a.to(DEV).repeat(times)[:rows], logits)
    ref.check(logits[:kinds], *want.grad(a, None, x.dtype), "grad")
    got = [op.logp, op.entropy, logits] + ([op.top_ids, op.top_logp] if top else [])
    if top:
        assert torch.equal(op.top_ids[:kinds].cpu(), want.top_ids)
        ref.check(op.top_logp[:kinds], want.top_logp, want.top_off, "top_logp")
    for first in range(kinds, rows, kinds):      # the same rows again
        for t in got:
            part = t[first:first + kinds]
            assert torch.equal(part, t[:part.shape[0]]), first
