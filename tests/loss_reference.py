"""The losses in 64 bits, with torch on the CPU, from their definitions in
include/bf16delta_loss.h, and how far a 32-bit computation may be from them.

Bounds.  u = 2^-24 is half a step of fp32; every 32-bit operation and every constant
rounded to 32 bits adds at most u of its result, exp2, log and log2 2u (one unit in
the last place).
  d_j = (x_j - m) / T   : 3u |d_j| (constant, difference, product), as a logarithm of any base
  S   = sum of e^d_j    : each term 3u |d_j| + 2u; its way through the running maxima
        adds no more than 3u |d_j| in all (the shifts add up to d_j) and 3u a
        shift; and u for each sum that it passes.  Weighted by p: 3u E|d| + u N,
        N = 2 + sums + 3 shifts
  ln S: that, 2u ln S for the logarithm
  logp = d_y - ln S     : the two, and u |logp|
  Q   = sum of p_j |d_j|: the terms' own 3u E d^2, Q times S's bound twice (in
        W and in its divisor), and u Q for the N sums and 8 more operations
  H   = ln S + Q        : the two, and 2u H
  g_j = p_j (A + B ln p_j) : p_j by the bound of ln p_j = d_j - ln S and 3u; A
        by H's and 4 operations, B's term by that of ln p_j and 4; 3 to join them
with 1 % on top for products of bounds.  Rounding to bf16 adds 2^-8 of the value.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8
TINY = 2.0 ** -118     # what fp32 cannot hold: p below 2^-126 times a coefficient below 2^8
F64 = torch.float64


def sums(vocab: int, f32: bool) -> int:
    """N of the above: a thread's elements, twice its turns, and the joins of lanes,
    waves and parts."""
    turns = -(-vocab // (4096 if f32 else 8192))
    return 2 + 32 * turns + 3 * (turns + 6 + 4 + 6 + 4 + 4 + 8)


class Rows:
    """Log probabilities of rows of logits: values and bounds.  x: (n, vocab), any type;
    tokens: n ids, all of rows that count (from 0 to vocab - 1)."""

    def __init__(self, x: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0,
                 top: int = 0):
        n_sums = sums(x.shape[1], x.dtype == torch.float32)
        x = x.to(F64)
        self.t = temperature
        self.tokens = tokens.long()
        m = x.amax(1, keepdim=True)
        self.d = (x - m) / temperature
        e = self.d.exp()
        s = e.sum(1, keepdim=True)
        self.p = e / s
        self.ln_s = s.log()
        d = self.d.clamp(min=-1e300)          # 0 * infinity
        self.q = (self.p * -d).sum(1, keepdim=True)
        self.entropy = self.ln_s + self.q
        s_off = U * (3 * self.q + n_sums)
        ln_off = s_off + 2 * U * self.ln_s
        self.lp = self.d - self.ln_s
        finite = self.d.abs().clamp(max=1e300)
        self.lp_off = 1.01 * (3 * U * finite + ln_off + U * self.lp.abs().clamp(max=1e300))
        self.h_off = 1.01 * (ln_off + 3 * U * (self.p * d * d).sum(1, keepdim=True)
                             + self.q * (2 * s_off + U * (n_sums + 8)) + 2 * U * self.entropy)
        self.logp, self.logp_off = self._at(self.lp), self._at(self.lp_off)
        if top:
            # stable: equal values stay in the order of their ids
            best = x.sort(dim=1, descending=True, stable=True)
            self.top_ids = best.indices[:, :top].clone()
            self.top_logp = self.lp.gather(1, self.top_ids)
            self.top_off = self.lp_off.gather(1, self.top_ids)
            free = best.values[:, :top] == -math.inf
            self.top_ids[free] = -1
            self.top_logp[free] = -math.inf

    def _at(self, v):
        return v.gather(1, self.tokens[:, None])[:, 0]

    def grad(self, a: torch.Tensor, h: torch.Tensor | None, dtype):
        """(gradient of the logits, bound) for 32-bit a and h."""
        a = a.to(F64)[:, None]
        h = torch.zeros_like(a) if h is None else h.to(F64)[:, None]
        lp = self.lp.clamp(min=-1e300)
        inner = torch.where(self.p > 0, a + h * (lp + self.entropy), 0.0)
        g = -self.p * inner / self.t
        size = a.abs() + h.abs() * (self.entropy + torch.where(self.p > 0, lp.abs(), 0.0))
        off = self.p / self.t * ((self.lp_off + 3 * U) * inner.abs()
                                 + h.abs() * (self.h_off + self.lp_off) + 8 * U * size)
        off = torch.where(self.p > 0, off, 0.0)
        at = torch.zeros_like(g)
        at.scatter_(1, self.tokens[:, None], a / self.t)
        g = g + at
        off = 1.01 * (off + 3 * U * at.abs() + 3 * U * g.abs()) + TINY * (1 + size) / self.t
        if dtype == torch.bfloat16:
            off = off * (1 + BF16) + g.abs() * BF16
        return g, off


def check(got: torch.Tensor, want: torch.Tensor, off, what: str) -> None:
    """got within off of want; infinities and NaN have to be the same."""
    got, want = got.detach().cpu().to(F64), want.to(F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = torch.as_tensor(off, dtype=F64).expand(want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= off))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()!r}, {want[i].item()!r}, {off[i].item()!r}")


def policy(logp, old, adv, weights=None, ref=None, entropy=None, clip=(0.2, 0.2), kl_coef=0.0,
           entropy_coef=0.0, scale=1.0) -> dict:
    """The clipped policy loss: values, and under "off" the bounds of the sums.

    The kernel computes in 64 bits too, so its numbers differ from these by their
    rounding to 32 bits and by a sum's order: 1e-13 of the terms' magnitudes (2^10
    operations of 2^-53 each)."""
    lp, old, adv = (t.to(F64) for t in (logp, old, adv))
    w = torch.ones_like(lp) if weights is None else weights.to(F64)
    live = w != 0
    u = lp - old
    r = u.exp()
    cut = ((adv > 0) & (u > math.log1p(clip[1]))) | ((adv < 0) & (u < math.log1p(-clip[0])))
    low, high = (torch.full_like(adv, b) for b in (1 - clip[0], min(1 + clip[1], 1e300)))
    bound = torch.where(adv > 0, high, low)     # 64-bit numbers: two Python ones would be fp32
    gain = torch.where(adv == 0, 0.0, torch.where(cut, bound * adv, r * adv))
    slope = torch.where(cut | (adv == 0), 0.0, -r * adv)
    each = -gain
    parts = gain.abs()
    if kl_coef:
        v = ref.to(F64) - lp
        k = torch.where(v == math.inf, math.inf, torch.expm1(v) - v)
        each, slope = each + kl_coef * k, slope - kl_coef * torch.expm1(v)
        parts = parts + abs(kl_coef) * k
    zero = torch.zeros_like(lp)
    h = zero if entropy is None else entropy.to(F64)
    if entropy_coef:
        each = each - entropy_coef * h
        parts = parts + abs(entropy_coef) * h.abs()
    moved = torch.where(u == math.inf, math.inf, torch.expm1(u) - u)
    total = lambda t: torch.where(live, w * t, 0.0).sum()
    weight = w.sum()
    mean = lambda t: total(t) / weight if weight != 0 else torch.zeros((), dtype=F64)
    found = {"loss": scale * total(each), "weight": weight, "kl": mean(moved),
             "clipped": mean(cut.to(F64)), "entropy": mean(h)}
    off = {k: U * abs(float(v)) + 1e-13 * float(p) for (k, v), p in zip(found.items(), (
        abs(scale) * total(parts).abs(), w.abs().sum(), mean(moved), 1.0, mean(h.abs())))}
    found["grad_logp"] = torch.where(live, scale * w * slope, 0.0)
    found["grad_entropy"] = torch.where(live, -scale * w * entropy_coef, 0.0)
    return found | {"off": off}


def balance(x, chosen, mask=None, balance_coef=0.01, z_coef=0.0, scale=1.0, dtype=None) -> dict:
    """The balance loss: values and bounds ("off", "grad_off").

    p as above: 3u |d| + (8 + log2 experts) u for its exponent, sum, reciprocal and
    product; a sum of p over rows adds u for each sum that a term passes (rows of a
    lane, lanes, waves) and 2^-33 a workgroup (at most 256) for its integer step."""
    dtype = dtype or x.dtype
    x = x.to(F64)
    rows, experts = x.shape
    live = torch.ones(rows, dtype=torch.bool) if mask is None else mask.bool()
    some = live & (x.amax(1) > -math.inf)
    n = max(int(live.sum()), 1)
    ids = chosen[live].flatten().long()
    counts = torch.zeros(experts, dtype=torch.int64)
    ids = ids[(ids >= 0) & (ids < experts)]
    counts.scatter_add_(0, ids, torch.ones_like(ids))
    f = counts.to(F64) / max(int(counts.sum()), 1)
    safe = torch.where(some[:, None], x, 0.0)
    m = safe.amax(1, keepdim=True)
    d = safe - m
    s = d.exp().sum(1, keepdim=True)
    keep = some.to(F64)[:, None]
    p = d.exp() / s * keep
    lse = (m + s.log()) * keep
    finite = torch.where(p > 0, d.abs(), 0.0)
    p_off = U * (3 * finite + 3 * (p * finite).sum(1, keepdim=True) + 8 + math.log2(experts) + 1)
    lse_off = U * (3 * (p * finite).sum(1, keepdim=True) + 4 + math.log2(experts)
                   + 3 * s.log() + lse.abs()) * keep
    joins = -(-rows // 4) // 64 + 64
    total = experts * (f * p.sum(0)).sum() / n
    total_off = experts / n * ((f * (p * p_off).sum(0)).sum() + U * joins * (f * p.sum(0)).sum()
                               + 256 * 2.0 ** -33) + U * total
    z = (lse ** 2).sum() / n
    z_off = (2 * lse.abs() * lse_off).sum() / n + 2 * U * z
    by_share, by_lse = scale * balance_coef * experts / n, scale * 2 * z_coef / n
    inner = (p * f).sum(1, keepdim=True)
    inner_off = (p * f * (p_off + 3 * U)).sum(1, keepdim=True)
    g = p * (by_share * (f - inner) + by_lse * lse)
    size = abs(by_share) * (f + inner) + abs(by_lse) * lse.abs()
    g_off = 1.01 * (p_off * g.abs() + p * (abs(by_share) * inner_off + abs(by_lse) * lse_off
                                           + 6 * U * size)) + TINY
    if dtype == torch.bfloat16:
        g_off = g_off * (1 + BF16) + g.abs() * BF16
    loss = balance_coef * total + z_coef * z
    return {"counts": counts, "tokens": torch.tensor(int(live.sum())), "balance": total, "z": z,
            "loss": loss, "grad": g,
            "off": {"balance": 1.01 * total_off, "z": 1.01 * z_off,
                    "loss": 1.01 * (abs(balance_coef) * total_off + abs(z_coef) * z_off)
                    + U * loss.abs()},
            "grad_off": g_off}
