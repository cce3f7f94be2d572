"""The optimizer step and the gradient norm in 64 bits, with numpy, from their
definitions in include/bf16delta_step.h, and how far a 32-bit computation may
be from them.

Bounds.  u = 2^-24 is half a step of fp32.  Every 32-bit operation, and every
constant rounded to 32 bits, adds at most u of its result:
  m   = beta1 m0 + rest1 g : 3u on the first term (constant, product, sum),
        4u on the second (constant, g = scale * grad, product, sum)
  v   = beta2 v0 + rest2 g g : 3u, and 6u (constant, g twice, two products, sum);
        both terms are positive
  d   = sqrt(v) root2 + eps : 3u from v (6u halved), 2u for the root (good to
        one unit in the last place), u each for root2, product, sum and eps, and u
        for a denormal v taken for 0: at most 11u of d
  upd = rate (m (1 / d)) : the bound of m carried through, 2u for the reciprocal, 2u
        for rate (lr / c1 and its product with lr_scale) and u each for the two
        products, beside d's 11u
  p   = p0 - (decay p0 + upd) : 5u of decay p0 (lr, lr_scale * weight_decay, their
        product, its product with p0, sum), u of upd for the sum, u of p for
        the difference
and 1 % on top for the products of bounds.  What is rounded to fewer bits after
that is compared through the rounding itself, which is monotone: it has to lie
between the roundings of value - bound and value + bound.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -146     # a few of the smallest fp32 steps, for values near zero
M64 = (1 << 64) - 1


# -------------------------------------------------------------- random bits ---

def _mix64(z: int) -> int:
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & M64
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & M64
    return z ^ (z >> 31)


def random_bits(start: int, n: int, seed: int, step: int) -> np.ndarray:
    """32 random bits for each of the elements numbered start .. start + n - 1."""
    key = _mix64((_mix64(seed & M64) + step) & M64)
    k0, k1 = np.uint32(key & 0xFFFFFFFF), np.uint32(key >> 32)
    e = np.uint64(start) + np.arange(n, dtype=np.uint64)
    high = (e >> np.uint64(32)).astype(np.uint32)
    x = e.astype(np.uint32) ^ k0
    x = (x ^ (x >> np.uint32(16))) * np.uint32(0xBF58476D) + (k1 + high * np.uint32(0x9E3779B9))
    x = (x ^ (x >> np.uint32(15))) * np.uint32(0x94D049BB)
    return x ^ (x >> np.uint32(16))


# ------------------------------------------------------------------ e4m3 ---

def e4m3_values() -> np.ndarray:
    """The values of codes 0 .. 255 (NaN for 0x7F and 0xFF)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where(c >= 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


E4M3 = e4m3_values()


def decode(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The values that 8-bit states stand for."""
    s = 2.0 ** (scale.astype(np.float64) - 127)
    return E4M3[codes] * np.repeat(s, 32)[:codes.size]


def scale_byte(top: np.ndarray) -> np.ndarray:
    """The smallest byte, at least 1, with top <= 448 * 2^(byte - 127)."""
    b = np.ones(top.shape, dtype=np.int64)
    pos = top > 0
    b[pos] = np.maximum(1, np.ceil(np.log2(top[pos] / 448.0) - 1e-9).astype(np.int64) + 127)
    low = pos & (top > 448.0 * 2.0 ** (b - 127.0))    # log2's own rounding
    return b + low


def block_top(x: np.ndarray) -> np.ndarray:
    """The largest finite magnitude of each block of 32."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = np.concatenate([a, np.zeros(-a.size % 32)])
    return a.reshape(-1, 32).max(axis=1) if a.size else np.zeros(0)


def round_e4m3(t: np.ndarray, r: np.ndarray, positive: bool) -> np.ndarray:
    """Magnitudes t (at most 448) to the e4m3 grid, up where the fraction of a step,
    cut to 16 bits, and r reach 2^16; `positive`: what is above 0 stays so."""
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(t, 2.0 ** -30))), -6.0) - 3)
    whole = np.floor(t / step)
    cut = np.floor((t / step - whole) * 65536)
    y = np.minimum((whole + (cut + r >= 65536)) * step, 448.0)
    return np.where((y == 0) & (t > 0), 2.0 ** -9, y) if positive else y


# ------------------------------------------------------------------- bf16 ---

def bf16_bits_nearest(x: np.ndarray) -> np.ndarray:
    """bf16 patterns (uint16) nearest to x, ties to even."""
    return _bf16(x, None)


def bf16_bits_random(x: np.ndarray, r: np.ndarray) -> np.ndarray:
    """bf16 patterns of x, away from zero where the fraction of a step, cut to
    16 bits, and r reach 2^16."""
    return _bf16(x, r)


def _bf16(x, r):
    a = np.abs(x)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -200))), -126.0)
    step = 2.0 ** (e - 7)
    k = a / step
    whole = np.floor(k)
    frac = k - whole
    if r is None:
        up = (frac > 0.5) | ((frac == 0.5) & (whole % 2 == 1))
    else:
        up = np.floor(frac * 65536) + r >= 65536
    y = ((whole + up) * step * np.sign(x)).astype(np.float32)
    return (y.view(np.uint32) >> 16).astype(np.uint16)


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# ------------------------------------------------------------------- step ---

class Tensor:
    """One tensor's step in 64 bits.  p0, g, m0, v0: float64 arrays holding the
    inputs' exact values; `scale`: the 32-bit factor of the gradients."""

    def __init__(self, p0, g, m0, v0, *, lr, beta1, beta2, eps, decay, t, scale=1.0):
        g = g * scale
        c1, c2 = -math.expm1(t * math.log(beta1)) if beta1 else 1.0, \
            -math.expm1(t * math.log(beta2)) if beta2 else 1.0
        a, b = beta1 * m0, (1 - beta1) * g
        self.m = a + b
        self.m_off = 1.01 * U * (3 * np.abs(a) + 4 * np.abs(b)) + TINY
        a, b = beta2 * v0, (1 - beta2) * g * g
        self.v = a + b
        self.v_off = 1.01 * U * (3 * a + 6 * b) + TINY
        d = np.sqrt(self.v / c2) + eps
        upd = lr * (self.m / c1) / d
        self.p = p0 - lr * decay * p0 - upd
        # sqrt(v) where v is itself only known to a few of the smallest fp32 steps
        d_off = 11 * U + np.sqrt(TINY / c2) / d
        self.p_off = 1.01 * (lr / c1 / d * self.m_off + np.abs(upd) * (6 * U + d_off)
                             + U * (5 * lr * decay * np.abs(p0) + np.abs(self.p))) + TINY


def check_f32(got: np.ndarray, want: np.ndarray, off: np.ndarray, what: str) -> None:
    bad = ~(np.abs(got.astype(np.float64) - want) <= off)
    assert not bad.any(), _say(what, bad, got, want, off)


def check_between(got: np.ndarray, low: np.ndarray, high: np.ndarray, what: str) -> None:
    bad = ~((got >= np.minimum(low, high)) & (got <= np.maximum(low, high)))
    assert not bad.any(), _say(what, bad, got, low, high)


def _say(what, bad, *arrays):
    i = int(np.flatnonzero(bad)[0])
    return f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: " + \
        ", ".join(repr(a[i]) for a in arrays)


def check_weights(got_bits: np.ndarray, t: Tensor, r, what: str) -> None:
    """r: None for the nearest, or the random halves."""
    low, high = (bf16_values(_bf16(t.p + s * t.p_off, r)) for s in (-1, 1))
    check_between(bf16_values(got_bits), low, high, what)


def check_state8(codes, scale, x, off, r, positive, what) -> None:
    """codes and scale bytes against the values x, known to within off."""
    n = x.size
    low, high = (scale_byte(np.maximum(block_top(np.maximum(np.abs(x) + s * off, 0.0)), 0.0))
                 for s in (-1, 1))
    check_between(scale.astype(np.int64), low, high, what + " scale")
    inverse = np.repeat(2.0 ** (127.0 - scale), 32)[:n]
    got = np.abs(E4M3[codes])
    low, high = (round_e4m3(np.clip(np.abs(x) + s * off, 0.0, None) * inverse, r, positive)
                 for s in (-1, 1))
    if positive:     # a v that the bound lets vanish may be held as the smallest code
        high = np.maximum(high, np.where(x > 0, 2.0 ** -9, 0.0))
    check_between(got, low, high, what)
    wrong = (np.signbit(E4M3[codes]) != (x < 0)) & (np.abs(x) > off) & (got > 0)
    assert not wrong.any(), what + " sign"
