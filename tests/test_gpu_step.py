"""The optimizer step and the gradient norm on the GPU (bf16delta_step.h), each
against its definition in 64 bits (tests/step_reference.py, which derives the
bounds), and the whole update: norm, step, compress, decompress."""
import math

import numpy as np
import pytest
import torch

import lossless_bf16_weight_xor_amd as bd
from lossless_bf16_weight_xor_amd import AdamWBatch, GradNormBatch
from tests import step_reference as ref
from tests.gpu_util import log, to_u16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

# every vector and scale-block edge, an empty tensor, the edges of a
# workgroup's chunk and of an element-number span, and a few chunks
SIZES = [1, 3, 4, 5, 31, 32, 33, 0, 63, 255, 511, 512, 513, 1023, 1024, 1025, 4095, 4096, 4097,
         8191, 3 * 4096 + 77, 20011]


def _gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def _normal(n, gen, std=1.0):
    return torch.randn(n, generator=gen, device=DEV) * std


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Model:
    """A batch of tensors with gradients and states, and what they were before."""

    def __init__(self, sizes, seed, bits, master, grads="mixed", spread=True, apart=False):
        gen = _gen(seed)
        self.sizes, self.bits = sizes, bits
        self.masters = [_normal(n, gen, 0.02) for n in sizes] if master else None
        self.weights = [x.to(torch.bfloat16) for x in
                        (self.masters or [_normal(n, gen, 0.02) for n in sizes])]
        self.out = [torch.full_like(w, 7.0) for w in self.weights] if apart else None
        self.grads = []
        for j, n in enumerate(sizes):
            g = _normal(n, gen, 1e-3)
            if spread and n:      # magnitudes over some decades, and some zeros
                g *= torch.exp(2 * _normal(n, gen))
                g[torch.rand(n, generator=gen, device=DEV) < 0.05] = 0
            kind = {"mixed": j % 2, "fp32": 0, "bf16": 1}[grads]
            self.grads.append(g.to(torch.bfloat16) if kind else g)
        m = [_normal(n, gen, 3e-4) * torch.exp(2 * _normal(n, gen)) for n in sizes]
        v = [(_normal(n, gen, 1e-3) * torch.exp(2 * _normal(n, gen))).square() for n in sizes]
        if bits == 32:
            self.states = (m, v)
        else:
            coded = [[_code(x) for x in s] for s in (m, v)]
            self.states = tuple([c[k] for c in coded[i]] for i, k in
                                ((0, 0), (1, 0), (0, 1), (1, 1)))
        self.before = self.snapshot()

    def batch(self, **kw):
        return AdamWBatch(self.weights, self.grads, masters=self.masters, out=self.out,
                          states=self.states, state_bits=self.bits, **kw)

    def snapshot(self):
        return {"w": [to_u16(x) for x in self.weights],
                "out": [to_u16(x) for x in (self.out or self.weights)],
                "p": [x.cpu().numpy().copy() for x in self.masters or []],
                "s": [[x.cpu().numpy().copy() for x in part] for part in self.states]}

    def values(self, snap, j):
        """(p0, m0, v0) of tensor j as float64."""
        p0 = snap["p"][j].astype(np.float64) if self.masters else ref.bf16_values(snap["w"][j])
        s = [part[j] for part in snap["s"]]
        if self.bits == 32:
            return p0, s[0].astype(np.float64), s[1].astype(np.float64)
        return p0, ref.decode(s[0], s[2]), ref.decode(s[1], s[3])

    def check(self, before, *, lr, betas, eps, step, decay, seed=0, scale=1.0, lr_scale=None):
        now = self.snapshot()
        start = 0
        for j, n in enumerate(self.sizes):
            p0, m0, v0 = self.values(before, j)
            t = ref.Tensor(p0, _np(self.grads[j]), m0, v0,
                           lr=lr * (lr_scale[j] if lr_scale else 1.0), beta1=betas[0],
                           beta2=betas[1], eps=eps, decay=decay[j], t=step, scale=scale)
            r = ref.random_bits(start, n, seed, step)
            start += -(-n // 512) * 512
            name = f"tensor {j} (n={n})"
            half = None if self.masters else ((r * np.uint32(0x9E3779B1)) >> np.uint32(16))
            ref.check_weights(now["out"][j], t, half, name + " weights")
            if self.masters:
                ref.check_f32(now["p"][j], t.p, t.p_off, name + " master")
            s = [part[j] for part in now["s"]]
            if self.bits == 32:
                ref.check_f32(s[0], t.m, t.m_off, name + " m")
                ref.check_f32(s[1], t.v, t.v_off, name + " v")
            else:
                ref.check_state8(s[0], s[2], t.m, t.m_off, r & np.uint32(0xFFFF), False,
                                 name + " m")
                ref.check_state8(s[1], s[3], t.v, t.v_off, r >> np.uint32(16), True, name + " v")
        return now


def _code(x):
    """x as (codes, scale bytes) of 8-bit states, rounded to the nearest."""
    n = x.numel()
    byte = ref.scale_byte(ref.block_top(_np(x)))
    t = _np(x) * np.repeat(2.0 ** (127.0 - byte), 32)[:n]
    code = torch.from_numpy(t.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    return code.to(DEV), torch.from_numpy(byte.astype(np.uint8)).to(DEV)


DECAY = [0.1 if j % 3 else 0.0 for j in range(len(SIZES))]


@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
@pytest.mark.parametrize("master", [True, False], ids=["master", "no master"])
@pytest.mark.parametrize("bits", [32, 8])
def test_step_matches_its_definition(bits, master, apart):
    log(f"step bits={bits} master={master} apart={apart}")
    m = Model(SIZES, 11 + bits, bits, master, apart=apart)
    batch = m.batch(weight_decay=DECAY)
    kw = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8)
    before = m.before
    for step in (7, 8):
        batch.run(step=step, seed=5, **kw)
        torch.cuda.synchronize()
        before = m.check(before, step=step, decay=DECAY, seed=5, **kw)
    if apart:
        assert all(np.array_equal(a, b) for a, b in zip(before["w"], m.before["w"]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas,eps,step", [((0.0, 0.0), 1e-8, 1), ((0.9, 0.999), 1e-12, 1),
                                            ((0.5, 0.99), 1e-3, 100000), ((0.99, 0.0), 1e-6, 3)])
def test_step_over_its_parameters(bits, betas, eps, step):
    log(f"step bits={bits} betas={betas} eps={eps} step={step}")
    sizes = [4097, 33, 1]
    m = Model(sizes, 3, bits, True)
    rates = [1.0, 0.5, 0.0]
    kw = dict(lr=1e-3, betas=betas, eps=eps)
    m.batch(weight_decay=0.2, lr_scale=rates).run(step=step, **kw)
    torch.cuda.synchronize()
    m.check(m.before, step=step, decay=[0.2] * 3, lr_scale=rates, **kw)


@pytest.mark.parametrize("master", [True, False], ids=["master", "no master"])
@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_around_the_tensors_is_written(bits, master):
    """Every array is a view into one buffer, with 16 to 31 guard bytes before and
    behind it: the guards keep their pattern, in a step, in one that is left
    out, and with the norm in between."""
    log(f"guards bits={bits} master={master}")
    m = Model(SIZES, 91, bits, master, apart=True)
    lists = [m.out, m.grads, *m.states] + ([m.masters] if master else [m.weights])
    total = sum(x.numel() * x.element_size() + 64 for part in lists for x in part)
    buffer = torch.full((total,), 0xA5, dtype=torch.uint8, device=DEV)
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)
    at = 16
    for part in lists:
        for j, x in enumerate(part):
            size = x.numel() * x.element_size()
            view = buffer[at:at + size].view(x.dtype)
            view.copy_(x)
            part[j] = view
            inside[at:at + size] = True
            at += -(-size // 16) * 16 + 16
    norm, batch = GradNormBatch(m.grads), m.batch(weight_decay=0.1)
    norm.run(1.0)
    batch.run(lr=1e-3, step=1, norm=norm)
    m.grads[-1][0] = math.nan
    norm.run(1.0)
    batch.run(lr=1e-3, step=2, norm=norm)
    torch.cuda.synchronize()
    assert norm.nonfinite.item() == 1
    assert bool((buffer[~inside] == 0xA5).all())


def test_a_fresh_state_starts_from_zeros():
    for bits in (32, 8):
        log(f"fresh states bits={bits}")
        m = Model([1000, 64, 0, 5], 9, bits, True)
        batch = AdamWBatch(m.weights, m.grads, masters=m.masters, state_bits=bits,
                           weight_decay=0.0)
        m.states = (batch.m, batch.v) if bits == 32 else (batch.m, batch.v, batch.m_scale,
                                                          batch.v_scale)
        before = m.snapshot()
        assert all(not x.any() for part in before["s"] for x in part)
        kw = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8)
        batch.run(step=1, **kw)
        torch.cuda.synchronize()
        m.check(before, step=1, decay=[0.0] * 4, **kw)


def test_a_tensor_of_more_than_two_to_the_33_elements():
    """Offsets beyond 32 bits, element numbers that use the high word, and more
    workgroups than one launch holds: slices around 2^32, around the launch's
    2^33 elements and at the end, the rest zeros."""
    log("2^33 elements")
    n = (1 << 33) + 4096 + 77
    zeros = lambda dtype, k=n: torch.zeros(k, dtype=dtype, device=DEV)
    w, g = zeros(torch.bfloat16), zeros(torch.bfloat16)
    states = (zeros(torch.uint8), zeros(torch.uint8), zeros(torch.uint8, -(-n // 32)),
              zeros(torch.uint8, -(-n // 32)))
    slices = [((1 << 32) - 1024, 2048), ((1 << 33) - 512, n - (1 << 33) + 512), (0, 256)]
    gen = _gen(17)
    for a, k in slices:
        w[a:a + k] = _normal(k, gen, 0.02).to(torch.bfloat16)
        g[a:a + k] = _normal(k, gen, 1e-3).to(torch.bfloat16)
    before = [(to_u16(w[a:a + k]), _np(g[a:a + k])) for a, k in slices]
    kw = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8)
    norm = GradNormBatch([g])
    norm.run()
    AdamWBatch([w], [g], states=[[x] for x in states], state_bits=8, weight_decay=0.1).run(
        step=3, seed=6, norm=norm, **kw)
    torch.cuda.synchronize()
    assert norm.norm.item() == pytest.approx(math.sqrt(sum(float((x ** 2).sum())
                                                           for _, x in before)), rel=1e-12)
    for (a, k), (bits, grad) in zip(slices, before):
        t = ref.Tensor(ref.bf16_values(bits), grad, np.zeros(k), np.zeros(k), lr=1e-3, beta1=0.9,
                       beta2=0.95, eps=1e-8, decay=0.1, t=3)
        r = ref.random_bits(a, k, 6, 3)
        ref.check_weights(to_u16(w[a:a + k]), t, (r * np.uint32(0x9E3779B1)) >> np.uint32(16),
                          f"weights from {a}")
        m, v, ms, vs = (x[a // per:-(-(a + k) // per)].cpu().numpy()
                        for x, per in zip(states, (1, 1, 32, 32)))
        ref.check_state8(m, ms, t.m, t.m_off, r & np.uint32(0xFFFF), False, f"m from {a}")
        ref.check_state8(v, vs, t.v, t.v_off, r >> np.uint32(16), True, f"v from {a}")
    assert not states[0][(1 << 32) + 1024:(1 << 32) + (1 << 20)].any()


def test_denormal_second_moments_beside_a_small_eps():
    """v below the smallest normal fp32 number still has its root where eps does
    not hide it (the exact root's variant): without it the updates would be 1e-4
    off.  Beside a far smaller eps, v itself may be lost: refused."""
    log("denormal v")
    for bits in (32, 8):
        m = Model([4096, 33], 5, bits, True, grads="fp32", spread=False)
        for j, g in enumerate(m.grads):
            g.mul_(1e-16)                      # g around 1e-19, v around 1e-39
            m.masters[j].zero_()
            for part in m.states:
                part[j].zero_()
        before = m.snapshot()
        kw = dict(lr=1e-3, betas=(0.9, 0.9), eps=1e-15)
        batch = m.batch(weight_decay=0.0)
        batch.run(step=1, **kw)
        torch.cuda.synchronize()
        m.check(before, step=1, decay=[0.0, 0.0], **kw)
        for g in m.grads:
            g.mul_(10.0)
        with pytest.raises(RuntimeError, match="EINVAL"):
            batch.run(lr=1e-3, step=1, betas=(0.9, 0.9), eps=1e-30)


def test_eight_bit_states_on_extreme_values():
    """Blocks of zeros, of one tiny value, of the largest floats, of values whose
    range passes that of e4m3, and the exact border 448 * 2^k."""
    log("extreme 8-bit states")
    n = 32 * 8
    g = torch.zeros(n, device=DEV)
    g[32] = 1e-22                       # m near the smallest scale, v far below fp32
    g[64:96] = 1e15 * torch.linspace(-1, 1, 32, device=DEV)
    g[96:128] = torch.logspace(-12, 3, 32, device=DEV)
    g[128:160] = 448.0 * 2.0 ** -10     # m and v exactly on and next to the border
    g[160:192] = 449.0 * 2.0 ** -10
    g[192:224] = -torch.logspace(-30, -20, 32, device=DEV)
    g[255] = 3.0
    w = [torch.ones(n, device=DEV).to(torch.bfloat16)]
    p = [torch.ones(n, device=DEV)]
    m = Model([n], 1, 8, True)
    m.grads, m.masters, m.weights = [g], p, w
    for part in m.states:
        part[0].zero_()
    before = m.snapshot()
    kw = dict(lr=1e-3, betas=(0.5, 0.5), eps=1e-8)
    m.batch(weight_decay=0.0).run(step=2, **kw)
    torch.cuda.synchronize()
    now = m.check(before, step=2, decay=[0.0], **kw)
    v = ref.decode(now["s"][1][0], now["s"][3][0])
    exact = 0.5 * _np(g) ** 2
    assert (v[exact > 1e-40] > 0).all()      # no positive v is lost


def test_eight_bit_rounding_keeps_averages():
    """Constant gradients for 120 steps, beta2 = 0.95: the average of v reaches g^2,
    and of m reaches g (rounded to the nearest, v would stop where a step adds
    less than half a step of the grid, near 0.6 g^2).  One rounding has a
    relative sd of at most 1/16: a step of the grid is at most 1/8 of the value,
    and the variance f (1 - f) of its fraction at most 1/4.  The averages carry
    that on for 1 / sqrt(1 - beta^2): at most 0.2 for v and 0.143 for m.  The mean
    of n elements is within 6 of its sds with near certainty."""
    log("8-bit averages")
    n = 1 << 16
    gen = _gen(2)
    g = (torch.rand(n, generator=gen, device=DEV) + 0.5) * 1e-3
    w = [torch.zeros(n, device=DEV).to(torch.bfloat16)]
    batch = AdamWBatch(w, [g], masters=[torch.zeros(n, device=DEV)], state_bits=8,
                       weight_decay=0.0)
    for t in range(1, 121):
        batch.run(lr=0.0, step=t, seed=77)
    torch.cuda.synchronize()
    m = ref.decode(batch.m[0].cpu().numpy(), batch.m_scale[0].cpu().numpy()) / _np(g)
    v = ref.decode(batch.v[0].cpu().numpy(), batch.v_scale[0].cpu().numpy()) / _np(g) ** 2
    for x, beta, sd in ((m, 0.9, 0.143), (v, 0.95, 0.2)):
        assert abs(x.mean() - (1 - beta ** 120)) < 6 * sd / math.sqrt(n), x.mean()
        assert x.std() < sd


def test_bf16_weights_without_a_master_move_on_average():
    """Updates of 2^-12, far below half of 1.5's bf16 step of 2^-7, 64 times: the
    mean weight moves by their sum.  A rounding's sd is at most half a step, so
    a weight's after 64 is at most 8 * 2^-8."""
    log("bf16 stochastic rounding")
    n = 1 << 16
    w = [torch.ones(n, device=DEV).to(torch.bfloat16) * 1.5]
    g = [torch.full((n,), -1.0, device=DEV)]
    batch = AdamWBatch(w, g, weight_decay=0.0)
    for t in range(1, 65):
        batch.run(lr=2.0 ** -12, step=t, betas=(0.0, 0.0), eps=1e-12, seed=3)
    torch.cuda.synchronize()
    got = _np(w[0]).mean() - 1.5
    assert abs(got - 64 * 2.0 ** -12) < 6 * 8 * 2.0 ** -8 / math.sqrt(n), got


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [True, False], ids=["master", "no master"])
def test_non_finite_gradients_poison_their_element_only(bits, master):
    log(f"non-finite bits={bits} master={master}")
    n = 4096 + 40
    clean = Model([n], 21, bits, master, grads="fp32")
    dirty = Model([n], 21, bits, master, grads="fp32")
    at = {5: math.nan, 40: math.inf, 41: -math.inf, n - 1: math.nan}
    for i, x in at.items():
        dirty.grads[0][i] = x
        clean.grads[0][i] = 0.0
        for part, k in zip(clean.states[:2], (0, 1)):
            part[0][i] = 0        # nothing of these elements reaches the blocks' scales
            dirty.states[k][0][i] = 0
    kw = dict(lr=1e-3, step=3, seed=9)
    for x in (clean, dirty):
        x.batch(weight_decay=0.1).run(**kw)
    torch.cuda.synchronize()
    a, b = clean.snapshot(), dirty.snapshot()
    keep = np.ones(n, dtype=bool)
    keep[list(at)] = False
    assert np.array_equal(a["out"][0][keep], b["out"][0][keep])
    if master:
        assert np.array_equal(a["p"][0][keep], b["p"][0][keep])
        assert np.isnan(b["p"][0][~keep]).all()
    assert np.isnan(ref.bf16_values(b["out"][0][~keep])).all()
    for k in (0, 1):
        assert np.array_equal(a["s"][k][0][keep], b["s"][k][0][keep])
        held = b["s"][k][0][~keep]
        if bits == 8:
            assert np.isnan(ref.E4M3[held]).all()
            assert np.array_equal(a["s"][k + 2][0], b["s"][k + 2][0])
        else:
            assert not np.isfinite(held).any()


def test_a_lost_first_moment_stays_in_its_element():
    """A NaN code in m alone: its block keeps the scale of the others."""
    log("NaN in m")
    n = 320
    a, b = (Model([n], 22, 8, True, grads="fp32") for _ in range(2))
    for x, code in ((a, 0), (b, 0xFF)):
        x.grads[0][70] = 0.0
        x.states[0][0][70] = code
    for x in (a, b):
        x.batch().run(lr=1e-3, step=3)
    torch.cuda.synchronize()
    x, y = a.snapshot(), b.snapshot()
    keep = np.arange(n) != 70
    for k in range(4):
        if k < 2:
            assert np.array_equal(x["s"][k][0][keep], y["s"][k][0][keep])
        else:
            assert np.array_equal(x["s"][k][0], y["s"][k][0])
    assert np.array_equal(x["p"][0][keep], y["p"][0][keep])
    assert np.isnan(y["p"][0][70]) and np.isnan(ref.E4M3[y["s"][0][0][70]])
    assert x["s"][1][0][70] == y["s"][1][0][70]


# ------------------------------------------------------------------- norm ---

def _norm_of(grads, c=1.0):
    return abs(c) * math.sqrt(math.fsum(float((_np(g) ** 2).sum()) for g in grads))


@pytest.mark.parametrize("sizes", [[1], [0, 3], [7, 8, 9], [8191, 8192, 8193], SIZES,
                                   [3 * 8192 * 2048 + 12345], [1 << 20] * 9])
def test_norm_matches_its_definition(sizes):
    log(f"norm sizes={sizes[:6]} ...")
    gen = _gen(len(sizes))
    grads = [_normal(n, gen, 1e-3).to(torch.bfloat16 if j % 2 else torch.float32)
             for j, n in enumerate(sizes)]
    want = _norm_of(grads)
    norm = GradNormBatch(grads)
    for max_norm, c in ((math.inf, 1.0), (want / 3, 1.0), (want * 2, -0.25), (1e-20, 3.0)):
        norm.run(max_norm, c)
        torch.cuda.synchronize()
        # n sums of 64-bit squares, in either order: at most n 2^-53 of the sum each
        off = (2 * sum(sizes) + 8) * 2.0 ** -53
        got = abs(c) * want
        assert abs(norm.norm.item() - got) <= off * got
        scale = c * min(1.0, max_norm / got) if got else c
        assert abs(norm.scale.item() - scale) <= (2.0 ** -24 + off + 2.0 ** -50) * abs(scale)
        assert norm.nonfinite.item() == 0
    a = norm.result.clone()
    norm.run(1e-20, 3.0)
    assert torch.equal(a.view(torch.int64), norm.result.view(torch.int64))


def test_norm_of_a_batch_beyond_the_caches():
    """More than 1 GiB of gradients: read from the first chunk on, nothing kept."""
    log("norm of 1.3 GiB")
    gen = _gen(3)
    grads = [_normal(n, gen, 1e-3).to(torch.bfloat16) for n in (400_000_003, 300_000_001, 77)]
    want = math.sqrt(sum(float(x.double().square().sum()) for g in grads
                         for x in g.split(1 << 26)))
    norm = GradNormBatch(grads)
    norm.run(1.0)
    a = norm.result.clone()
    norm.run(1.0)
    torch.cuda.synchronize()
    assert abs(norm.norm.item() - want) <= 1e-7 * 2.0 ** -10 * want
    assert torch.equal(a.view(torch.int64), norm.result.view(torch.int64))


def test_norm_of_huge_and_tiny_gradients_is_finite():
    log("norm range")
    big = [torch.full((5000,), 3e38, device=DEV), torch.full((9,), -1e38, device=DEV)]
    norm = GradNormBatch(big)
    norm.run(1.0)
    want = _norm_of(big)
    assert abs(norm.norm.item() - want) < 1e-12 * want and norm.nonfinite.item() == 0
    assert norm.scale.item() == pytest.approx(1.0 / want, rel=1e-4, abs=2e-45)
    small = [torch.full((70,), 1e-40, device=DEV)]
    norm = GradNormBatch(small)
    norm.run()
    assert abs(norm.norm.item() - _norm_of(small)) < 1e-12 * _norm_of(small)
    assert norm.scale.item() == 1.0


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_flags_a_non_finite_gradient_anywhere(value, dtype):
    log(f"norm flag {value} {dtype}")
    grads = [torch.ones(n, device=DEV, dtype=dtype) for n in (5, 8192 + 3, 100000)]
    norm = GradNormBatch(grads)
    for j, i in ((0, 0), (0, 4), (1, 8191), (1, 8194), (2, 99999), (2, 50000)):
        grads[j][i] = value
        norm.run(1.0)
        assert norm.nonfinite.item() == 1, (j, i)
        grads[j][i] = 1
    norm.run(1.0)
    assert norm.nonfinite.item() == 0


# --------------------------------------------------------------- together ---

@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_uses_the_norm_on_the_device(bits):
    log(f"clipped step bits={bits}")
    m = Model(SIZES, 31, bits, True, apart=True)
    norm = GradNormBatch(m.grads)
    batch = m.batch(weight_decay=DECAY)
    kw = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8)
    norm.run(max_norm=_norm_of(m.grads) / 10, grad_scale=0.5)
    batch.run(step=5, norm=norm, **kw)
    torch.cuda.synchronize()
    assert norm.scale.item() == pytest.approx(0.1, rel=1e-6)
    m.check(m.before, step=5, decay=DECAY, scale=norm.scale.item(), **kw)


def test_the_norm_of_parts_is_combined_through_the_views():
    """Two halves of a model, as two ranks hold them: each one's norm without
    clipping, the whole's norm, scale and flag written back into the views."""
    log("norm of parts")
    parts = [Model([5000, 33], 32, 32, True), Model([4097], 33, 32, True)]
    norms = [GradNormBatch(m.grads) for m in parts]
    kw = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8)
    for poison in (False, True):
        if poison:
            parts[1].grads[0][3] = math.inf
        for norm in norms:
            norm.run()
        total = (norms[0].norm.square() + norms[1].norm.square()).sqrt()
        bad = torch.maximum(norms[0].nonfinite, norms[1].nonfinite)
        for norm in norms:
            norm.norm.copy_(total)
            norm.scale.copy_((0.01 / total).clamp(max=1.0))
            norm.nonfinite.copy_(bad)
        before = [m.snapshot() for m in parts]
        for m, norm in zip(parts, norms):
            m.batch(weight_decay=0.1).run(step=2, norm=norm, **kw)
        torch.cuda.synchronize()
        for m, norm, old in zip(parts, norms, before):
            if poison:
                assert all(np.array_equal(i, j) for i, j in zip(m.snapshot()["p"], old["p"]))
            else:
                want = 0.01 / _norm_of(parts[0].grads + parts[1].grads)
                assert norm.scale.item() == pytest.approx(want, rel=1e-6) and want < 1
                m.check(old, step=2, decay=[0.1] * 2, scale=norm.scale.item(), **kw)


@pytest.mark.parametrize("apart", [False, True], ids=["in place", "apart"])
@pytest.mark.parametrize("master", [True, False], ids=["master", "no master"])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_with_non_finite_gradients_is_left_out(bits, master, apart):
    log(f"left out bits={bits} master={master} apart={apart}")
    m = Model(SIZES, 41, bits, master, apart=apart)
    m.grads[-1][17] = math.inf
    norm = GradNormBatch(m.grads)
    norm.run(max_norm=1.0)
    m.batch().run(lr=1.0, step=1, norm=norm)
    torch.cuda.synchronize()
    now = m.snapshot()
    for j in range(len(SIZES)):
        want = ref.bf16_bits_nearest(m.before["p"][j].astype(np.float64)) if master \
            else m.before["w"][j]
        assert np.array_equal(now["out"][j], want)
        assert np.array_equal(now["w"][j], m.before["w"][j])
        for a, b in zip(now["s"], m.before["s"]):
            assert np.array_equal(a[j], b[j])
        if master:
            assert np.array_equal(now["p"][j], m.before["p"][j])


@pytest.mark.parametrize("bits,master", [(32, True), (8, True), (8, False)])
def test_update_from_gradients_to_the_receiver(bits, master):
    """norm -> step into the other working copy -> compress -> decompress on a
    receiver, for four steps with the two copies taking turns: the receiver
    follows the trainer bit for bit."""
    log(f"update bits={bits} master={master}")
    sizes = [20011, 4096, 0, 333, 8192 * 3]
    m = Model(sizes, 51, bits, master, apart=True)
    other = [w.clone() for w in m.weights]
    norm = GradNormBatch(m.grads)
    turns = [AdamWBatch(a, m.grads, masters=m.masters, out=b, states=m.states, state_bits=bits)
             for a, b in ((m.weights, other), (other, m.weights))]
    receiver = [w.clone() for w in m.weights]
    gen = _gen(5)
    for t in range(1, 5):
        for g in m.grads:
            if g.numel():
                g.copy_(_normal(g.numel(), gen, 1e-2))
        norm.run(max_norm=1.0)
        step = turns[(t - 1) % 2]
        step.run(lr=1e-3, step=t, seed=8, norm=norm)
        payloads = bd.compress_batch(step.pairs())
        res = bd.decompress_batch([(w, p, cs) for w, (p, cs, _) in zip(receiver, payloads)])
        assert all(r["status"] == bd.OK for r in res)
        changed = sum(r["n_changed"] for r in res)
        assert changed > 0
        for w, new in zip(receiver, step.out):
            assert torch.equal(w.view(torch.int16), new.view(torch.int16))


@pytest.mark.parametrize("bits,master", [(32, True), (8, False)])
def test_captured_steps_are_those_run_eagerly(bits, master):
    """norm and step captured once, with rate and step number on the device, and
    replayed with eager work in between; every replay against an eager twin."""
    log(f"graph bits={bits} master={master}")
    sizes = [20011, 333, 0, 4096]
    a, b = (Model(sizes, 61, bits, master) for _ in range(2))
    norms = [GradNormBatch(x.grads) for x in (a, b)]
    batches = [x.batch() for x in (a, b)]
    lr = torch.tensor(1e-3, device=DEV)
    step = torch.tensor(0, dtype=torch.int64, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        norms[0].run(max_norm=0.5)
        batches[0].run(lr=lr, step=step, seed=4, norm=norms[0])
    gen = _gen(6)
    for t in range(1, 5):
        for x, y in zip(a.grads, b.grads):
            if x.numel():
                x.copy_(_normal(x.numel(), gen, 1e-2))
                y.copy_(x)
        lr.fill_(1e-3 / t)
        graph.replay()
        norms[1].run(max_norm=0.5)
        batches[1].run(lr=float(lr.item()), step=t, seed=4, norm=norms[1])
        torch.cuda.synchronize()
        x, y = a.snapshot(), b.snapshot()
        for key in ("w", "p"):
            assert all(np.array_equal(i, j) for i, j in zip(x[key], y[key])), (t, key)
        for i, j in zip(x["s"], y["s"]):
            assert all(np.array_equal(k, l) for k, l in zip(i, j)), t
        assert torch.equal(norms[0].result, norms[1].result)


def test_two_graphs_of_one_batch_take_turns():
    """Graphs that share a batch, its norm and their workspace, replayed in turn
    with eager calls of the same batch in between."""
    log("two graphs")
    sizes = [20011, 333]
    a, b = (Model(sizes, 62, 8, True) for _ in range(2))
    (na, ba), (nb, bb) = ((GradNormBatch(x.grads), x.batch()) for x in (a, b))
    one = lambda norm, batch, t: (norm.run(max_norm=0.5), batch.run(lr=1e-3, step=t, norm=norm))
    graphs = []
    for t in (3, 4):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one(na, ba, t)
        graphs.append(g)
    for t in (3, 4, 5, 4, 3, 3, 4, 5):
        graphs[t - 3].replay() if t < 5 else one(na, ba, t)
        one(nb, bb, t)
        torch.cuda.synchronize()
        x, y = a.snapshot(), b.snapshot()
        assert all(np.array_equal(i, j) for i, j in zip(x["out"], y["out"])), t
        assert all(np.array_equal(k, l) for i, j in zip(x["s"], y["s"]) for k, l in zip(i, j)), t
        assert torch.equal(na.result, nb.result)


@pytest.mark.parametrize("betas,step", [((0.0, 0.0), 1), ((0.9, 0.999), 1), ((0.9, 0.95), 0),
                                        ((0.99, 0.9999), 12345678901)])
def test_rate_and_step_number_from_the_device(betas, step):
    """The kernel's own bias corrections; a step word of 0 counts as 1."""
    log(f"device numbers betas={betas} step={step}")
    sizes = [4097, 33, 0, 1000]
    for bits in (32, 8):
        for lr_there, step_there in ((True, True), (True, False), (False, True)):
            if step == 0 and not step_there:
                continue
            m = Model(sizes, 7, bits, False)
            kw = dict(betas=betas, eps=1e-8, seed=12)
            m.batch(weight_decay=0.3).run(
                lr=torch.tensor(0.25, device=DEV) if lr_there else 0.25,
                step=torch.tensor([step], device=DEV) if step_there else step, **kw)
            torch.cuda.synchronize()
            m.check(m.before, lr=0.25, step=max(step, 1), decay=[0.3] * 4, **kw)


def test_device_numbers_of_another_kind_are_refused():
    log("device numbers refused")
    m = Model([64], 7, 32, True)
    batch = m.batch()
    for lr in (torch.tensor(1.0), torch.ones(2, device=DEV),
               torch.tensor(1.0, dtype=torch.float64, device=DEV)):
        with pytest.raises(TypeError):
            batch.run(lr=lr, step=1)
    for step in (torch.tensor(1), torch.tensor(1, dtype=torch.int32, device=DEV)):
        with pytest.raises(TypeError):
            batch.run(lr=1.0, step=step)
    for step in (0, -1):
        with pytest.raises(RuntimeError, match="EINVAL"):
            batch.run(lr=1.0, step=step)


def test_lists_that_do_not_fit_are_refused():
    log("lists refused")
    m = Model([64, 40], 7, 8, True)
    good = dict(masters=m.masters, states=m.states, state_bits=8)
    cut = [m.grads[0], m.grads[1][:39]]
    for change, error in (
            (dict(masters=[x.half() for x in m.masters]), TypeError),
            (dict(masters=[x.cpu() for x in m.masters]), TypeError),
            (dict(masters=m.masters[::-1]), ValueError),
            (dict(out=[torch.empty(128, dtype=torch.bfloat16, device=DEV)[::2], m.weights[1]]),
             ValueError),
            (dict(out=[torch.empty(65, dtype=torch.bfloat16, device=DEV)[1:], m.weights[1]]),
             ValueError),
            (dict(states=m.states[:2]), ValueError),
            (dict(states=(m.states[0], m.states[1], m.states[2], m.states[2][:1])), ValueError),
            (dict(state_bits=32), ValueError),
            (dict(weight_decay=[0.1]), ValueError),
            (dict(weight_decay=-0.1), ValueError),
            (dict(lr_scale=math.nan), ValueError)):
        with pytest.raises(error):
            AdamWBatch(m.weights, m.grads, **{**good, **change})
    with pytest.raises(ValueError):
        AdamWBatch(m.weights, cut, **good)
    with pytest.raises(TypeError):
        GradNormBatch([m.grads[0].half()])
    with pytest.raises(ValueError):
        m.batch().pairs()
    norm = GradNormBatch(m.grads)
    for bad in (0.0, -1.0, math.nan):
        with pytest.raises(ValueError):
            norm.run(bad)
    with pytest.raises(ValueError):
        norm.run(1.0, math.inf)


def test_runs_on_another_stream():
    log("another stream")
    a, b = (Model(SIZES, 71, 8, True) for _ in range(2))
    side = torch.cuda.Stream()
    norm, batch = GradNormBatch(a.grads), a.batch()
    with torch.cuda.stream(side):
        norm.run(0.1)
        batch.run(lr=1e-3, step=2, norm=norm)
    side.synchronize()
    norm2, batch2 = GradNormBatch(b.grads), b.batch()
    norm2.run(0.1)
    batch2.run(lr=1e-3, step=2, norm=norm2)
    torch.cuda.synchronize()
    x, y = a.snapshot(), b.snapshot()
    assert all(np.array_equal(i, j) for i, j in zip(x["out"], y["out"]))
    assert all(np.array_equal(k, l) for i, j in zip(x["s"], y["s"]) for k, l in zip(i, j))


def test_a_capture_refuses_to_prepare():
    log("prepare in a capture")
    grads = [torch.zeros(64, device=DEV)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = torch.zeros(1, device=DEV)
    with torch.cuda.graph(graph, stream=side):
        keep.add_(1)
        with pytest.raises(RuntimeError, match="EINVAL"):
            GradNormBatch(grads)
    graph.replay()
    torch.cuda.synchronize()
    assert keep.item() == 1


def test_a_shared_tensor_listed_twice_is_refused():
    log("shared tensors")
    m = Model([100, 100], 81, 32, True)
    for change in ("weights", "masters"):
        x = Model([100, 100], 81, 32, True)
        getattr(x, change)[1] = getattr(x, change)[0]
        if change == "weights":
            x.out = x.weights
        with pytest.raises(RuntimeError, match="EINVAL"):
            x.batch()
    m.grads[1] = m.grads[0]        # a gradient is only read
    m.batch()
