"""The trainer's step that makes the new weights: cases, plain forms and inputs.

Operators: the AdamW step over many tensors with 32-bit or 8-bit states, and
the global gradient norm with its clip factor.  A case lists the tensors of a
decoder stack (hidden, ffn, layers, vocab) as one flat arena per quantity,
each tensor starting on a multiple of 512 elements and the gaps holding zeros;
the matrices come first (with weight decay), the vectors after them (without).
The plain forms work on the arenas, the framework's calls on the list of
tensors in them.  Every case's gradients are finite.
"""
import math

import torch

own = False

SPAN = 512            # a tensor starts on a multiple of this many elements
BLOCK = 32            # elements that share a scale byte (8-bit states)
LR, BETA1, BETA2, EPS, DECAY, MAX_NORM = 1e-4, 0.9, 0.95, 1e-8, 0.1, 1.0
M32, M64 = (1 << 32) - 1, (1 << 64) - 1


def _case(name, op, hidden, ffn, layers, vocab, grad="bf16", bits=32, master=True, clip=False):
    return {"name": name, "op": op, "hidden": hidden, "ffn": ffn, "layers": layers,
            "vocab": vocab, "grad": grad, "bits": bits, "master": master, "clip": clip}


def listed():
    return [
        # the gradients of a tiny model, where the launch is all there is
        _case("norm tiny", "norm", 96, 259, 2, 0),
        # eight 7B-shaped layers with their embedding, bf16 gradients
        _case("norm bf16 8 layers", "norm", 4096, 11008, 8, 32000),
        # one wide layer of a 70B-shaped model, gradients accumulated in fp32
        _case("norm fp32 wide layer", "norm", 8192, 28672, 1, 0, grad="fp32"),
        # a tiny model's whole step: latency
        _case("step32 tiny", "step", 96, 259, 2, 0),
        # one 7B-shaped layer, the usual mixed-precision set-up
        _case("step32 layer", "step", 4096, 11008, 1, 0),
        # four 7B-shaped layers, fp32 gradients, clipped by their global norm
        _case("step32 clipped fp32", "step", 4096, 11008, 4, 0, grad="fp32", clip=True),
        # bf16 weights without a master copy, sizes that divide nothing
        _case("step32 no master odd", "step", 1283, 3517, 5, 0, master=False),
        # a tiny model's whole step with 8-bit states: latency
        _case("step8 tiny", "step", 96, 259, 2, 0, bits=8),
        # one 7B-shaped layer with 8-bit states
        _case("step8 layer", "step", 4096, 11008, 1, 0, bits=8),
        # four 7B-shaped layers, 8-bit states and no master copy, clipped
        _case("step8 no master clipped", "step", 4096, 11008, 4, 0, bits=8, master=False,
              clip=True),
        # fp32 gradients, 8-bit states, sizes that divide nothing
        _case("step8 fp32 odd", "step", 1283, 3517, 5, 0, grad="fp32", bits=8),
        # an embedding alone: one large tensor
        _case("step8 embedding", "step", 4096, 0, 0, 32000, bits=8),
    ]


def draw(rng):
    op = rng.choice(["norm", "step", "step", "step"])
    while True:
        hidden = round(math.exp(rng.uniform(math.log(48), math.log(6144))))
        ffn = round(hidden * rng.uniform(1.5, 4.0))
        layers = rng.randint(1, 12)
        vocab = rng.choice([0, 0, round(math.exp(rng.uniform(math.log(500), math.log(64000))))])
        n = layers * (4 * hidden * hidden + 3 * hidden * ffn) + vocab * hidden
        if n <= 600_000_000:
            break
    case = _case("", op, hidden, ffn, layers, vocab, grad=rng.choice(["bf16", "fp32"]),
                 bits=rng.choice([32, 8]), master=rng.random() < 0.6, clip=rng.random() < 0.5)
    del case["name"]
    return case


def _tensors(case):
    """(elements of each tensor, how many of the tensors have weight decay)."""
    h, f, layers, vocab = case["hidden"], case["ffn"], case["layers"], case["vocab"]
    matrices = [vocab * h] * (vocab > 0) + ([h * h] * 4 + [f * h] * 3) * layers
    return matrices + [h] * (2 * layers + (vocab > 0)), len(matrices)


def _layout(case):
    """(elements and start of each tensor, decayed tensors, start of the vectors, arena size)."""
    sizes, matrices = _tensors(case)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // SPAN) * SPAN
    return sizes, starts, matrices, starts[matrices], at


def _nearest_block_scaled(x):
    """(e4m3 codes, E8M0 scale bytes) of x, as a checkpoint of 8-bit states holds it."""
    byte = _scale_byte(x.abs().view(-1, BLOCK).amax(1))
    codes = (x.view(-1, BLOCK) * _power_of_two(254 - byte)[:, None]).to(torch.float8_e4m3fn)
    return codes.view(-1), byte.to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    sizes, starts, matrices, vectors_at, total = _layout(case)

    def normal():
        return torch.randn(total, generator=gen, device=dev)

    # gradients whose size differs from row to row (log-normal), some rows
    # without any gradient so far (tokens that have not occurred)
    rows = torch.randn(total // SPAN, 1, generator=gen, device=dev).exp_().mul_(1e-3)
    rows *= torch.rand(total // SPAN, 1, generator=gen, device=dev) > 0.03
    live = torch.ones(total, dtype=torch.bool, device=dev)
    for start, n in zip(starts, sizes):
        live[start + n:start + -(-n // SPAN) * SPAN] = False

    def spread(x):
        return x.view(-1, SPAN).mul_(rows).view(-1).mul_(live)

    grad = spread(normal())
    s = {"case": case, "vectors_at": vectors_at, "step": 40 + seed % 1000, "seed": seed,
         "grad": grad if case["grad"] == "fp32" else grad.to(torch.bfloat16)}
    del grad

    def views(t, per=1):
        return [t[a // per:a // per + -(-n // per)] for a, n in zip(starts, sizes)]

    if case["op"] == "step":
        master = normal().mul_(0.02).mul_(live)
        s["weights"] = master.to(torch.bfloat16)
        s["master"] = master if case["master"] else None
        del master
        m = spread(normal().mul_(0.25))
        v = spread(spread(torch.rand(total, generator=gen, device=dev).add_(0.25)))
        s["m_scale"] = s["v_scale"] = None
        if case["bits"] == 8:
            m, s["m_scale"] = _nearest_block_scaled(m)
            v, s["v_scale"] = _nearest_block_scaled(v)
        s["m"], s["v"] = m, v
    if own:
        import lossless_bf16_weight_xor_amd as bd
        grads = views(s["grad"])
        if case["op"] == "norm" or case["clip"]:
            s["norm"] = bd.GradNormBatch(grads)
        if case["op"] == "step":
            scales = (views(s["m_scale"], BLOCK), views(s["v_scale"], BLOCK)) \
                if case["bits"] == 8 else ()
            s["batch"] = bd.AdamWBatch(
                views(s["weights"]), grads,
                masters=views(s["master"]) if case["master"] else None,
                states=(views(s["m"]), views(s["v"]), *scales), state_bits=case["bits"],
                weight_decay=[DECAY if j < matrices else 0.0 for j in range(len(sizes))])
    return s


def run(state):
    case = state["case"]
    found = {}
    norm = None
    if case["op"] == "norm" or case["clip"]:
        if own:
            norm = state["norm"]
            norm.run(max_norm=MAX_NORM)
            found = {"norm": norm.norm, "scale": norm.scale, "nonfinite": norm.nonfinite}
        else:
            found = _plain_norm(state["grad"])
    if case["op"] == "step":
        if own:
            state["batch"].run(lr=LR, step=state["step"], betas=(BETA1, BETA2), eps=EPS,
                               seed=state["seed"], norm=norm)
        else:
            _plain_step(state, found.get("scale"))
        state["step"] += 1
        found |= {"weights": state["weights"], "master": state["master"],
                  "m": state["m"], "v": state["v"]}
        if case["bits"] == 8:
            found |= {k: state[k].view(torch.float8_e8m0fnu) for k in ("m_scale", "v_scale")}
    return found


# ------------------------------------------------------------ plain forms ---

def _plain_norm(grad):
    norm = grad.float().square().sum(dtype=torch.float64).sqrt()
    return {"norm": norm, "scale": (MAX_NORM / norm).clamp(max=1.0).float(),
            "nonfinite": (~torch.isfinite(norm)).int()}


def _plain_step(s, scale):
    case, t = s["case"], s["step"]
    c1, c2 = -math.expm1(t * math.log(BETA1)), -math.expm1(t * math.log(BETA2))
    g = s["grad"].float()
    if scale is not None:
        g = g * scale
    m, v = s["m"], s["v"]
    if case["bits"] == 8:
        m, v = _decode(m, s["m_scale"]), _decode(v, s["v_scale"])
    p = s["master"] if case["master"] else s["weights"].float()
    m.mul_(BETA1).add_(g, alpha=1 - BETA1)
    v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    update = m / v.sqrt().mul_(1 / math.sqrt(c2)).add_(EPS)
    update.mul_(LR / c1)
    at = s["vectors_at"]
    update[:at].add_(p[:at], alpha=LR * DECAY)
    p.sub_(update)
    del update, g
    random = None
    if case["bits"] == 8 or not case["master"]:
        random = _random_bits(p.numel(), s["seed"], t, p.device)
    if case["master"]:
        s["weights"].copy_(p)
    else:
        r = ((random * _signed(0x9E3779B1)) >> 16) & 0xFFFF
        s["weights"].copy_(((p.view(torch.int32) + r) & -0x10000).view(torch.float32))
    if case["bits"] == 8:
        _encode(m, random & 0xFFFF, False, s["m"], s["m_scale"])
        _encode(v, (random >> 16) & 0xFFFF, True, s["v"], s["v_scale"])


def _power_of_two(byte):
    """2^(byte - 127), byte from 1 to 254."""
    return (byte.int() << 23).view(torch.float32)


def _scale_byte(top):
    """The smallest byte (from 1) with top <= 448 * 2^(byte - 127)."""
    return (((top.view(torch.int32) + 0x1FFFFF) >> 23) - 8).clamp(min=1)


def _decode(codes, scale):
    return (codes.float().view(-1, BLOCK) * _power_of_two(scale)[:, None]).view(-1)


def _encode(x, r, positive, codes, scale):
    """x rounded to e4m3 times a power of two per block, up where the fraction of a
    step, cut to 16 bits, and the random number r reach 2^16; a positive v stays positive."""
    byte = _scale_byte(x.abs().view(-1, BLOCK).amax(1))
    t = (x.abs().view(-1, BLOCK) * _power_of_two(254 - byte)[:, None]).view(-1)
    normal = ((t.view(torch.int32) + (r << 4)) & -0x100000).view(torch.float32)
    small = (((t * 2.0 ** 25).int() + r) >> 16).float() * 2.0 ** -9
    y = torch.where(t >= 2.0 ** -6, normal, small)
    if positive:
        y = torch.where((y == 0) & (x > 0), 2.0 ** -9, y)
    codes.copy_(torch.copysign(y, x).to(torch.float8_e4m3fn))
    scale.copy_(byte)


def _mix64(z):
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & M64
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & M64
    return z ^ (z >> 31)


def _signed(x):
    return x - (1 << 32) if x >> 31 else x


def _random_bits(n, seed, step, dev):
    """32 random bits per element of the arena (below 2^31 elements), as int32, from
    seed, step and place; products and sums wrap."""
    key = _mix64((_mix64(seed) + step) & M64)
    x = torch.arange(n, dtype=torch.int32, device=dev) ^ _signed(key & M32)
    x = (x ^ ((x >> 16) & 0xFFFF)).mul_(_signed(0xBF58476D)).add_(_signed(key >> 32))
    x = (x ^ ((x >> 15) & 0x1FFFF)).mul_(_signed(0x94D049BB))
    return x ^ ((x >> 16) & 0xFFFF)


# ---------------------------------------------------- definition in 64 bits ---

def _exact_random(first, n, seed, step, dev):
    def mix(z):
        for shift, factor in ((30, 0xBF58476D1CE4E5B9), (27, 0x94D049BB133111EB)):
            z ^= z >> shift
            z = z * factor % (1 << 64)
        return z ^ z >> 31

    key = mix((mix(seed) + step) % (1 << 64))
    low, high = key % (1 << 32), key >> 32

    def times(a, factor):     # modulo 2^32, in two halves that stay below 2^63
        return (a * (factor % 65536) + ((a * (factor >> 16)) % 65536) * 65536) % (1 << 32)

    x = torch.arange(first, first + n, device=dev).bitwise_xor(low)
    x = times(x.bitwise_xor(x // 65536), 0xBF58476D).add(high).remainder(1 << 32)
    x = times(x.bitwise_xor(x // 32768), 0x94D049BB)
    return x.bitwise_xor(x // 65536)


def _exact_block(x, r, positive):
    """(e4m3 values, scales) of one slice in 64 bits."""
    x = x.reshape(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    mantissa, exponent = torch.frexp(top / 448)       # top <= 448 * 2^k
    k = torch.where(mantissa == 0.5, exponent - 1, exponent)
    k = torch.where(top > 0, k, torch.full_like(k, -126)).clamp(min=-126)
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), k)
    t = x.abs() / scale
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device),
                     (torch.frexp(t)[1] - 1).clamp(min=-6) - 3)
    whole = torch.floor(t / step)
    cut = torch.floor((t / step - whole) * 65536)
    y = (whole + (cut + r.reshape(-1, BLOCK) >= 65536)) * step
    if positive:
        y = torch.where((y == 0) & (x > 0), torch.full_like(y, 2.0 ** -9), y)
    return (y * x.sign()).reshape(-1), scale.reshape(-1)


def exact(case, seed):
    s = prepare(case, seed)
    total = s["grad"].numel()
    found, factor = {}, 1.0
    if case["op"] == "norm" or case["clip"]:
        squares = torch.zeros((), dtype=torch.float64, device=s["grad"].device)
        for at in range(0, total, 1 << 26):
            squares += (s["grad"][at:at + (1 << 26)].double() ** 2).sum()
        norm = squares ** 0.5
        factor = torch.where(norm > MAX_NORM, MAX_NORM / norm, torch.ones_like(norm))
        found = {"norm": norm, "scale": factor, "nonfinite": torch.zeros_like(norm).int()}
    if case["op"] == "norm":
        return found
    dev, t = s["grad"].device, s["step"]
    bits8, master = case["bits"] == 8, case["master"]
    out = {k: [] for k in ("weights", "m", "v") + ("master",) * master
           + ("m_scale", "v_scale") * bits8}
    for a in range(0, total, 1 << 26):
        b = min(total, a + (1 << 26))
        g = s["grad"][a:b].double() * factor
        if bits8:
            m, v = ((s[k][a:b].double().reshape(-1, BLOCK)
                     * torch.pow(2.0, s[k + "_scale"][a // BLOCK:b // BLOCK].double() - 127)
                     .reshape(-1, 1)).reshape(-1) for k in ("m", "v"))
        else:
            m, v = s["m"][a:b].double(), s["v"][a:b].double()
        p = (s["master"] if master else s["weights"])[a:b].double()
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        wd = torch.where(torch.arange(a, b, device=dev) < s["vectors_at"], DECAY, 0.0)
        p = p - LR * wd.double() * p - LR * (m / (1 - BETA1 ** t)) / (
            (v / (1 - BETA2 ** t)) ** 0.5 + EPS)
        r = _exact_random(a, b - a, seed, t, dev) if bits8 or not master else None
        if master:
            out["master"].append(p)
            out["weights"].append(p)
        else:
            step = torch.pow(2.0, (torch.frexp(p)[1] - 8).double())
            whole = torch.floor(p.abs() / step)
            cut = torch.floor((p.abs() / step - whole) * 65536)
            up = cut + (r * 0x9E3779B1 % (1 << 32)) // 65536 >= 65536
            out["weights"].append((whole + up) * step * p.sign())
        if bits8:
            for k, x, bits, positive in (("m", m, r % 65536, False), ("v", v, r // 65536, True)):
                y, scale = _exact_block(x, bits, positive)
                out[k].append(y)
                out[k + "_scale"].append(scale)
        else:
            out["m"].append(m)
            out["v"].append(v)
    found["master"] = None
    for k in list(out):
        found[k] = torch.cat(out.pop(k))
    return found


def work(case):
    n = sum(_tensors(case)[0])
    grad = 2 if case["grad"] == "bf16" else 4
    if case["op"] == "norm":
        return {"bytes": n * grad, "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 * (1 + 1 / BLOCK)
    weights = 4 + 4 + 2 if case["master"] else 2 + 2
    return {"bytes": n * (grad + state + weights), "flops": 15 * n}
