"""The losses of a policy update, between a model's logits and the gradients that the
optimizer step takes: cases, plain forms and inputs.

Operators: log probabilities of given tokens with their entropy and the top
alternatives ("logp"); the whole way from logits to their gradient through the
clipped policy loss ("train"); that loss alone ("policy"); and the balance loss of
a router with its per-expert counts and gradient ("balance").  Logits hold some
entries of -infinity (a vocabulary padded to a round size), some tokens are left
out (prompts, padding: id -1), and no ratio lies on a border of the clip range,
where 32 bits decide either way.
"""
import math

import torch

own = False

CLIP_LOW, CLIP_HIGH = 0.2, 0.28
KL, ENTROPY = 0.02, 0.003       # coefficients of the policy loss, where a case has them
BALANCE, Z = 0.01, 0.001        # and of the router's
NEAR = 1e-3                     # log ratios keep this far from the clip range's borders


def _logits(name, op, rows, vocab, dtype="bf16", entropy=True, top=0, temperature=1.0, kl=False):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype,
            "entropy": entropy, "top": top, "temperature": temperature, "kl": kl}


def _tokens(name, rows, entropy=False, kl=False):
    return {"name": name, "op": "policy", "rows": rows, "entropy": entropy, "kl": kl}


def _router(name, rows, experts, choices, dtype="fp32", z=False):
    return {"name": name, "op": "balance", "rows": rows, "experts": experts, "choices": choices,
            "dtype": dtype, "z": z}


def listed():
    return [
        # one sampled token with the usual handful of alternatives: latency
        _logits("logp one token", "logp", 1, 32000, entropy=False, top=5),
        # a decoding batch with a large vocabulary and many alternatives
        _logits("logp 96 tokens top 20", "logp", 96, 131072, top=20),
        # prompts scored under a sampling temperature, fp32 logits, sizes that divide nothing
        _logits("logp prompts odd fp32", "logp", 1021, 50021, dtype="fp32", temperature=0.7),
        # a tiny model's update: latency of the three calls
        _logits("train tiny fp32", "train", 24, 1003, dtype="fp32"),
        # a micro-batch of the 7B-shaped model, with an entropy bonus
        _logits("train 4096 tokens", "train", 4096, 32000),
        # rows that start on odd elements, no entropy
        _logits("train odd rows", "train", 2039, 100003, entropy=False),
        # a large vocabulary in fp32, entropy bonus and reference policy
        _logits("train wide fp32", "train", 4096, 131072, dtype="fp32", kl=True),
        # the loss of one micro-batch: latency
        _tokens("policy 4096 tokens", 4096),
        # the loss of a whole batch at once, with every term
        _tokens("policy whole batch", 1000003, entropy=True, kl=True),
        # a small router: latency
        _router("balance tiny", 64, 8, 2, dtype="bf16"),
        # one layer's router over a batch
        _router("balance layer", 65536, 64, 8, z=True),
        # many experts, a number that divides nothing
        _router("balance wide odd", 32771, 257, 6, dtype="bf16", z=True),
    ]


def _spread(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["logp", "logp", "train", "train", "policy", "balance"])
    if op == "policy":
        case = _tokens("", _spread(rng, 1, 1000000), rng.random() < 0.5, rng.random() < 0.5)
    elif op == "balance":
        experts = _spread(rng, 4, 384)
        case = _router("", _spread(rng, 1, 65536), experts, rng.randint(1, min(8, experts)),
                       rng.choice(["bf16", "fp32"]), rng.random() < 0.5)
    else:
        top = rng.choice([0, 1, 5, 20]) if op == "logp" else 0
        while True:
            rows, vocab = _spread(rng, 1, 256 if top else 8192), _spread(rng, 300, 160000)
            if rows * vocab <= 4096 * 131072:
                break
        case = _logits("", op, rows, vocab, rng.choice(["bf16", "fp32"]), rng.random() < 0.6, top,
                       rng.choice([1.0, 1.0, 0.7, 1.3]), op == "train" and rng.random() < 0.4)
    del case["name"]
    return case


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)

    def normal(*size):
        return torch.randn(*size, generator=gen, device=dev)

    def uniform(*size):
        return torch.rand(*size, generator=gen, device=dev)

    n = case["rows"]
    s = {"case": case}
    if case["op"] == "balance":
        # experts that are preferred overall, tokens of unequal decision
        logits = normal(n, case["experts"]).mul_(1 + uniform(n, 1)).add_(normal(case["experts"]))
        s["logits"] = logits.to(_type(case))
        s["chosen"] = s["logits"].float().topk(case["choices"], dim=1).indices
        s["mask"] = uniform(n) > 0.06       # the rest is padding
        s["out"] = torch.empty_like(s["logits"])
    if case["op"] in ("logp", "train"):
        vocab = case["vocab"]
        # flat and peaked rows; the last entries are no tokens
        logits = normal(n, vocab).mul_(0.5 + 2.5 * uniform(n, 1))
        logits[:, vocab - vocab // 250:] = -math.inf
        tokens = (uniform(n) * (vocab - vocab // 250)).long().clamp(max=vocab - vocab // 250 - 1)
        # most tokens are ones that the model would draw
        at = tokens[:, None]
        logits.scatter_add_(1, at, (4 + 8 * uniform(n))[:, None])
        s["logits"] = logits.to(_type(case))
        del logits
        s["tokens"] = torch.where(uniform(n) < 0.05, -1, tokens)
        s["tokens"][0] = tokens[0]
    if case["op"] in ("train", "policy"):
        if case["op"] == "train":
            s["out"] = torch.empty_like(s["logits"])
            step = max(1, (1 << 26) // case["vocab"])
            logp = torch.cat([_plain_logp(s["logits"][a:a + step], s["tokens"][a:a + step],
                                          case["temperature"], False, 0)["logp"]
                              for a in range(0, n, step)])
        else:
            logp = -normal(n).square_()
            s["logp"] = logp
            s["entropy"] = 3 * uniform(n) if case["entropy"] else None
        ratio = 0.15 * normal(n)
        for border in (math.log1p(-CLIP_LOW), math.log1p(CLIP_HIGH)):
            ratio = torch.where((ratio - border).abs() < NEAR, 0.0, ratio)
        s["old"] = logp - ratio
        s["ref"] = logp + 0.3 * normal(n) if case["kl"] else None
        s["advantages"] = normal(n).add_(0.25)
        s["weights"] = (uniform(n) > 0.1).float()
        s["weights"][0] = 1.0
        if case["op"] == "train":
            s["weights"] *= s["tokens"] >= 0
    if own:
        import lossless_bf16_weight_xor_amd as bd
        if case["op"] in ("logp", "train"):
            s["probs"] = bd.TokenLogProbs(n, case["vocab"], dev, entropy=case["entropy"],
                                          top=case["top"])
        if case["op"] in ("train", "policy"):
            s["loss"] = bd.PolicyLoss(n, dev)
        if case["op"] == "balance":
            s["router"] = bd.RouterBalance(n, case["experts"], dev, balance_coef=BALANCE,
                                           z_coef=Z if case["z"] else 0.0)
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    case = s["case"]
    if case["op"] == "balance":
        router = s["router"]
        router.run(s["logits"], s["chosen"], mask=s["mask"])
        router.backward(s["logits"], s["out"], mask=s["mask"])
        return {"counts": router.counts, "tokens": router.tokens, "loss": router.loss,
                "balance": router.balance, "z": router.z, "grad": s["out"]}
    found = {}
    if case["op"] in ("logp", "train"):
        probs = s["probs"]
        probs.run(s["logits"], s["tokens"], temperature=case["temperature"])
        found["logp"] = probs.logp
        if case["entropy"]:
            found["entropy"] = probs.entropy
        if case["top"]:
            found |= {"top_ids": probs.top_ids, "top_logp": probs.top_logp}
        if case["op"] == "logp":
            return found
    loss = s["loss"]
    logp, entropy = (found["logp"], found.get("entropy")) if case["op"] == "train" \
        else (s["logp"], s["entropy"])
    loss.run(logp, s["old"], s["advantages"], weights=s["weights"], ref_logp=s["ref"],
             entropy=entropy, clip=(CLIP_LOW, CLIP_HIGH), kl_coef=KL if case["kl"] else 0.0,
             entropy_coef=ENTROPY if case["entropy"] else 0.0, scale=1 / case["rows"])
    grad_entropy = loss.grad_entropy if case["entropy"] else None
    found |= {"loss": loss.loss, "grad_logp": loss.grad_logp}
    if case["op"] == "policy":
        found |= {"weight": loss.weight, "kl": loss.kl, "clipped": loss.clipped}
        if case["entropy"]:
            found |= {"grad_entropy": grad_entropy, "mean_entropy": loss.entropy}
        return found
    probs.backward(s["logits"], s["tokens"], loss.grad_logp, s["out"], grad_entropy=grad_entropy)
    return found | {"grad": s["out"]}


# ------------------------------------------------------------ plain forms ---

def _plain(s):
    case = s["case"]
    if case["op"] == "balance":
        return _plain_balance(s["logits"], s["chosen"], s["mask"], Z if case["z"] else 0.0)
    if case["op"] == "policy":
        return _plain_policy(s, s["logp"], s["entropy"])
    found = _plain_logp(s["logits"], s["tokens"], case["temperature"], case["entropy"],
                        case["top"])
    if case["op"] == "logp":
        return found
    loss = _plain_policy(s, found["logp"], found.get("entropy"))
    grad = _plain_grad(s["logits"], s["tokens"], case["temperature"], loss["grad_logp"],
                       loss.get("grad_entropy"))
    return found | {"loss": loss["loss"], "grad_logp": loss["grad_logp"], "grad": grad}


def _plain_logp(logits, tokens, temperature, entropy, top):
    x = logits.float()
    d = (x - x.amax(1, keepdim=True)) / temperature
    e = d.exp()
    total = e.sum(1)
    live = tokens >= 0
    own_d = d.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    found = {"logp": torch.where(live, own_d - total.log(), 0.0)}
    if entropy:
        e *= d.clamp(min=-1e4)
        found["entropy"] = torch.where(live, total.log() - e.sum(1) / total, 0.0)
    if top:
        # the order of the values, then the lowest id, as one integer
        bits = (x + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 32)
        order -= torch.arange(x.shape[1], device=x.device)
        ids = torch.remainder(-order.topk(top, dim=1).values, 1 << 32)
        found["top_ids"] = torch.where(live[:, None], ids, -1)
        found["top_logp"] = torch.where(live[:, None], d.gather(1, ids) - total.log()[:, None],
                                        -math.inf)
    return found


def _plain_grad(logits, tokens, temperature, grad_logp, grad_entropy):
    x = logits.float()
    d = (x - x.amax(1, keepdim=True)) / temperature
    d -= d.exp().sum(1, keepdim=True).log()
    p = d.exp()
    live = (tokens >= 0).float()[:, None]
    a = grad_logp[:, None] * live
    if grad_entropy is None:
        g = -a * p
    else:
        d.clamp_(min=-1e4)
        d += (p * -d).sum(1, keepdim=True)
        g = p * (-a - grad_entropy[:, None] * live * d)
    g.scatter_add_(1, tokens.clamp(min=0)[:, None], a)
    return g.div_(temperature).to(logits.dtype)


def _plain_policy(s, logp, entropy):
    """In 64 bits: close to 1, a ratio's distance from a border and from 1 matters."""
    case, w = s["case"], s["weights"].double()
    scale = 1 / case["rows"]
    change = logp.double() - s["old"].double()
    ratio, adv = change.exp(), s["advantages"].double()
    bounded = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    cut = bounded * adv < ratio * adv
    each = -torch.where(cut, bounded * adv, ratio * adv)
    slope = torch.where(cut, 0.0, -ratio * adv)
    if case["kl"]:
        away = s["ref"].double() - logp.double()
        each = each + KL * (torch.expm1(away) - away)
        slope = slope - KL * torch.expm1(away)
    found = {}
    if entropy is not None:
        each = each - ENTROPY * entropy.double()
        found["grad_entropy"] = (-scale * ENTROPY * w).float()
        found["mean_entropy"] = ((w * entropy.double()).sum() / w.sum()).float()
    return found | {
        "loss": (scale * (w * each).sum()).float(), "grad_logp": (scale * w * slope).float(),
        "weight": w.sum().float(), "clipped": ((w * cut).sum() / w.sum()).float(),
        "kl": ((w * (torch.expm1(change) - change)).sum() / w.sum()).float()}


def _plain_balance(logits, chosen, mask, z_coef):
    experts = logits.shape[1]
    keep = mask.float()[:, None]
    tokens = mask.sum()
    counts = torch.zeros(experts, dtype=torch.int64, device=logits.device)
    counts.scatter_add_(0, chosen.flatten(), mask.long()[:, None].expand(chosen.shape).flatten())
    share = counts.float() / counts.sum().clamp(min=1)
    n = tokens.clamp(min=1).float()
    x = logits.float()
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(1, keepdim=True)
    p = e / total * keep
    lse = (m + total.log()) * keep
    balance = experts * (share * p.sum(0)).sum() / n
    z = lse.square().sum() / n
    inner = BALANCE * experts * (share - (p * share).sum(1, keepdim=True)) + 2 * z_coef * lse
    return {"counts": counts, "tokens": tokens, "balance": balance, "z": z,
            "loss": BALANCE * balance + z_coef * z, "grad": (p * inner / n).to(logits.dtype)}


# ---------------------------------------------------- definition in 64 bits ---

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(s)
    if case["op"] == "policy":
        return _exact_policy(s, s["logp"].double(),
                             None if s["entropy"] is None else s["entropy"].double())
    logits, tokens, t = s["logits"], s["tokens"], case["temperature"]
    step = max(1, (1 << 26) // case["vocab"])
    rows = [slice(a, a + step) for a in range(0, case["rows"], step)]
    parts = {"logp": [], "entropy": [], "top_logp": []}
    for r in rows:
        y = torch.log_softmax(logits[r].double() / t, dim=1)
        drop = tokens[r] < 0
        logp = y[torch.arange(y.shape[0], device=y.device), tokens[r].clamp(min=0)]
        parts["logp"].append(logp.masked_fill(drop, 0.0))
        parts["entropy"].append(torch.special.entr(y.exp()).sum(1).masked_fill(drop, 0.0))
        if case["top"]:
            best = y.sort(dim=1, descending=True).values[:, :case["top"]]
            parts["top_logp"].append(best.masked_fill(drop[:, None], -math.inf))
    logp, entropy = torch.cat(parts["logp"]), torch.cat(parts["entropy"])
    found = {"logp": logp}
    if case["entropy"]:
        found["entropy"] = entropy
    if case["top"]:
        found |= {"top_ids": None, "top_logp": torch.cat(parts["top_logp"])}
    if case["op"] == "logp":
        return found
    loss = _exact_policy(s, logp, entropy if case["entropy"] else None)
    grad = []
    for r in rows:
        y = torch.log_softmax(logits[r].double() / t, dim=1)
        keep = (tokens[r] >= 0).double()
        a = loss["grad_logp"][r] * keep / t
        g = y.exp() * -a[:, None]
        if case["entropy"]:
            h = loss["grad_entropy"][r] * keep / t
            # p (ln p + H), with p ln p = 0 where p is 0
            g -= h[:, None] * (y.exp() * entropy[r][:, None] - torch.special.entr(y.exp()))
        at = torch.arange(g.shape[0], device=g.device)
        g[at, tokens[r].clamp(min=0)] += a
        grad.append(g)
    return found | {"loss": loss["loss"], "grad_logp": loss["grad_logp"],
                    "grad": torch.cat(grad)}


def _exact_policy(s, logp, entropy):
    case = s["case"]
    w, adv, old = (s[k].double() for k in ("weights", "advantages", "old"))
    log_ratio = logp - old
    high = (log_ratio > math.log1p(CLIP_HIGH)) & (adv > 0)
    low = (log_ratio < math.log1p(-CLIP_LOW)) & (adv < 0)
    gain = torch.exp(log_ratio) * adv
    slope = -gain.masked_fill(high | low, 0.0)
    gain = torch.where(high, (1 + CLIP_HIGH) * adv, torch.where(low, (1 - CLIP_LOW) * adv, gain))
    loss = -(w * gain).sum()
    if case["kl"]:
        u = s["ref"].double() - logp
        loss += KL * (w * (u.exp() - u - 1)).sum()
        slope += KL * (1 - u.exp())
    n, found = case["rows"], {}
    if entropy is not None:
        loss -= ENTROPY * (w * entropy).sum()
        found = {"grad_entropy": -ENTROPY * w / n, "mean_entropy": (w * entropy).sum() / w.sum()}
    return found | {"loss": loss / n, "grad_logp": slope * w / n, "weight": w.sum(),
                    "clipped": w[high | low].sum() / w.sum(),
                    "kl": (w * (log_ratio.exp() - log_ratio - 1)).sum() / w.sum()}


def _exact_balance(s):
    live = s["mask"]
    experts = s["logits"].shape[1]
    y = torch.log_softmax(s["logits"].double(), dim=1)
    p = y.exp()
    lse = torch.logsumexp(s["logits"].double(), dim=1)
    n = max(1, int(live.sum()))
    counts = torch.bincount(s["chosen"][live].flatten(), minlength=experts)
    f = counts.double() / max(1, int(counts.sum()))
    balance = experts * (f @ p[live].sum(0)) / n
    z = lse[live].square().sum() / n
    zc = Z if s["case"]["z"] else 0.0
    grad = p * (BALANCE * experts * (f - (p @ f)[:, None]) + 2 * zc * lse[:, None]) / n
    return {"counts": counts, "tokens": None, "balance": balance, "z": z,
            "loss": BALANCE * balance + zc * z, "grad": grad * live[:, None]}


def work(case):
    """Logits count once where they are read and once where their gradient is written;
    about ten operations an element for a softmax and its sums, as many for the gradient."""
    n = case["rows"]
    if case["op"] == "policy":
        arrays = 5 + 2 * case["entropy"] + case["kl"]
        return {"bytes": 4 * n * arrays, "flops": 30 * n}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "balance":
        e = n * case["experts"]
        return {"bytes": 2 * e * size + n * (8 * case["choices"] + 1) + 8 * case["experts"],
                "flops": 20 * e}
    e = n * case["vocab"]
    row = 8 + 4 + 4 * case["entropy"] + 12 * case["top"]
    if case["op"] == "logp":
        return {"bytes": e * size + n * row, "flops": 10 * e}
    return {"bytes": 2 * e * size + n * (row + 4 * (4 + case["kl"])), "flops": 20 * e}
