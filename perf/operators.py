"""Cases of the token-model operators: embedding lookup and its gradient, matrix products
grouped by expert in their three directions, the preference loss and the clipped policy
loss, each loss with its gradient.

`run` makes one pass through one operator.  With `own` it calls this package on the
buffers that a training or serving program keeps; without it computes the same in plain
32-bit torch operations, rounded once at the end.  `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SPREAD = 2.0          # standard deviation of the synthetic logits
TEMPERATURE = 0.9     # of the policy loss

# --------------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding step of 32 sequences: the latency of a lookup
        dict(name="embed decode", op="embed", rows=32, vocab=32000, dim=2048, table="bf16",
             out="bf16"),
        # a packed prompt batch read from an FP32 master table
        dict(name="embed prompt", op="embed", rows=16384, vocab=128000, dim=4096, table="f32",
             out="bf16"),
        # a training batch's table gradient, every row of it written
        dict(name="embed grad", op="embed_grad", rows=8192, vocab=32000, dim=2048, table="f32",
             out="bf16"),
        # long batch, row length odd: no row but the first starts on a 16-byte boundary
        dict(name="embed grad odd", op="embed_grad", rows=40001, vocab=65537, dim=1001,
             table="f32", out="f16"),
        # one decoding step through many experts: the weights' bytes are what counts
        dict(name="experts decode", op="group", rows=64, groups=64, k=2048, n=1024, dtype="bf16",
             skew=0.5),
        # a training batch through 32 experts, skewed routing
        dict(name="experts train", op="group", rows=16384, groups=32, k=2048, n=2816,
             dtype="bf16", skew=0.5),
        # gradient of the rows, few large experts
        dict(name="experts dx", op="group_dx", rows=8192, groups=8, k=4096, n=2048, dtype="f16",
             skew=0.3),
        # gradient of the weights: the ragged length is the one summed over
        dict(name="experts dw", op="group_dw", rows=16384, groups=32, k=2048, n=2816,
             dtype="bf16", skew=0.5),
        # two short pairs, a vocabulary row that is no multiple of 16 bytes
        dict(name="preference short", op="preference", rows=150, pairs=2, vocab=32003,
             dtype="bf16", kind=0, mean=False),
        # a training batch of 16 pairs over a large vocabulary
        dict(name="preference batch", op="preference", rows=12288, pairs=16, vocab=128000,
             dtype="bf16", kind=0, mean=False),
        # a small step on FP32 logits
        dict(name="policy short", op="policy", rows=192, vocab=32000, dtype="f32"),
        # a training batch of sampled answers
        dict(name="policy batch", op="policy", rows=8192, vocab=128000, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "group", "group_dx", "group_dw", "preference",
                     "policy"])
    if op in ("embed", "embed_grad"):
        rows, vocab, dim = _log(rng, 1, 65536), _log(rng, 64, 131072), _log(rng, 8, 8192)
        if rng.random() < 0.6:
            dim = max(8, dim // 8 * 8)
        rows = min(rows, (1 << 27) // dim)
        vocab = min(vocab, (1 << 28) // dim)
        return dict(op=op, rows=rows, vocab=vocab, dim=dim,
                    table="f32" if op == "embed_grad" else rng.choice(["bf16", "f16", "f32"]),
                    out=rng.choice(["bf16", "f16", "f32"]))
    if op.startswith("group"):
        rows, groups = _log(rng, 1, 16384), _log(rng, 1, 128)
        k, n = _log(rng, 64, 4096), _log(rng, 64, 4096)
        if rng.random() < 0.75:
            k, n = k // 8 * 8, n // 8 * 8
        groups = max(1, min(groups, (1 << 28) // (k * n)))
        return dict(op=op, rows=rows, groups=groups, k=k, n=n, dtype=rng.choice(["bf16", "f16"]),
                    skew=round(rng.uniform(0.0, 1.0), 2))
    vocab = _log(rng, 100, 131072)
    if rng.random() < 0.5:
        vocab = max(104, vocab // 8 * 8)
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "policy":
        return dict(op=op, rows=min(_log(rng, 1, 16384), (1 << 29) // vocab), vocab=vocab,
                    dtype=dtype)
    pairs = _log(rng, 1, 64)
    rows = min(2 * pairs * _log(rng, 1, 512), (1 << 29) // vocab)
    return dict(op=op, rows=rows, pairs=pairs, vocab=vocab, dtype=dtype, kind=rng.choice([0, 1]),
                mean=rng.random() < 0.3)


# --------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _split(rows, parts, skew, seed):
    """`parts` ragged lengths that sum to rows, as offsets (some parts may be empty)."""
    rng = np.random.default_rng(seed)
    p = (1.0 + np.arange(parts)) ** -skew * rng.gamma(4.0, size=parts)
    counts = rng.multinomial(rows, rng.permutation(p / p.sum()))
    off = np.zeros(parts + 1, np.int32)
    np.cumsum(counts, out=off[1:])
    return torch.from_numpy(off).cuda(), int(counts.max())


def _token_ids(rows, vocab, g):
    """Token numbers whose frequency falls as one over their rank."""
    u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp_(0, vocab - 1)


def _logits(c, g):
    """Logits, sampled tokens (a tenth of the rows masked) and each row's log probability
    to within the noise of a reference model's."""
    x = torch.randn(c["rows"], c["vocab"], generator=g, device="cuda", dtype=DT[c["dtype"]])
    x *= SPREAD
    t = torch.randint(0, c["vocab"], (c["rows"],), generator=g, device="cuda")
    lp = x.gather(1, t[:, None])[:, 0].float() - math.log(c["vocab"]) - SPREAD ** 2 / 2
    masked = torch.rand(c["rows"], generator=g, device="cuda") < 0.1
    return x, torch.where(masked, -100, t), lp, masked


def prepare(case, seed):
    c, g, s = case, _gen(seed), dict(case)
    op = c["op"]
    if op in ("embed", "embed_grad"):
        s["ids"] = _token_ids(c["rows"], c["vocab"], g)
        s["scale"] = math.sqrt(c["dim"])
        if op == "embed":
            s["weights"] = torch.randn(c["vocab"], c["dim"], generator=g, device="cuda",
                                       dtype=DT[c["table"]])
            s["result"] = torch.empty(c["rows"], c["dim"], device="cuda", dtype=DT[c["out"]])
        else:
            s["dout"] = torch.randn(c["rows"], c["dim"], generator=g, device="cuda",
                                    dtype=DT[c["out"]])
            s["result"] = torch.empty(c["vocab"], c["dim"], device="cuda", dtype=DT[c["table"]])
        if own:
            import communication_avoiding_step_gb300 as casgd
            s["ws"] = casgd.embed_workspace(c["rows"], c["vocab"], c["dim"])
        return s
    if op.startswith("group"):
        dt = DT[c["dtype"]]
        s["offsets"], s["longest"] = _split(c["rows"], c["groups"], c["skew"], seed)

        def rnd(*shape):
            return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

        x, w, y = (c["rows"], c["k"]), (c["groups"], c["n"], c["k"]), (c["rows"], c["n"])
        if op == "group":
            s["a"], s["b"], s["result"] = rnd(*x), rnd(*w), torch.empty(y, device="cuda", dtype=dt)
        elif op == "group_dx":
            s["a"], s["b"], s["result"] = rnd(*y), rnd(*w), torch.empty(x, device="cuda", dtype=dt)
        else:
            s["a"], s["b"], s["result"] = rnd(*y), rnd(*x), torch.empty(w, device="cuda", dtype=dt)
        if op != "group_dw":
            s["b"] *= c["k"] ** -0.5
        if own:
            import communication_avoiding_step_gb300 as casgd
            t = {"group": ("a", "b", "result"), "group_dx": ("result", "b", "a"),
                 "group_dw": ("b", "result", "a")}[op]
            s["ws"] = casgd.group_workspace(*(s[k] for k in t))
        return s
    s["logits"], s["targets"], lp, masked = _logits(c, g)
    s["grad"] = torch.empty_like(s["logits"])
    noise = torch.randn(2, c["rows"], generator=g, device="cuda")
    if op == "preference":
        s["offsets"], _ = _split(c["rows"], 2 * c["pairs"], 0.0, seed)
        lp = torch.where(masked, 0.0, lp + 0.2 * noise[0])
        seq = torch.bucketize(torch.arange(c["rows"], device="cuda"), s["offsets"][1:].long(),
                              right=True)
        s["ref"] = torch.zeros(2 * c["pairs"], device="cuda", dtype=torch.float64).index_add_(
            0, seq, lp.double()).float()
        if c["mean"]:
            n = torch.bincount(seq[~masked], minlength=2 * c["pairs"]).clamp(min=1)
            s["ref"] /= n
        if own:
            import communication_avoiding_step_gb300 as casgd
            s["out"] = casgd.PreferenceOut.alloc(c["pairs"])
            s["ws"] = casgd.preference_workspace(c["rows"], c["pairs"])
        return s
    # policy: the sampled tokens' log probabilities under the sampling and reference models
    lp = (lp + math.log(c["vocab"]) + SPREAD ** 2 / 2) / TEMPERATURE \
        - math.log(c["vocab"]) - (SPREAD / TEMPERATURE) ** 2 / 2
    s["old"], s["ref"] = lp + 0.15 * noise[0], lp + 0.3 * noise[1]
    s["adv"] = torch.randn(c["rows"], generator=g, device="cuda")
    s["weights"] = torch.where(masked, 0.0, 1.0 / c["rows"])
    if own:
        import communication_avoiding_step_gb300 as casgd
        s["out"] = casgd.PolicyOut.alloc(c["rows"])
        s["ws"] = casgd.policy_workspace(c["rows"])
    return s


# --------------------------------------------------------------------------- one pass

BETA, SMOOTHING = 0.1, 0.05          # preference loss
KL, CLIP_LOW, CLIP_HIGH = 0.05, 0.2, 0.28   # policy loss


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import communication_avoiding_step_gb300 as casgd
    op = s["op"]
    if op == "embed":
        return casgd.embed(s["weights"], s["ids"], s["result"], s["ws"], scale=s["scale"])
    if op == "embed_grad":
        return casgd.embed_grad(s["dout"], s["ids"], s["result"], s["ws"], scale=s["scale"])
    if op == "group":
        return casgd.group_product(s["a"], s["b"], s["offsets"], s["result"], s["ws"])
    if op == "group_dx":
        return casgd.group_product_dx(s["a"], s["b"], s["offsets"], s["result"], s["ws"])
    if op == "group_dw":
        return casgd.group_product_dw(s["a"], s["b"], s["offsets"], s["result"], s["ws"])
    if op == "preference":
        o = casgd.preference_loss(s["logits"], s["targets"], s["offsets"], s["ref"], s["grad"],
                                  s["out"], s["ws"], beta=BETA, kind=s["kind"],
                                  smoothing=SMOOTHING, mean=s["mean"])
        return {"loss": o.loss, "margin": o.margin, "logp": o.logp, "grad": s["grad"]}
    o = casgd.policy_loss(s["logits"], s["targets"], s["weights"], s["old"], s["adv"], s["grad"],
                          s["out"], s["ws"], ref_logp=s["ref"], kl=KL, clip_low=CLIP_LOW,
                          clip_high=CLIP_HIGH, temperature=TEMPERATURE)
    return {"loss": o.stats[:1], "kl": o.stats[1:2], "logp": o.logp, "grad": s["grad"]}


def _padded(a, offsets, longest):
    """Rows of each group side by side, groups padded with zeros to the longest."""
    j = torch.arange(longest, device=a.device)
    at = offsets[:-1, None].long() + j
    ok = at < offsets[1:, None]
    return torch.where(ok[..., None], a[at.clamp(max=a.shape[0] - 1)].float(), 0.0), at, ok


def _row_softmax(x, targets):
    """exp(x - max) of each row, its sum, and the targets' log probabilities (0: masked)."""
    keep = targets >= 0
    t = targets.clamp(min=0)[:, None]
    m = x.amax(1, keepdim=True)
    xt = x.gather(1, t) - m
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True)
    return e, z, t, keep, torch.where(keep, (xt - torch.log(z))[:, 0], 0.0)


def _row_grad(e, z, t, coef):
    """coef * (softmax - onehot), in the place of e."""
    e /= z
    e.scatter_add_(1, t, torch.full_like(t, -1.0, dtype=e.dtype))
    return e.mul_(coef[:, None])


def _glm(z, kind):
    """l(z, 1), l(z, -1) and their derivatives: logistic, or least squares."""
    if kind == 0:
        soft = torch.clamp(-z, min=0) + torch.log1p(torch.exp(-z.abs()))
        return soft, soft + z, -1 / (1 + torch.exp(z)), 1 / (1 + torch.exp(-z))
    return 0.5 * (z - 1) ** 2, 0.5 * (z + 1) ** 2, z - 1, z + 1


def _preference(s, x):
    ns = 2 * s["pairs"]
    e, z, t, keep, lp = _row_softmax(x, s["targets"])
    seq = torch.bucketize(torch.arange(s["rows"], device=x.device), s["offsets"][1:].long(),
                          right=True)
    logp = torch.zeros(ns, device=x.device, dtype=x.dtype).index_add_(0, seq, lp)
    per = torch.ones_like(logp)
    if s["mean"]:
        per = 1 / torch.zeros_like(logp).index_add_(0, seq, keep.to(x.dtype)).clamp(min=1)
        logp = logp * per
    d = logp - s["ref"].to(x.dtype)
    margin = BETA * (d[0::2] - d[1::2])
    lpos, lneg, gpos, gneg = _glm(margin, s["kind"])
    loss = ((1 - SMOOTHING) * lpos + SMOOTHING * lneg).mean()
    g = ((1 - SMOOTHING) * gpos + SMOOTHING * gneg) * BETA / s["pairs"]
    # dlogp / dlogits = onehot - softmax
    coef = torch.stack([-g, g], 1).reshape(-1) * per
    return {"loss": loss[None], "margin": margin, "logp": logp,
            "grad": _row_grad(e, z, t, torch.where(keep, coef[seq], 0.0))}


def _policy(s, x):
    def as_x(k):
        return s[k].to(x.dtype)
    e, z, t, keep, lp = _row_softmax(x / TEMPERATURE, s["targets"])
    w, adv = torch.where(keep, as_x("weights"), 0.0), as_x("adv")
    ratio = torch.exp(lp - as_x("old"))
    away = as_x("ref") - lp
    kl = torch.exp(away) - away - 1
    inside = torch.where(adv >= 0, ratio <= 1 + CLIP_HIGH, ratio >= 1 - CLIP_LOW)
    surrogate = torch.minimum(ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv)
    g = torch.where(inside, -ratio * adv, 0.0) + KL * (1 - torch.exp(away))
    return {"loss": (w * (KL * kl - surrogate)).sum()[None], "kl": (w * kl).sum()[None],
            "logp": lp, "grad": _row_grad(e, z, t, -g * w / TEMPERATURE)}


def _run_plain(s):
    op = s["op"]
    if op == "embed":
        return (s["weights"][s["ids"]].float() * s["scale"]).to(s["result"].dtype)
    if op == "embed_grad":
        out = torch.zeros(s["vocab"], s["dim"], device="cuda")
        out.index_add_(0, s["ids"], s["dout"].float() * s["scale"])
        return out.to(s["result"].dtype)
    if op in ("group", "group_dx"):
        a, at, ok = _padded(s["a"], s["offsets"], s["longest"])
        w = s["b"].float()
        y = torch.bmm(a, w.transpose(1, 2) if op == "group" else w)
        return y[ok].to(s["result"].dtype)
    if op == "group_dw":
        a, _, _ = _padded(s["a"], s["offsets"], s["longest"])
        b, _, _ = _padded(s["b"], s["offsets"], s["longest"])
        return torch.bmm(a.transpose(1, 2), b).to(s["result"].dtype)
    r = (_preference if op == "preference" else _policy)(s, s["logits"].float())
    r["grad"] = r["grad"].to(s["grad"].dtype)
    return r


# --------------------------------------------------------------------------- 64 bits


def _exact_rows(x, targets, inv_t):
    """64-bit log probabilities of the targets, and softmax of each row, in slabs of rows."""
    p = torch.empty(x.shape, device=x.device, dtype=torch.float64)
    lp = torch.zeros(x.shape[0], device=x.device, dtype=torch.float64)
    slab = max(1, (1 << 27) // x.shape[1])
    for i in range(0, x.shape[0], slab):
        l = torch.log_softmax(x[i:i + slab].double() * inv_t, 1)
        at = targets[i:i + slab]
        lp[i:i + slab] = torch.where(at >= 0, l.gather(1, at.clamp(min=0)[:, None])[:, 0], 0.0)
        p[i:i + slab] = torch.exp(l)
    return p, lp


def _exact_grad(p, targets, g):
    """sum of g * lp differentiated by the logits: g (onehot - softmax)."""
    rows = torch.arange(p.shape[0], device=p.device)
    g = torch.where(targets >= 0, g, 0.0)
    p *= -g[:, None]
    p[rows, targets.clamp(min=0)] += g
    return p


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    s.pop("result", None)
    if op == "embed":
        return s["weights"][s["ids"]].double() * s["scale"]
    if op == "embed_grad":
        out = torch.zeros(s["vocab"], s["dim"], device="cuda", dtype=torch.float64)
        return out.index_put_((s["ids"],), s["dout"].double() * s["scale"], accumulate=True)
    if op.startswith("group"):
        off = s["offsets"].tolist()
        parts = []
        for e in range(s["groups"]):
            a = s["a"][off[e]:off[e + 1]].double()
            if op == "group":
                parts.append(a @ s["b"][e].double().T)
            elif op == "group_dx":
                parts.append(a @ s["b"][e].double())
            else:
                parts.append(a.T @ s["b"][off[e]:off[e + 1]].double())
        return torch.stack(parts) if op == "group_dw" else torch.cat(parts)
    del s["grad"]
    x, t = s["logits"], s["targets"]
    if op == "preference":
        p, lp = _exact_rows(x, t, 1.0)
        off = s["offsets"].tolist()
        logp, per = [], []
        for a, b in zip(off[:-1], off[1:]):
            n = max(1, int((t[a:b] >= 0).sum())) if s["mean"] else 1
            logp.append(lp[a:b].sum() / n)
            per.append(1.0 / n)
        logp = torch.stack(logp)
        d = (logp - s["ref"].double()).view(-1, 2)
        z = (BETA * (d[:, 0] - d[:, 1])).requires_grad_()
        if s["kind"] == 0:
            l = -(1 - SMOOTHING) * torch.nn.functional.logsigmoid(z) \
                - SMOOTHING * torch.nn.functional.logsigmoid(-z)
        else:
            l = (1 - SMOOTHING) * (z - 1) ** 2 / 2 + SMOOTHING * (z + 1) ** 2 / 2
        loss = l.sum() / s["pairs"]
        dz, = torch.autograd.grad(loss, z)
        g = torch.zeros(s["rows"], device="cuda", dtype=torch.float64)
        for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
            g[a:b] = dz[i // 2] * (BETA if i % 2 == 0 else -BETA) * per[i]
        return {"loss": loss.detach()[None], "margin": z.detach(), "logp": logp,
                "grad": _exact_grad(p, t, g)}
    p, lp = _exact_rows(x, t, 1 / TEMPERATURE)
    q = lp.clone().requires_grad_()
    w = torch.where(t >= 0, s["weights"].double(), 0.0)
    adv = s["adv"].double()
    ratio = torch.exp(q - s["old"].double())
    away = s["ref"].double() - q
    kl = (w * (torch.exp(away) - away - 1)).sum()
    clipped = torch.clamp(ratio, 1 - CLIP_LOW, 1 + CLIP_HIGH)
    loss = KL * kl - (w * torch.minimum(ratio * adv, clipped * adv)).sum()
    g, = torch.autograd.grad(loss, q)
    return {"loss": loss.detach()[None], "kl": kl.detach()[None], "logp": lp,
            "grad": _exact_grad(p, t, g / TEMPERATURE)}


# --------------------------------------------------------------------------- floors

SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def _distinct(rows, vocab):
    """Expected number of different tokens among `rows` of _token_ids."""
    k = np.arange(vocab, dtype=np.float64)
    p = np.log1p(1 / (k + 1)) / math.log(vocab + 1.0)
    return float(-np.expm1(rows * np.log1p(-p)).sum())


def work(case):
    c, op = case, case["op"]
    if op == "embed":
        return {"bytes": c["dim"] * (_distinct(c["rows"], c["vocab"]) * SIZE[c["table"]]
                                     + c["rows"] * SIZE[c["out"]]) + 8 * c["rows"],
                "flops": c["rows"] * c["dim"]}
    if op == "embed_grad":
        return {"bytes": c["dim"] * (c["rows"] * SIZE[c["out"]] + c["vocab"] * SIZE[c["table"]])
                + 8 * c["rows"], "flops": 2 * c["rows"] * c["dim"]}
    if op.startswith("group"):
        # groups that no row is routed to need no weights read (their gradient is written)
        read = c["groups"] if op == "group_dw" else \
            c["groups"] * -math.expm1(c["rows"] * math.log1p(-1.0 / (c["groups"] + 1e-9))) \
            if c["groups"] > 1 else 1
        return {"bytes": SIZE[c["dtype"]] * (c["rows"] * (c["k"] + c["n"])
                                             + read * c["n"] * c["k"]),
                "flops": 2 * c["rows"] * c["k"] * c["n"]}
    n = c["rows"] * c["vocab"]
    # a tenth of the rows is masked: not read, but its gradient is written
    return {"bytes": 1.9 * n * SIZE[c["dtype"]], "flops": 5 * n}
