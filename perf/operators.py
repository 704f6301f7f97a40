"""The training operators around the optimizer, as cases to measure: embedding lookup and its gradient by sorted
tokens, residual addition with RMS norm (with an 8-bit output, and its gradient), and the clipped policy loss with a
KL term from logits (with its gradient, and the token log-probabilities alone).

`run` computes a case in elementary torch operations in 32 bits; with `own` set it makes the calls a user makes of
newton_schulz_momentum_gb300."""

import math

import torch

own = False

FP8_MAX = 448.0  # largest finite value of e4m3
EPS = 1e-6
LIVE = 0.85  # share of a policy case's rows with a weight above 0
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    """Sizes: the Llama-3-8B set of the benchmark (hidden 4096, vocabulary 128256) and generic ones."""
    return [
        # One new token of one sequence: the lookup at its smallest, where the launch is what counts.
        {"name": "embed_1_token", "op": "embed", "n": 1, "rows": 128256, "dim": 4096, "type": "bf16", "out": "bf16"},
        # The lookup of one training step's tokens in the optimizer's fp32 table.
        {"name": "embed_16k", "op": "embed", "n": 16384, "rows": 128256, "dim": 4096, "type": "f32", "out": "bf16"},
        # The gradient of that table: dense fp32, as AdamW reads it; most of its rows had no token.
        {"name": "embed_grad_16k", "op": "embed_grad", "n": 16384, "rows": 128256, "dim": 4096, "type": "bf16",
         "pad": 0},
        # A small model's table of odd sizes with fp32 gradients and a padding token, more tokens than rows.
        {"name": "embed_grad_odd", "op": "embed_grad", "n": 20011, "rows": 5003, "dim": 1027, "type": "f32",
         "pad": 3},
        # Single-token decoding: one row, its output in 8 bits for the next product.
        {"name": "norm_1_row_fp8", "op": "norm", "n": 1, "dim": 4096, "type": "bf16", "residual": True, "group": 128},
        # One training step's tokens through the norm in front of a layer.
        {"name": "norm_16k", "op": "norm", "n": 16384, "dim": 4096, "type": "bf16", "residual": True, "group": 0},
        # Prefill of a wide model with ragged groups of scales, fp32 residual stream.
        {"name": "norm_fp8_odd", "op": "norm", "n": 3001, "dim": 8200, "type": "f32", "residual": True, "group": 128},
        # The norm's backward pass over a training step's tokens, the residual's gradient joining in.
        {"name": "norm_grad_16k", "op": "norm_grad", "n": 16384, "dim": 4096, "type": "bf16", "residual": True},
        # Many narrow rows (the norm of each head's queries), odd width, no residual.
        {"name": "norm_grad_heads", "op": "norm_grad", "n": 65537, "dim": 129, "type": "f32", "residual": False},
        # A handful of sampled tokens: few rows, each long.
        {"name": "policy_8_tokens", "op": "policy", "n": 8, "vocab": 128256, "type": "bf16", "kl": 0.05, "temp": 1.0},
        # The loss over one optimisation step's tokens: the largest case.
        {"name": "policy_8k", "op": "policy", "n": 8192, "vocab": 128256, "type": "bf16", "kl": 0.05, "temp": 1.0},
        # fp32 logits of an odd vocabulary (no row but the first is aligned), with a temperature and no KL term.
        {"name": "policy_odd_f32", "op": "policy", "n": 1025, "vocab": 50257, "type": "f32", "kl": 0.0, "temp": 0.7},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, evenly spread over the logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "policy", "policy", "logp"])
    kind = rng.choice(["bf16", "f32"])
    if op in ("embed", "embed_grad"):
        rows, dim = _spread(rng, 500, 128256), _spread(rng, 32, 8192)
        dim = min(dim, 128256 * 4096 // rows)
        n = min(_spread(rng, 1, 32768), max(1, (1 << 27) // dim))
        case = {"op": op, "n": n, "rows": rows, "dim": dim, "type": kind}
        if op == "embed":
            return case | {"out": rng.choice(["bf16", "f32"])}
        return case | {"pad": rng.choice([-1, 0, rng.randrange(rows)])}
    if op in ("norm", "norm_grad"):
        dim = _spread(rng, 32, 16384)
        n = min(_spread(rng, 1, 65536), (1 << 27) // dim)
        case = {"op": op, "n": n, "dim": dim, "type": kind, "residual": rng.random() < 0.75}
        return case if op == "norm_grad" else case | {"group": rng.choice([0, 32, 128])}
    vocab = _spread(rng, 500, 262144)
    n = min(_spread(rng, 1, 16384), 2_000_000_000 // (vocab * SIZE[kind]))
    case = {"op": op, "n": n, "vocab": vocab, "type": kind, "temp": rng.choice([1.0, 0.7, 1.3])}
    return case if op == "logp" else case | {"kl": rng.choice([0.0, 0.05, 0.1])}


# ---- inputs


def _tokens(n, rows, g):
    """Token ids whose frequency falls with the id as in natural text: about log(1 + 1 / v) / log(rows)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(rows + 1)) - 1).long().clamp_(0, rows - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)

    op, n, kind = case["op"], case["n"], TYPES[case["type"]]
    s = {"case": case}
    if op == "embed":
        s["table"] = normal(case["rows"], case["dim"], std=0.02, dtype=kind)
        s["ids"] = _tokens(n, case["rows"], g)
        s["scale"] = math.sqrt(case["dim"])
    elif op == "embed_grad":
        s["grad_out"] = normal(n, case["dim"], std=1e-3, dtype=kind)
        s["ids"] = _tokens(n, case["rows"], g)
        s["scale"] = math.sqrt(case["dim"])
    elif op == "norm":
        s["x"] = normal(n, case["dim"], dtype=kind)
        s["residual"] = normal(n, case["dim"], std=3.0, dtype=kind) if case["residual"] else None
        s["gain"] = normal(case["dim"], std=0.2) + 1.0
    elif op == "norm_grad":
        s["dy"] = normal(n, case["dim"], std=1e-3, dtype=kind)
        s["h"] = normal(n, case["dim"], std=3.0, dtype=kind)
        s["dh"] = normal(n, case["dim"], std=1e-3, dtype=kind) if case["residual"] else None
        s["gain"] = normal(case["dim"], std=0.2) + 1.0
    else:
        vocab, temp = case["vocab"], case["temp"]
        z = normal(n, vocab, std=2.0, dtype=kind)
        a = torch.randint(0, vocab, (n,), generator=g, device="cuda")
        at = torch.arange(n, device="cuda")
        # The sampled token stands out from the rest by as much as sampled tokens do.
        z[at, a] += (torch.rand(n, generator=g, device="cuda") * 12.0).to(kind)
        s["logits"], s["targets"] = z, a
        if op == "policy":
            lp = torch.empty(n, device="cuda")
            for i in range(0, n, 512):
                t = z[i:i + 512].float() / temp
                lp[i:i + 512] = t.gather(1, a[i:i + 512, None])[:, 0] - torch.logsumexp(t, 1)
            s["old_logp"] = lp + normal(n, std=0.15)
            s["ref_logp"] = lp + normal(n, std=0.3) if case["kl"] else None
            s["advantages"] = normal(n)
            live = (torch.rand(n, generator=g, device="cuda") < LIVE).float()  # the others are prompt or padding
            live[0] = 1.0
            s["weights"] = live / live.sum()
    return s


# ---- the plain form


def _plain_embed_grad(s, case):
    ids = s["ids"]
    d = s["grad_out"].float() * s["scale"]
    if case["pad"] >= 0:
        d = d * (ids != case["pad"]).float()[:, None]
    return torch.zeros(case["rows"], case["dim"], device="cuda").index_add_(0, ids, d)


def _plain_quantize(y, group):
    n, dim = y.shape
    parts = -(-dim // group)
    full = torch.zeros(n, parts * group, device=y.device)
    full[:, :dim] = y
    full = full.view(n, parts, group)
    top = full.abs().amax(2)
    scales = torch.where(top > 0, top / FP8_MAX, torch.ones_like(top))
    q = (full / scales[:, :, None]).view(n, parts * group)[:, :dim].to(torch.float8_e4m3fn)
    return q.contiguous(), scales


def _plain_norm(s, case):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["gain"]
    got = {} if s["residual"] is None else {"h": h.to(s["x"].dtype)}
    if case["group"]:
        q, scales = _plain_quantize(y, case["group"])
        return got | {"q": q, "scales": scales}
    return got | {"y": y.to(s["x"].dtype)}


def _plain_norm_grad(s):
    dy, h = s["dy"].float(), s["h"].float()
    rho = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    hat, d = h * rho, dy * s["gain"]
    dx = rho * (d - hat * (d * hat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dgain": (dy * hat).sum(0)}


def _plain_logp(s, case):
    z = s["logits"].float()
    if case["temp"] != 1.0:
        z = z / case["temp"]
    e = z - z.amax(1, keepdim=True)
    p = torch.exp(e)
    total = p.sum(1, keepdim=True)
    logp = e.gather(1, s["targets"][:, None])[:, 0] - torch.log(total[:, 0])
    return logp, p, total


def _plain_policy(s, case):
    logp, p, total = _plain_logp(s, case)
    w, adv, ref = s["weights"], s["advantages"], s["ref_logp"]
    live = w != 0
    logp = torch.where(live, logp, torch.zeros_like(logp))
    r = torch.exp(logp - s["old_logp"])
    whole, cut = r * adv, torch.clamp(r, 0.8, 1.2) * adv
    each = -torch.minimum(whole, cut)
    c = -whole * (whole <= cut).float()
    if ref is not None:
        d = ref - logp
        each = each + case["kl"] * (torch.exp(d) - d - 1.0)
        c = c + case["kl"] * (1.0 - torch.exp(d))
    c = torch.where(live, c * w, torch.zeros_like(c)) / case["temp"]
    loss = torch.where(live, each * w, torch.zeros_like(each)).sum()
    d = p.mul_((-c / total[:, 0])[:, None])
    d.scatter_add_(1, s["targets"][:, None], c[:, None])
    return {"loss": loss, "logp": logp, "dlogits": d.to(s["logits"].dtype)}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import newton_schulz_momentum_gb300 as dm
        if op == "embed":
            return dm.embedding(s["table"], s["ids"], scale=s["scale"], dtype=TYPES[case["out"]])
        if op == "embed_grad":
            return dm.embedding_grad(s["grad_out"], s["ids"], case["rows"], scale=s["scale"], padding_idx=case["pad"])
        if op == "norm" and case["group"]:
            q, scales, h = dm.add_rmsnorm_fp8(s["x"], s["residual"], s["gain"], eps=EPS, group=case["group"])
            return {"q": q, "scales": scales} | ({} if s["residual"] is None else {"h": h})
        if op == "norm":
            y, h = dm.add_rmsnorm(s["x"], s["residual"], s["gain"], eps=EPS)
            return {"y": y} | ({} if s["residual"] is None else {"h": h})
        if op == "norm_grad":
            dx, dgain = dm.add_rmsnorm_grad(s["dy"], s["h"], s["gain"], dh=s["dh"], eps=EPS)
            return {"dx": dx, "dgain": dgain}
        if op == "logp":
            return dm.token_logprobs(s["logits"], s["targets"], temperature=case["temp"])
        loss, logp, dlogits = dm.policy_loss(s["logits"], s["targets"], s["old_logp"], s["advantages"], s["weights"],
                                             ref_logp=s["ref_logp"], clip_low=0.2, clip_high=0.2, kl_coef=case["kl"],
                                             temperature=case["temp"])
        return {"loss": loss, "logp": logp, "dlogits": dlogits}
    if op == "embed":
        return (s["table"][s["ids"]].float() * s["scale"]).to(TYPES[case["out"]])
    if op == "embed_grad":
        return _plain_embed_grad(s, case)
    if op == "norm":
        return _plain_norm(s, case)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "logp":
        return _plain_logp(s, case)[0]
    return _plain_policy(s, case)


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return torch.nn.functional.embedding(s["ids"], s["table"].double()) * s["scale"]
    if op == "embed_grad":
        # Tokens in the order of their ids, each id's gradients one run of the list, added run by run.
        ids, order = torch.sort(s["ids"], stable=True)
        got = torch.zeros(case["rows"], case["dim"], device="cuda", dtype=torch.float64)
        distinct, counts = torch.unique_consecutive(ids, return_counts=True)
        first = torch.cumsum(counts, 0) - counts
        for k in range(0, case["dim"], 512):
            d = s["grad_out"][:, k:k + 512].double()[order] * s["scale"]
            got[distinct, k:k + 512] = torch.segment_reduce(d, "sum", lengths=counts, axis=0)
        assert int(first[-1] + counts[-1]) == case["n"]
        if case["pad"] >= 0:
            got[case["pad"]] = 0.0
        return got
    if op == "norm":
        h = s["x"].double() + (0.0 if s["residual"] is None else s["residual"].double())
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["dim"] + EPS) * s["gain"].double()
        got = {} if s["residual"] is None else {"h": h}
        if not case["group"]:
            return got | {"y": y}
        pieces = torch.split(y, case["group"], 1)
        tops = [p.abs().max(1).values for p in pieces]
        scales = [torch.where(t == 0, 1.0, t / FP8_MAX) for t in tops]
        q = torch.cat([p / c[:, None] for p, c in zip(pieces, scales)], 1)
        return got | {"q": q.float().to(torch.float8_e4m3fn).double(), "scales": torch.stack(scales, 1)}
    if op == "norm_grad":
        dy, h, gain = s["dy"].double(), s["h"].double(), s["gain"].double()
        ms = h.pow(2).sum(1) / case["dim"] + EPS
        along = torch.einsum("nd,d,nd->n", dy, gain, h) / case["dim"]
        dx = (dy * gain) * ms.pow(-0.5)[:, None] - h * (along * ms.pow(-1.5))[:, None]
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(),
                "dgain": torch.einsum("nd,nd,n->d", dy, h, ms.pow(-0.5))}
    n, vocab, temp = case["n"], case["vocab"], case["temp"]
    rows = max(1, (1 << 26) // vocab)
    logp = torch.empty(n, device="cuda", dtype=torch.float64)
    for i in range(0, n, rows):
        ls = torch.log_softmax(s["logits"][i:i + rows].double() / temp, 1)
        logp[i:i + rows] = torch.gather(ls, 1, s["targets"][i:i + rows, None]).squeeze(1)
    if op == "logp":
        return logp
    w, adv = s["weights"].double(), s["advantages"].double()
    logp = torch.where(w == 0, 0.0, logp)
    r = (logp - s["old_logp"].double()).exp()
    inside = torch.where(adv >= 0, r <= 1.2, r >= 0.8)  # where the clipped value is not the smaller one
    each = -adv * torch.where(inside, r, torch.where(adv >= 0, 1.2, 0.8))
    c = torch.where(inside, -adv * r, 0.0)
    if s["ref_logp"] is not None:
        d = s["ref_logp"].double() - logp
        each = each + case["kl"] * (torch.expm1(d) - d)
        c = c - case["kl"] * torch.expm1(d)
    c = c * w / temp
    dlogits = torch.empty(n, vocab, device="cuda", dtype=torch.float64)
    for i in range(0, n, rows):
        p = torch.softmax(s["logits"][i:i + rows].double() / temp, 1)
        p[torch.arange(p.shape[0], device="cuda"), s["targets"][i:i + rows]] -= 1.0
        dlogits[i:i + rows] = p * -c[i:i + rows, None]
    return {"loss": (each * w).sum(), "logp": logp, "dlogits": dlogits}


# ---- what a pass cannot do without


def work(case):
    op, n, size = case["op"], case["n"], SIZE[case["type"]]
    if op == "embed":
        # Each distinct row once; their expected number follows from the distribution of the ids.
        every = math.log(case["rows"] + 1)
        distinct = sum(1.0 - (1.0 - math.log1p(1.0 / (v + 1)) / every) ** n for v in range(case["rows"]))
        return {"bytes": case["dim"] * (distinct * size + n * SIZE[case["out"]]) + 8 * n, "flops": n * case["dim"]}
    if op == "embed_grad":
        return {"bytes": case["dim"] * (n * size + 4 * case["rows"]) + 8 * n, "flops": n * case["dim"]}
    if op == "norm":
        item = size + (2 * size if case["residual"] else 0) + (1 if case["group"] else size)
        scales = 4 * n * -(-case["dim"] // case["group"]) if case["group"] else 0
        return {"bytes": n * case["dim"] * item + scales + 4 * case["dim"], "flops": 5 * n * case["dim"]}
    if op == "norm_grad":
        item = size * (4 if case["residual"] else 3)
        return {"bytes": n * case["dim"] * item + 8 * case["dim"], "flops": 10 * n * case["dim"]}
    if op == "logp":
        return {"bytes": n * (case["vocab"] * size + 12), "flops": 4 * n * case["vocab"]}
    # Rows of weight 0 are written, with zeros, and need no reading.
    live = 1 + LIVE * (n - 1)
    return {"bytes": (live + n) * case["vocab"] * size + 28 * n, "flops": 8 * live * case["vocab"]}
