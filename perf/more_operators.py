"""The operators between a model's norms and its loss, as cases to measure: the norm of each head's queries and keys
with the position rotation, causal attention over packed prompts with grouped heads, and log-probabilities with
entropy and top alternatives, each with its gradient.

`run` computes a case in elementary torch operations in 32 bits (angles in 64); with `own` set it makes the calls a
user makes of newton_schulz_momentum_gb300."""

import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
LIVE = 0.85  # share of a training batch's rows that have a target; the others are prompt or padding
BANNED = 0.01  # share of logits at -infinity where a grammar rules tokens out
CHUNK = 1 << 27  # elements of a score matrix that the plain form holds at a time


def listed():
    """Sizes: the heads of the Llama-3-8B set of the benchmark (32 query and 8 key heads of 128, vocabulary 128256) and
    generic ones."""
    return [
        # Single-token decoding: one token's heads, where the launch is what counts.
        {"name": "rotary_1_token", "op": "rotary", "n": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rotary_dim": 128,
         "type": "bf16", "norm": True, "axes": 1, "interleaved": False, "far": 1 << 20},
        # One training step's tokens, text and image patches mixed: positions of three axes.
        {"name": "rotary_16k_axes", "op": "rotary", "n": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary_dim": 128, "type": "bf16", "norm": True, "axes": 3, "interleaved": False, "far": 4096},
        # The backward pass of the norm and rotation over that step's tokens.
        {"name": "rotary_grad_16k", "op": "rotary_grad", "n": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary_dim": 128, "type": "bf16", "norm": True, "axes": 3, "interleaved": False, "far": 4096},
        # A small fp32 model of odd sizes whose heads turn a quarter of their columns, by neighbours.
        {"name": "rotary_grad_odd", "op": "rotary_grad", "n": 8191, "heads": 9, "kv_heads": 3, "dim": 78,
         "rotary_dim": 20, "type": "f32", "norm": True, "axes": 1, "interleaved": True, "far": 2048},
        # A short turn of one conversation: a prompt shorter than a tile.
        {"name": "attention_turn", "op": "attention", "n": 61, "sequences": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "causal": True, "shape_seed": 0},
        # One long prompt.
        {"name": "attention_8k", "op": "attention", "n": 8192, "sequences": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "causal": True, "shape_seed": 0},
        # A small model's training step: sequences of odd lengths packed one behind the other, seven query heads to a
        # key head.
        {"name": "attention_grad_packed", "op": "attention_grad", "n": 16001, "sequences": 37, "heads": 14,
         "kv_heads": 2, "dim": 64, "causal": True, "shape_seed": 5},
        # A training step on one long sequence: the largest case.
        {"name": "attention_grad_8k", "op": "attention_grad", "n": 8192, "sequences": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "causal": True, "shape_seed": 0},
        # A handful of sampled tokens, with the alternatives a client is shown.
        {"name": "stats_8_tokens", "op": "stats", "n": 8, "vocab": 128256, "type": "bf16", "top": 20, "temp": 1.0,
         "banned": False, "live": False},
        # The scoring of one optimisation step's tokens.
        {"name": "stats_8k", "op": "stats", "n": 8192, "vocab": 128256, "type": "bf16", "top": 5, "temp": 1.0,
         "banned": False, "live": True},
        # The gradient of the log-probabilities and of an entropy bonus over an optimisation step's tokens.
        {"name": "stats_grad_4k", "op": "stats_grad", "n": 4096, "vocab": 128256, "type": "bf16", "temp": 1.0,
         "banned": False, "live": True},
        # fp32 logits of an odd vocabulary (no row but the first is aligned) with tokens ruled out, at a temperature.
        {"name": "stats_grad_odd", "op": "stats_grad", "n": 1025, "vocab": 50257, "type": "f32", "temp": 0.7,
         "banned": True, "live": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, evenly spread over the logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_grad", "attention", "attention_grad", "stats", "stats_grad"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    if op in ("rotary", "rotary_grad"):
        dim = rng.choice([32, 64, 96, 128, 128, 256, 2 * _spread(rng, 16, 128)])
        rotary_dim = rng.choice([dim, dim, dim // 4 * 2, 2])
        axes = rng.choice([1, 3]) if rotary_dim >= 6 else 1
        n = min(_spread(rng, 1, 32768), (1 << 26) // ((heads + kv_heads) * dim))
        return {"op": op, "n": n, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rotary_dim": rotary_dim,
                "type": rng.choice(["bf16", "f32"]), "norm": rng.random() < 0.75, "axes": axes,
                "interleaved": rng.random() < 0.3, "far": _spread(rng, 100, 1 << 24)}
    if op in ("attention", "attention_grad"):
        dim = rng.choice([64, 128, 128, 8 * rng.randrange(2, 17)])
        n = _spread(rng, 1, 16384)
        sequences = min(n, _spread(rng, 1, 64))
        case = {"op": op, "n": n, "sequences": sequences, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "causal": rng.random() < 0.75, "shape_seed": rng.randrange(1 << 16)}
        # No more work than the longest listed prompt's.
        while sum(s * s for s in _lengths(case)) * heads * dim > 8192 * 8192 * 32 * 128 // (1 if case["causal"] else 2):
            case["n"] = case["n"] * 3 // 4
        return case
    vocab = _spread(rng, 500, 262144)
    kind = rng.choice(["bf16", "f32"])
    case = {"op": op, "n": min(_spread(rng, 1, 16384), 1_000_000_000 // (vocab * SIZE[kind])), "vocab": vocab,
            "type": kind, "temp": rng.choice([1.0, 0.7, 1.3]), "banned": rng.random() < 0.3, "live": rng.random() < 0.5}
    return case | ({"top": rng.choice([0, 1, 5, 20, 32])} if op == "stats" else {})


def _lengths(case):
    """Lengths of the packed sequences: shares drawn evenly over a factor of 50, as prompts of one batch have, some of
    them empty."""
    if case["sequences"] == 1:
        return [case["n"]]
    rng = random.Random(case["shape_seed"])
    shares = [math.exp(rng.uniform(0.0, math.log(50.0))) * (rng.random() > 0.05) + 1e-9 for _ in range(case["sequences"])]
    ends, total, sofar = [], sum(shares), 0.0
    for s in shares:
        sofar += s
        ends.append(round(case["n"] * sofar / total))
    ends[-1] = case["n"]
    return [b - a for a, b in zip([0] + ends, ends)]


# ---- inputs


def _sections(case):
    """How many of the rotation's frequencies follow each axis: time a quarter, height and width the rest."""
    half = case["rotary_dim"] // 2
    if case["axes"] == 1:
        return None
    time = max(1, half // 4)
    high = (half - time + 1) // 2
    return (time, high, half - time - high)


def _positions(case, g):
    """Positions of a sequence that begins somewhere in the window; with three axes every other run of 256 tokens is an
    image of 16 x 16 patches, whose axes differ."""
    n = case["n"]
    first = int(torch.randint(0, case["far"], (1,), generator=g, device="cuda"))
    at = torch.arange(n, device="cuda") + first
    if case["axes"] == 1:
        return at
    k = torch.arange(n, device="cuda")
    image = (k // 256) % 2 == 1
    start = at - k % 256
    return torch.stack([torch.where(image, start, at), torch.where(image, start + k % 256 // 16, at),
                        torch.where(image, start + k % 16, at)])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)

    op, n = case["op"], case["n"]
    s = {"case": case}
    if op in ("rotary", "rotary_grad"):
        kind, hq, hk, dim = TYPES[case["type"]], case["heads"], case["kv_heads"], case["dim"]
        # Queries and keys lie in the product that makes them together with the values.
        qkv = normal(n, hq + 2 * hk, dim, dtype=kind)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_gain"] = normal(dim, std=0.2) + 1.0 if case["norm"] else None
        s["k_gain"] = normal(dim, std=0.2) + 1.0 if case["norm"] else None
        s["positions"], s["sections"] = _positions(case, g), _sections(case)
        if op == "rotary_grad":
            s["dq_out"], s["dk_out"] = normal(n, hq, dim, std=1e-3, dtype=kind), normal(n, hk, dim, std=1e-3, dtype=kind)
        return s
    if op in ("attention", "attention_grad"):
        hq, hk, dim = case["heads"], case["kv_heads"], case["dim"]
        # What a norm and a rotation leave: rows of unit mean square, keys that share some of the queries' direction.
        s["q"], s["k"] = normal(n, hq, dim, dtype=torch.bfloat16), normal(n, hk, dim, dtype=torch.bfloat16)
        s["v"] = normal(n, hk + 1, dim, dtype=torch.bfloat16)[:, 1:]
        s["k"] += (0.2 * s["q"][:, ::hq // hk].float()).to(torch.bfloat16)
        ends = torch.tensor([0] + _lengths(case)).cumsum(0)
        s["ends"] = ends.tolist()
        s["offsets"] = None if case["sequences"] == 1 else ends.to(torch.int32).cuda()
        s["scale"] = dim ** -0.5
        if op == "attention_grad":
            s["dout"] = normal(n, hq, dim, std=1e-3, dtype=torch.bfloat16)
            s["out"], s["lse"] = _plain_attention(s, case)
        return s
    vocab, kind = case["vocab"], TYPES[case["type"]]
    z = normal(n, vocab, std=2.0, dtype=kind)
    a = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    at = torch.arange(n, device="cuda")
    if case["banned"]:
        for i in range(0, n, 512):
            z[i:i + 512].masked_fill_(torch.rand(min(512, n - i), vocab, generator=g, device="cuda") < BANNED, -math.inf)
        z[at, a] = normal(n, std=2.0).to(kind)
    # The sampled token stands out from the rest by as much as sampled tokens do.
    z[at, a] += (torch.rand(n, generator=g, device="cuda") * 12.0).to(kind)
    if case["live"]:
        a = torch.where(torch.rand(n, generator=g, device="cuda") < LIVE, a, -1)
    s["logits"], s["targets"] = z, a
    if op == "stats_grad":
        got = _plain_stats(s, case, 0)
        s["norm"], s["entropy"] = got["norm"], got["entropy"]
        s["dlogp"], s["dentropy"] = normal(n, std=1.0 / n), normal(n, std=0.1 / n)
    return s


# ---- the plain form


def _turns(s, case):
    """cos and sin of every token's angles, n x 1 x rotary_dim / 2."""
    half = case["rotary_dim"] // 2
    freqs = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    pos = s["positions"].double()
    if case["axes"] == 1:
        angle = pos[:, None] * freqs
    else:
        angle = torch.cat([pos[i, :, None] * f for i, f in enumerate(torch.split(freqs, list(s["sections"])))], 1)
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _turn(z, cos, sin, case):
    rd = case["rotary_dim"]
    if case["interleaved"]:
        a, b = z[..., 0:rd:2], z[..., 1:rd:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = z[..., :rd // 2], z[..., rd // 2:rd]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, z[..., rd:]], -1)


def _plain_rotary(s, case):
    cos, sin = _turns(s, case)
    got = {}
    for name in ("q", "k"):
        z = s[name].float()
        if case["norm"]:
            z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s[name + "_gain"]
        got[name + "_out"] = _turn(z, cos, sin, case).to(s[name].dtype)
    return got


def _plain_rotary_grad(s, case):
    cos, sin = _turns(s, case)
    got = {}
    for name in ("q", "k"):
        d = _turn(s[f"d{name}_out"].float(), cos, -sin, case)
        if case["norm"]:
            x = s[name].float()
            rho = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            hat = x * rho
            got[f"d{name}_gain"] = (d * hat).sum((0, 1))
            d = d * s[name + "_gain"]
            d = rho * (d - hat * (d * hat).mean(-1, keepdim=True))
        got["d" + name] = d.to(s[name].dtype)
    return {name: got[name] for name in ("dq", "dk", "dq_gain", "dk_gain") if name in got}


def _pieces(s, case):
    """(tokens of a sequence, its query heads in pieces that fit)."""
    group = case["heads"] // case["kv_heads"]
    for b, e in zip(s["ends"], s["ends"][1:]):
        if e > b:
            step = max(1, CHUNK // ((e - b) ** 2 * group))
            for h in range(0, case["kv_heads"], step):
                yield b, e, h, min(h + step, case["kv_heads"])


def _scores(s, case, b, e, h0, h1):
    """(queries, keys, values, scores) of a piece: key head x group x tokens."""
    group = case["heads"] // case["kv_heads"]
    q = s["q"][b:e, h0 * group:h1 * group].float().transpose(0, 1).reshape(h1 - h0, group * (e - b), -1)
    k, v = s["k"][b:e, h0:h1].float().transpose(0, 1), s["v"][b:e, h0:h1].float().transpose(0, 1)
    x = torch.matmul(q, k.transpose(1, 2)).mul_(s["scale"]).view(h1 - h0, group, e - b, e - b)
    if case["causal"]:
        x.masked_fill_(torch.ones(e - b, e - b, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    return q, k, v, x.view(h1 - h0, group * (e - b), e - b)


def _plain_attention(s, case):
    group = case["heads"] // case["kv_heads"]
    out = torch.empty(case["n"], case["heads"], case["dim"], device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(case["heads"], case["n"], device="cuda")
    for b, e, h0, h1 in _pieces(s, case):
        _, _, v, x = _scores(s, case, b, e, h0, h1)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x.sub_(m))
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / total
        out[b:e, h0 * group:h1 * group] = o.view((h1 - h0) * group, e - b, -1).transpose(0, 1).to(torch.bfloat16)
        lse[h0 * group:h1 * group, b:e] = (m + torch.log(total)).view((h1 - h0) * group, e - b)
    return out, lse


def _plain_attention_grad(s, case):
    group = case["heads"] // case["kv_heads"]
    dq, dk, dv = (torch.empty(s[t].shape, device="cuda", dtype=torch.bfloat16) for t in "qkv")
    for b, e, h0, h1 in _pieces(s, case):
        q, k, v, x = _scores(s, case, b, e, h0, h1)
        do = s["dout"][b:e, h0 * group:h1 * group].float().transpose(0, 1).reshape(q.shape)
        p = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
        p = p.div_(p.sum(-1, keepdim=True))
        dv[b:e, h0:h1] = torch.matmul(p.transpose(1, 2), do).transpose(0, 1).to(torch.bfloat16)
        dp = torch.matmul(do, v.transpose(1, 2))
        ds = dp.sub_((dp * p).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
        dk[b:e, h0:h1] = torch.matmul(ds.transpose(1, 2), q).transpose(0, 1).to(torch.bfloat16)
        d = torch.matmul(ds, k).view((h1 - h0) * group, e - b, -1)
        dq[b:e, h0 * group:h1 * group] = d.transpose(0, 1).to(torch.bfloat16)
    return {"dq": dq, "dk": dk, "dv": dv}


def _plain_stats(s, case, top):
    n, vocab = s["logits"].shape
    logp, entropy = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    norm = torch.zeros(n, 2, device="cuda")
    top_logp = torch.zeros(n, top, device="cuda")
    top_ids = torch.full((n, top), -1, device="cuda", dtype=torch.int64)
    step = max(1, CHUNK // vocab)
    for i in range(0, n, step):
        x, a = s["logits"][i:i + step].float(), s["targets"][i:i + step]
        live = a >= 0
        m = x.amax(1, keepdim=True)
        z = (x - m) / case["temp"]
        p = torch.exp(z)
        total = p.sum(1)
        each = torch.where(p > 0, p * z, torch.zeros_like(p)).sum(1)
        lp = z.gather(1, a.clamp(min=0)[:, None])[:, 0] - torch.log(total)
        logp[i:i + step] = torch.where(live, lp, torch.zeros_like(lp))
        entropy[i:i + step] = torch.where(live, torch.log(total) - each / total, torch.zeros_like(lp))
        norm[i:i + step] = torch.where(live[:, None], torch.stack([m[:, 0], total], 1), torch.zeros(1, 2, device="cuda"))
        for t in range(top):
            at = x.argmax(1, keepdim=True)  # the first of equals
            top_logp[i:i + step, t] = torch.where(live, z.gather(1, at)[:, 0] - torch.log(total), torch.zeros_like(lp))
            top_ids[i:i + step, t] = torch.where(live, at[:, 0], torch.full_like(a, -1))
            x.scatter_(1, at, -math.inf)
    return {"logp": logp, "entropy": entropy, "top_logp": top_logp, "top_ids": top_ids, "norm": norm}


def _plain_stats_grad(s, case):
    n, vocab = s["logits"].shape
    out = torch.empty_like(s["logits"])
    step = max(1, CHUNK // vocab)
    for i in range(0, n, step):
        a = s["targets"][i:i + step]
        m, total = s["norm"][i:i + step].split(1, 1)
        lp = (s["logits"][i:i + step].float() - m) / case["temp"] - torch.log(total)
        p = torch.exp(lp)
        g, ge = s["dlogp"][i:i + step, None], s["dentropy"][i:i + step, None]
        d = torch.where(p > 0, -p * (g + ge * (lp + s["entropy"][i:i + step, None])), torch.zeros_like(p))
        d.scatter_add_(1, a.clamp(min=0)[:, None], g)
        out[i:i + step] = torch.where(a[:, None] >= 0, d / case["temp"], torch.zeros_like(d)).to(out.dtype)
    return out


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import newton_schulz_momentum_gb300 as dm
        if op in ("rotary", "rotary_grad"):
            options = dict(q_gain=s["q_gain"], k_gain=s["k_gain"], norm=case["norm"], rotary_dim=case["rotary_dim"],
                           base=10000.0, sections=s["sections"], interleaved=case["interleaved"], eps=EPS)
            if op == "rotary":
                q, k = dm.qk_norm_rotary(s["q"], s["k"], s["positions"], **options)
                return {"q_out": q, "k_out": k}
            dq, dk, dqg, dkg = dm.qk_norm_rotary_grad(s["dq_out"], s["dk_out"], s["q"], s["k"], s["positions"], **options)
            return {"dq": dq, "dk": dk} | ({"dq_gain": dqg, "dk_gain": dkg} if case["norm"] else {})
        if op == "attention":
            out, lse = dm.attention(s["q"], s["k"], s["v"], offsets=s["offsets"], causal=case["causal"], scale=s["scale"])
            return {"out": out, "lse": lse}
        if op == "attention_grad":
            dq, dk, dv = dm.attention_grad(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], offsets=s["offsets"],
                                           causal=case["causal"], scale=s["scale"])
            return {"dq": dq, "dk": dk, "dv": dv}
        if op == "stats":
            return dm.token_stats(s["logits"], s["targets"], top=case["top"], temperature=case["temp"])._asdict()
        return dm.token_stats_grad(s["logits"], s["targets"], s["norm"], s["entropy"], dlogp=s["dlogp"],
                                   dentropy=s["dentropy"], temperature=case["temp"])
    if op == "rotary":
        return _plain_rotary(s, case)
    if op == "rotary_grad":
        return _plain_rotary_grad(s, case)
    if op == "attention":
        out, lse = _plain_attention(s, case)
        return {"out": out, "lse": lse}
    if op == "attention_grad":
        return _plain_attention_grad(s, case)
    if op == "stats":
        return _plain_stats(s, case, case["top"])
    return _plain_stats_grad(s, case)


# ---- the definitions in 64 bits


def _exact_turns(s, case):
    """Each token's turn as a complex number of modulus 1, n x 1 x rotary_dim / 2."""
    half = case["rotary_dim"] // 2
    parts = _sections(case) or (half,)
    pos = s["positions"].view(case["axes"], case["n"])
    axis = [i for i, count in enumerate(parts) for _ in range(count)]
    angle = torch.stack([pos[axis[j]].double() * math.exp(-math.log(10000.0) * j / half) for j in range(half)], 1)
    return torch.polar(torch.ones_like(angle), angle)[:, None]


def _exact_turn(z, turn, case):
    rd = case["rotary_dim"]
    pairs = z[..., :rd].unflatten(-1, (rd // 2, 2) if case["interleaved"] else (2, rd // 2))
    if not case["interleaved"]:
        pairs = pairs.transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    if not case["interleaved"]:
        turned = turned.transpose(-1, -2)
    return torch.cat([turned.flatten(-2), z[..., rd:]], -1)


def _exact_rotary(s, case):
    turn = _exact_turns(s, case)
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        if case["norm"]:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS) * s[name + "_gain"].double()
        got[name + "_out"] = _exact_turn(x, turn, case)
    return got


def _exact_rotary_grad(s, case):
    back = _exact_turns(s, case).conj()
    got = {}
    for name in ("q", "k"):
        d = _exact_turn(s[f"d{name}_out"].double(), back, case)
        if case["norm"]:
            x, gain = s[name].double(), s[name + "_gain"].double()
            ms = x.pow(2).sum(-1) / case["dim"] + EPS
            got[f"d{name}_gain"] = torch.einsum("nhd,nhd,nh->d", d, x, ms.pow(-0.5))
            along = torch.einsum("nhd,d,nhd->nh", d, gain, x) / case["dim"]
            d = d * gain * ms.pow(-0.5)[..., None] - x * (along * ms.pow(-1.5))[..., None]
        got["d" + name] = d
    return {name: got[name] for name in ("dq", "dk", "dq_gain", "dk_gain") if name in got}


def _exact_attention(s, case, grad):
    """Head by head, queries in blocks; a block of a causal sequence meets the keys up to its end."""
    n, hq, hk, dim = case["n"], case["heads"], case["kv_heads"], case["dim"]
    out = {"out": torch.empty(n, hq, dim, device="cuda", dtype=torch.float64),
           "lse": torch.empty(hq, n, device="cuda", dtype=torch.float64)}
    if grad:
        out = {name: torch.zeros(n, h, dim, device="cuda", dtype=torch.float64) for name, h in
               (("dq", hq), ("dk", hk), ("dv", hk))}
    for b, e in zip(s["ends"], s["ends"][1:]):
        rows = max(1, min(1024, (1 << 24) // max(1, e - b)))
        for h in range(hq):
            kv = h // (hq // hk)
            k, v = s["k"][b:e, kv].double(), s["v"][b:e, kv].double()
            for i in range(b, e, rows):
                j = min(i + rows, e)
                until = (j if case["causal"] else e) - b
                x = s["q"][i:j, h].double() @ k[:until].T * s["scale"]
                if case["causal"]:
                    ahead = torch.arange(until, device="cuda") > torch.arange(i - b, j - b, device="cuda")[:, None]
                    x = torch.where(ahead, -math.inf, x)
                total = torch.logsumexp(x, 1)
                p = torch.exp(x - total[:, None])
                if not grad:
                    out["out"][i:j, h], out["lse"][h, i:j] = p @ v[:until], total
                    continue
                do = s["dout"][i:j, h].double()
                dp = do @ v[:until].T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
                out["dq"][i:j, h] = ds @ k[:until]
                out["dk"][b:b + until, kv] += ds.T @ s["q"][i:j, h].double()
                out["dv"][b:b + until, kv] += p.T @ do
    return out


def _exact_stats(s, case):
    n, vocab, top = case["n"], case["vocab"], case["top"]
    f64 = dict(device="cuda", dtype=torch.float64)
    got = {"logp": torch.zeros(n, **f64), "entropy": torch.zeros(n, **f64), "top_logp": torch.zeros(n, top, **f64),
           "top_ids": torch.full((n, top), -1, device="cuda"), "norm": torch.zeros(n, 2, **f64)}
    rows = max(1, (1 << 25) // vocab)
    for i in range(0, n, rows):
        x, a = s["logits"][i:i + rows].double(), s["targets"][i:i + rows]
        ls = torch.log_softmax(x / case["temp"], 1)
        every = torch.special.entr(torch.exp(ls)).sum(1)
        live = a >= 0
        got["logp"][i:i + rows][live] = ls[live].gather(1, a[live, None])[:, 0]
        got["entropy"][i:i + rows][live] = every[live]
        high = x.max(1).values
        got["norm"][i:i + rows][live] = torch.stack(
            [high, torch.exp(torch.logsumexp(x / case["temp"], 1) - high / case["temp"])], 1)[live]
        if top:
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
            got["top_ids"][i:i + rows][live] = ids[live]
            got["top_logp"][i:i + rows][live] = ls.gather(1, ids)[live]
    return got


def _exact_stats_grad(s, case):
    n, vocab = case["n"], case["vocab"]
    got = torch.zeros(n, vocab, device="cuda", dtype=torch.float64)
    rows = max(1, (1 << 25) // vocab)
    for i in range(0, n, rows):
        a = s["targets"][i:i + rows]
        ls = torch.log_softmax(s["logits"][i:i + rows].double() / case["temp"], 1)
        p = torch.exp(ls)
        every = torch.special.entr(p).sum(1, keepdim=True)
        ge = s["dentropy"][i:i + rows, None].double()
        d = -s["dlogp"][i:i + rows, None].double() * p + ge * (torch.special.entr(p) - p * every)
        live = (a >= 0).nonzero()[:, 0]
        d[live, a[live]] += s["dlogp"][i:i + rows][live].double()
        got[i + live] = d[live] / case["temp"]
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return _exact_rotary(s, case)
    if op == "rotary_grad":
        return _exact_rotary_grad(s, case)
    if op in ("attention", "attention_grad"):
        return _exact_attention(s, case, op == "attention_grad")
    return _exact_stats(s, case) if op == "stats" else _exact_stats_grad(s, case)


# ---- what a pass cannot do without


def work(case):
    op, n = case["op"], case["n"]
    if op in ("rotary", "rotary_grad"):
        every = n * (case["heads"] + case["kv_heads"]) * case["dim"]
        passes = 2 if op == "rotary" else 3 if case["norm"] else 2
        return {"bytes": every * SIZE[case["type"]] * passes + 8 * n * case["axes"],
                "flops": every * (8 if op == "rotary" else 14)}
    if op in ("attention", "attention_grad"):
        hq, hk, dim = case["heads"], case["kv_heads"], case["dim"]
        pairs = sum(v * (v + 1) // 2 if case["causal"] else v * v for v in _lengths(case)) * hq
        if op == "attention":
            return {"bytes": 2 * n * dim * (2 * hq + 2 * hk) + 4 * n * hq, "flops": 4 * dim * pairs}
        return {"bytes": 2 * n * dim * (4 * hq + 4 * hk) + 4 * n * hq, "flops": 10 * dim * pairs}
    live = LIVE * n if case["live"] else n
    row = case["vocab"] * SIZE[case["type"]]
    if op == "stats":
        return {"bytes": live * row + n * (24 + 12 * case["top"]), "flops": 6 * live * case["vocab"]}
    # Rows without a target are written, with zeros, and need no reading.
    return {"bytes": (live + n) * row + 28 * n, "flops": 8 * live * case["vocab"]}
