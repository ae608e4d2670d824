"""Cases of the operators that make a model of decoder layers: rotary positions, products with weights that are not
quantised (projections, the output head) and the log probabilities that a server answers with.

``rotary``    q and k turned by their positions: pairs of channels (a, b) become scale (a cos - b sin, b cos + a sin)
              with the angle position * frequency; neighbouring channels or the two halves are pairs, channels behind
              the turned part are copied
``linear``    y = resid + act(W x + bias) * mul, W [O x I] in bfloat16
``logprobs``  log softmax of scale * logits at given tokens, its entropy, and the k largest entries of each row
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_ctx = []


def _context():
    """The library context, made once, as a server keeps it."""
    if not _ctx:
        from int4_grouped_expert_router_gb300 import binding
        _ctx.append((binding, binding.coli_init(0)))
    return _ctx[0]


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    turn = dict(q_heads=64, k_heads=8, hd=128, rot=128, layout="half", base=10000.0, scaling="none", dtype="bf16", where="plan")
    lin = dict(bias=False, act="none", mul=False, resid=False, x="bf16", y="bf16")
    return [
        # one request decodes one token: the smallest call
        dict(name="rotary one request", op="rotary", T=1, B=1, far=5000, **turn),
        # a decode step of a full batch at far positions, neighbouring channels, half of the head turned
        dict(name="rotary batch far", op="rotary", T=64, B=64, far=1000000, **turn | dict(rot=64, layout="neighbours", base=1e6)),
        # ragged prompts, frequencies scaled by parts for a long context
        dict(name="rotary prompts", op="rotary", T=8191, B=5, far=60000, **turn | dict(base=500000.0, scaling="parts")),
        # packed rows in binary32 with positions of their own, a head whose turned part is not a whole vector
        dict(name="rotary f32 packed", op="rotary", T=3001, B=1, far=8192,
             **turn | dict(q_heads=20, k_heads=20, hd=80, rot=36, dtype="f32", where="given", scaling="linear")),
        # the output projection of one decoded token at the width of the decode layer, into the residual
        dict(name="linear one token", op="linear", S=1, I=6144, O=6144, **lin | dict(resid=True)),
        # the output head for a decode batch: binary32 logits over an odd vocabulary
        dict(name="linear head", op="linear", S=24, I=6144, O=50021, **lin | dict(y="f32")),
        # the gate of a dense block in binary32 for a short prompt: silu(gate) * up
        dict(name="linear gate f32", op="linear", S=301, I=6144, O=2048, **lin | dict(bias=True, act="silu", mul=True, x="f32", y="f32")),
        # a long prompt through a projection with everything behind it
        dict(name="linear prompt", op="linear", S=4096, I=6144, O=6144, **lin | dict(bias=True, act="gelu", resid=True)),
        # one decoded token: its log probability, the entropy, five alternatives
        dict(name="logprobs one token", op="logprobs", S=1, V=50021, k=5, n=1, dtype="f32", scale=1.25),
        # a decode batch of a large vocabulary in bfloat16, where many entries tie
        dict(name="logprobs batch", op="logprobs", S=64, V=151001, k=20, n=1, dtype="bf16", scale=1.0),
        # the tokens of a prompt are scored
        dict(name="logprobs prompt", op="logprobs", S=2048, V=65536, k=1, n=1, dtype="f32", scale=1.0),
        # fifty candidate answers are scored for each of a few requests
        dict(name="logprobs candidates", op="logprobs", S=15, V=32003, k=32, n=50, dtype="f32", scale=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "linear", "linear", "logprobs"])
    if op == "rotary":
        hd = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        k_heads = rng.choice([1, 2, 4, 8, 20])
        q_heads = k_heads * rng.choice([1, 4, 5, 8])
        T = min(_log(rng, 1, 16384), 70_000_000 // ((q_heads + k_heads) * hd))
        return dict(op=op, T=T, B=min(T, _log(rng, 1, 64)), far=_log(rng, 100, 1000000), q_heads=q_heads, k_heads=k_heads,
                    hd=hd, rot=rng.choice([hd, hd, hd // 2, 2 * rng.randint(1, hd // 2)]),
                    layout=rng.choice(["half", "neighbours"]), base=rng.choice([10000.0, 500000.0, 1e6]),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    where=rng.choice(["plan", "given"]))
    if op == "linear":
        S = rng.choice([1, _log(rng, 2, 64), _log(rng, 64, 4096)])
        I = _log(rng, 64, 8192)
        I = max(64, I // 64 * 64) if rng.random() < 0.7 else I  # whole tiles, or any width
        O = _log(rng, 64, 60000)
        x = rng.choice(["bf16", "bf16", "f32"])
        # no more products than the largest listed case
        O = max(1, min(O, 150_000_000_000 // (S * I * (2 if x == "f32" else 1))))
        return dict(op=op, S=S, I=I, O=O, bias=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu", "relu2"]),
                    mul=rng.random() < 0.3, resid=rng.random() < 0.5, x=x, y=rng.choice(["bf16", "f32", x]))
    S = _log(rng, 1, 2048)
    V = min(_log(rng, 100, 200000), 134_000_000 // S)
    return dict(op=op, S=S, V=V, k=rng.choice([0, 1, 5, 20, 32]), n=rng.choice([1, 1, 2, 50]), dtype=rng.choice(["bf16", "f32"]),
                scale=rng.choice([1.0, 1.25, 0.7]))


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _uniform(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


# How the scaled kinds are called in the cases, with what they take.
SCALED = {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
          "parts": dict(factor=8.0, original_len=8192, low=1.0, high=4.0)}


def _frequencies(c):
    """Radians per position of each pair, in 64 bits."""
    rot, base, s = c["rot"], c["base"], SCALED[c["scaling"]]
    if c["scaling"] == "base" and rot > 2:
        base = base * s["factor"] ** (rot / (rot - 2))
    f = base ** (-2 * torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
    if c["scaling"] == "linear":
        f = f / s["factor"]
    if c["scaling"] == "parts":  # fast pairs stay, slow ones are stretched, a ramp in the turns that they make lies between
        turns = s["original_len"] * f / (2 * math.pi)
        stay = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        f = f * (stay + (1 - stay) / s["factor"])
    return f


def _ragged(total, parts):
    """`total` rows among `parts` sequences, none of them empty, not alike."""
    weight = [1 + (7 * b) % 5 for b in range(parts)]
    rows = [max(1, (total - parts) * w // sum(weight) + 1) for w in weight]
    rows[0] += total - sum(rows)
    return rows


def _inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 29)
    if c["op"] == "rotary":
        T, B, dt = c["T"], c["B"], DTYPES[c["dtype"]]
        qkv = torch.randn(T, c["q_heads"] + 2 * c["k_heads"], c["hd"], device="cuda", generator=g).to(dt)
        i = dict(q=qkv[:, :c["q_heads"]], k=qkv[:, c["q_heads"]:c["q_heads"] + c["k_heads"]])  # slices of a fused projection
        if c["where"] == "given":  # documents one after another in the rows, each from a position of its own
            first = torch.randint(0, c["far"], (T,), device="cuda", generator=g)
            at = torch.arange(T, device="cuda")
            i["positions"] = (first[at // 97 * 97] + at % 97).to(torch.int32)
            return i
        rows = _ragged(T, B)
        start = [0]
        for m in rows:
            start.append(start[-1] + m)
        more = torch.randint(0, c["far"], (B,), device="cuda", generator=g)
        i["lens"] = (torch.tensor(rows, device="cuda") + more).to(torch.int32)
        i["q_start"] = None if T == B else torch.tensor(start, dtype=torch.int32, device="cuda")
        return i
    if c["op"] == "linear":
        S, I, O = c["S"], c["I"], c["O"]
        loud = 1 + 9 * (_uniform(g, I) > 0.99).float()  # a few loud channels, as a residual stream has them
        y = DTYPES[c["y"]]
        return dict(x=(_normal(g, S, I) * loud).to(DTYPES[c["x"]]), w=(_normal(g, O, I) * 0.02).to(torch.bfloat16),
                    bias=_normal(g, O) if c["bias"] else None, mul=_normal(g, S, O).to(y) if c["mul"] else None,
                    resid=_normal(g, S, O).to(y) if c["resid"] else None)
    S, V = c["S"], c["V"]
    logits = torch.empty(S, V, dtype=DTYPES[c["dtype"]], device="cuda")
    step = max(1, 16_000_000 // V)
    for at in range(0, S, step):  # rows of differing sharpness, some entries forbidden
        z = _normal(g, min(step, S - at), V).mul_(0.5 + 4 * _uniform(g, min(step, S - at), 1))
        logits[at:at + step] = z.masked_fill_(_uniform(g, *z.shape) > 0.98, -math.inf)
    tokens = torch.randint(0, V, (S, c["n"]), device="cuda", generator=g, dtype=torch.int32)
    return dict(logits=logits, tokens=tokens)


def prepare(case, seed):
    c = case
    s = dict(_inputs(c, seed), case=c)
    if c["op"] == "rotary":
        s["freqs"] = _frequencies(c)
        if own:
            B, _ = _context()
            s["freqs"] = B.coli_rotary_freqs(c["rot"], c["base"], scaling=c["scaling"], **SCALED[c["scaling"]])
            s["out"] = [torch.empty(s[n].shape, dtype=s[n].dtype, device="cuda") for n in ("q", "k")]
            s["plan"] = {n: s[n] for n in ("positions", "lens", "q_start") if n in s}
        elif c["where"] == "plan":
            start = s["q_start"] if s["q_start"] is not None else torch.arange(c["B"] + 1, dtype=torch.int32, device="cuda")
            row = torch.arange(c["T"], device="cuda")
            seq = torch.searchsorted(start[1:].contiguous(), row.to(torch.int32), right=True)
            s["positions"] = s["lens"][seq] - (start[seq + 1] - row)
    if c["op"] == "linear" and own:
        B, ctx = _context()
        s["handle"] = _Uploaded(B, ctx, s.pop("w"))
        s["y"] = torch.empty(c["S"], c["O"], dtype=DTYPES[c["y"]], device="cuda")
    if c["op"] == "logprobs" and own:
        S, k = c["S"], c["k"]
        s["out"] = dict(logp=torch.empty(S, c["n"], device="cuda"), entropy=torch.empty(S, device="cuda"),
                        top_id=torch.empty(S, k, dtype=torch.int32, device="cuda") if k else None,
                        top_logp=torch.empty(S, k, device="cuda") if k else None)
    return s


class _Uploaded:
    """A weight that the library holds, freed with the state that holds it."""

    def __init__(self, B, ctx, w):
        self.B, self.ctx, self.handle = B, ctx, B.coli_dense_upload(ctx, w)

    def __del__(self):
        self.B.coli_dense_free(self.ctx, self.handle)


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------

def _rotary(s):
    c, half = s["case"], s["case"]["rot"] // 2
    angle = s["positions"].double()[:, None] * s["freqs"]  # in 64 bits: far positions turn many times
    cos, sin = (t.float()[:, None] for t in (torch.cos(angle), torch.sin(angle)))
    out = []
    for x in (s["q"], s["k"]):
        y = x.float()
        part = y[..., :c["rot"]]
        a, b = (part[..., :half], part[..., half:]) if c["layout"] == "half" else (part[..., 0::2], part[..., 1::2])
        u, v = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat((u, v), -1) if c["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
        out.append(torch.cat((turned, y[..., c["rot"]:]), -1).to(x.dtype))
    return out


def _act(z, kind):
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if kind == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "relu":
        return torch.clamp(z, min=0)
    if kind == "relu2":
        return torch.square(torch.clamp(z, min=0))
    return z


def _linear(s):
    c = s["case"]
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _act(z, c["act"])
    if s["mul"] is not None:
        z = z * s["mul"].float()
    if s["resid"] is not None:
        z = z + s["resid"].float()
    return z.to(DTYPES[c["y"]])


def _logprobs(s):
    c = s["case"]
    x = s["logits"].float()
    z = x * c["scale"]
    top = z.amax(-1, keepdim=True)
    d = z - top
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    mean = torch.where(e > 0, d * e, torch.zeros_like(e)).sum(-1, keepdim=True) / total
    out = [torch.gather(d, 1, s["tokens"].long()) - log_total, (log_total - mean)[:, 0]]
    if c["k"]:
        at = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["k"]]  # ties: the lowest index first
        out += [at.to(torch.int32), torch.gather(d, 1, at) - log_total]
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        B, ctx = _context()
        c = s["case"]
        if op == "rotary":
            B.coli_rotary(ctx, s["q"], s["k"], s["freqs"], *s["out"], interleaved=c["layout"] == "neighbours", **s["plan"])
            return s["out"]
        if op == "linear":
            B.coli_dense_linear(ctx, s["handle"].handle, s["x"], s["y"], bias=s["bias"], act=c["act"], mul=s["mul"], resid=s["resid"])
            return s["y"]
        B.coli_logprobs(ctx, s["logits"], tokens=s["tokens"], scale=c["scale"], **s["out"])
        return [t for t in s["out"].values() if t is not None]
    return {"rotary": _rotary, "linear": _linear, "logprobs": _logprobs}[op](s)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "rotary":
        cells = c["T"] * (c["q_heads"] + c["k_heads"]) * c["hd"]
        plan = 4 * c["T"] if c["where"] == "given" else 4 * (2 * c["B"] + 1)
        return {"bytes": 2 * cells * size[c["dtype"]] + plan + 4 * c["rot"],
                "flops": 3 * cells * c["rot"] // c["hd"]}
    if c["op"] == "linear":
        S, I, O = c["S"], c["I"], c["O"]
        return {"bytes": 2 * O * I + S * I * size[c["x"]] + S * O * size[c["y"]] * (1 + c["mul"] + c["resid"]) + 4 * O * c["bias"],
                "flops": 2 * S * I * O}
    cells = c["S"] * c["V"]
    return {"bytes": cells * size[c["dtype"]] + 4 * c["S"] * (2 * c["n"] + 1 + 2 * c["k"]), "flops": 6 * cells}


# ---------------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    c, i = case, _inputs(case, seed)
    if c["op"] == "rotary":
        if "positions" in i:
            at = i["positions"].double()
        else:
            start = i["q_start"].tolist() if i["q_start"] is not None else list(range(c["B"] + 1))
            at = torch.cat([torch.arange(n - (e - b), n, dtype=torch.float64, device="cuda")
                            for n, b, e in zip(i["lens"].tolist(), start, start[1:])])
        unit = torch.polar(torch.ones(c["T"], c["rot"] // 2, dtype=torch.float64, device="cuda"), torch.outer(at, _frequencies(c)))
        out = []
        for x in (i["q"], i["k"]):
            y = x.double().clone()
            whole = y[..., :c["rot"]]
            if c["layout"] == "half":
                z = torch.complex(*whole.chunk(2, -1)) * unit[:, None]
                y[..., :c["rot"]] = torch.cat((z.real, z.imag), -1)
            else:
                z = torch.view_as_complex(whole.unflatten(-1, (-1, 2)).contiguous()) * unit[:, None]
                y[..., :c["rot"]] = torch.view_as_real(z).flatten(-2)
            out.append(y)
        return out
    if c["op"] == "linear":
        z = torch.einsum("si,oi->so", i["x"].double(), i["w"].double())
        if c["bias"]:
            z += i["bias"].double()
        if c["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif c["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif c["act"] == "gelu_tanh":
            z = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        elif c["act"] in ("relu", "relu2"):
            z = torch.where(z > 0, z ** (2 if c["act"] == "relu2" else 1), 0.0)
        if c["mul"]:
            z = z * i["mul"].double()
        return z + i["resid"].double() if c["resid"] else z
    rows = []
    for x, tokens in zip(i["logits"], i["tokens"]):
        p = torch.log_softmax(x.double() * c["scale"], 0)
        rows.append([p[tokens.long()], torch.special.entr(p.exp()).sum()])
        if c["k"]:
            # an order of (value, index) pairs that no two entries share
            most = torch.topk(x.double(), c["k"]).values[-1]
            near = torch.nonzero(x.double() >= most).flatten().tolist()
            values = x.double()[near].tolist()
            best = sorted(zip(values, near), key=lambda t: (-t[0], t[1]))[:c["k"]]
            ids = torch.tensor([t for _, t in best], device="cuda")
            rows[-1] += [ids.to(torch.int32), p[ids]]
    return [torch.stack(t) for t in zip(*rows)]
