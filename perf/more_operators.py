"""Cases of the operators that make a node's gradient: activations kept in 8 bits and the
backward passes that read them, linear layers of experts on ragged runs of rows, and the norm
and position rotation of queries and keys. `run` computes a case in plain torch operations in
32 bits, or, where `own` is true, by the framework's kernels.

An activation in 8 bits: whole numbers c of at most 127, and for every 128 columns of a row an
exponent byte b, standing for c 2^(b - 127), with the least b for which the group's largest
magnitude rounds to 127 at most.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
GROUP = 128                       # columns that share an exponent
LEAST = {"f32": -126, "bf16": -126, "f16": -24}  # exponents: the type holds every c 2^e
MOST = {"f32": 121, "bf16": 121, "f16": 9}
NORM_EPS, HEAD_EPS = 1e-5, 1e-6


def listed():
    return [
        # a ragged batch in single precision, its rows a slice of a wider activation
        {"name": "store_odd_f32", "op": "store", "rows": 1237, "dim": 777, "pad": 23,
         "type": "f32"},
        # the activations of one training step of a large model
        {"name": "store_large", "op": "store", "rows": 16384, "dim": 4096, "pad": 0,
         "type": "bf16"},
        # an odd width and an odd number of positions
        {"name": "norm8_odd_f16", "op": "norm8", "rows": 3001, "dim": 1023, "pad": 0,
         "type": "f16"},
        # the norm's gradients in one training step of a large model
        {"name": "norm8_large", "op": "norm8", "rows": 16384, "dim": 4096, "pad": 0,
         "type": "bf16"},
        # a batch of single tokens: the weights are what is read
        {"name": "experts_tokens", "op": "experts", "rows": 64, "left": 0, "experts": 8,
         "n": 2048, "k": 1024, "type": "bf16"},
        # the first matrix of a layer of experts in one training step
        {"name": "experts_large", "op": "experts", "rows": 16384, "left": 0, "experts": 8,
         "n": 4096, "k": 2048, "type": "bf16"},
        # odd sizes, and rows behind the last expert's
        {"name": "experts_back_odd_f16", "op": "experts_back", "rows": 1237, "left": 37,
         "experts": 5, "n": 777, "k": 333, "stored": False, "type": "f16"},
        # both gradients of such a layer in one training step, its input kept in 8 bits
        {"name": "experts_back8_large", "op": "experts_back", "rows": 16384, "left": 0,
         "experts": 4, "n": 2048, "k": 4096, "stored": True, "type": "bf16"},
        # one position of a model that answers token by token: latency
        {"name": "heads_token", "op": "heads", "rows": 1, "q": 32, "kv": 8, "dim": 128,
         "turned": 128, "pairs": False, "type": "bf16"},
        # all positions of one training step of a large model
        {"name": "heads_large", "op": "heads", "rows": 16384, "q": 32, "kv": 8, "dim": 128,
         "turned": 128, "pairs": False, "type": "bf16"},
        # a small model in single precision, neighbouring elements turned, half of a head
        {"name": "heads_back_odd_f32", "op": "heads_back", "rows": 1501, "q": 6, "kv": 2,
         "dim": 80, "turned": 40, "pairs": True, "type": "f32"},
        # the gradients of one training step of a large model
        {"name": "heads_back_large", "op": "heads_back", "rows": 16384, "q": 32, "kv": 8,
         "dim": 128, "turned": 128, "pairs": False, "type": "bf16"},
    ]


def _size(rng, low, high):
    """Log-uniform in [low, high]; half of the sizes are odd, the others multiples of 64."""
    v = int(math.exp(rng.uniform(math.log(low), math.log(high))))
    return v | 1 if rng.random() < 0.5 or v < 64 else v // 128 * 128 + 64


def draw(rng):
    op = rng.choice(["store", "norm8", "experts", "experts_back", "heads", "heads_back"])
    if op in ("store", "norm8"):
        dim = _size(rng, 32, 8192)
        rows = int(math.exp(rng.uniform(0.0, math.log(16384 * 4096 / 2 / dim))))
        return {"op": op, "rows": min(rows, 65536) | 1, "dim": dim,
                "pad": rng.choice([0, 0, 8, 13]), "type": rng.choice(["f32", "bf16", "f16"])}
    if op in ("heads", "heads_back"):
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 96, 112, 128, 192, 256, 2 * rng.randint(8, 100)])
        turned = rng.choice([dim, dim, dim // 4 * 2])
        q = kv * rng.choice([1, 2, 4, 7])
        most = 16384 * 40 * 128 / 2 / ((q + kv) * dim)
        return {"op": op, "rows": int(math.exp(rng.uniform(0.0, math.log(most)))) | 1, "q": q,
                "kv": kv, "dim": dim, "turned": turned, "pairs": rng.random() < 0.5,
                "type": rng.choice(["f32", "bf16", "f16"])}
    n, k, experts = _size(rng, 64, 4096), _size(rng, 64, 4096), rng.choice([1, 2, 5, 8, 16, 33])
    most = min(16384, 16384 * 4096 * 2048 / 2 / (n * k))
    rows = int(math.exp(rng.uniform(0.0, math.log(most)))) | 1
    c = {"op": op, "rows": rows, "left": rng.choice([0, 0, rows // 9]), "experts": experts,
         "n": n, "k": k, "type": rng.choice(["bf16", "f16"])}
    if op == "experts_back":
        c["stored"] = rng.random() < 0.5
    return c


# --------------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _activations(gen, rows, dim, pad):
    """Features of unequal spread and an offset, as a residual stream has; a slice of a
    wider array where pad is not 0."""
    wide = dim + pad
    x = _normal(gen, rows, wide).mul_(torch.exp(0.5 * _normal(gen, wide)))
    return x.add_(0.5 * _normal(gen, wide))[:, :dim]


def _in_groups(x):
    """x [rows, dim] as [rows, groups, 128], zeros behind the last column."""
    rows, dim = x.shape
    groups = -(-dim // GROUP)
    padded = torch.zeros(rows, groups * GROUP, dtype=x.dtype, device=x.device)
    padded[:, :dim] = x
    return padded.view(rows, groups, GROUP)


def _store(x, kind):
    """The 8-bit form of x in plain torch: (codes int8 [rows, dim rounded up to 16], exponent
    bytes uint8 [rows, groups])."""
    rows, dim = x.shape
    g = _in_groups(x.float())
    fraction, power = torch.frexp(g.abs().amax(2))  # the largest: fraction 2^power
    e = torch.where(fraction * 128 < 127.5, power - 7, power - 6)
    e = torch.where(fraction == 0, LEAST[kind], e.clamp(LEAST[kind], MOST[kind]))
    # by two powers of two, each of them a number
    half = e[:, :, None] // 2
    c = torch.ldexp(torch.ldexp(g, -half), half - e[:, :, None])
    c = c.round().clamp(-127, 127).to(torch.int8).view(rows, -1)
    width = -(-dim // 16) * 16
    codes = torch.zeros(rows, width, dtype=torch.int8, device=x.device)
    codes[:, :dim] = c[:, :dim]
    return codes, (e + 127).to(torch.uint8)


def _restore(codes, exponents, dim):
    """What the 8-bit form stands for, in 32 bits."""
    g = _in_groups(codes[:, :dim].float())
    e = exponents.to(torch.int32)[:, :, None] - 127
    half = e // 2
    return torch.ldexp(torch.ldexp(g, half), e - half).view(codes.shape[0], -1)[:, :dim]


def _runs(seed, experts, rows):
    """Where the experts' runs of rows begin and end, unequal as a router's choices are."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    share = torch.exp(0.7 * torch.randn(experts, generator=gen))
    ends = (share.cumsum(0) / share.sum() * rows).round().long()
    return [0] + ends.tolist()[:-1] + [rows]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = DTYPES[case["type"]]
    s, op, rows = {"case": dict(case)}, case["op"], case["rows"]
    if op in ("store", "norm8"):
        dim, pad = case["dim"], case["pad"]
        x = _activations(gen, rows, dim, pad)
        if op == "store":
            s["x"] = torch.empty(rows, dim + pad, dtype=t, device=DEV)[:, :dim].copy_(x)
            return s
        x = x.to(t)
        s["codes"], s["exponents"] = _store(x, case["type"])
        x = x.float()
        s["mean"] = x.mean(1)
        s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + NORM_EPS)
        s["weight"] = (1.0 + 0.1 * _normal(gen, dim)).to(t)
        s["dy"] = (0.1 * _normal(gen, rows, dim + pad)).to(t)[:, :dim]
        return s
    if op in ("experts", "experts_back"):
        e, n, k = case["experts"], case["n"], case["k"]
        s["runs"] = _runs(seed, e, rows - case["left"])
        s["offsets"] = torch.tensor(s["runs"], dtype=torch.int32, device=DEV)
        s["weight"] = _normal(gen, e, n, k).mul_(k ** -0.5).to(t)
        x = _activations(gen, rows, k, 0).to(t)
        if op == "experts":
            s["x"], s["y"] = x, torch.zeros(rows, n, dtype=t, device=DEV)
            return s
        if case["stored"]:
            s["codes"], s["exponents"] = _store(x, case["type"])
        else:
            s["x"] = x
        s["dy"] = (0.01 * _normal(gen, rows, n)).to(t)
        s["dx"] = torch.zeros(rows, k, dtype=t, device=DEV)
        return s
    q, kv, dim = case["q"], case["kv"], case["dim"]
    # one projection for queries, keys and values; the first two are slices of its result
    both = _activations(gen, rows, (q + 2 * kv) * dim, 0).to(t).view(rows, q + 2 * kv, dim)
    s["q"], s["k"] = both[:, :q], both[:, q:q + kv]
    s["q_weight"] = (1.0 + 0.1 * _normal(gen, dim)).to(t)
    s["k_weight"] = (1.0 + 0.1 * _normal(gen, dim)).to(t)
    # several documents one after the other, one of them far along a long one
    start = torch.randint(0, 1 << 20, (1,), generator=gen, device=DEV)
    at = torch.arange(rows, device=DEV)
    s["positions"] = torch.where(at < rows // 2, at + start, at - rows // 2).to(torch.int32)
    half = torch.arange(case["turned"] // 2, device=DEV, dtype=torch.float64)
    s["freqs"] = (10000.0 ** (-half / max(1, case["turned"] // 2))).float()
    if op == "heads_back":
        s["dq"] = (0.1 * _normal(gen, rows, q, dim)).to(t)
        s["dk"] = (0.1 * _normal(gen, rows, kv, dim)).to(t)
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_store(s):
    kind = s["case"]["type"]
    return _restore(*_store(s["x"], kind), s["case"]["dim"]).to(DTYPES[kind])


def _plain_norm8(s):
    x, dy = _restore(s["codes"], s["exponents"], s["case"]["dim"]), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    d = dy * s["weight"].float()
    dx = rstd * (d - d.sum(1, keepdim=True) / x.shape[1]
                 - xh * ((d * xh).sum(1, keepdim=True) / x.shape[1]))
    return dx.to(s["dy"].dtype), (dy * xh).sum(0), dy.sum(0)


def _plain_experts(s):
    for e, (a, b) in enumerate(zip(s["runs"], s["runs"][1:])):  # a matrix of its own for each
        s["y"][a:b] = s["x"][a:b].float() @ s["weight"][e].float().t()
    return s["y"]


def _plain_experts_back(s):
    if s["case"]["stored"]:
        x = _restore(s["codes"], s["exponents"], s["case"]["k"])
    else:
        x = s["x"].float()
    dw = torch.empty(s["weight"].shape, dtype=torch.float32, device=DEV)
    for e, (a, b) in enumerate(zip(s["runs"], s["runs"][1:])):
        dy = s["dy"][a:b].float()
        s["dx"][a:b] = dy @ s["weight"][e].float()
        torch.matmul(dy.t(), x[a:b], out=dw[e])
    return s["dx"], dw


def _split(x, s):
    """The two members of each turned pair, and what is not turned."""
    turned = s["case"]["turned"]
    r = x[..., :turned]
    if s["case"]["pairs"]:
        return r[..., 0::2], r[..., 1::2], x[..., turned:]
    return r[..., :turned // 2], r[..., turned // 2:], x[..., turned:]


def _joined(a, b, rest, s):
    if s["case"]["pairs"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _cos_sin(s):
    angle = s["positions"].double()[:, None, None] * s["freqs"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _plain_heads(s):
    cos, sin = _cos_sin(s)

    def one(x, weight):
        x = x.float()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + HEAD_EPS)
        a, b, rest = _split(x * r * weight.float(), s)
        return _joined(a * cos - b * sin, a * sin + b * cos, rest, s)
    t = s["q"].dtype
    return one(s["q"], s["q_weight"]).to(t), one(s["k"], s["k_weight"]).to(t)


def _plain_heads_back(s):
    cos, sin = _cos_sin(s)

    def one(dy, x, weight):
        x = x.float()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + HEAD_EPS)
        a, b, rest = _split(dy.float(), s)
        g = _joined(a * cos + b * sin, b * cos - a * sin, rest, s)
        xh, d = x * r, g * weight.float()
        dx = r * (d - xh * ((d * xh).sum(-1, keepdim=True) / x.shape[-1]))
        return dx.to(dy.dtype), (g * xh).sum((0, 1))
    dq, wq = one(s["dq"], s["q"], s["q_weight"])
    dk, wk = one(s["dk"], s["k"], s["k_weight"])
    return dq, dk, wq, wk


# --------------------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        plain = {"store": _plain_store, "norm8": _plain_norm8, "experts": _plain_experts,
                 "experts_back": _plain_experts_back, "heads": _plain_heads,
                 "heads_back": _plain_heads_back}
        return plain[op](s)
    from top_gradient_compression_gb300 import api
    if op == "store":
        return api.restore8(api.checkpoint8(s["x"]))
    if op == "heads":
        return api.head_norm_rotary(s["q"], s["k"], s["positions"], s["freqs"], s["q_weight"],
                                    s["k_weight"], HEAD_EPS, s["case"]["pairs"])
    if "ws" not in s:  # kept by a training loop from step to step
        c = s["case"]
        if op == "norm8":
            size = api.layer_norm_backward_workspace_size(c["rows"], c["dim"])
        elif op == "heads_back":
            size = api.head_norm_rotary_backward_workspace_size(c["rows"], c["q"], c["kv"],
                                                                c["dim"])
        else:
            size = api.expert_linear_workspace_size(c["rows"], c["experts"], c["n"], c["k"])
        s["ws"] = api.workspace(size, DEV)
    if op == "norm8":
        x = api.Checkpoint8(s["codes"], s["exponents"], s["case"]["dim"], s["dy"].dtype)
        return api.layer_norm_backward(s["dy"], x, s["mean"], s["rstd"], s["weight"], ws=s["ws"])
    if op == "experts":
        return api.expert_linear(s["x"], s["weight"], s["offsets"], out=s["y"], ws=s["ws"])
    if op == "experts_back":
        x = s["x"] if "x" in s else api.Checkpoint8(s["codes"], s["exponents"], s["case"]["k"],
                                                    s["dy"].dtype)
        return api.expert_linear_backward(s["dy"], x, s["weight"], s["offsets"], dx=s["dx"],
                                          ws=s["ws"])
    return api.head_norm_rotary_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"],
                                         s["freqs"], s["q_weight"], s["k_weight"], HEAD_EPS,
                                         s["case"]["pairs"], ws=s["ws"])


# --------------------------------------------------------------------------- what it takes
def work(case):
    op, rows, e = case["op"], case["rows"], BYTES[case["type"]]
    if op in ("store", "norm8"):
        n = rows * case["dim"]
        eight = n + rows * -(-case["dim"] // GROUP)
        if op == "store":  # written, and read back
            return {"bytes": 2 * n * e + 2 * eight, "flops": 5 * n}
        return {"bytes": 2 * n * e + eight + case["dim"] * (e + 8) + 8 * rows, "flops": 15 * n}
    if op in ("experts", "experts_back"):
        rows -= case["left"]
        n, k = case["n"], case["k"]
        used = min(case["experts"], rows) * n * k  # weights of experts that have rows
        if op == "experts":
            return {"bytes": e * (rows * (n + k) + used), "flops": 2 * rows * n * k}
        x = rows * (k + -(-k // GROUP)) if case["stored"] else rows * k * e
        return {"bytes": e * (rows * (n + k) + used) + x + 4 * case["experts"] * n * k,
                "flops": 4 * rows * n * k}
    n = rows * (case["q"] + case["kv"]) * case["dim"]
    if op == "heads":
        return {"bytes": 2 * n * e + 4 * rows + 2 * case["dim"] * e, "flops": 7 * n}
    return {"bytes": 3 * n * e + 4 * rows + 2 * case["dim"] * (e + 4), "flops": 16 * n}


# --------------------------------------------------------------------------- 64 bits
def _exact_values(codes, exponents, dim):
    scale = torch.pow(2.0, exponents.double() - 127.0).repeat_interleave(GROUP, 1)[:, :dim]
    return codes[:, :dim].double() * scale


def _exact_store(x, kind):
    x = x.double()
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], GROUP):
        part = x[:, c:c + GROUP]
        top = part.abs().max(1, keepdim=True).values
        e = torch.floor(torch.log2(top / 127.5)) + 1.0  # top 2^-e < 127.5
        e = e.clamp(LEAST[kind], MOST[kind])
        out[:, c:c + GROUP] = torch.round(part * 2.0 ** -e).clamp(-127, 127) * 2.0 ** e
    return out


def _exact_heads(s, backward):
    phase = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                        s["positions"].double()[:, None] * s["freqs"].double()[None, :])
    phase = phase[:, None, :].conj() if backward else phase[:, None, :]
    turned, pairs = s["case"]["turned"], s["case"]["pairs"]

    def turn(x):
        head = x[..., :turned]
        z = head.unflatten(-1, (-1, 2)) if pairs else head.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * phase)
        z = z.flatten(-2) if pairs else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., turned:]], -1)

    def norm(x):
        return (x.square().mean(-1, keepdim=True) + HEAD_EPS).rsqrt()
    if not backward:
        return tuple(turn(s[i].double() * norm(s[i].double()) * s[i + "_weight"].double())
                     for i in ("q", "k"))
    dx, dw = [], []
    for i in ("q", "k"):
        x, g = s[i].double(), turn(s["d" + i].double())
        r, u = norm(x), g * s[i + "_weight"].double()
        dx.append(r * u - r ** 3 * x * (u * x).mean(-1, keepdim=True))
        dw.append(torch.einsum("thd,thd->d", g, x * r))
    return (*dx, *dw)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "store":
        return _exact_store(s["x"], case["type"])
    if op == "norm8":
        x = _exact_values(s["codes"], s["exponents"], case["dim"])
        dy, rstd = s["dy"].double(), s["rstd"].double()
        xh = (x - s["mean"].double()[:, None]) * rstd[:, None]
        d = dy * s["weight"].double()
        dx = (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True)) * rstd[:, None]
        return dx, torch.einsum("rd,rd->d", dy, xh), dy.sum(0)
    if op in ("heads", "heads_back"):
        return _exact_heads(s, op == "heads_back")
    of = torch.bucketize(torch.arange(case["rows"], device=DEV), s["offsets"], right=True) - 1
    w = s["weight"].double()
    if op == "experts":
        y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            r = (of == e).nonzero()[:, 0]
            y[r] = torch.einsum("rk,nk->rn", s["x"][r].double(), w[e])
        return y
    x = _exact_values(s["codes"], s["exponents"], case["k"]) if case["stored"] else s["x"].double()
    dx = torch.zeros(case["rows"], case["k"], dtype=torch.float64, device=DEV)
    dw = torch.zeros_like(w)
    for e in range(case["experts"]):
        r = (of == e).nonzero()[:, 0]
        dy = s["dy"][r].double()
        dx[r] = torch.einsum("rn,nk->rk", dy, w[e])
        dw[e] = torch.einsum("rn,rk->nk", dy, x[r])
    return dx, dw
