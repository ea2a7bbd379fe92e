"""Cases of the operators at the two ends of a training step's gradient exchange.

Layer norm and its backward pass make part of the gradient that the nodes exchange;
the orthogonalised update (Newton-Schulz) and the weight step built on it use the
reduced gradient. `run` computes a case in plain torch operations in 32 bits, or, where
`own` is true, by the framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
# a, b, c of the quintic step x -> a x + b x^3 + c x^5 on the singular values, five times
COEFFS = [(3.4445, -4.7750, 2.0315)] * 5
MU, DECAY = 0.95, 0.1


def listed():
    return [
        # one position of a model that answers token by token: latency
        {"name": "ln_token", "op": "ln", "rows": 1, "dim": 1024, "pad": 0, "type": "bf16"},
        # a ragged batch in single precision, its rows a slice of a wider activation
        {"name": "ln_ragged_f32", "op": "ln", "rows": 1237, "dim": 777, "pad": 23, "type": "f32"},
        # the activations of one training step of a large model
        {"name": "ln_large", "op": "ln", "rows": 16384, "dim": 4096, "pad": 0, "type": "bf16"},
        # a small model's batch: the two launches' latency counts
        {"name": "ln_bwd_small", "op": "ln_bwd", "rows": 64, "dim": 512, "pad": 0, "type": "f32"},
        # an odd width and an odd number of positions
        {"name": "ln_bwd_odd_f16", "op": "ln_bwd", "rows": 3001, "dim": 1023, "pad": 0,
         "type": "f16"},
        # the activations of one training step of a large model, both gradients
        {"name": "ln_bwd_large", "op": "ln_bwd", "rows": 16384, "dim": 4096, "pad": 0,
         "type": "bf16"},
        # a small layer: fifteen dependent products of a few tiles each
        {"name": "ortho_small", "op": "ortho", "batch": 1, "m": 256, "n": 256, "type": "f32"},
        # tall layers of odd sizes, three of them in one call
        {"name": "ortho_odd_tall", "op": "ortho", "batch": 3, "m": 1000, "n": 333, "type": "bf16"},
        # a large model's attention projection
        {"name": "ortho_large", "op": "ortho", "batch": 1, "m": 4096, "n": 4096, "type": "f32"},
        # the weight step of a small layer
        {"name": "muon_small", "op": "muon", "batch": 1, "m": 512, "n": 512, "type": "f32"},
        # the same layer of eight blocks of a model, 16-bit weights, one call
        {"name": "muon_blocks", "op": "muon", "batch": 8, "m": 1024, "n": 1024, "type": "bf16"},
        # a large model's feed-forward matrix
        {"name": "muon_large", "op": "muon", "batch": 1, "m": 4096, "n": 16384, "type": "f32"},
    ]


def _size(rng, low, high):
    """Log-uniform in [low, high]; half of the sizes are odd, the others multiples of 64."""
    v = int(math.exp(rng.uniform(math.log(low), math.log(high))))
    return v | 1 if rng.random() < 0.5 or v < 64 else v // 128 * 128 + 64


def draw(rng):
    op = rng.choice(["ln", "ln_bwd", "ortho", "muon"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("ln", "ln_bwd"):
        dim = _size(rng, 32, 8192)
        rows = int(math.exp(rng.uniform(0.0, math.log(16384 * 4096 / 2 / dim))))
        return {"op": op, "rows": min(rows, 65536) | 1, "dim": dim,
                "pad": rng.choice([0, 0, 8, 13]), "type": kind}
    m, n = _size(rng, 16, 4096), _size(rng, 16, 16384)
    if rng.random() < 0.5:
        m, n = n, m
    most = max(1, min(16, 4096 ** 3 // (min(m, n) ** 2 * max(m, n))))
    return {"op": op, "batch": rng.randint(1, most), "m": m, "n": n, "type": kind}


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _gradients(gen, batch, m, n):
    """Gradients of linear layers: a few strong directions, a tail that decays with the
    direction's rank, and noise of the examples."""
    r = min(m, n, 64)
    decay = torch.arange(1, r + 1, device=DEV, dtype=torch.float32).rsqrt()
    g = torch.baddbmm(_normal(gen, batch, m, n), _normal(gen, batch, m, r) * decay,
                      _normal(gen, batch, r, n), beta=1.0)
    return g.mul_(1e-3)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = DTYPES[case["type"]]
    s = {"case": dict(case)}
    if case["op"] in ("ln", "ln_bwd"):
        rows, dim, wide = case["rows"], case["dim"], case["dim"] + case["pad"]
        # features of unequal spread and an offset, as a residual stream has
        spread = torch.exp(0.5 * _normal(gen, wide))
        x = _normal(gen, rows, wide).mul_(spread).add_(0.5 * _normal(gen, wide))
        s["x"] = x.to(t)[:, :dim]
        s["weight"] = (1.0 + 0.1 * _normal(gen, dim)).to(t)
        s["bias"] = (0.1 * _normal(gen, dim)).to(t)
        if case["op"] == "ln_bwd":
            s["dy"] = (0.1 * _normal(gen, rows, wide)).to(t)[:, :dim]
            xs = s["x"].float()
            s["mean"] = xs.mean(1)
            s["rstd"] = torch.rsqrt(xs.var(1, unbiased=False) + EPS)
        return s
    batch, m, n = case["batch"], case["m"], case["n"]
    g = _gradients(gen, batch, m, n)
    if case["op"] == "ortho":
        s["g"] = g.to(t)
        return s
    # a step in mid-training: momentum of a few steps, weights of unit gain, and an update
    # whose entries' size (0.2 of the rate) does not depend on the layer's shape
    s["grad"] = g
    s["momentum"] = _gradients(gen, batch, m, n).mul_(4.0)
    s["weight"] = _normal(gen, batch, m, n).mul_(n ** -0.5).to(t)
    s["lr"], s["scale"] = 5e-4, 0.2 * max(m, n) ** 0.5
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    x = s["x"].float()
    mean = x.sum(1, keepdim=True) / x.shape[1]
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).sum(1, keepdim=True) / x.shape[1] + EPS)
    y = xc * rstd * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_norm_backward(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    d = dy * s["weight"].float()
    dx = rstd * (d - d.sum(1, keepdim=True) / x.shape[1]
                 - xh * ((d * xh).sum(1, keepdim=True) / x.shape[1]))
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _plain_orthogonal(g):
    tall = g.shape[1] > g.shape[2]
    x = g.float()
    x = x.transpose(1, 2) if tall else x
    x = x / torch.sqrt((x * x).sum((1, 2), keepdim=True))
    for a, b, c in COEFFS:  # each step needs the one before it
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.transpose(1, 2) if tall else x


def _plain_muon(s):
    s["momentum"].mul_(MU).add_(s["grad"])
    o = _plain_orthogonal(s["grad"] + MU * s["momentum"])
    w = s["weight"].float() * (1.0 - s["lr"] * DECAY) - (s["lr"] * s["scale"]) * o
    s["weight"].copy_(w)
    return s["weight"], s["momentum"]


# --------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "ln":
            return _plain_norm(state)
        if op == "ln_bwd":
            return _plain_norm_backward(state)
        if op == "ortho":
            return _plain_orthogonal(state["g"]).to(torch.bfloat16)
        return _plain_muon(state)
    from top_gradient_compression_gb300 import api
    if op == "ln":
        return api.layer_norm(state["x"], state["weight"], state["bias"], EPS)
    if op == "ln_bwd":
        if "ws" not in state:  # kept by a training loop from step to step
            x = state["x"]
            state["ws"] = api.workspace(
                api.layer_norm_backward_workspace_size(x.shape[0], x.shape[1]), x.device)
        return api.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"],
                                       state["weight"], ws=state["ws"])
    if "ws" not in state:  # kept by a training loop from step to step
        t = state["g"] if op == "ortho" else state["grad"]
        state["ws"] = api.workspace(api.orthogonalize_workspace_size(*t.shape), t.device)
    if op == "ortho":
        return api.orthogonalize(state["g"], COEFFS, ws=state["ws"])
    return api.muon_step(state["weight"], state["grad"], state["momentum"], lr=state["lr"],
                         mu=MU, nesterov=True, weight_decay=DECAY, scale=state["scale"],
                         coeffs=COEFFS, ws=state["ws"])


# --------------------------------------------------------------------------- what it takes
def work(case):
    if case["op"] in ("ln", "ln_bwd"):
        n, e = case["rows"] * case["dim"], BYTES[case["type"]]
        if case["op"] == "ln":
            return {"bytes": 2 * n * e + 2 * case["dim"] * e + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + case["dim"] * (e + 8) + 8 * case["rows"], "flops": 14 * n}
    k, l = sorted((case["m"], case["n"]))
    elements = case["batch"] * k * l
    # a step: the symmetric products x x' and s s at half a product's cost, and p x
    flops = len(COEFFS) * case["batch"] * (k * k * l + k ** 3 + 2 * k * k * l)
    e = BYTES[case["type"]]
    moved = e + 2 if case["op"] == "ortho" else 4 + 8 + 2 * e
    return {"bytes": elements * moved, "flops": flops}


# --------------------------------------------------------------------------- 64 bits
def _exact_orthogonal(g):
    """The steps as one polynomial of the Gram matrix: with q_k(G) the product of the first
    k factors a + b S + c S^2, S_k = q_k G q_k, and the result is q x / |x|."""
    x = g.double()
    if x.shape[1] > x.shape[2]:
        return _exact_orthogonal(g.transpose(1, 2)).transpose(1, 2)
    x = x / torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True)
    eye = torch.eye(x.shape[1], dtype=torch.float64, device=x.device)
    gram = torch.bmm(x, x.mT)
    q = eye.expand_as(gram)
    for a, b, c in COEFFS:
        p = a * eye + torch.bmm(gram, b * eye + c * gram)
        q = torch.bmm(p, q)
        gram = torch.bmm(torch.bmm(p, gram), p)
    return torch.bmm(q, x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ln", "ln_bwd"):
        x = s["x"].double()
        w, b = s["weight"].double(), s["bias"].double()
        if case["op"] == "ln":
            mean = x.mean(1)
            rstd = (x.var(1, unbiased=False) + EPS).pow(-0.5)
            return torch.addcmul(b, (x - mean[:, None]) * rstd[:, None], w), mean, rstd
        dy, mean, rstd = s["dy"].double(), s["mean"].double(), s["rstd"].double()
        xh = (x - mean[:, None]) * rstd[:, None]
        d = dy * w
        dx = (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True)) * rstd[:, None]
        return dx, torch.einsum("rd,rd->d", dy, xh), dy.sum(0)
    if case["op"] == "ortho":
        return _exact_orthogonal(s["g"])
    g, m = s["grad"].double(), s["momentum"].double()
    m = MU * m + g
    w = s["weight"].double()
    w = w - s["lr"] * (DECAY * w + s["scale"] * _exact_orthogonal(g + MU * m))
    return w, m
