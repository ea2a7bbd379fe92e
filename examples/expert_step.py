"""A data-parallel training step of a block with attention and a layer of experts, on one GPU.

P nodes see different examples. In each step

1. every node runs layer norm, one projection to queries, keys and values (a linear layer of one
   expert), their norm and rotation, attention (plain torch), and a linear layer of experts, each on
   its own run of the tokens; between the forward and the backward pass it keeps the inputs of the
   norm and of both linear layers in 8 bits;
2. the backward pass writes all weights' gradients into the node's row of the flat gradient [P][N];
3. each row keeps its largest components per layer (``topk_ef_segments``), and the P streams are
   summed into a dense vector (``sparse_reduce``);
4. the matrices take orthogonalised momentum steps (``muon_step``, the experts' as one batch), the
   norms' weights plain ones.

    python examples/expert_step.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from top_gradient_compression_gb300 import api  # noqa: E402

HALF = torch.bfloat16


class Block:
    """The block's sizes, its parameters and where their gradients lie in a flat one."""

    def __init__(self, dim=96, q=4, kv=2, head=24, out=80, experts=3, tokens=96, device="cuda:0"):
        self.dim, self.q, self.kv, self.head, self.out = dim, q, kv, head, out
        self.experts, self.tokens, self.device = experts, tokens, device
        gen = torch.Generator(device=device).manual_seed(1)

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device=device)
        self.normal = normal
        self.shapes = {"weight": (dim,), "bias": (dim,), "project": ((q + 2 * kv) * head, dim),
                       "q_weight": (head,), "k_weight": (head,),
                       "experts": (experts, out, q * head)}
        self.params = {"weight": torch.ones(dim, device=device),
                       "bias": torch.zeros(dim, device=device),
                       "project": normal(*self.shapes["project"]) / dim ** 0.5,
                       "q_weight": torch.ones(head, device=device),
                       "k_weight": torch.ones(head, device=device),
                       "experts": normal(*self.shapes["experts"]) / (q * head) ** 0.5}
        self.begin = np.cumsum([0] + [int(np.prod(s)) for s in self.shapes.values()])
        # the tokens come sorted by their experts, whose runs are unequal; the last two have none
        cuts = [(tokens - 2) * e * (e + 1) // (experts * (experts + 1))
                for e in range(experts + 1)]
        self.offsets = torch.tensor(cuts, dtype=torch.int32, device=device)
        self.positions = torch.arange(tokens, dtype=torch.int32, device=device)
        half = torch.arange(head // 2, dtype=torch.float64, device=device)
        self.freqs = (100.0 ** (-half / (head // 2))).float()
        size = max(api.expert_linear_workspace_size(tokens, 1, (q + 2 * kv) * head, dim),
                   api.expert_linear_workspace_size(tokens, experts, out, q * head),
                   api.layer_norm_backward_workspace_size(tokens, dim),
                   api.head_norm_rotary_backward_workspace_size(tokens, q, kv, head))
        self.ws = api.workspace(size, device)

    def views(self, flat):
        """The parameters' views of a flat vector."""
        return {name: flat[a:b].view(shape) for (name, shape), a, b in
                zip(self.shapes.items(), self.begin, self.begin[1:])}

    def forward(self, x):
        """(y, what the backward pass needs)."""
        p, s = self.params, {}
        normed, s["mean"], s["rstd"] = api.layer_norm(x, p["weight"], p["bias"])
        s["x"] = api.checkpoint8(x)
        h = normed.to(HALF)
        s["h"] = api.checkpoint8(h)
        s["project"], s["experts"] = p["project"].to(HALF), p["experts"].to(HALF)
        qkv = api.expert_linear(h, s["project"], ws=self.ws).view(self.tokens, -1, self.head)
        s["q"], s["k"] = qkv[:, :self.q], qkv[:, self.q:self.q + self.kv]
        q, k = api.head_norm_rotary(s["q"], s["k"], self.positions, self.freqs, p["q_weight"],
                                    p["k_weight"])
        # attention, every query of a group with its key: [kv, group, tokens, head]
        s["qh"] = q.float().view(self.tokens, self.kv, -1, self.head).permute(1, 2, 0, 3)
        s["kh"] = k.float().transpose(0, 1)[:, None]
        s["vh"] = qkv[:, self.q + self.kv:].float().transpose(0, 1)[:, None]
        score = s["qh"] @ s["kh"].mT / self.head ** 0.5
        later = torch.ones_like(score, dtype=torch.bool).triu(1)
        s["prob"] = score.masked_fill(later, float("-inf")).softmax(-1)
        o = (s["prob"] @ s["vh"]).permute(2, 0, 1, 3).reshape(self.tokens, -1).to(HALF)
        s["o"] = api.checkpoint8(o)
        y = torch.zeros(self.tokens, self.out, dtype=HALF, device=self.device)
        return api.expert_linear(o, s["experts"], self.offsets, out=y, ws=self.ws), s

    def backward(self, dy, s, flat):
        """All gradients into `flat`; returns x's."""
        g = self.views(flat)
        do = torch.zeros(self.tokens, self.q * self.head, dtype=HALF, device=self.device)
        api.expert_linear_backward(dy, s["o"], s["experts"], self.offsets, dx=do,
                                   dweight=g["experts"], ws=self.ws)
        do = do.float().view(self.tokens, self.kv, -1, self.head).permute(1, 2, 0, 3)
        dv = (s["prob"].mT @ do).sum(1)
        dprob = do @ s["vh"].mT
        ds = s["prob"] * (dprob - (dprob * s["prob"]).sum(-1, keepdim=True)) / self.head ** 0.5
        dq = (ds @ s["kh"]).permute(2, 0, 1, 3).reshape(self.tokens, self.q, self.head).to(HALF)
        dk = (ds.mT @ s["qh"]).sum(1).transpose(0, 1).to(HALF)
        dqkv = torch.empty(self.tokens, self.q + 2 * self.kv, self.head, dtype=HALF,
                           device=self.device)
        dqkv[:, self.q + self.kv:] = dv.transpose(0, 1)
        api.head_norm_rotary_backward(
            dq, dk.contiguous(), s["q"], s["k"], self.positions, self.freqs,
            self.params["q_weight"], self.params["k_weight"], dq_out=dqkv[:, :self.q],
            dk_out=dqkv[:, self.q:self.q + self.kv], dq_weight=g["q_weight"],
            dk_weight=g["k_weight"], ws=self.ws)
        dh, _ = api.expert_linear_backward(dqkv.view(self.tokens, -1), s["h"], s["project"],
                                           dweight=g["project"], ws=self.ws)
        return api.layer_norm_backward(dh.float(), s["x"], s["mean"], s["rstd"],
                                       self.params["weight"], dweight=g["weight"],
                                       dbias=g["bias"], ws=self.ws)[0]


def train(steps: int = 40, nodes: int = 4, lr: float = 0.02, device: str = "cuda:0", **sizes):
    """Fits the outputs of another block of the same form; returns the loss of every step."""
    block = Block(device=device, **sizes)
    teacher = Block(device=device, **sizes)
    teacher.params["project"] = teacher.normal(*block.shapes["project"]) / block.dim ** 0.5
    teacher.params["experts"] = teacher.normal(*block.shapes["experts"]) / block.dim ** 0.5
    x = block.normal(nodes, block.tokens, block.dim)
    target = [teacher.forward(x[p])[0].float() for p in range(nodes)]

    begin = block.begin.astype(np.uint64)
    keep = np.maximum(1, np.diff(block.begin) // 4).astype(np.uint32)
    n = int(begin[-1])
    grad = torch.zeros(nodes, n, device=device)
    residual = torch.zeros_like(grad)
    summed = api.reduce_out(n, device, 0, 1)
    topk_ws = api.workspace(api.topk_ef_segments_workspace_size(nodes, n, begin, keep), device)
    sum_ws = api.workspace(api.reduce_workspace_size(nodes, n), device)
    momentum = {k: torch.zeros_like(block.params[k]) for k in ("project", "experts")}
    muon_ws = {k: api.workspace(api.orthogonalize_workspace_size(
        *((1,) + tuple(m.shape))[-3:]), device) for k, m in momentum.items()}

    losses = []
    for _ in range(steps):
        loss = torch.zeros((), device=device)
        for p in range(nodes):
            y, kept = block.forward(x[p])
            off = y.float() - target[p]
            loss += off.square().mean() / nodes
            block.backward((off * (2.0 / (off.numel() * nodes))).to(HALF), kept, grad[p])
        streams = api.topk_ef_segments(grad, residual, begin, keep, ws=topk_ws)
        total = block.views(api.sparse_reduce(*streams, n, 0, 1, out=summed, ws=sum_ws).dense)
        for name, param in block.params.items():
            if name in momentum:
                api.muon_step(param, total[name], momentum[name], lr=lr, ws=muon_ws[name])
            else:
                param -= lr * total[name]
        losses.append(loss)
    for ws in (block.ws, topk_ws, sum_ws, *muon_ws.values()):
        status = api.get_status(ws)
        if status:
            raise RuntimeError(api.STATUS[status])
    return [float(v) for v in losses]


if __name__ == "__main__":
    curve = train()
    for step in range(0, len(curve), 10):
        print(f"step {step:3d}  loss {curve[step]:.5f}")
    print(f"last      loss {curve[-1]:.5f}")
