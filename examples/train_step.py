"""A data-parallel training step around the sparse gradient exchange, on one GPU.

P nodes share a layer norm and a linear layer and see different examples. In each step

1. every node runs layer norm, the linear layer and their backward pass; the norm's weight
   gradients go straight into the node's row of the flat gradient [P][N];
2. each row keeps its largest components per layer, the rest staying in the error-feedback
   residual (``topk_ef_segments``);
3. the P streams are summed into a dense vector (``sparse_reduce`` with a dense result);
4. the norm's parameters take a plain gradient step, and the matrix an orthogonalised
   momentum step on its slice of the vector (``muon_step``).

    python examples/train_step.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from top_gradient_compression_gb300 import api  # noqa: E402


def train(steps: int = 60, nodes: int = 4, examples: int = 256, dim: int = 192, out: int = 160,
          lr: float = 0.02, device: str = "cuda:0"):
    """Fits a fixed teacher of the same form; returns the loss of every step."""
    gen = torch.Generator(device=device).manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)
    teacher = normal(out, dim) / dim ** 0.5
    x = normal(nodes, examples, dim) * torch.exp(normal(dim)) + normal(dim)
    weight, bias = torch.ones(dim, device=device), torch.zeros(dim, device=device)
    matrix = 0.1 * normal(out, dim) / dim ** 0.5
    target = [api.layer_norm(x[p])[0] @ teacher.t() for p in range(nodes)]

    # the flat gradient's layers: weight, bias, matrix
    begin = np.array([0, dim, 2 * dim, 2 * dim + out * dim], np.uint64)
    keep = np.array([dim // 4, dim // 4, out * dim // 10], np.uint32)
    n = int(begin[-1])
    grad = torch.zeros(nodes, n, device=device)
    residual = torch.zeros_like(grad)
    momentum = torch.zeros_like(matrix)
    norm_ws = api.workspace(api.layer_norm_backward_workspace_size(examples, dim), device)
    topk_ws = api.workspace(api.topk_ef_segments_workspace_size(nodes, n, begin, keep), device)
    sum_ws = api.workspace(api.reduce_workspace_size(nodes, n), device)
    muon_ws = api.workspace(api.orthogonalize_workspace_size(1, out, dim), device)
    summed = api.reduce_out(n, device, 0, 1)

    losses = []
    for _ in range(steps):
        loss = torch.zeros((), device=device)
        for p in range(nodes):
            h, mean, rstd = api.layer_norm(x[p], weight, bias)
            off = h @ matrix.t() - target[p]
            loss += off.square().mean() / nodes
            dy = off * (2.0 / (off.numel() * nodes))
            torch.mm(dy.t(), h, out=grad[p, 2 * dim:].view(out, dim))
            api.layer_norm_backward(dy @ matrix, x[p], mean, rstd, weight, dweight=grad[p, :dim],
                                    dbias=grad[p, dim:2 * dim], ws=norm_ws)
        streams = api.topk_ef_segments(grad, residual, begin, keep, ws=topk_ws)
        total = api.sparse_reduce(*streams, n, 0, 1, out=summed, ws=sum_ws).dense
        weight -= lr * total[:dim]
        bias -= lr * total[dim:2 * dim]
        api.muon_step(matrix, total[2 * dim:].view(out, dim), momentum, lr=lr, ws=muon_ws)
        losses.append(loss)
    for ws in (topk_ws, sum_ws, muon_ws):
        status = api.get_status(ws)
        if status:
            raise RuntimeError(api.STATUS[status])
    return [float(v) for v in losses]


if __name__ == "__main__":
    curve = train()
    for step in range(0, len(curve), 10):
        print(f"step {step:3d}  loss {curve[step]:.5f}")
    print(f"last      loss {curve[-1]:.5f}")
