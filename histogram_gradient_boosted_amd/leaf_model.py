"""A small model of learned vectors on top of grown trees, as an example of the
vector verbs run together: `python -m histogram_gradient_boosted_amd.leaf_model`.

Each bin of a row is a token with a learned vector (embed); the row's vectors
side by side are normalised (layer_norm) and sent to the leaf that each tree
gives the row (route, route_gather).  A leaf is an expert with a learned scale
for every value; the answers come back with the leaves' learned weights applied
(route_combine), and the score is their mean.  The gradients are the verbs' own,
called in the opposite order; nothing here needs torch.autograd.
"""
from __future__ import annotations

from dataclasses import dataclass, field
from typing import Dict, List, NamedTuple

import numpy as np

from .binding import Context, Route
from .tree import DeviceLevel


def leaves_of(levels: List[DeviceLevel], n_rows: int, device, first: int = 0):
    """(int32 [n_rows]: the deepest node of a grown tree that holds each row,
    numbered from `first` on, level by level; the number after the last)."""
    import torch
    leaf = torch.full((n_rows,), first, dtype=torch.int32, device=device)
    first += 1
    for level in levels[1:]:
        counts = torch.from_numpy(np.diff(level.offsets)).to(device)
        node = torch.repeat_interleave(torch.arange(first, first + level.n_nodes, dtype=torch.int32, device=device), counts)
        leaf[level.rows[: node.numel()].long()] = node
        first += level.n_nodes
    return leaf, first


def tokens_of(bins: np.ndarray, n_slots: int, device):
    """The tokens [n_rows, F] of a binned matrix [F, n_rows]: a feature's first
    token is its number times n_slots."""
    import torch
    F = bins.shape[0]
    first = torch.arange(F, dtype=torch.int32, device=device) * n_slots
    return (torch.from_numpy(bins.T.astype(np.int32)).to(device) + first).contiguous()


class Saved(NamedTuple):
    """What the forward pass keeps for the gradients."""
    tokens: object
    experts: object
    x: object
    mean: object
    rstd: object
    route: Route
    place: object     # the expert of each place
    sorted: object    # the rows in the experts' order
    scales: object    # the expert's scales, by place
    answers: object
    share: object


@dataclass
class LeafModel:
    """Parameters are float32; `dtype` is the vectors' type.  `state` is the
    optimiser's: running means of each gradient and its square, and the steps."""
    ctx: Context
    n_features: int
    n_slots: int
    n_leaves: int
    dim: int
    dtype: object
    params: Dict[str, object]
    state: Dict[str, object] = field(default_factory=dict)

    @classmethod
    def make(cls, ctx: Context, n_features: int, n_slots: int, n_leaves: int, dim: int, dtype=None, seed: int = 0):
        import torch
        gen = torch.Generator(device="cpu").manual_seed(seed)
        dev, width = torch.device("cuda", ctx.device), n_features * dim

        def normal(*shape, std):
            return (torch.randn(shape, generator=gen) * std).to(dev)

        params = {"table": normal(n_features * n_slots, dim, std=dim ** -0.5),
                  "weight": torch.ones(width, device=dev), "bias": torch.zeros(width, device=dev),
                  "leaf": normal(n_leaves, width, std=0.1), "gate": torch.ones(n_leaves, 1, device=dev)}
        return cls(ctx, n_features, n_slots, n_leaves, dim, dtype or torch.float32, params)

    def forward(self, tokens, experts):
        """Scores [n] of rows with `tokens` [n, F] and `experts` [n, trees]."""
        import torch
        c, p, n = self.ctx, self.params, tokens.shape[0]
        x = c.embed(p["table"], tokens, scale=self.dim ** 0.5, dtype=self.dtype).view(n, -1)
        y, mean, rstd = c.layer_norm(x, p["weight"], p["bias"])
        route = c.route(experts, self.n_leaves)
        flat = torch.cat([experts.reshape(-1), experts.new_full((1,), -1)])   # order's -1 finds the last: no expert
        place = flat[route.order.long()]
        rows = c.route_gather(y, route)
        scales = c.embed(p["leaf"], place, dtype=self.dtype)
        answers = rows * scales
        share = c.embed(p["gate"], experts).view(experts.shape)
        out = c.route_combine(answers, route, share)
        return out.float().mean(1), Saved(tokens, experts, x, mean, rstd, route, place, rows, scales, answers, share)

    def backward(self, d_score, s: Saved):
        """The parameters' gradients from the scores'."""
        c, p = self.ctx, self.params
        n, width = s.x.shape
        grad = {}
        d_out = (d_score / width).to(self.dtype).unsqueeze(1).expand(n, width).contiguous()
        d_answers, d_share = c.route_combine_backward(d_out, s.answers, s.route, s.share)
        grad["gate"] = c.embed_backward(d_share.unsqueeze(-1), s.experts, self.n_leaves)
        grad["leaf"] = c.embed_backward(d_answers * s.sorted, s.place, self.n_leaves, dtype=p["leaf"].dtype)
        d_y = c.route_gather_backward(d_answers * s.scales, s.route)
        d_x, grad["weight"], grad["bias"] = c.layer_norm_backward(d_y, s.x, s.mean, s.rstd, p["weight"])
        grad["table"] = c.embed_backward(d_x.view(n, self.n_features, self.dim), s.tokens, p["table"].shape[0],
                                         scale=self.dim ** 0.5, dtype=p["table"].dtype)
        return grad

    def step(self, tokens, experts, label, rate: float):
        """One step on the mean squared error, which it returns: each parameter
        goes against its gradient's running mean, over the root of the mean
        square (0.9 and 0.999 kept of each a step)."""
        import torch
        score, saved = self.forward(tokens, experts)
        error = score - label
        grad = self.backward(error * (2.0 / error.shape[0]), saved)
        t = self.state["steps"] = self.state.get("steps", 0) + 1
        for name, g in grad.items():
            if t == 1:
                self.state[name] = torch.zeros_like(g), torch.zeros_like(g)
            mean, square = self.state[name]
            mean.lerp_(g, 0.1)
            square.lerp_(g * g, 0.001)
            self.params[name].addcdiv_(mean, (square / (1 - 0.999 ** t)).sqrt_().add_(1e-8), value=-rate / (1 - 0.9 ** t))
        return (error * error).mean()


def example(n_rows: int = 100_000, n_features: int = 12, n_bins: int = 64, trees: int = 2, depth: int = 5, dim: int = 16,
            steps: int = 60, rate: float = 0.02, seed: int = 0, dtype=None):
    """Grows `trees` trees on residuals, then trains a LeafModel on what they
    leave; returns the losses of its steps."""
    import torch

    from . import synth
    from .tree import grow_tree_device
    w = synth.random_small(seed, n_rows, n_features, n_bins, False, 2)
    dev = torch.device("cuda", 0)
    ctx = Context(0)
    ctx.upload_bins(w.bins, w.n_bins, w.has_missing)
    b = torch.from_numpy(w.bins.astype(np.float32)).to(dev) / n_bins
    label = torch.sin(6 * b[0]) + b[1] * b[2] - (b[3] > 0.5).float() * b[4]
    label = (label - label.mean()) / label.std()
    hess = torch.ones(n_rows, device=dev)
    left, experts, n_leaves = label.clone(), [], 0
    for _ in range(trees):
        levels = grow_tree_device(ctx, -left, hess, depth, w.lam, w.gamma)
        leaf, end = leaves_of(levels, n_rows, dev, n_leaves)
        node = (leaf - n_leaves).long()
        n_leaves = end
        count = torch.zeros(int(node.max()) + 1, device=dev).index_add_(0, node, hess)
        value = torch.zeros_like(count).index_add_(0, node, left) / (count + w.lam)
        left = left - value[node]
        experts.append(leaf)
    experts = torch.stack(experts, 1).contiguous()
    model = LeafModel.make(ctx, n_features, w.n_slots, n_leaves, dim, dtype or torch.bfloat16, seed)
    tokens = tokens_of(w.bins, w.n_slots, dev)
    losses = [float(model.step(tokens, experts, left, rate)) for _ in range(steps)]
    ctx.sync()
    ctx.close()
    return losses


if __name__ == "__main__":
    result = example()
    print(f"mean squared error of what the trees leave: {result[0]:.4f} before the first step, {result[-1]:.4f} after {len(result) - 1}")
