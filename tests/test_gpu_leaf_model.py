"""The example model: its gradients against torch's autograd of the same
formulas in 64 bits, and a training run on grown trees."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch as _torch
    from histogram_gradient_boosted_amd import binding
    if not _torch.cuda.is_available() or not binding.available():
        pytest.skip("no HIP device")
    return _torch


def plain(torch, p, tokens, experts, dim):
    """The model's formulas, elementwise, differentiable."""
    n = tokens.shape[0]
    x = (p["table"][tokens.long()] * dim ** 0.5).reshape(n, -1)
    m = x.mean(1, keepdim=True)
    y = (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + 1e-5) * p["weight"] + p["bias"]
    e = experts.long().clamp(min=0)
    live = (experts >= 0).unsqueeze(-1)
    return (y.unsqueeze(1) * p["leaf"][e] * p["gate"][e] * live).sum(1).mean(1)


@pytest.mark.parametrize("n,features,slots,leaves,trees,dim", [(1, 1, 3, 1, 1, 4), (50, 3, 7, 9, 2, 5), (3000, 6, 33, 62, 3, 8)])
def test_gradients_are_those_of_the_formulas(torch, n, features, slots, leaves, trees, dim):
    from histogram_gradient_boosted_amd.binding import Context
    from histogram_gradient_boosted_amd.leaf_model import LeafModel
    g = torch.Generator(device="cuda").manual_seed(n)
    ctx = Context(0)
    model = LeafModel.make(ctx, features, slots, leaves, dim, torch.float32, seed=1)
    tokens = (torch.randint(0, slots, (n, features), generator=g, device="cuda")
              + torch.arange(features, device="cuda") * slots).int()
    experts = torch.randint(-1 if n > 1 else 0, leaves, (n, trees), generator=g, device="cuda").int()
    d_score = torch.randn(n, generator=g, device="cuda")
    score, saved = model.forward(tokens, experts)
    grad = model.backward(d_score, saved)
    ctx.sync()
    p = {k: v.double().requires_grad_() for k, v in model.params.items()}
    want = plain(torch, p, tokens, experts, dim)
    want.backward(d_score.double())
    # 32-bit roundings along the way, each relative to sums of magnitudes that exceed a
    # result by up to the terms that cancel in it: bounded by the largest gradient of the kind
    def near(got, ref, what):
        off, size = (got.double() - ref).abs().max(), ref.abs().max() + ref.abs().mean() + 1e-6
        assert float(off) <= float(size) * 64 * (n * trees) ** 0.5 * U + 1e-9, (what, float(off), float(size))
    near(score, want.detach(), "score")
    for k in p:
        near(grad[k], p[k].grad, k)
    ctx.close()


def test_example_learns_what_the_trees_leave(torch):
    from histogram_gradient_boosted_amd import leaf_model
    losses = leaf_model.example(n_rows=20_000, steps=40)
    assert np.isfinite(losses).all() and losses[-1] < 0.9 * losses[0]


def test_leaves_of_a_grown_tree(torch):
    """Every row's node is the deepest that holds it."""
    from histogram_gradient_boosted_amd import synth
    from histogram_gradient_boosted_amd.binding import Context
    from histogram_gradient_boosted_amd.leaf_model import leaves_of
    from histogram_gradient_boosted_amd.tree import grow_tree_device
    w = synth.random_small(3, 5000, 4, 32, True, 2)
    ctx = Context(0)
    ctx.upload_bins(w.bins, w.n_bins, w.has_missing)
    levels = grow_tree_device(ctx, torch.from_numpy(w.grad).cuda(), torch.from_numpy(w.hess).cuda(), 4, w.lam, w.gamma)
    leaf, end = leaves_of(levels, 5000, "cuda", 10)
    want, first = np.full(5000, 10), 11
    for level in levels[1:]:
        rows = level.rows.cpu().numpy()
        for k in range(level.n_nodes):
            want[rows[level.offsets[k]:level.offsets[k + 1]]] = first + k
        first += level.n_nodes
    assert end == first and np.array_equal(leaf.cpu().numpy(), want)
    ctx.close()
