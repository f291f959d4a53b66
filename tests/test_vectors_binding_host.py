"""What the binding of the vector verbs refuses before any device call, on host
tensors: these checks come before the one for the device."""
import pytest
import torch

from histogram_gradient_boosted_amd import binding


@pytest.fixture()
def ctx():
    c = binding.Context.__new__(binding.Context)   # no device: only the checks run
    c._torch, c._lib, c.device = torch, binding.load(), 0
    return c


def calls(ctx, x):
    """Every verb, given x ([4, 8]) as its vectors."""
    i = torch.zeros(4, 2, dtype=torch.int32)
    r = binding.Route(i.reshape(-1), i, torch.zeros(4, dtype=torch.int32))
    return (lambda: ctx.embed(x, i), lambda: ctx.embed_backward(x, i[:, 0], 5), lambda: ctx.layer_norm(x),
            lambda: ctx.layer_norm_backward(x, x, x[:, 0], x[:, 0]), lambda: ctx.route_gather(x, r),
            lambda: ctx.route_combine(x, r), lambda: ctx.route_gather_backward(x, r),
            lambda: ctx.route_combine_backward(x, x, r))


def test_views_that_torch_would_negate_are_refused(ctx):
    """conj().imag is a view whose values are those in memory with the other sign."""
    z = torch.ones(4, 1, dtype=torch.complex64)
    x = z.conj().imag
    assert x.is_neg() and float(x[0, 0]) == 0
    for call in calls(ctx, x):
        with pytest.raises(ValueError, match="resolve_neg"):
            call()
    for call in calls(ctx, x.resolve_neg()):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_layer_norm_backward_takes_a_truth_value_for_bias(ctx):
    """layer_norm has the bias itself at that name; here a tensor, or what has no truth value, is refused first."""
    import numpy as np
    x = torch.zeros(4, 8)
    for bias in (torch.ones(8), torch.zeros(1), torch.ones(1)):
        with pytest.raises(ValueError, match="bias"):
            ctx.layer_norm_backward(x, x, x[:, 0], x[:, 0], None, bias)
    with pytest.raises(ValueError, match="bias"):
        ctx.layer_norm_backward(x, x, x[:, 0], x[:, 0], None, np.ones(8))
    for bias in (True, False, 1, None):
        with pytest.raises(ValueError, match="CUDA tensor"):
            ctx.layer_norm_backward(x, x, x[:, 0], x[:, 0], None, bias)


def test_tensors_whose_gradient_would_be_lost_are_refused(ctx):
    """The verbs record nothing for autograd, so a result would have no gradient and not say so."""
    x = torch.zeros(4, 8, requires_grad=True)
    for call in calls(ctx, x):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    with torch.no_grad():
        for call in calls(ctx, x):
            with pytest.raises(ValueError, match="CUDA tensor"):
                call()
    for call in calls(ctx, x.detach()):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
