"""The vector verbs on contexts: what a sync reports when several things went
wrong before it, and contexts side by side."""
import sys

import numpy as np
import pytest

from histogram_gradient_boosted_amd import synth

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-vectors-contexts]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch():
    import torch as _torch
    from histogram_gradient_boosted_amd import binding
    if not _torch.cuda.is_available() or not binding.available():
        pytest.skip("no HIP device")
    return _torch


@pytest.fixture(scope="module")
def hgb(torch):
    from histogram_gradient_boosted_amd import binding
    return binding


@pytest.fixture()
def ctx(hgb):
    c = hgb.Context(0)
    yield c
    c.close()


def bad_token(torch, ctx):
    ctx.embed(torch.ones(3, 4, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda"))


def bad_expert(torch, ctx):
    ctx.route(torch.tensor([[0], [3]], dtype=torch.int32, device="cuda"), 3)


def reports(hgb, ctx, *words):
    """The next sync fails with these words in its message."""
    with pytest.raises(hgb.HGBError) as e:
        ctx.sync()
    for w in words:
        assert w in str(e.value), str(e.value)
    return e.value.status


def test_a_sync_reports_tokens_and_experts(torch, hgb, ctx):
    bad_token(torch, ctx)
    bad_expert(torch, ctx)
    assert reports(hgb, ctx, "token", "expert") == hgb.HGB_E_INVALID
    ctx.sync()
    bad_token(torch, ctx)
    assert reports(hgb, ctx, "token") == hgb.HGB_E_INVALID
    bad_expert(torch, ctx)
    assert reports(hgb, ctx, "expert") == hgb.HGB_E_INVALID
    ctx.sync()


@pytest.mark.parametrize("bad", [bad_token, bad_expert])
def test_a_row_index_is_reported_and_then_the_token(torch, hgb, ctx, bad):
    w = synth.random_small(65, 1000, 4, 64, False, 0)
    ctx.upload_bins(w.bins, w.n_bins, w.has_missing)
    ctx.begin_tree(torch.from_numpy(w.grad).cuda(), torch.from_numpy(w.hess).cuda())
    hist = torch.empty((1, 4, 64, 2), dtype=torch.int64, device="cuda")
    rows = torch.tensor([0, 1, 1000, 2], dtype=torch.int32, device="cuda")
    ctx.build_level(hist, rows, np.array([0, 4], np.int32))
    bad(torch, ctx)
    assert reports(hgb, ctx, "row index") == hgb.HGB_E_INVALID
    assert reports(hgb, ctx, bad.__name__[4:]) == hgb.HGB_E_INVALID
    ctx.sync()


@pytest.mark.parametrize("bad", [bad_token, bad_expert])
def test_a_tree_that_is_not_finite_is_reported_and_then_the_token(torch, hgb, ctx, bad):
    w = synth.random_small(66, 1000, 4, 64, False, 0)
    ctx.set_async_begin(True)
    ctx.upload_bins(w.bins, w.n_bins, w.has_missing)
    g = torch.from_numpy(w.grad).cuda()
    g[7] = float("nan")
    ctx.begin_tree(g, torch.from_numpy(w.hess).cuda())
    bad(torch, ctx)
    assert reports(hgb, ctx) == hgb.HGB_E_NONFINITE
    assert reports(hgb, ctx, bad.__name__[4:]) == hgb.HGB_E_INVALID
    ctx.sync()


def test_two_contexts_sort_by_digits_of_different_widths(torch, hgb):
    """Turn by turn, sorts whose kernels take 139 and 83 KB of LDS."""
    a, b = hgb.Context(0), hgb.Context(0)
    n = 1_100_000
    g = torch.Generator(device="cuda").manual_seed(1)
    e = torch.randint(0, 200, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    want = torch.sort(e.view(-1), stable=True).indices.int()
    for c, experts in ((a, 1023), (b, 200), (a, 1023), (b, 1023), (a, 200)):
        say("experts", experts)
        assert torch.equal(c.route(e, experts).order, want)
    a.sync()
    b.sync()
    a.close()
    b.close()


def test_a_closed_context_is_refused_as_a_null_one(torch, hgb):
    ctx = hgb.Context(0)
    x, i = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    r = ctx.route(i, 3)
    y = ctx.route_gather(x, r)
    _, mean, rstd = ctx.layer_norm(x)
    ctx.close()
    for call in (lambda: ctx.embed(x, i), lambda: ctx.embed_backward(x, i[:, 0].contiguous(), 5), lambda: ctx.layer_norm(x),
                 lambda: ctx.layer_norm_backward(x, x, mean, rstd), lambda: ctx.route(i, 3), lambda: ctx.route_gather(x, r),
                 lambda: ctx.route_combine(y, r), lambda: ctx.route_gather_backward(y, r),
                 lambda: ctx.route_combine_backward(x, y, r), ctx.sync):
        with pytest.raises(hgb.HGBError, match="null context"):
            call()
