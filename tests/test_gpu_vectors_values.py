"""The vector verbs on values that must reach nothing, or everything they should:
rows of bad tokens, sorts of millions of slots, NaN and infinities in the layer
norm's gradients.  Plain forms in 64 bits; u = 2^-24 bounds a 32-bit rounding."""
import sys

import pytest
import test_gpu_vectors as base

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def say(*a):
    print("[gpu-vectors-values]", *a, flush=True)
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


@pytest.fixture(scope="module")
def ctx(hgb):
    c = hgb.Context(0)
    yield c
    c.sync()
    c.close()


@pytest.mark.parametrize("n,dim,kind", [(20, 7, "float32"), (50, 12, "float32"), (3000, 12, "bfloat16"), (20000, 33, "float32"),
                                        (300000, 5, "float16"), (1100000, 3, "float32")])
def test_rows_of_tokens_out_of_range_reach_nothing(torch, hgb, n, dim, kind):
    """Their gradients are NaN: one that was added to any token would show."""
    say("bad tokens", n, dim, kind)
    ctx = hgb.Context(0)
    g = torch.Generator(device="cuda").manual_seed(n)
    t, vocab = getattr(torch, kind), 40
    tok = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    bad = torch.rand(n, generator=g, device="cuda") < 0.1
    bad[[0, n // 2, n - 1]] = True
    values = torch.tensor([vocab, -5, 2 ** 31 - 1, -2 ** 31, vocab + 24, 1 << 16, 63, -2], dtype=torch.int32, device="cuda")
    tok = torch.where(bad, values[torch.arange(n, device="cuda") % 8], tok)
    table = torch.randn(vocab, dim, generator=g, device="cuda").to(t)
    out = ctx.embed(table, tok)
    with pytest.raises(hgb.HGBError, match="token"):
        ctx.sync()
    want = table[tok.long().clamp(0, vocab - 1)]
    want[bad] = 0
    assert torch.equal(out, want)

    grad = torch.randn(n, dim, generator=g, device="cuda").to(t)
    grad[bad] = float("nan")
    got = ctx.embed_backward(grad, tok, vocab, dtype=torch.float32)
    with pytest.raises(hgb.HGBError, match="token"):
        ctx.sync()
    ctx.sync()
    at, rows = tok[~bad].long(), grad[~bad].double()
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, at, rows)
    size = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, at, rows.abs())
    count = torch.bincount(at, minlength=vocab).double().unsqueeze(-1)
    base.check(torch, got, want, size * (count + 2) * U, "embed_backward")
    ctx.close()


# slots past 2^18 (four keys a thread), 2^20 (eight) and 2^22 (several tiles a block)
@pytest.mark.parametrize("rows,top,experts,dim,kind,drop", [(131201, 2, 1023, 2, "f32", 0.1), (300007, 4, 64, 3, "bf16", 0.0),
                                                            (262144, 5, 1023, 1, "f16", 0.3), (70001, 64, 1023, 1, "f32", 0.1),
                                                            (4200001, 1, 3, 2, "bf16", 0.2), (150000, 8, 1, 1, "f32", 1.0)])
def test_route_of_many_slots(torch, ctx, rows, top, experts, dim, kind, drop):
    base.test_route_and_back(torch, ctx, rows, top, experts, dim, kind, drop, 0)


@pytest.mark.parametrize("rows,dim,kind", [(40, 3, "float32"), (40, 20, "bfloat16"), (40, 333, "float32"), (20, 1792, "bfloat16"),
                                           (20, 2051, "float16"), (12, 9001, "float32"), (12, 20001, "bfloat16")])
def test_layer_norm_gradients_of_bad_values(torch, ctx, rows, dim, kind):
    """A NaN or an infinity spoils its own row's gradient, and what its values are summed into, and nothing else."""
    say("norm gradients of bad values", rows, dim, kind)
    t = getattr(torch, kind)
    g = torch.Generator(device="cuda").manual_seed(dim)
    x, grad = (torch.randn(rows, dim, generator=g, device="cuda").to(t) for _ in range(2))
    w = torch.rand(dim, generator=g, device="cuda") + 0.5
    good = x.clone()
    _, mean, rstd = ctx.layer_norm(good, w)
    clean = ctx.layer_norm_backward(grad, good, mean, rstd, w)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[[1, 4, rows - 1]] = False

    # in the gradient: dx of its rows; dweight and dbias of its columns
    for value in (float("nan"), float("inf")):
        spoilt = grad.clone()
        spoilt[1, 0] = spoilt[4, dim - 1] = spoilt[rows - 1, dim // 2] = value
        dx, dw, db = ctx.layer_norm_backward(spoilt, x, mean, rstd, w)
        assert torch.equal(dx[rest], clean[0][rest])
        assert bool(dx[~rest].isnan().any(1).all())
        column = torch.ones(dim, dtype=torch.bool, device="cuda")
        column[[0, dim - 1, dim // 2]] = False
        for got, want in ((dw, clean[1]), (db, clean[2])):
            assert torch.equal(got[column], want[column]) and not bool(torch.isfinite(got[~column]).any())

    # in x, with the statistics that the forward pass gives such rows: no value of h there is a number
    for value in (float("nan"), float("inf")):
        x = good.clone()
        x[1, 0] = x[4, dim - 1] = x[rows - 1, dim // 2] = value
        _, m, r = ctx.layer_norm(x, w)
        dx, dw, db = ctx.layer_norm_backward(grad, x, m, r, w)
        assert torch.equal(dx[rest], clean[0][rest])
        assert bool(dx[~rest].isnan().all()) and bool(dw.isnan().all())
        assert torch.equal(db, clean[2])

    # infinite statistics of a row of gradients that are zero: 0 * inf, in its row and dweight, not in dbias
    x, spoilt, r = good, grad.clone(), rstd.clone()
    spoilt[4], r[4] = 0, float("inf")
    dx, dw, db = ctx.layer_norm_backward(spoilt, x, mean, r, w)
    rest[:] = True
    rest[4] = False
    assert torch.equal(dx[rest], clean[0][rest]) and bool(dx[4].isnan().all())
    assert bool(dw.isnan().all()) and bool(torch.isfinite(db).all())
    ctx.sync()
