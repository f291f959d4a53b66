"""The vector verbs against plain 64-bit forms: token embedding, layer norm and
rows sorted by expert, with their gradients, at the sizes, types, strides and
masks where they can go wrong.

Tolerances are the operations' rounding bounds: u = 2^-24 for each 32-bit
operation (a sum of k terms, one after the other, is off by at most k u times
the sum of their magnitudes), and half a step of the output's type for its one
rounding (with the smallest subnormal's half where the type underflows)."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def say(*a):
    print("[gpu-vectors]", *a, flush=True)
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


def dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def half_step(torch, dtype):
    """(relative, absolute) error of one rounding to dtype."""
    f = torch.finfo(dtype)
    return f.eps / 2, f.tiny * f.eps / 2


def gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(torch, g, *shape, dtype=None, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype or torch.float32)


def strided(torch, t, extra, shift=0):
    """The same values in rows `extra` values further apart, `shift` values into the buffer."""
    n, d = t.shape
    buf = torch.full((shift + n * (d + extra) + 1,), 7.0, dtype=t.dtype, device=t.device)
    v = buf[shift:shift + n * (d + extra)].view(n, d + extra)[:, :d]
    v.copy_(t)
    return v


def check(torch, got, want, bound, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs() - bound
    assert bool((off <= 0).all()), f"{what}: {float((got - want).abs().max()):.3g} off, {float(off.max()):.3g} over the bound"


# -- embedding -----------------------------------------------------------------

def tokens_of(torch, g, n, vocab, kind):
    if kind == "one":      # a single token, n times
        return torch.full((n,), vocab // 2, dtype=torch.int32, device="cuda")
    if kind == "each":     # every token once, as far as they go
        return (torch.arange(n, device="cuda") * 7919 % vocab).int()
    u = torch.rand(n, generator=g, device="cuda").double()
    return ((torch.exp(u * math.log(vocab + 1.0)) - 1).long().clamp_(max=vocab - 1)).int()   # a few frequent, many rare


EMBED = [
    # n, vocab, dim, kind, table type, vector type, pad, extra stride, shift
    (0, 5, 8, "skewed", "f32", "f32", -1, 0, 0),
    (1, 1, 1, "one", "f32", "f32", -1, 0, 0),
    (1, 9, 64, "one", "bf16", "bf16", -1, 0, 0),
    (63, 100, 7, "skewed", "f16", "f16", 0, 0, 0),
    (65, 3, 129, "skewed", "f32", "bf16", 1, 3, 1),
    (1000, 1000, 64, "each", "f32", "f32", -1, 0, 0),
    (1025, 17, 8, "skewed", "bf16", "bf16", -1, 5, 3),
    (4097, 300, 520, "skewed", "f32", "f16", 0, 0, 0),
    (16384, 70000, 16, "skewed", "bf16", "bf16", -1, 0, 0),
    (16385, 70000, 33, "skewed", "f32", "bf16", 2, 0, 1),
    (40000, 2, 9, "skewed", "f32", "f32", -1, 0, 0),
    (40001, 1 << 20, 4, "skewed", "f32", "f16", -1, 0, 0),
    (50000, 11, 65, "one", "bf16", "bf16", -1, 0, 0),
    (300000, 7196, 64, "skewed", "f32", "bf16", -1, 0, 0),
    (3, 5, 5001, "skewed", "f16", "f16", -1, 1, 0),
]


@pytest.mark.parametrize("n,vocab,dim,kind,tt,vt,pad,extra,shift", EMBED)
def test_embed_and_its_gradient(torch, ctx, n, vocab, dim, kind, tt, vt, pad, extra, shift):
    say("embed", n, vocab, dim, kind, tt, vt)
    g = gen(torch, n + vocab)
    tok = tokens_of(torch, g, n, vocab, kind)
    table = randn(torch, g, vocab, dim, dtype=dt(torch, tt))
    grad = randn(torch, g, n, dim, dtype=dt(torch, vt))
    if extra or shift:
        table, grad = strided(torch, table, extra, shift), strided(torch, grad, extra, shift)
    scale = 1.7
    rel, tiny = half_step(torch, dt(torch, vt))
    out = ctx.embed(table, tok, scale=scale, pad=pad, dtype=dt(torch, vt))
    live = (tok != pad).unsqueeze(-1)
    s32 = float(torch.tensor(scale, dtype=torch.float32))
    want = table.double()[tok.long()] * s32 * live
    check(torch, out, want, want.abs() * (rel + U) * 1.001 + tiny, "embed")
    if out.numel():
        assert bool((out[tok == pad] == 0).all())

    dtable = ctx.embed_backward(grad, tok, vocab, scale=scale, pad=pad, dtype=dt(torch, tt))
    gd = grad.double() * live
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, tok.long(), gd) * s32
    size = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, tok.long(), gd.abs()) * s32
    count = torch.bincount(tok.long(), minlength=vocab).double().unsqueeze(-1)
    rel, tiny = half_step(torch, dt(torch, tt))
    check(torch, dtable, want, size * (count + 2) * U + want.abs() * rel * 1.001 + tiny, "embed_backward")
    absent = torch.bincount(tok[tok != pad].long(), minlength=vocab) == 0
    assert bool((dtable[absent] == 0).all())
    again = ctx.embed_backward(grad, tok, vocab, scale=scale, pad=pad, dtype=dt(torch, tt))
    assert torch.equal(dtable, again), "the same call gives the same bits"
    ctx.sync()


def test_embed_is_linear_and_its_gradient_its_transpose(torch, ctx):
    """<grad, embed(table + d) - embed(table)> = <dtable, d>, in 32 bits."""
    g = gen(torch, 3)
    tok = tokens_of(torch, g, 5000, 333, "skewed")
    table, d, grad = (randn(torch, g, *s) for s in ((333, 40), (333, 40), (5000, 40)))
    dtable = ctx.embed_backward(grad, tok, 333, scale=0.5)
    one, two = ctx.embed(table, tok, scale=0.5), ctx.embed(table + d, tok, scale=0.5)
    left = (grad.double() * (two.double() - one.double())).sum()
    right = (dtable.double() * d.double()).sum()
    # each product's rounding, summed over its values; a token's sum has at most 5000 terms
    bound = U * ((grad.abs() * (two.abs() + one.abs())).double().sum() * 3
                 + 5002 * (ctx.embed_backward(grad.abs(), tok, 333, scale=0.5) * d.abs()).double().sum())
    assert abs(float(left - right)) <= float(bound)


def test_embed_strided_outputs(torch, ctx):
    """Outputs with rows apart: what lies between the rows is left alone."""
    g = gen(torch, 4)
    for n, vocab, dim in ((100, 60, 24), (17000, 300, 9)):
        tok = tokens_of(torch, g, n, vocab, "skewed")
        table, grad = randn(torch, g, vocab, dim), randn(torch, g, n, dim)
        wide = torch.full((n, dim + 5), 3.0, device="cuda")
        ctx.embed(table, tok, out=wide[:, :dim])
        assert torch.equal(wide[:, :dim], ctx.embed(table, tok)) and bool((wide[:, dim:] == 3).all())
        wide = torch.full((vocab, dim + 5), 3.0, device="cuda")
        ctx.embed_backward(grad, tok, vocab, out=wide[:, :dim])
        assert torch.equal(wide[:, :dim], ctx.embed_backward(grad, tok, vocab)) and bool((wide[:, dim:] == 3).all())


@pytest.mark.parametrize("n", [50, 3000, 20000])
def test_embed_tokens_out_of_range_are_padding_and_reported(torch, hgb, n):
    ctx = hgb.Context(0)
    g = gen(torch, n)
    tok = torch.randint(0, 40, (n,), generator=g, device="cuda").int()
    bad = tok.clone()
    bad[n // 2], bad[n - 1], bad[0] = 40, -5, 2 ** 31 - 1
    table, grad = randn(torch, g, 40, 12), randn(torch, g, n, 12)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[n // 2, n - 1, 0]] = False
    for call in (lambda t: ctx.embed(table, t), lambda t: ctx.embed_backward(grad * keep.unsqueeze(-1), t, 40)):
        good = call(tok)
        ctx.sync()
        got = call(bad)
        with pytest.raises(hgb.HGBError, match="token"):
            ctx.sync()
        ctx.sync()   # reported once
        if good.shape[0] == n:
            good = good * keep.unsqueeze(-1)
        # a sum loses terms that are zero: its chunks, and with them its roundings, may differ
        assert bool(((got - good).abs() <= n * U * 8 * n ** 0.5).all())
    ctx.close()


def test_embed_gradient_leaves_out_bad_values_at_padding(torch, ctx):
    """NaN and infinities in padded rows do not reach the table's gradient."""
    g = gen(torch, 8)
    for n in (200, 30000):
        tok = tokens_of(torch, g, n, 50, "skewed")
        tok[::3] = 13
        grad = randn(torch, g, n, 20)
        clean = grad.clone()
        clean[tok == 13] = 0
        grad[tok == 13] = float("nan")
        grad[0] = float("inf")
        got = ctx.embed_backward(grad, tok, 50, pad=13)
        assert torch.equal(got, ctx.embed_backward(clean, tok, 50, pad=13))
        assert bool((got[13] == 0).all())


def test_embed_many_tokens_of_one_value(torch, ctx):
    """Nine million tokens: several tiles a block, and every index in its place."""
    n, vocab = 9_000_001, 5000
    g = gen(torch, 5)
    tok = torch.randint(0, vocab, (n,), generator=g, device="cuda").int()
    grad = torch.randint(-3, 4, (n, 1), generator=g, device="cuda").float()
    want = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_add_(0, tok.long(), grad[:, 0].double())
    got = ctx.embed_backward(grad, tok, vocab)   # whole numbers below 2^24: exact
    assert torch.equal(got[:, 0].double(), want)


def test_embed_rows_past_32_bits(torch, ctx):
    """A table whose element offsets pass 2^32."""
    stride, vocab = 1 << 16, 66000
    try:
        buf = torch.empty(stride * vocab, dtype=torch.bfloat16, device="cuda")
    except RuntimeError:
        pytest.skip("the table does not fit this device's memory")
    table = buf.view(vocab, stride)[:, :24]
    g = gen(torch, 6)
    tok = torch.tensor([0, 65999, 32768, 65537, 65535], dtype=torch.int32, device="cuda")
    rows = randn(torch, g, 5, 24, dtype=torch.bfloat16)
    for i in range(5):
        table[int(tok[i])] = rows[i]
    assert torch.equal(ctx.embed(table, tok), rows)
    ctx.embed_backward(rows, tok, vocab, out=table)
    assert torch.equal(table[tok.long()], rows)
    assert float(table.double().abs().sum()) == float(rows.double().abs().sum())


# -- layer norm ------------------------------------------------------------------

NORM = [
    # rows, dim, type, parameters' type, extra stride, shift
    (0, 8, "f32", "f32", 0, 0),
    (1, 1, "f32", "f32", 0, 0),
    (1, 7, "bf16", "f32", 0, 0),
    (5, 64, "f32", "f32", 0, 0),
    (130, 8, "f16", "f16", 0, 0),
    (257, 129, "bf16", "bf16", 3, 1),
    (33, 333, "f32", "f32", 1, 1),
    (100, 512, "f16", "f32", 0, 0),
    (67, 1000, "bf16", "f32", 0, 0),
    (300, 1792, "bf16", "f32", 0, 0),
    (31, 2049, "f16", "f32", 0, 3),
    (9, 4100, "f32", "f32", 0, 0),
    (12, 8192, "bf16", "bf16", 8, 0),
    (5, 16385, "f32", "f32", 0, 0),
    (3, 40003, "bf16", "f32", 0, 1),
    (5000, 24, "f32", "f32", 0, 0),
]


def norm_case(torch, rows, dim, kind, pk, extra, shift):
    g = gen(torch, rows * 31 + dim)
    x = (randn(torch, g, rows, dim) * (0.5 + torch.rand(rows, 1, generator=g, device="cuda"))
         + 3 * randn(torch, g, rows, 1)).to(dt(torch, kind))
    grad = randn(torch, g, rows, dim, dtype=dt(torch, kind))
    w = (1 + 0.2 * randn(torch, g, dim)).to(dt(torch, pk))
    b = (0.2 * randn(torch, g, dim)).to(dt(torch, pk))
    if extra or shift:
        x, grad = strided(torch, x, extra, shift), strided(torch, grad, extra, shift)
    return x, grad, w, b


def terms(dim):
    """Roundings one after the other in a row's sum: a lane's values (at least 64
    lanes, or 32 values a lane), then a tree."""
    return dim / 64 + 48


# every case with both parameters; some with one or none
NORM_CASES = [(*c, "both") for c in NORM] + [(*c, which) for c in NORM if c[1] in (7, 129, 1792, 40003)
                                             for which in ("none", "weight", "bias")]


@pytest.mark.parametrize("rows,dim,kind,pk,extra,shift,which", NORM_CASES)
def test_layer_norm_and_its_gradient(torch, ctx, rows, dim, kind, pk, extra, shift, which):
    say("norm", rows, dim, kind, pk, which)
    x, grad, w, b = norm_case(torch, rows, dim, kind, pk, extra, shift)
    w = w if which in ("both", "weight") else None
    b = b if which in ("both", "bias") else None
    eps = 1e-5
    rel, tiny = half_step(torch, x.dtype)
    k = terms(dim)
    y, mean, rstd = ctx.layer_norm(x, w, b, eps)
    xd = x.double()
    wd = w.double() if w is not None else torch.ones(dim, dtype=torch.float64, device="cuda")
    bd = b.double() if b is not None else torch.zeros(dim, dtype=torch.float64, device="cuda")
    m = xd.mean(1, keepdim=True)
    var = ((xd - m) ** 2).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + float(torch.tensor(eps)))
    dm = (k + 2) * U * xd.abs().mean(1, keepdim=True)
    # the mean's error adds its square to the variance (the deviations sum to zero), and roundings of the deviations
    dvar = (k + 8) * U * var + dm * dm + 2 * U * dm * torch.sqrt(var)
    dr = r * (0.5 * dvar / (var + eps) * 1.01 + 4 * U)
    if dim > 1:
        check(torch, mean, m[:, 0], dm[:, 0], "mean")
        check(torch, rstd, r[:, 0], dr[:, 0], "rstd")
    want = (xd - m) * r * wd + bd
    h = ((xd - m) * r).abs()
    bound = wd.abs() * (r * dm + (xd - m).abs() * dr + 4 * U * h) + 2 * U * (h * wd.abs() + bd.abs())
    check(torch, y, want, bound * 1.01 + want.abs() * rel * 1.001 + tiny, "y")

    dx, dw, db = ctx.layer_norm_backward(grad, x, mean, rstd, w, bias=which != "weight")
    md, rd, gd = mean.double()[:, None], rstd.double()[:, None], grad.double()
    h = (xd - md) * rd
    a = gd * wd
    ma, mb = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    want = rd * (a - ma - h * mb)
    big_a, big_b = a.abs().mean(1, keepdim=True), (a * h).abs().mean(1, keepdim=True)
    bound = rd * ((k + 4) * U * big_a + h.abs() * (k + 8) * U * big_b + 6 * U * (a.abs() + big_a + h.abs() * big_b))
    check(torch, dx, want, bound + want.abs() * rel * 1.001 + tiny, "dx")
    prel, ptiny = half_step(torch, w.dtype if w is not None else torch.float32)
    for got, term, name in ((dw, gd * h, "dweight"), (db, gd, "dbias")):
        if got is None:
            assert (name == "dweight") == (w is None) or which == "weight"
            continue
        want = term.sum(0)
        check(torch, got, want, (rows + 8) * U * term.abs().sum(0) + want.abs() * prel * 1.001 + ptiny, name)
    again = ctx.layer_norm_backward(grad, x, mean, rstd, w, bias=which != "weight")
    assert all(p is q is None or torch.equal(p, q) for p, q in zip((dx, dw, db), again)), "the same call, the same bits"


# the widths at which the launch changes its shape, and rows enough for several to a wave
NORM_SHAPES = [(40000, 20, "bf16"), (4500, 512, "f16"), (4300, 513, "f32"), (4300, 1024, "bf16"), (4300, 1025, "f16"),
               (2300, 1500, "f32"), (2300, 2048, "bf16"), (1100, 2050, "f16"), (1100, 4096, "f32"), (1100, 4097, "bf16"),
               (1100, 6000, "f32"), (600, 8192, "f16"), (600, 8193, "bf16"), (600, 16384, "f32"), (300, 16385, "bf16")]


@pytest.mark.parametrize("rows,dim,kind", NORM_SHAPES)
def test_layer_norm_over_many_rows(torch, ctx, rows, dim, kind):
    test_layer_norm_and_its_gradient(torch, ctx, rows, dim, kind, "f32", 0, 0, "both")


def test_layer_norm_gradient_against_differences(torch, ctx):
    """<grad, norm(x + t d) - norm(x - t d)> / 2t in 64 bits against <dx, d> and <dweight, e>."""
    g = gen(torch, 12)
    x, grad, d = (randn(torch, g, 40, 200) for _ in range(3))
    w, b, e = 1 + 0.3 * randn(torch, g, 200), randn(torch, g, 200), randn(torch, g, 200)

    def plain(x, w):
        m = x.mean(1, keepdim=True)
        return (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + 1e-5) * w + b.double()

    _, mean, rstd = ctx.layer_norm(x, w, b)
    dx, dw, db = ctx.layer_norm_backward(grad, x, mean, rstd, w)
    t = 1e-4
    diff = (grad.double() * (plain(x.double() + t * d, w.double()) - plain(x.double() - t * d, w.double()))).sum() / (2 * t)
    got = (dx.double() * d.double()).sum()
    size = (dx.abs() * d.abs()).double().sum()
    # 32-bit roundings of each value (at most 300 u of the row's size) and the difference's own t^2 term
    assert abs(float(got - diff)) <= float(size) * (300 * U + 10 * t * t)
    diff = (grad.double() * (plain(x.double(), (w + e).double()) - plain(x.double(), w.double()))).sum()
    assert abs(float((dw.double() * e).sum() - diff)) <= float((grad.abs().sum(0) * 5 * e.abs()).sum()) * 50 * U
    assert abs(float(db.double().sum() - grad.double().sum())) <= float(grad.abs().sum()) * 50 * U


def test_layer_norm_of_hard_rows(torch, ctx):
    """Constant rows, rows far from zero, rows with a NaN or an infinity beside good ones."""
    for dim in (64, 1000, 1792, 20000):
        x = torch.zeros(6, dim, device="cuda")
        x[1] = 5.0
        x[2] = 1e4 + torch.arange(dim, device="cuda") % 2       # 1e4 and 1e4 + 1: variance 1/4
        x[3, 0] = float("nan")
        x[4, dim - 1] = float("inf")
        x[5] = (torch.arange(dim, device="cuda") % 2).float()
        y, mean, rstd = ctx.layer_norm(x)
        assert bool((y[:2] == 0).all())
        assert bool((rstd[:2] == torch.tensor(1 / math.sqrt(1e-5), device="cuda").float()).all()) or \
            bool(((rstd[:2].double() * math.sqrt(1e-5) - 1).abs() <= 8 * U).all())
        # x - mean loses the mean's rounding: half a unit of 1e4 (2^-11), once, beside 1/2
        assert bool(((y[2].abs() - 1).abs() <= 2 * terms(dim) * U * 1e4 + 1e-4).all())
        assert bool(y[3].isnan().all()) and bool(y[4].isnan().any())
        assert bool(torch.isfinite(y[5]).all())
        assert torch.equal(y[5], ctx.layer_norm(x[5:])[0][0]), "a row does not depend on its neighbours"


# -- rows sorted by expert ----------------------------------------------------------

ROUTE = [
    # rows, top, experts, dim, type, share dropped, extra stride
    (0, 2, 4, 8, "f32", 0.0, 0),
    (1, 1, 1, 1, "f32", 0.0, 0),
    (1, 2, 64, 512, "bf16", 0.0, 0),
    (3, 2, 64, 33, "f16", 0.0, 0),
    (64, 1, 7, 129, "f32", 0.3, 3),
    (513, 2, 1023, 16, "bf16", 0.1, 0),
    (700, 3, 5, 1000, "bf16", 1.0, 0),      # every slot dropped
    (2048, 8, 64, 64, "f32", 0.1, 0),
    (2049, 8, 64, 24, "bf16", 0.0, 8),
    (6000, 4, 1023, 40, "f16", 0.5, 0),
    (9000, 2, 2, 2100, "bf16", 0.0, 0),
    (40000, 3, 300, 8, "f32", 0.05, 0),
    (5, 64, 100, 72, "f32", 0.2, 1),
]


@pytest.mark.parametrize("rows,top,experts,dim,kind,drop,extra", ROUTE)
def test_route_and_back(torch, ctx, rows, top, experts, dim, kind, drop, extra):
    say("route", rows, top, experts, dim, kind, drop)
    g = gen(torch, rows + 7 * top + experts)
    e = (torch.rand(rows, top, generator=g, device="cuda") ** 2 * experts).int().clamp_(max=experts - 1)
    e[torch.rand(rows, top, generator=g, device="cuda") < drop] = -1
    w = torch.rand(rows, top, generator=g, device="cuda")
    t = dt(torch, kind)
    x, y, grad, gs = (randn(torch, g, n, dim, dtype=t) for n in (rows, rows * top, rows, rows * top))
    if extra:
        x, y, grad, gs = (strided(torch, v, extra, 1) for v in (x, y, grad, gs))
    r = ctx.route(e, experts)
    flat = e.reshape(-1).long().cpu()
    key = torch.where(flat < 0, torch.tensor(experts), flat)
    order = torch.sort(key, stable=True).indices
    first = torch.searchsorted(key[order].contiguous(), torch.arange(experts + 1))
    used = int(first[-1])
    place = torch.full((rows * top,), -1)
    place[order[:used]] = torch.arange(used)
    order[used:] = -1
    assert torch.equal(r.offsets.cpu().long(), first)
    assert torch.equal(r.order.cpu().long(), order)
    assert torch.equal(r.position.cpu().long(), place.reshape(rows, top))
    pos = place.reshape(rows, top).cuda()
    live = (pos >= 0).unsqueeze(-1)
    rel, tiny = half_step(torch, t)

    xs = ctx.route_gather(x, r)
    want = torch.zeros(rows * top, dim, dtype=t, device="cuda")
    want[:used] = x[(order[:used] // top).cuda()]
    assert torch.equal(xs, want)

    def sums(v, weights):
        rows_ = torch.where(live, v.double()[pos.clamp(min=0)], torch.zeros((), dtype=torch.float64, device="cuda")) \
            if rows else torch.zeros(0, top, dim, dtype=torch.float64, device="cuda")
        rows_ = rows_ * weights.double().unsqueeze(-1)
        return rows_.sum(1), rows_.abs().sum(1)

    for got, v, weights in ((ctx.route_combine(y, r, w), y, w), (ctx.route_combine(y, r), y, torch.ones_like(w)),
                            (ctx.route_gather_backward(gs, r), gs, torch.ones_like(w))):
        want, size = sums(v, weights)
        check(torch, got, want, size * (top + 2) * U + want.abs() * rel * 1.001 + tiny, "combine")

    dy, dw = ctx.route_combine_backward(grad, y, r, w)
    want = torch.zeros(rows * top, dim, dtype=torch.float64, device="cuda")
    slot = order[:used].cuda()
    want[:used] = grad.double()[slot // top] * w.reshape(-1)[slot].double().unsqueeze(-1)
    check(torch, dy, want, want.abs() * (rel + U) * 1.001 + tiny, "dy")
    prod = torch.where(live, y.double()[pos.clamp(min=0)] if rows else want.reshape(0, top, dim),
                       torch.zeros((), dtype=torch.float64, device="cuda")) * grad.double().unsqueeze(1)
    check(torch, dw, prod.sum(-1), prod.abs().sum(-1) * (terms(dim) + 4) * U, "dweights")
    dy1, none = ctx.route_combine_backward(grad, y, r)
    assert none is None and torch.equal(dy1, ctx.route_gather(grad, r))
    ctx.sync()


def test_route_experts_out_of_range_are_dropped_and_reported(torch, hgb):
    ctx = hgb.Context(0)
    for rows in (10, 9000):
        g = gen(torch, rows)
        e = torch.randint(0, 6, (rows, 2), generator=g, device="cuda").int()
        e[3, 1], e[rows - 1, 0] = 6, -7
        good = e.clone()
        good[3, 1] = good[rows - 1, 0] = -1
        a = ctx.route(good, 6)
        ctx.sync()
        b = ctx.route(e, 6)
        with pytest.raises(hgb.HGBError, match="expert"):
            ctx.sync()
        ctx.sync()
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    ctx.close()


def test_route_positions_out_of_range_are_dropped(torch, ctx, hgb):
    """A position that is no place is skipped by every verb that reads it."""
    g = gen(torch, 2)
    x, y = randn(torch, g, 6, 40), randn(torch, g, 12, 40)
    e = torch.arange(12, device="cuda").reshape(6, 2).int() % 4
    r = ctx.route(e, 4)
    bad = r.position.clone()
    bad[2, 1], bad[4, 0] = 12, 2 ** 31 - 1
    keep = torch.ones(6, 2, device="cuda")
    keep[2, 1] = keep[4, 0] = 0
    rb = hgb.Route(r.order, bad, r.offsets)
    assert torch.equal(ctx.route_combine(y, rb), ctx.route_combine(y, r, keep))
    out = torch.zeros(12, 40, device="cuda")
    ctx.route_gather(x, rb, out=out)
    want = ctx.route_gather(x, r)
    want[r.position[2, 1].long()] = 0
    want[r.position[4, 0].long()] = 0
    assert torch.equal(out, want)
    _, dw = ctx.route_combine_backward(x, y, rb, torch.ones(6, 2, device="cuda"))
    assert float(dw[2, 1]) == 0 and float(dw[4, 0]) == 0


def test_route_leaves_out_bad_values_of_dropped_slots(torch, ctx):
    """Places past the last routed slot hold NaN: no sum reads them."""
    g = gen(torch, 9)
    e = torch.randint(0, 4, (50, 3), generator=g, device="cuda").int()
    e[::2, 1] = -1
    e[7] = -1
    r = ctx.route(e, 4)
    used = int(r.offsets[-1])
    y = randn(torch, g, 150, 20)
    y[used:] = float("nan")
    out = ctx.route_combine(y, r, torch.rand(50, 3, generator=g, device="cuda"))
    assert bool(torch.isfinite(out).all()) and bool((out[7] == 0).all())
    dy, dw = ctx.route_combine_backward(randn(torch, g, 50, 20), y, r, torch.rand(50, 3, generator=g, device="cuda"))
    assert bool(torch.isfinite(dy).all()) and bool((dy[used:] == 0).all()) and bool((dw[7] == 0).all())


# -- calls of more bytes than the caches keep, whose outputs are stored past them ---

@pytest.mark.parametrize("n,vocab,dim,tt,vt,extra", [(1700001, 7196, 64, "f32", "bf16", 0), (100, 262144, 512, "bf16", "bf16", 0),
                                                     (700000, 999, 100, "f32", "f32", 4), (150001, 300, 700, "f16", "f16", 1)])
def test_large_embed(torch, ctx, n, vocab, dim, tt, vt, extra):
    test_embed_and_its_gradient(torch, ctx, n, vocab, dim, "skewed", tt, vt, 3, extra, 0)


@pytest.mark.parametrize("rows,dim,kind", [(34001, 1500, "bf16"), (60000, 501, "f32"), (150001, 400, "f16")])
def test_large_layer_norm(torch, ctx, rows, dim, kind):
    test_layer_norm_and_its_gradient(torch, ctx, rows, dim, kind, "f32", 0, 0, "both")


@pytest.mark.parametrize("rows,top,dim,kind", [(20001, 4, 1024, "bf16"), (15000, 5, 603, "f32")])
def test_large_route(torch, ctx, rows, top, dim, kind):
    test_route_and_back(torch, ctx, rows, top, 64, dim, kind, 0.1, 0)


# -- streams, graphs, refusals ------------------------------------------------------

def step(torch, ctx, table, tok, w, b, e, share, n, top):
    """One pass through all the verbs, forward and back."""
    v = ctx.embed(table, tok, scale=2.0)
    x = v.reshape(n, -1)
    y, mean, rstd = ctx.layer_norm(x, w, b)
    r = ctx.route(e, 8)
    xs = ctx.route_gather(y, r)
    out = ctx.route_combine(xs, r, share)
    dys, dshare = ctx.route_combine_backward(out, xs, r, share)
    dy = ctx.route_gather_backward(dys, r)
    dx, dw, db = ctx.layer_norm_backward(dy, x, mean, rstd, w)
    dtable = ctx.embed_backward(dx.reshape(v.shape), tok, table.shape[0], scale=2.0)
    return [v, y, mean, rstd, *r, xs, out, dys, dshare, dy, dx, dw, db, dtable]


def step_inputs(torch, seed, n, top=2):
    g = gen(torch, seed)
    table = randn(torch, g, 200, 16)
    tok = torch.randint(0, 200, (n, 10), generator=g, device="cuda").int()
    w, b = 1 + randn(torch, g, 160) * 0.1, randn(torch, g, 160)
    e = torch.randint(-1, 8, (n, top), generator=g, device="cuda").int()
    share = torch.rand(n, top, generator=g, device="cuda")
    return table, tok, w, b, e, share, n, top


@pytest.mark.parametrize("n", [50, 10000])
def test_on_another_stream(torch, hgb, n):
    """A context on a side stream, its tensors made and read on the current one, without a wait by the caller."""
    ref = hgb.Context(0)
    side = torch.cuda.Stream()
    ctx = hgb.Context(0, stream=side)
    for seed in range(6):
        args = step_inputs(torch, seed, n)
        got = [t.clone() for t in step(torch, ctx, *args)]
        args = None
        want = step(torch, ref, *step_inputs(torch, seed, n))
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    ctx.sync()
    ctx.close()
    ref.close()


@pytest.mark.parametrize("n", [50, 10000])
def test_captured_into_a_graph(torch, hgb, n):
    """Every verb captured; each replay on new inputs against an eager pass, with eager work in between."""
    side = torch.cuda.Stream()
    ctx = hgb.Context(0, stream=side)
    args = step_inputs(torch, 100, n)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(torch, ctx, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step(torch, ctx, *args)
    for seed in range(5):
        fresh = step_inputs(torch, seed, n)
        for dst, src in zip(args[:6], fresh[:6]):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = step(torch, ctx, *fresh)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), seed
    ctx.sync()
    ctx.close()


def test_refusals(torch, ctx, hgb):
    f = lambda *s, dtype=None: torch.zeros(s, dtype=dtype or torch.float32, device="cuda")   # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    r = ctx.route(i(4, 2), 3)
    for call in (
        lambda: ctx.embed(f(4, 8), i(3).long()),
        lambda: ctx.embed(f(4, 8).cpu(), i(3)),
        lambda: ctx.embed(f(4, 8, dtype=torch.float64), i(3)),
        lambda: ctx.embed(f(8), i(3)),
        lambda: ctx.embed(f(4, 8).T, i(3)),
        lambda: ctx.embed(f(4, 8), i(3), out=f(2, 8)),
        lambda: ctx.embed(f(4, 8), i(3), out=f(3, 7)),
        lambda: ctx.embed(f(4, 0), i(3)),
        lambda: ctx.embed_backward(f(3, 8), i(4), 5),
        lambda: ctx.embed_backward(f(1, 8).expand(3, 8), i(3), 5),
        lambda: ctx.layer_norm(f(4, 8), f(7)),
        lambda: ctx.layer_norm(f(4, 8), f(8, dtype=torch.bfloat16)),
        lambda: ctx.layer_norm(f(4, 8, dtype=torch.bfloat16), f(8), f(8, dtype=torch.bfloat16)),
        lambda: ctx.layer_norm_backward(f(4, 8), f(4, 8), f(3), f(4)),
        lambda: ctx.layer_norm_backward(f(4, 8), f(4, 8, dtype=torch.bfloat16), f(4), f(4)),
        lambda: ctx.route(i(4), 3),
        lambda: ctx.route_gather(f(5, 8), r),
        lambda: ctx.route_combine(f(4, 8), r),
        lambda: ctx.route_combine(f(8, 8), r, f(4, 1)),
        lambda: ctx.route_combine(f(8, 8), r, f(4, 2, dtype=torch.bfloat16)),
        lambda: ctx.route_combine_backward(f(4, 8), f(8, 9), r),
    ):
        with pytest.raises(ValueError):
            call()
    table = f(4, 8)
    for call, word in (
        (lambda: ctx.embed(f(4, 8, dtype=torch.bfloat16), i(3), dtype=torch.float32), "type"),
        (lambda: ctx.embed(f(0, 8), i(3)), "vocab"),
        (lambda: ctx.embed(table, i(4), out=table), "overlaps"),
        (lambda: ctx.embed_backward(f(3, 8), i(3), 0), "limits"),
        (lambda: ctx.embed_backward(f(3, 8), i(3), 5, dtype=torch.bfloat16), "out"),
        (lambda: ctx.layer_norm(f(4, 8), eps=-1.0), "eps"),
        (lambda: ctx.layer_norm(f(4, 8), eps=float("nan")), "eps"),
        (lambda: ctx.layer_norm(table, out=table), "overlaps"),
        (lambda: ctx.route(i(4, 2), 0), "limits"),
        (lambda: ctx.route(i(4, 2), 1024), "limits"),
        (lambda: ctx.route(i(4, 65), 10), "limits"),
    ):
        with pytest.raises(hgb.HGBError, match=word):
            call()
    ctx.sync()
