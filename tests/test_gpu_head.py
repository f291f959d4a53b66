"""Cross entropy and distillation over a vocabulary, with their gradients,
against plain 64-bit forms, at the sizes, types, strides and masks where they
can go wrong.

Tolerances: u = 2^-24 for each 32-bit operation.  A logit is a sum of dim
products, off by (dim + 2) u times the sum of their magnitudes.  exp2 and log2
are taken of such logits (in units of log2: two more roundings of the value),
and sums of exponentials of up to 128 terms a part and of the parts; so lse is
off by the largest logit's error and u times a count of those roundings.  The
logits' gradient is rounded once more, to half a step of the inputs' type
(beside a 32-bit table gradient: half a step squared), and a product of it is
off by its length in u."""
import pytest

from test_gpu_vectors import U, check, ctx, dt, gen, half_step, hgb, randn, strided, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-head]", *a, flush=True)


HEADS = [
    # n, vocab, dim, type, dtable's type, scale, pads, extra stride, shift
    (1, 1, 1, "f32", "f32", 1.0, 0.0, 0, 0),
    (1, 7, 3, "bf16", "bf16", 1.0, 0.0, 0, 0),
    (2, 2, 8, "f16", "f32", 0.5, 0.0, 0, 0),
    (3, 300, 64, "bf16", "f32", 1.0, 0.3, 0, 0),
    (31, 1000, 40, "f32", "f32", 1.3, 0.3, 0, 0),
    (32, 256, 64, "f16", "f16", 1.0, 0.0, 0, 0),
    (33, 257, 65, "bf16", "bf16", 1.0, 0.2, 0, 0),
    (8, 7196, 64, "f32", "f32", 1.0, 0.0, 0, 0),
    (64, 5000, 16, "bf16", "bf16", 2.0, 0.0, 8, 0),
    (255, 513, 72, "f16", "f16", 1.0, 0.9, 3, 1),
    (256, 256, 128, "bf16", "f32", 1.0, 0.0, 0, 0),
    (257, 511, 129, "f32", "f32", -0.7, 0.1, 2, 3),
    (300, 4000, 200, "bf16", "bf16", 1.0, 0.1, 0, 0),
    (1000, 1023, 129, "f16", "f16", 1.0, 0.1, 0, 0),
    (520, 2500, 520, "f32", "f32", 1.0, 0.0, 0, 0),
    (700, 1300, 333, "bf16", "f32", 1.0, 0.2, 0, 1),
    (4099, 40, 24, "bf16", "bf16", 1.0, 0.1, 0, 0),
    (5000, 2, 257, "f16", "f32", 1.0, 0.1, 0, 0),
    (40, 20000, 1030, "bf16", "bf16", 1.0, 0.0, 0, 0),
]


def problem(torch, n, vocab, dim, kind, extra, shift, seed):
    g = gen(torch, seed)
    x = randn(torch, g, n, dim, dtype=dt(torch, kind))
    table = randn(torch, g, vocab, dim, dtype=dt(torch, kind), scale=2.0 / dim ** 0.5)
    token = (torch.rand(n, generator=g, device="cuda") ** 2 * vocab).int().clamp_(max=vocab - 1)
    x = (x.float() + table[token.long()].float() * 2).to(x.dtype)
    if extra or shift:
        x, table = strided(torch, x, extra, shift), strided(torch, table, extra, shift)
    return g, x, table, token


class Plain:
    """The logits in 64 bits, and how far 32-bit ones may be off them."""

    def __init__(self, torch, x, table, scale):
        xd, wd = x.double(), table.double()
        self.z = xd @ wd.T * scale
        n, vocab = self.z.shape
        dim = x.shape[1]
        self.lse = torch.logsumexp(self.z, 1)
        self.z_off = ((dim + 2) * U * abs(scale) * (xd.abs() @ wd.abs().T)).amax(1)
        top = self.z.abs().amax(1)
        parts = 4 * ((vocab + 255) // 256)
        self.lse_off = self.z_off + U * (128 + parts + 8 * top + 4 * self.lse.abs() + 8)
        self.q_off = self.z_off + U * (8 * top + 8 * self.lse.abs() + 8)   # of exp(z - lse), relative


def check_grads(torch, got, x, table, dz, off, kind, out_kind, top_rate, what):
    """dx and dtable of the logits' gradient dz, whose values are off by `off` before they are rounded."""
    xd, wd = x.double(), table.double()
    n, vocab = dz.shape
    live = (dz != 0).any(1, keepdim=True)
    step = half_step(torch, dt(torch, kind))[0] if kind != "f32" else 0.0
    floor = float(top_rate) * 2.0 ** -39 if kind == "f16" else 0.0   # half of fp16's smallest, over the factor that dz is held with
    rel, tiny = half_step(torch, dt(torch, kind))
    size = dz.abs()
    err = off + size * step * 1.001 + floor * live
    want = dz @ wd
    bound = err @ wd.abs() + (vocab + 300) * U * (size @ wd.abs())
    check(torch, got[0], want, bound * (1 + rel) + want.abs() * rel * 1.001 + tiny, what + " dx")
    step2 = step if out_kind == kind else step * step
    err = off + size * step2 * 1.001 + floor * live
    want = dz.T @ xd
    bound = err.T @ xd.abs() + (2 * n + 300) * U * (size.T @ xd.abs())
    rel, tiny = half_step(torch, dt(torch, out_kind))
    check(torch, got[1], want, bound * (1 + rel) + want.abs() * rel * 1.001 + tiny, what + " dtable")


@pytest.mark.parametrize("n,vocab,dim,kind,out_kind,scale,pads,extra,shift", HEADS)
def test_cross_entropy_and_its_gradients(torch, ctx, n, vocab, dim, kind, out_kind, scale, pads, extra, shift):
    say("cross_entropy", n, vocab, dim, kind, out_kind)
    g, x, table, target = problem(torch, n, vocab, dim, kind, extra, shift, n + vocab + dim)
    target[torch.rand(n, generator=g, device="cuda") < pads] = -1
    scale = float(torch.tensor(scale))
    p = Plain(torch, x, table, scale)
    loss, lse = ctx.cross_entropy(x, table, target, scale)
    live, at = target >= 0, target.clamp(min=0).long()
    check(torch, lse, p.lse, p.lse_off, "lse")
    want = torch.where(live, p.lse - p.z.gather(1, at[:, None])[:, 0], 0.0)
    check(torch, loss, want, p.lse_off + p.z_off + 4 * U * p.z.abs().amax(1), "loss")
    assert bool((loss[~live] == 0).all())

    say("  gradients")
    grad = randn(torch, g, n) * (64.0 if kind == "f16" else 1.0)
    out = None
    if extra:
        out = torch.full((n, dim + extra), 9.0, dtype=x.dtype, device="cuda")[:, :dim]
    got = ctx.cross_entropy_backward(grad, x, table, target, lse, scale, dtype=dt(torch, out_kind), out=out)
    q = torch.exp(p.z - lse.double()[:, None])
    dz = q.clone()
    dz[torch.arange(n, device="cuda"), at] -= 1
    rate = (torch.where(live, grad.double(), 0.0) * scale)[:, None]
    check_grads(torch, got, x, table, dz * rate, q * p.q_off[:, None] * rate.abs() + 2 * U * dz.abs() * rate.abs(), kind, out_kind,
                rate.abs().max(), "cross_entropy_backward")
    assert bool((got[0][~live] == 0).all())
    if extra:
        assert bool((out.as_strided((n, extra), (dim + extra, 1), out.storage_offset() + dim) == 9.0).all())
    again = ctx.cross_entropy_backward(grad, x, table, target, lse, scale, dtype=dt(torch, out_kind))
    assert torch.equal(again[0], got[0].contiguous()) and torch.equal(again[1], got[1])
    ctx.sync()


@pytest.mark.parametrize("top,heat", [(1, 1.0), (7, 2.0), (64, 0.5), (65, 3.0), (256, 1.0)])
@pytest.mark.parametrize("n,vocab,dim,kind,out_kind,scale,pads,extra,shift", HEADS[::2])
def test_distill_and_its_gradients(torch, ctx, n, vocab, dim, kind, out_kind, scale, pads, extra, shift, top, heat):
    say("distill", n, vocab, dim, kind, out_kind, top, heat)
    g, x, table, token = problem(torch, n, vocab, dim, kind, extra, shift, n + vocab + dim + top)
    # tokens at random, so that a row has some twice where the vocabulary is small
    tokens = (torch.rand(n, top, generator=g, device="cuda") * vocab).int().clamp_(max=vocab - 1)
    tokens[:, 0] = token
    tokens[torch.rand(n, top, generator=g, device="cuda") < 0.1] = -1
    tokens[torch.rand(n, generator=g, device="cuda") < pads] = -1
    teacher = randn(torch, g, n, top, dtype=dt(torch, "f32" if top % 2 else kind), scale=2.0)
    teacher[torch.rand(n, top, generator=g, device="cuda") < 0.1] = float("-inf")
    p = Plain(torch, x, table, 1.0 / heat)
    loss, lse, picked = ctx.distill(x, table, tokens, teacher, heat)
    check(torch, lse, p.lse, p.lse_off, "lse")
    at = tokens.clamp(min=0).long()
    z = p.z.gather(1, at)
    check(torch, picked, torch.where(tokens >= 0, z, 0.0), (p.z_off + 4 * U * p.z.abs().amax(1))[:, None].expand(n, top), "picked")
    live = (tokens >= 0) & (teacher > float("-inf"))
    some = live.any(1)
    t = torch.where(live, teacher.double() / heat, float("-inf"))
    logp = torch.where(live, torch.log_softmax(t, 1), 0.0)
    prob = torch.where(live, torch.nan_to_num(torch.softmax(t, 1), nan=0.0), 0.0)
    want = heat * heat * (prob * (logp - z + p.lse[:, None])).sum(1) * some
    size = (prob * (logp.abs() + z.abs() + p.lse.abs()[:, None])).sum(1)
    teacher_off = U * (16 + 4 * torch.where(live, t, 0.0).abs().amax(1) + top)   # of p, relative, and of log p
    off = heat * heat * (p.lse_off + p.z_off + 4 * U * p.z.abs().amax(1) + teacher_off * (1 + size) + (top + 8) * U * size)
    check(torch, loss, want, off, "loss")
    assert bool((loss[~some] == 0).all())

    say("  gradients")
    grad = randn(torch, g, n) * (64.0 if kind == "f16" else 1.0)
    got = ctx.distill_backward(grad, x, table, tokens, teacher, lse, picked, heat, dtype=dt(torch, out_kind))
    q = torch.exp(p.z - lse.double()[:, None])
    big = torch.zeros_like(q).scatter_add_(1, at, prob)
    rate = (torch.where(some, grad.double(), 0.0) * heat)[:, None]
    off = (q * p.q_off[:, None] + big * teacher_off[:, None] + 4 * U * (q + big)) * rate.abs()
    check_grads(torch, got, x, table, (q - big) * rate, off, kind, out_kind, rate.abs().max(), "distill_backward")
    again = ctx.distill_backward(grad, x, table, tokens, teacher, lse, picked, heat, dtype=dt(torch, out_kind))
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    ctx.sync()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("heat", [0.5, 1.0, 4.0])
def test_teachers_of_the_types_lowest_and_largest_values(torch, ctx, kind, heat):
    """A teacher masked with its type's lowest value, whole rows too: over the temperature that is no longer finite."""
    g, x, table, _ = problem(torch, 5, 300, 16, kind, 0, 0, 3)
    low, inf = torch.finfo(dt(torch, kind)).min, float("inf")
    teacher = torch.full((5, 6), low, device="cuda")
    teacher[1, 2] = 1.0
    teacher[2, :3] = -inf
    teacher[3, :2] = torch.tensor([1.0, 2.0], device="cuda")
    teacher[4] = -low
    tokens = torch.randperm(300, generator=g, device="cuda")[:30].view(5, 6).int()
    p = Plain(torch, x, table, 1.0 / heat)
    loss, lse, picked = ctx.distill(x, table, tokens, teacher.to(dt(torch, kind)), heat)
    prob = torch.softmax((teacher.double() - teacher.double().amax(1, keepdim=True)) / heat, 1)
    logp = torch.where(prob > 0, prob.log(), 0.0)
    z = p.z.gather(1, tokens.long())
    size = (prob * (logp.abs() + z.abs() + p.lse.abs()[:, None])).sum(1)
    teacher_off = 24 * U
    off = heat * heat * (p.lse_off + p.z_off + 4 * U * p.z.abs().amax(1) + (teacher_off + 14 * U) * (1 + size))
    check(torch, loss, heat * heat * (prob * (logp - z + p.lse[:, None])).sum(1), off, "loss")
    got = ctx.distill_backward(torch.ones(5, device="cuda"), x, table, tokens, teacher.to(dt(torch, kind)), lse, picked, heat)
    q = torch.exp(p.z - lse.double()[:, None])
    big = torch.zeros_like(q).scatter_add_(1, tokens.long(), prob)
    off = (q * p.q_off[:, None] + big * teacher_off + 4 * U * (q + big)) * heat
    check_grads(torch, got, x, table, (q - big) * heat, off, kind, kind, heat, "distill_backward")
    ctx.sync()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_rows_without_a_target_reach_nothing(torch, ctx, kind):
    """NaN and infinities in padded rows, and beside what is read."""
    n, vocab, dim = 300, 700, 40
    g, x, table, target = problem(torch, n, vocab, dim, kind, 0, 0, 4)
    dead = torch.rand(n, generator=g, device="cuda") < 0.4
    target[dead] = -1
    grad = randn(torch, g, n)
    tokens = target[:, None].repeat(1, 3).contiguous()
    teacher = randn(torch, g, n, 3)
    results = []
    for fill in (0.0, float("nan"), float("inf")):
        xs = strided(torch, x, 5, 3)
        xs.as_strided((n, 5), (dim + 5, 1), xs.storage_offset() + dim).fill_(fill)
        xs[dead] = fill
        loss, lse = ctx.cross_entropy(xs, table, target)
        dx, dw = ctx.cross_entropy_backward(grad, xs, table, target, lse)
        l2, lse2, picked = ctx.distill(xs, table, tokens, teacher)
        dx2, dw2 = ctx.distill_backward(grad, xs, table, tokens, teacher, lse2, picked)
        results.append((loss, lse[~dead], dx, dw, l2, lse2[~dead], dx2, dw2))
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
    assert bool((results[0][2][dead] == 0).all()) and bool(results[0][3].isfinite().all())


def test_all_rows_padded_and_no_rows(torch, ctx):
    table = torch.randn(50, 24, device="cuda")
    for n in (0, 1, 40):
        x = torch.randn(n, 24, device="cuda")
        target = torch.full((n,), 7, dtype=torch.int32, device="cuda")
        loss, lse = ctx.cross_entropy(x, table, target, pad=7)
        assert loss.shape == lse.shape == (n,) and bool((loss == 0).all()) and bool(lse.isfinite().all())
        dx, dw = ctx.cross_entropy_backward(torch.ones(n, device="cuda"), x, table, target, lse, pad=7)
        assert dx.shape == (n, 24) and bool((dx == 0).all()) and dw.shape == (50, 24) and bool((dw == 0).all())
        tokens = torch.full((n, 5), -1, dtype=torch.int32, device="cuda")
        loss, lse, picked = ctx.distill(x, table, tokens, torch.zeros(n, 5, device="cuda"))
        assert bool((loss == 0).all()) and bool((picked == 0).all())
        dx, dw = ctx.distill_backward(torch.ones(n, device="cuda"), x, table, tokens, torch.zeros(n, 5, device="cuda"), lse, picked)
        assert bool((dx == 0).all()) and bool((dw == 0).all())
    ctx.sync()


def test_tokens_out_of_range_count_as_padding_and_are_reported(torch, hgb, ctx):
    g, x, table, target = problem(torch, 60, 90, 16, "f32", 0, 0, 8)
    want, lse = ctx.cross_entropy(x, table, target)
    grad = torch.ones(60, device="cuda")
    clean = ctx.cross_entropy_backward(grad, x, table, target, lse)
    ctx.sync()
    bad = target.clone()
    bad[5], bad[6] = 90, -2
    pads = target.clone()
    pads[5] = pads[6] = -1
    loss, _ = ctx.cross_entropy(x, table, bad)
    assert float(loss[5]) == 0 and float(loss[6]) == 0 and torch.equal(loss[7:], want[7:])
    with pytest.raises(hgb.HGBError, match="token"):
        ctx.sync()
    a, b = ctx.cross_entropy_backward(grad, x, table, bad, lse), ctx.cross_entropy_backward(grad, x, table, pads, lse)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[0][7:], clean[0][7:])
    with pytest.raises(hgb.HGBError, match="token"):
        ctx.sync()
    tokens = bad[:, None].repeat(1, 2).contiguous()
    tokens[:, 1] = 3
    teacher = torch.zeros(60, 2, device="cuda")
    loss, lse, picked = ctx.distill(x, table, tokens, teacher)
    assert float(picked[5, 0]) == 0 and float(loss[5]) > 0
    with pytest.raises(hgb.HGBError, match="token"):
        ctx.sync()
    ctx.distill_backward(grad, x, table, tokens, teacher, lse, picked)
    with pytest.raises(hgb.HGBError, match="token"):
        ctx.sync()
    ctx.sync()


def test_extreme_logits(torch, ctx):
    """One token far above all others, and rows of equal ones: no overflow, and gradients that vanish or are even."""
    x = torch.tensor([[300.0, 0.0], [0.0, 0.0], [-300.0, 1.0]], device="cuda")
    table = torch.zeros(1000, 2, device="cuda")
    table[17, 0] = 300.0
    target = torch.tensor([17, 5, 17], dtype=torch.int32, device="cuda")
    loss, lse = ctx.cross_entropy(x, table, target)
    want = torch.logsumexp(x.double() @ table.double().T, 1) - (x.double() @ table.double().T).gather(1, target[:, None].long())[:, 0]
    check(torch, loss, want, 90000.0 * 16 * U + 1e-5, "loss")
    dx, dw = ctx.cross_entropy_backward(torch.ones(3, device="cuda"), x, table, target, lse)
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all()) and float(dx[0].abs().max()) < 2
    assert float(loss[0]) >= 0 and float(loss[0]) < 0.02


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_gradients_against_differences(torch, ctx, kind):
    """The losses' change along a direction of x, from the forward verbs."""
    g, x, table, target = problem(torch, 70, 500, 48, "bf16", 0, 0, 21)
    x, table = x.float(), table.float()
    way = randn(torch, g, 70, 48)
    tokens = torch.stack([target, (target + 3) % 500, (target + 50) % 500], 1).contiguous()
    teacher = randn(torch, g, 70, 3)
    h = 2.0 ** -6
    one = torch.ones(70, device="cuda")
    for heat in (None, 2.0):
        def at(step):
            if heat is None:
                return ctx.cross_entropy(x + step * way, table, target)[0].double()
            return ctx.distill(x + step * way, table, tokens, teacher, heat)[0].double()

        xs, ws = x.to(dt(torch, kind)), table.to(dt(torch, kind))
        if heat is None:
            dx, _ = ctx.cross_entropy_backward(one, xs, ws, target, ctx.cross_entropy(xs, ws, target)[1])
        else:
            _, lse, picked = ctx.distill(xs, ws, tokens, teacher, heat)
            dx, _ = ctx.distill_backward(one, xs, ws, tokens, teacher, lse, picked, heat)
        rate = (at(h) - at(-h)) / (2 * h)
        y = (way.double() @ table.double().T).abs().amax(1)   # of the logits' change
        rel = half_step(torch, dt(torch, kind))[0]
        # the third derivative of log sum exp is below 8 y^3; the losses' roundings over the step; inputs, dz and dx of fewer bits
        wide = (way.double().abs() * (table.double().abs().amax(0))).sum(1)
        bound = h * h / 6 * 8 * y ** 3 + 2000 * U * 40 / h + 8 * rel * wide * (0 if kind == "f32" else 1) + 1e-3
        assert bool(((dx.double() * way).sum(1) - rate).abs().le(bound).all()), (kind, heat)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab", [(1, 1), (3, 65), (40, 200), (70, 129), (300, 257), (300, 1600)])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_logits_all_far_from_zero(torch, ctx, kind, n, vocab, scale):
    """Every logit near -600 or 600: places behind the vocabulary must not count as logits of zero."""
    g = gen(torch, 71)
    for side in (-1.0, 1.0):
        x = torch.ones(n, 8, dtype=dt(torch, kind), device="cuda") + randn(torch, g, n, 8, dtype=dt(torch, kind), scale=0.05)
        table = (75.0 * side * torch.ones(vocab, 8, device="cuda") + randn(torch, g, vocab, 8)).to(dt(torch, kind))
        target = (torch.rand(n, generator=g, device="cuda") * vocab).int().clamp_(max=vocab - 1)
        p = Plain(torch, x, table, scale)
        loss, lse = ctx.cross_entropy(x, table, target, scale)
        check(torch, lse, p.lse, p.lse_off, "lse")
        want = p.lse - p.z.gather(1, target[:, None].long())[:, 0]
        check(torch, loss, want, p.lse_off + p.z_off + 4 * U * p.z.abs().amax(1), "loss")
        grad = torch.ones(n, device="cuda")
        got = ctx.cross_entropy_backward(grad, x, table, target, lse, scale)
        q = torch.exp(p.z - lse.double()[:, None])
        dz = q.clone()
        dz[torch.arange(n, device="cuda"), target.long()] -= 1
        check_grads(torch, got, x, table, dz * scale, q * p.q_off[:, None] + 2 * U * dz.abs(), kind, kind, 1.0, "far")
    ctx.sync()


def test_batches_of_rows_and_other_streams(torch, hgb, ctx):
    g, x, table, target = problem(torch, 60, 90, 16, "bf16", 0, 0, 8)
    want, lse = ctx.cross_entropy(x, table, target)
    got = ctx.cross_entropy(x.view(3, 20, 16), table, target.view(3, 20))
    assert got[0].shape == (3, 20) and torch.equal(got[0].view(-1), want)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        a = ctx.cross_entropy(x, table, target)[0]
        b = ctx.cross_entropy_backward(torch.ones(60, device="cuda"), x, table, target, lse)[1]
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(a, want)
    assert torch.equal(b, ctx.cross_entropy_backward(torch.ones(60, device="cuda"), x, table, target, lse)[1])
