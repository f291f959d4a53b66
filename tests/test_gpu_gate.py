"""The gate and its gradient against plain 64-bit forms, at the sizes, types,
strides, ties and masks where they can go wrong.

Tolerances: u = 2^-24 for each 32-bit operation.  A share is scale * s / sum
with exponentials of differences d of 32-bit logits, off by (2 + 2 |d|) u each
(d up to the largest that leaves a share that counts, 104 before it underflows
to nothing), so by 2 (2 + 2 * 104) u = 420 u relative and 2^-126 absolute at
most; a gradient is a share times a difference of sums of `top` such terms."""
import pytest

from test_gpu_vectors import U, check, ctx, dt, gen, half_step, hgb, randn, strided, torch  # noqa: F401

pytestmark = pytest.mark.gpu

SHARE = 420 * U


def say(*a):
    print("[gpu-gate]", *a, flush=True)


def reference(torch, logits, top, score, bias, groups, keep, best, renormalise, scale):
    """The definition in 64 bits; ties to the lower index by stable sorts."""
    z = logits.double()
    low = torch.full((), float("-inf"), dtype=torch.float64, device=z.device)
    masked = ~(z < float("inf")) | (z == float("-inf"))
    z = torch.where(masked, low, z)
    if score == "softmax":
        s = torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
    else:
        s = torch.sigmoid(z)
    key = s.clone() if bias is not None or groups > 1 else z.clone()   # the scores' order, also where they round to the same
    if bias is not None:
        b = bias.double()
        masked = masked | ~(b < float("inf")) | (b == float("-inf"))
        key = key + torch.where(b.isfinite(), b, torch.zeros_like(b))
    key = torch.where(masked, low, key)
    if groups > 1:
        n, e = key.shape
        by = key.view(n, groups, -1)
        worth = torch.sort(by, -1, descending=True).values[..., :best].sum(-1)
        order = torch.sort(worth, dim=-1, descending=True, stable=True).indices[:, :keep]
        kept = torch.zeros(n, groups, dtype=torch.bool, device=z.device).scatter_(1, order, True)
        key = torch.where(kept.unsqueeze(-1), by, low).reshape(n, e)
    chosen = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :top]
    live = key.gather(1, chosen) > low
    zc = torch.where(live, z.gather(1, chosen), low)
    if renormalise:
        log = zc if score == "softmax" else torch.nn.functional.logsigmoid(zc)
        share = torch.nan_to_num(torch.softmax(log, 1), nan=0.0)
    else:
        share = s.gather(1, chosen) * live
    return torch.where(live, chosen, -1), scale * share


GATES = [
    # n, experts, top, score, bias, groups, keep, best, renormalise, type, extra stride
    (1, 1, 1, "softmax", False, 1, 1, 2, True, "f32", 0),
    (3, 64, 2, "softmax", False, 1, 1, 2, True, "bf16", 0),
    (3, 2, 2, "sigmoid", True, 1, 1, 2, False, "f16", 0),
    (7, 5, 3, "softmax", True, 5, 3, 1, False, "f32", 0),
    (100, 8, 3, "softmax", True, 2, 1, 2, True, "bf16", 3),
    (257, 9, 4, "sigmoid", False, 3, 2, 2, True, "f16", 1),
    (1000, 60, 6, "softmax", False, 1, 1, 2, False, "f32", 0),
    (1000, 64, 8, "sigmoid", True, 8, 4, 2, True, "f32", 0),
    (999, 65, 7, "softmax", True, 5, 2, 2, False, "bf16", 0),
    (4097, 256, 8, "sigmoid", True, 8, 4, 2, True, "bf16", 0),
    (4097, 256, 8, "softmax", True, 8, 3, 1, True, "f32", 5),
    (500, 333, 16, "softmax", True, 3, 2, 2, True, "f16", 0),
    (300, 512, 64, "sigmoid", False, 1, 1, 2, True, "bf16", 0),
    (300, 513, 9, "softmax", False, 1, 1, 2, False, "f32", 0),
    (211, 1023, 10, "sigmoid", True, 11, 5, 2, False, "f32", 0),
    (211, 1023, 64, "softmax", True, 1023, 700, 1, True, "f16", 1),
]


def inputs(torch, n, experts, kind, extra, bias, seed, masks=0.0):
    g = gen(torch, seed)
    logits = randn(torch, g, n, experts, dtype=dt(torch, kind), scale=1.5)
    if masks:
        logits[torch.rand(n, experts, generator=g, device="cuda") < masks] = float("-inf")
    if extra:
        logits = strided(torch, logits, extra, 1)
    return g, logits, randn(torch, g, experts, scale=0.1) if bias else None


@pytest.mark.parametrize("masks", [0.0, 0.4, 0.95])
@pytest.mark.parametrize("n,experts,top,score,bias,groups,keep,best,renormalise,kind,extra", GATES)
def test_gate(torch, ctx, n, experts, top, score, bias, groups, keep, best, renormalise, kind, extra, masks):
    say("gate", n, experts, top, score, groups, kind, masks)
    _, logits, b = inputs(torch, n, experts, kind, extra, bias, n + experts, masks)
    chosen, share = ctx.gate(logits, top, score, b, groups, keep, best, renormalise, 1.7)
    want, ws = reference(torch, logits, top, score, b, groups, keep, best, renormalise, float(torch.tensor(1.7)))
    assert torch.equal(chosen.long(), want)
    check(torch, share, ws, ws.abs() * SHARE + 2.0 ** -120, "share")
    again = ctx.gate(logits, top, score, b, groups, keep, best, renormalise, 1.7)
    assert torch.equal(again[0], chosen) and torch.equal(again[1], share)
    ctx.sync()


def test_gate_of_no_rows(torch, ctx):
    chosen, share = ctx.gate(torch.empty(0, 9, device="cuda"), 3)
    assert chosen.shape == share.shape == (0, 3)
    d = ctx.gate_backward(share, torch.empty(0, 9, device="cuda"), chosen)
    assert d.shape == (0, 9)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_expert_and_group(torch, ctx, score):
    z = torch.zeros(5, 40, device="cuda")
    z[1] = torch.arange(40, device="cuda") // 10 % 2   # two equal groups above two equal ones
    z[2, 7::8] = 1.0
    z[3, 39] = -1.0
    z[4] = torch.finfo(torch.float32).min
    for bias in (None, torch.zeros(40, device="cuda")):
        for groups, keep in ((1, 1), (4, 2)):
            got = ctx.gate(z, 6, score, bias, groups, keep)
            want = reference(torch, z, 6, score, bias, groups, keep, 2, True, 1.0)
            assert torch.equal(got[0].long(), want[0]), (score, groups, got[0], want[0])
            check(torch, got[1], want[1], want[1] * SHARE + 2.0 ** -120, "share")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups", [(64, 4), (32, 4), (30, 5), (256, 8), (9, 3)])
def test_biases_of_the_lowest_and_largest_values(torch, ctx, score, experts, groups):
    """Two such keys are not finite in sum, and a group of them is still worth more than a masked one."""
    g = gen(torch, 19)
    most, per = torch.finfo(torch.float32).max, experts // groups
    z = randn(torch, g, 70, experts)
    low = torch.full((experts,), -most, device="cuda")
    low[:per] = float("-inf")
    mixed = low.clone()
    mixed[-1] = 0.0
    high = torch.zeros(experts, device="cuda")
    high[per:] = most
    last = low.clone()
    last[per:] = float("-inf")
    last[-per:] = -most
    for bias in (low, mixed, high, last):
        for keep in (1, 2):
            got = ctx.gate(z, 2, score, bias, groups, keep)
            want = reference(torch, z, 2, score, bias, groups, keep, 2, True, 1.0)
            assert torch.equal(got[0].long(), want[0]), (keep, got[0][0], want[0][0])
            check(torch, got[1], want[1], want[1] * SHARE + 2.0 ** -120, "share")
    ctx.sync()


def test_keys_closer_than_32_bits_hold_are_told_apart(torch, ctx):
    """The second expert's key is the larger by about 2^-30, and the lower index has the lesser."""
    n = 4096
    g = gen(torch, 5)
    z = randn(torch, g, n, 16)
    z[:, 1] = z[:, 0] - 2.0 ** -12
    s = torch.sigmoid(z.double())
    bias = torch.zeros(16, device="cuda")
    bias[2:] = -4.0
    step = (s[:, 0] - s[:, 1])
    for row in range(0, n, 512):   # one bias for all rows: taken for this row's difference, rounded up
        b = bias.clone()
        b[1] = torch.nextafter(step[row].float(), torch.ones((), device="cuda"))
        got = ctx.gate(z, 3, "sigmoid", b)
        want = reference(torch, z, 3, "sigmoid", b, 1, 1, 2, True, 1.0)
        assert torch.equal(got[0].long(), want[0])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_bad_logits_are_masked_and_reported(torch, hgb, ctx, kind):
    g = gen(torch, 9)
    z = randn(torch, g, 50, 33, dtype=dt(torch, kind))
    clean = ctx.gate(z, 4)
    ctx.sync()
    z[3, 5], z[3, 6], z[7] = float("nan"), float("inf"), float("nan")
    for score, bias in (("softmax", None), ("sigmoid", torch.zeros(33, device="cuda"))):
        chosen, share = ctx.gate(z, 4, score, bias)
        want, ws = reference(torch, z, 4, score, bias, 1, 1, 2, True, 1.0)
        assert torch.equal(chosen.long(), want) and bool((chosen[7] == -1).all()) and bool((share[7] == 0).all())
        check(torch, share, ws, ws * SHARE + 2.0 ** -120, "share")
        with pytest.raises(hgb.HGBError, match="NaN or .infinity"):
            ctx.sync()
        ctx.sync()
    others = [r for r in range(50) if r not in (3, 7)]
    assert torch.equal(ctx.gate(z, 4)[0][others], clean[0][others])
    with pytest.raises(hgb.HGBError):
        ctx.sync()
    bias = torch.zeros(33, device="cuda")
    bias[0], bias[1] = float("nan"), float("-inf")
    z = randn(torch, g, 50, 33, dtype=dt(torch, kind))
    assert not bool((ctx.gate(z, 8, "softmax", bias)[0] < 2).any())
    with pytest.raises(hgb.HGBError, match="bias"):
        ctx.sync()
    bias[0] = float("-inf")   # a mask, and no error
    assert not bool((ctx.gate(z, 8, "softmax", bias)[0] < 2).any())
    ctx.sync()


def grad_reference(torch, grad, logits, chosen, score, renormalise, scale):
    """Through autograd in 64 bits, for the given experts."""
    z = torch.where(logits.double() < float("inf"), logits.double(), float("-inf")).requires_grad_()
    live, at = chosen >= 0, chosen.clamp(min=0).long()
    live = live & (z.detach().gather(1, at) > float("-inf"))
    safe = torch.where(torch.isinf(z), torch.full_like(z, -1e4), z)   # a mask, of no gradient
    log = torch.log_softmax(safe, 1) if score == "softmax" else torch.nn.functional.logsigmoid(safe)
    log = torch.where(live, log.gather(1, at), -1e300)
    share = torch.softmax(log, 1) if renormalise else torch.exp(log)
    (scale * share * live * torch.where(live, grad.double(), 0.0)).sum().backward()
    out = torch.where(torch.isinf(z.detach()), 0.0, z.grad)
    big = (share.detach() * live).abs()
    return out, big


@pytest.mark.parametrize("masks", [0.0, 0.4, 0.95])
@pytest.mark.parametrize("n,experts,top,score,bias,groups,keep,best,renormalise,kind,extra", GATES)
def test_gate_backward(torch, ctx, n, experts, top, score, bias, groups, keep, best, renormalise, kind, extra, masks):
    say("gate_backward", n, experts, top, score, kind, masks)
    g, logits, b = inputs(torch, n, experts, kind, extra, bias, n + experts, masks)
    chosen, _ = ctx.gate(logits, top, score, b, groups, keep, best, renormalise, 1.7)
    grad = randn(torch, g, n, top)
    out = None
    if extra:
        out = torch.full((n, experts + 3), 9.0, dtype=logits.dtype, device="cuda")[:, :experts]
    got = ctx.gate_backward(grad, logits, chosen, score, renormalise, 1.7, out=out)
    want, share = grad_reference(torch, grad, logits, chosen, score, renormalise, float(torch.tensor(1.7)))
    rel, tiny = half_step(torch, logits.dtype)
    # each term is scale * share * (g - the mean g): both off by the shares' error, the mean by top more roundings
    size = 1.7 * grad.abs().max(1, keepdim=True).values.double() * share.amax(1, keepdim=True)
    check(torch, got, want, size * (4 * SHARE + 2 * top * U) + want.abs() * rel + tiny, "dlogits")
    if extra:
        assert bool((out.as_strided((n, 3), (experts + 3, 1), out.storage_offset() + experts) == 9.0).all())
    assert torch.equal(ctx.gate_backward(grad, logits, chosen, score, renormalise, 1.7), got.contiguous())
    ctx.sync()


def test_gate_backward_against_differences(torch, ctx):
    """The shares' change along a direction, from the forward verb itself."""
    g = gen(torch, 77)
    for score, renormalise in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        z = randn(torch, g, 64, 24)
        chosen, _ = ctx.gate(z, 4, score, renormalise=renormalise)
        grad, way = randn(torch, g, 64, 4), randn(torch, g, 64, 24)
        d = ctx.gate_backward(grad, z, chosen, score, renormalise)
        h = 2.0 ** -7

        def along(step):
            c, s = ctx.gate(z + step * way, 24, score, renormalise=False)   # all of them: the choice does not matter
            s = s.double().gather(1, c.argsort(1)).gather(1, chosen.long())
            return ((s / s.sum(1, keepdim=True) if renormalise else s) * grad).sum(1)

        rate = (along(h) - along(-h)) / (2 * h)
        # the third derivative of a softmax or sigmoid along `way` is below 3 (2 max |way|)^3 share; rounding 4 SHARE / h
        bound = (h * h / 6 * 3 * (2 * way.abs().amax(1)) ** 3 + 4 * SHARE / h) * grad.abs().sum(1)
        assert bool(((d * way).sum(1) - rate).abs().le(bound).all()), (score, renormalise)


def test_gate_backward_of_bad_and_repeated_experts(torch, hgb, ctx):
    g = gen(torch, 3)
    z = randn(torch, g, 6, 10)
    grad = randn(torch, g, 6, 3)
    chosen = torch.tensor([[1, 2, 3], [4, 4, 4], [-1, 5, -1], [-1, -1, -1], [0, 9, 2], [7, 6, 5]], dtype=torch.int32, device="cuda")
    got = ctx.gate_backward(grad, z, chosen, "sigmoid", False)
    s = torch.sigmoid(z.double())
    want = torch.zeros_like(s).scatter_add_(1, chosen.clamp(min=0).long(), grad.double() * (chosen >= 0)) * s * (1 - s)
    check(torch, got, want, want.abs() * SHARE + 3e-6, "dlogits")
    ctx.sync()
    chosen[4, 0], chosen[5, 1] = 10, -2
    got = ctx.gate_backward(grad, z, chosen, "sigmoid", False)
    assert float(got[4, 0]) == 0 and float(got[5, 6]) == 0 and torch.equal(got[:4] != 0, want[:4] != 0)
    with pytest.raises(hgb.HGBError, match="expert"):
        ctx.sync()
