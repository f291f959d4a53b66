"""The losses' gradients where the rows' gradients differ by many orders, are
very large or small, or not finite.

fp16's logits' gradient is held times a power of two that brings the largest
finite rate (grad times the scale) to 2^14 to 2^15, and its smallest step is
2^-24: off by 2^-39 of that rate at most, which no row's own size lessens.
Below rates of 2^-112 the power stays 2^126, and the step is 2^-151."""
import pytest

from test_gpu_head import Plain, problem
from test_gpu_vectors import U, check, ctx, dt, half_step, hgb, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-head-rates]", *a, flush=True)


def gradients(torch, ctx, grad, n, vocab, dim, kind, out_kind):
    """Of both losses: (dx, dtable) twice, and the calls' arguments."""
    _, x, table, target = problem(torch, n, vocab, dim, kind, 0, 0, n + vocab + dim)
    _, lse = ctx.cross_entropy(x, table, target)
    tokens = torch.stack([target, (target + 1) % vocab, (target + 5) % vocab], 1).contiguous()
    teacher = torch.tensor([2.0, 1.0, 0.0], device="cuda").expand(n, 3).contiguous()
    _, lse2, picked = ctx.distill(x, table, tokens, teacher, 1.0)
    return (ctx.cross_entropy_backward(grad, x, table, target, lse, dtype=dt(torch, out_kind)),
            ctx.distill_backward(grad, x, table, tokens, teacher, lse2, picked, 1.0, dtype=dt(torch, out_kind)), x, table, target, lse)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("n,vocab,dim", [(7, 300, 64), (300, 1000, 72)])
def test_a_rate_that_is_not_finite_changes_no_other_row(torch, ctx, n, vocab, dim, bad, kind):
    say("not finite", n, vocab, dim, bad, kind)
    g = torch.Generator(device="cuda").manual_seed(4)
    grad = torch.randn(n, generator=g, device="cuda") * 1000
    grad[2] = 0.0
    clean = gradients(torch, ctx, grad, n, vocab, dim, kind, "f32")
    grad[2] = bad
    got = gradients(torch, ctx, grad, n, vocab, dim, kind, "f32")
    others = [r for r in range(n) if r != 2]
    for k in (0, 1):
        assert bool(clean[k][0].isfinite().all())
        assert torch.equal(got[k][0][others], clean[k][0][others])
        assert not bool(got[k][0][2].isfinite().all())
    ctx.sync()


@pytest.mark.parametrize("kind,log_rate", [("f16", -130), ("f16", -120), ("f16", -100), ("f16", -60), ("f16", 60), ("f16", 100), ("f16", 119),
                                           ("bf16", -60), ("bf16", 114), ("f32", -60), ("f32", 114)])
@pytest.mark.parametrize("n,vocab,dim", [(7, 300, 64), (300, 1000, 72)])
def test_rates_of_any_size(torch, ctx, n, vocab, dim, kind, log_rate):
    """dtable in 32 bits holds what rates of 2^-130 to 2^119 give (fp16), or of 2^-60 on (the others, which have 32 bits' exponents)."""
    say("rates of 2 to the", log_rate, n, vocab, dim, kind)
    g = torch.Generator(device="cuda").manual_seed(5)
    grad = (0.5 + torch.rand(n, generator=g, device="cuda")) * 2.0 ** log_rate
    (got, _, x, table, target, lse) = gradients(torch, ctx, grad, n, vocab, dim, kind, "f32")
    against(torch, got, grad, x, table, target, lse, kind, max(2.0 * 2.0 ** log_rate, 2.0 ** -112))
    ctx.sync()


@pytest.mark.parametrize("out_kind", ["own", "f32"])
@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n,vocab,dim", [(40, 300, 64), (300, 20000, 72)])
def test_rates_that_span_many_orders(torch, ctx, n, vocab, dim, kind, out_kind):
    say("many orders", n, vocab, dim, kind, out_kind)
    g = torch.Generator(device="cuda").manual_seed(6)
    grad = torch.randn(n, generator=g, device="cuda") * 2.0 ** (-20 * torch.rand(n, generator=g, device="cuda"))
    out = kind if out_kind == "own" else "f32"
    (got, _, x, table, target, lse) = gradients(torch, ctx, grad, n, vocab, dim, kind, out)
    against(torch, got, grad, x, table, target, lse, kind, grad.abs().max(), out)
    ctx.sync()


def against(torch, got, grad, x, table, target, lse, kind, top_rate, out_kind="f32"):
    """The cross entropy's gradients against the formula's in 64 bits; of dx the rows that x's type holds."""
    n, vocab = x.shape[0], table.shape[0]
    p = Plain(torch, x, table, 1.0)
    q = torch.exp(p.z - lse.double()[:, None])
    rate = grad.double()[:, None]
    dz = q.clone()
    dz[torch.arange(n, device="cuda"), target.long()] -= 1
    off = (q * p.q_off[:, None] + 2 * U * dz.abs()) * rate.abs()
    held = ((dz * rate) @ table.double()).abs().amax(1) < torch.finfo(x.dtype).max / 2
    dx = torch.where(held[:, None], got[0], 0)
    some = torch.where(held[:, None], dz * rate, 0)
    step, floor = half_step(torch, x.dtype)[0], float(top_rate) * 2.0 ** -39 if kind == "f16" else 0.0
    rel, tiny = half_step(torch, x.dtype)
    size = some.abs()
    err = off * held[:, None] + size * (0.0 if kind == "f32" else step) * 1.001 + floor
    want = some @ table.double()
    bound = err @ table.double().abs() + (vocab + 300) * U * (size @ table.double().abs())
    check(torch, dx, want, bound * (1 + rel) + want.abs() * rel * 1.001 + tiny, "dx")
    size = (dz * rate).abs()
    step = 0.0 if kind == "f32" else step if out_kind == kind else step * step
    err = off + size * step * 1.001 + floor
    want = (dz * rate).T @ x.double()
    bound = err.T @ x.double().abs() + (2 * n + 300) * U * (size.T @ x.double().abs())
    rel, tiny = half_step(torch, dt(torch, out_kind))
    check(torch, got[1], want, bound * (1 + rel) + want.abs() * rel * 1.001 + tiny, "dtable")
