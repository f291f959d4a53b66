"""A 32-bit table gradient of 16-bit inputs: the logits' gradient is a factor of
it in 24 bits (bf16: three parts of 8) or 22 (fp16: two of 11).

Each row of x holds a single one, in a column of its own, so that a value of
dtable is one value of dz, not a sum: what is off is the logits' error, as in
test_gpu_head.py, and dz's rounding to its parts: half a step each, 2^-8 of what
the part before left for bf16 and 2^-11 for fp16."""
import pytest

from test_gpu_head import Plain
from test_gpu_vectors import U, check, ctx, dt, hgb, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-head-planes]", *a, flush=True)


@pytest.mark.parametrize("kind,left", [("bf16", 2.0 ** -24), ("f16", 2.0 ** -22)])
@pytest.mark.parametrize("n,vocab", [(24, 300), (64, 1000), (512, 40000)])
def test_the_tables_gradient_has_more_bits_than_its_inputs(torch, ctx, n, vocab, kind, left):
    say(n, vocab, kind)
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.eye(n, device="cuda").to(dt(torch, kind))
    table = torch.randn(vocab, n, generator=g, device="cuda").to(dt(torch, kind))
    target = torch.randint(0, vocab, (n,), generator=g, device="cuda").int()
    grad = 0.5 + torch.rand(n, generator=g, device="cuda")
    floor = 2.0 ** -38 if kind == "f16" else 0.0   # half of fp16's smallest, over the factor that dz is held with
    p = Plain(torch, x, table, 1.0)
    rate = grad.double()[:, None]
    row = torch.arange(n, device="cuda")

    _, lse = ctx.cross_entropy(x, table, target)
    _, got = ctx.cross_entropy_backward(grad, x, table, target, lse, dtype=torch.float32)
    q = torch.exp(p.z - lse.double()[:, None])
    dz = q.clone()
    dz[row, target.long()] -= 1
    off = (q * p.q_off[:, None] + 2 * U * dz.abs()) * rate
    check(torch, got, (dz * rate).T, (off + (dz * rate).abs() * (left + 2 * U) + floor).T, "cross_entropy_backward")

    tokens = torch.stack([target, (target + 1) % vocab, (target + 7) % vocab], 1).contiguous()
    teacher = torch.randn(n, 3, generator=g, device="cuda")
    _, lse, picked = ctx.distill(x, table, tokens, teacher, 1.0)
    _, got = ctx.distill_backward(grad, x, table, tokens, teacher, lse, picked, 1.0, dtype=torch.float32)
    q = torch.exp(p.z - lse.double()[:, None])
    big = torch.zeros_like(q).scatter_add_(1, tokens.long(), torch.softmax(teacher.double(), 1))
    off = (q * p.q_off[:, None] + big * U * (19 + 4 * teacher.double().abs().amax(1, keepdim=True)) + 4 * U * (q + big)) * rate
    check(torch, got, ((q - big) * rate).T, (off + ((q - big) * rate).abs() * (left + 2 * U) + floor).T, "distill_backward")
    ctx.sync()
