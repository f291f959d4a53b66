"""The gate where logits tie at zero or lie among the smallest numbers.

The choice is compared with stable sorts in 64 bits, on the host (whose
conversions keep the smallest numbers); shares as in test_gpu_gate.py."""
import pytest

from test_gpu_gate import SHARE, reference
from test_gpu_vectors import check, ctx, dt, hgb, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-gate-ties]", *a, flush=True)


def compare(torch, ctx, z, top, score, groups, keep):
    got = ctx.gate(z.cuda(), top, score, None, groups, keep)
    want = reference(torch, z.double() + 0.0, top, score, None, groups, keep, 2, True, 1.0)   # + 0: one zero
    wrong = (got[0].cpu().long() != want[0]).any(1)
    row = int(wrong.int().argmax())
    assert not bool(wrong.any()), (int(wrong.sum()), got[0][row], want[0][row])
    check(torch, got[1].cpu(), want[1], want[1] * SHARE + 2.0 ** -120, "share")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("experts,groups,keep", [(9, 1, 1), (16, 1, 1), (64, 1, 1), (64, 8, 3), (129, 1, 1), (256, 1, 1), (333, 3, 2), (513, 1, 1), (1023, 1, 1)])
def test_zeros_of_both_signs_tie(torch, ctx, experts, groups, keep, kind):
    """Zeros at random places among negatives: the lowest places are chosen."""
    say(experts, groups, kind)
    g = torch.Generator().manual_seed(experts + groups)
    for zeros in (2, 5, experts // 2):
        z = -torch.rand(400, experts, generator=g) - 0.5
        at = torch.rand(400, experts, generator=g).argsort(1)[:, :zeros]
        z.scatter_(1, at, torch.where(torch.rand(400, zeros, generator=g) < 0.5, -0.0, 0.0))
        for top in (1, 2, 8):
            for score in ("softmax", "sigmoid"):
                compare(torch, ctx, z.to(dt(torch, kind)), top, score, groups, keep)
    ctx.sync()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("experts", [8, 16, 64, 256, 1023])
def test_the_smallest_numbers_are_in_order(torch, ctx, experts, kind):
    """Logits of a few units of the type's smallest number, of both signs: the
    largest first, and of equal ones the lowest place."""
    say(experts, kind)
    g = torch.Generator().manual_seed(experts)
    f = torch.finfo(dt(torch, kind))
    unit = f.tiny * f.eps
    for units in (1, 3, 40):
        z = torch.randint(-units, units + 1, (400, experts), generator=g).double() * unit
        z = z.to(dt(torch, kind))
        assert float(z.double().abs().max()) == units * unit
        for top in (1, 8):
            compare(torch, ctx, z, top, "softmax", 1, 1)
    ctx.sync()
