"""The gate's gradient of experts that a row names several times: the same
bits every time, in the slots' order."""
import pytest

from test_gpu_vectors import ctx, hgb, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-gate-repeats]", *a, flush=True)


@pytest.mark.parametrize("experts,top", [(1, 3), (5, 64), (8, 7), (9, 16), (64, 4), (200, 33), (256, 64), (1023, 64)])
def test_an_expert_named_several_times_sums_its_slots_in_order(torch, ctx, experts, top):
    """At logits of zero a sigmoid's slot gives grad / 4 exactly, so the sum's
    bits show its order; the gradients are of many sizes."""
    say("named several times", experts, top)
    g = torch.Generator().manual_seed(experts * 64 + top)
    n = 300
    names = torch.randint(0, min(experts, 4), (n, top), generator=g).int() * max(1, experts // 4)
    names[::3] = names[::3, :1]   # one expert in every slot
    names[1::3, ::2] = -1
    grad = torch.randn(n, top, generator=g) * 2.0 ** torch.randint(-14, 15, (n, top), generator=g)
    want = torch.zeros(n, experts)
    row = torch.arange(n)
    for k in range(top):   # slot after slot, each sum rounded to 32 bits
        at = names[:, k].clamp(min=0).long()
        want[row, at] += torch.where(names[:, k] >= 0, grad[:, k] / 4, 0.0)
    got = ctx.gate_backward(grad.cuda(), torch.zeros(n, experts, device="cuda"), names.cuda(), "sigmoid", False)
    assert torch.equal(got.cpu(), want)
    ctx.sync()
