"""What the binding of the gate and the losses refuses on the device."""
import pytest

from test_gpu_vectors import ctx, hgb, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [-1, 0, 65, 1024, 2 ** 31 - 1])
def test_gate_refuses_a_top_before_it_allocates(torch, hgb, ctx, top):
    """2^31 slots of 100,000 rows would be 1.7 PB."""
    free = torch.cuda.memory_allocated()
    with pytest.raises(hgb.HGBError, match="top"):
        ctx.gate(torch.zeros(100_000, 1000, dtype=torch.bfloat16, device="cuda"), top)
    assert torch.cuda.memory_allocated() == free
    ctx.sync()
