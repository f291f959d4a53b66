"""Gradients of no rows: the table's is zeros, also of the smallest tables."""
import pytest

from test_gpu_vectors import ctx, dt, hgb, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,out_kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("vocab,dim", [(1, 1), (1, 3), (3, 1), (3, 4), (3, 5), (4, 4), (17, 1), (300, 33)])
def test_the_tables_gradient_of_no_rows_is_zero(torch, ctx, vocab, dim, kind, out_kind):
    x, table = torch.empty(0, dim, dtype=dt(torch, kind), device="cuda"), torch.ones(vocab, dim, dtype=dt(torch, kind), device="cuda")
    none, tokens = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    junk = torch.full((4096,), 7.0, device="cuda")   # what a fresh output may hold
    del junk
    dx, dtable = ctx.cross_entropy_backward(none, x, table, tokens, none, dtype=dt(torch, out_kind))
    assert dx.shape == (0, dim) and dtable.shape == (vocab, dim) and bool((dtable == 0).all())
    slots, teacher = tokens.view(0, 1).expand(0, 2).contiguous(), torch.empty(0, 2, dtype=dt(torch, kind), device="cuda")
    dx, dtable = ctx.distill_backward(none, x, table, slots, teacher, none, torch.empty(0, 2, device="cuda"), dtype=dt(torch, out_kind))
    assert dx.shape == (0, dim) and dtable.shape == (vocab, dim) and bool((dtable == 0).all())
    ctx.sync()
