"""The vector verbs on arguments side by side in one buffer: the same bits as on
buffers of their own, and every other column left as it was."""
import sys

import pytest

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-vectors-packed]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch():
    import torch as _torch
    from histogram_gradient_boosted_amd import binding
    if not _torch.cuda.is_available() or not binding.available():
        pytest.skip("no HIP device")
    return _torch


@pytest.fixture(scope="module")
def ctx(torch):
    from histogram_gradient_boosted_amd import binding
    c = binding.Context(0)
    yield c
    c.sync()
    c.close()


# rows, dim, type; the last calls are large enough to store past the caches
CASES = [(1, 8, "float32"), (50, 9, "bfloat16"), (300, 40, "float16"), (3000, 333, "float32"), (777, 1025, "bfloat16"),
         (90001, 520, "bfloat16"), (70001, 301, "float32")]


@pytest.mark.parametrize("n,dim,kind", CASES)
def test_side_by_side(torch, ctx, n, dim, kind):
    say(n, dim, kind)
    t = getattr(torch, kind)
    g = torch.Generator(device="cuda").manual_seed(n + dim)

    def place(rows, parts, first):
        """`parts` matrices [rows, dim] in one buffer, three values apart, the `first` ones filled."""
        buf = torch.full((rows, parts * (dim + 3)), 7.0, dtype=t, device="cuda")
        views = [buf[:, k * (dim + 3):k * (dim + 3) + dim] for k in range(parts)]
        for v in views[:first]:
            v.copy_(torch.randn(rows, dim, generator=g, device="cuda"))
        return buf, views

    def check(buf, out, want, call):
        """call() writes `want` into out, a view of buf, and nothing else."""
        rest = buf.clone()
        got = call()
        assert torch.equal(out, want)
        column = out.storage_offset()
        rest[:, column:column + dim] = out
        assert torch.equal(buf, rest), "the other columns"
        return got

    w, b = (torch.rand(dim, generator=g, device="cuda") for _ in range(2))
    buf, (x, grad, out) = place(n, 3, 2)
    want = ctx.layer_norm(x.contiguous(), w, b)
    got = check(buf, out, want[0], lambda: ctx.layer_norm(x, w, b, out=out))
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    _, mean, rstd = want
    want = ctx.layer_norm_backward(grad.contiguous(), x.contiguous(), mean, rstd, w)
    got = check(buf, out, want[0], lambda: ctx.layer_norm_backward(grad, x, mean, rstd, w, out=out))
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])

    tok = torch.randint(0, n, (n,), generator=g, device="cuda").int()
    check(buf, out, ctx.embed(x.contiguous(), tok), lambda: ctx.embed(x, tok, out=out))
    check(buf, out, ctx.embed_backward(grad.contiguous(), tok, n), lambda: ctx.embed_backward(grad, tok, n, out=out))

    # x and its sums in the even rows' halves of the sorted rows' buffer
    top = 2
    e = torch.randint(-1, 5, (n, top), generator=g, device="cuda").int()
    share = torch.rand(n, top, generator=g, device="cuda")
    r = ctx.route(e, 5)
    buf, (y, ys) = place(n * top, 2, 2)
    x, want = y[:n], ctx.route_gather(y[:n].contiguous(), r)
    check(buf, ys, want, lambda: ctx.route_gather(x, r, out=ys))
    want = ctx.route_combine(ys.contiguous(), r, share)
    rest = buf.clone()
    ctx.route_combine(ys, r, share, out=x)
    rest[:n, :dim] = want
    assert torch.equal(buf, rest)
    buf, (grad, y, dy) = place(n * top, 3, 2)
    grad = grad[:n]
    want = ctx.route_combine_backward(grad.contiguous(), y.contiguous(), r, share)
    got = check(buf, dy, want[0], lambda: ctx.route_combine_backward(grad, y, r, share, out=dy))
    assert torch.equal(got[1], want[1])
    ctx.sync()


def test_shared_bytes_are_refused(torch, ctx):
    from histogram_gradient_boosted_amd.binding import HGBError
    buf = torch.zeros(10, 16, device="cuda")
    for a, b in ((buf[:, :8], buf[:, 7:15]), (buf[:9, 8:], buf.view(-1)[15:15 + 9 * 16].view(9, 16)[:, :8])):
        with pytest.raises(HGBError, match="overlaps"):
            ctx.layer_norm(a, out=b)
    ctx.sync()
