"""The vector verbs where sizes and offsets pass 32 bits: more blocks than one
dimension of a grid holds, and rows past 2^32 elements."""
import gc
import sys

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CHUNK = 1 << 20


def say(*a):
    print("[gpu-vectors-large]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch():
    import torch as _torch
    from histogram_gradient_boosted_amd import binding
    if not _torch.cuda.is_available() or not binding.available():
        pytest.skip("no HIP device")
    return _torch


@pytest.fixture()
def ctx(torch):
    from histogram_gradient_boosted_amd import binding
    c = binding.Context(0)
    yield c
    c.sync()
    c.close()
    gc.collect()
    torch.cuda.empty_cache()


def room(torch, gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def pieces(n):
    return ((a, min(a + CHUNK, n)) for a in range(0, n, CHUNK))


def test_embed_of_many_wide_rows(torch, ctx):
    """2^24 rows and more of 129 vectors each: as many blocks."""
    room(torch, 48)
    n, dim = (1 << 24) + 1001, 1025
    say("embed", n, dim)
    g = gen(torch, 1)
    table = torch.randn(7, dim, generator=g, device="cuda").bfloat16()
    tok = torch.randint(0, 7, (n,), generator=g, device="cuda", dtype=torch.int32)
    out = ctx.embed(table, tok)
    ctx.sync()
    for a, b in pieces(n):
        assert torch.equal(out[a:b], table[tok[a:b].long()]), a


def test_routing_of_many_wide_rows(torch, ctx):
    """The same there and back, one expert a row: the rows come back as they were."""
    room(torch, 120)
    n, dim = (1 << 24) + 1001, 1025
    say("route", n, dim)
    g = gen(torch, 2)
    x = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    e = torch.randint(0, 50, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    r = ctx.route(e, 50)
    xs = ctx.route_gather(x, r)
    ctx.sync()
    for a, b in pieces(n):
        assert torch.equal(xs[a:b], x[r.order[a:b].long()]), a
    back = ctx.route_combine(xs, r)
    ctx.sync()
    for a, b in pieces(n):
        assert torch.equal(back[a:b], x[a:b]), a
    back.zero_()
    ctx.route_gather_backward(xs, r, out=back)
    ctx.sync()
    for a, b in pieces(n):
        assert torch.equal(back[a:b], x[a:b]), a


def test_combine_gradient_of_many_slots(torch, ctx):
    """2^26 slots and more, a wave each, and the sort of as many."""
    room(torch, 120)
    n, top, dim, experts = (1 << 23) + 1001, 8, 257, 1023
    slots = n * top
    say("combine gradient", slots, dim)
    g = gen(torch, 3)
    e = torch.randint(-1, experts, (n, top), generator=g, device="cuda", dtype=torch.int32)
    r = ctx.route(e, experts)
    key = torch.where(e < 0, experts, e).reshape(-1)
    used = int(r.offsets[-1])
    assert used == int((e >= 0).sum()) and bool((r.order[used:] == -1).all())
    order = r.order[:used].long()
    sorted_key = key[order].long() * slots + order
    assert bool((sorted_key[1:] > sorted_key[:-1]).all()), "by expert, then by slot"
    assert torch.equal(r.position.view(-1)[order], torch.arange(used, dtype=torch.int32, device="cuda"))
    assert torch.equal(r.position < 0, e < 0)
    assert torch.equal(r.offsets[1:].long() - r.offsets[:-1].long(), torch.bincount(key.long(), minlength=experts + 1)[:experts])
    del key, order, sorted_key
    grad = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.empty(slots, dim, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(n, top, generator=g, device="cuda")
    dy, dw = ctx.route_combine_backward(grad, y, r, w)
    ctx.sync()
    flat = w.view(-1)
    for a, b in pieces(slots):
        s = r.order[a:b].long()
        live = (s >= 0).unsqueeze(-1)
        s = s.clamp(min=0)
        rows = grad[s // top]
        # one rounding of the product, one to 16 bits
        assert torch.equal(dy[a:b], torch.where(live, rows.float() * flat[s].unsqueeze(-1), 0.0).bfloat16()), a
        prod = rows.float() * y[a:b].float()   # exact: 8 bits by 8
        kept = live[:, 0]
        off = (dw.view(-1)[s].double() - prod.sum(1, dtype=torch.float64)).abs()
        # a lane adds up to 16 values of 257, then 6 sums over lanes
        bound = prod.abs().sum(1, dtype=torch.float64) * 24 * U
        assert bool((off <= bound)[kept].all()), a
    assert bool((dw[e < 0] == 0).all())


def test_layer_norm_and_routing_past_32_bits(torch, ctx):
    """Rows 2^16 elements apart, 66,000 of them: the same as the rows side by side."""
    room(torch, 40)
    stride, n, dim = 1 << 16, 66000, 24
    g = gen(torch, 4)

    def apart(dtype=torch.bfloat16):
        return torch.empty(n * stride, dtype=dtype, device="cuda").view(n, stride)[:, :dim]

    x, grad, out = apart(), apart(), apart()
    x.copy_(torch.randn(n, dim, generator=g, device="cuda"))
    grad.copy_(torch.randn(n, dim, generator=g, device="cuda"))
    w, b = torch.rand(dim, generator=g, device="cuda"), torch.rand(dim, generator=g, device="cuda")
    y, mean, rstd = ctx.layer_norm(x, w, b, out=out)
    close = ctx.layer_norm(x.contiguous(), w, b)
    assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd), close))
    got = ctx.layer_norm_backward(grad, x, mean, rstd, w, out=out)
    assert all(torch.equal(p, q) for p, q in
               zip(got, ctx.layer_norm_backward(grad.contiguous(), x.contiguous(), mean, rstd, w)))
    r = ctx.route(torch.randint(0, 9, (n, 1), generator=g, device="cuda", dtype=torch.int32), 9)
    share = torch.rand(n, 1, generator=g, device="cuda")
    assert torch.equal(ctx.route_gather(x, r, out=out), ctx.route_gather(x.contiguous(), r))
    assert torch.equal(ctx.route_combine(x, r, share, out=out), ctx.route_combine(x.contiguous(), r, share))
    got = ctx.route_combine_backward(grad, x, r, share, out=out)
    want = ctx.route_combine_backward(grad.contiguous(), x.contiguous(), r, share)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    # and the gradient of an embedding, read from such rows
    tok = torch.randint(0, 40, (n,), generator=g, device="cuda", dtype=torch.int32)
    assert torch.equal(ctx.embed_backward(grad, tok, 40), ctx.embed_backward(grad.contiguous(), tok, 40))
