"""The gate and the head's losses as programs call them: as a run of verbs with
the routing between them, captured and replayed, over several pieces of the
vocabulary and of the rows, into a caller's buffers, at the largest tops."""
import pytest

from test_gpu_gate import SHARE
from test_gpu_head import Plain, check_grads, problem
from test_gpu_vectors import U, check, ctx, dt, gen, half_step, hgb, randn, strided, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-head-calls]", *a, flush=True)


class Model:
    """Tokens to vectors, normalised, through some of the experts (a learned
    scale each) and on to the next token: every verb's forward and backward."""

    def __init__(self, torch, ctx, vocab, dim, experts, dtype, seed):
        g = gen(torch, seed)
        self.torch, self.ctx, self.dtype = torch, ctx, dtype
        self.table = randn(torch, g, vocab, dim, dtype=dtype, scale=dim ** -0.5)
        self.gate = randn(torch, g, experts, dim, scale=dim ** -0.5)
        self.scales = 1 + 0.2 * randn(torch, g, experts, dim)
        self.balance = 0.05 * randn(torch, g, experts)

    def loss(self, tokens, targets, grad, teacher=None):
        """Losses and the parameters' gradients of the sum of grad * loss."""
        torch, c = self.torch, self.ctx
        experts, dim = self.scales.shape
        x = c.embed(self.table, tokens, scale=dim ** 0.5)
        y, mean, rstd = c.layer_norm(x)
        logits = y.float() @ self.gate.T
        chosen, share = c.gate(logits, 2, "sigmoid", self.balance, groups=2, keep=1)
        route = c.route(chosen, experts)
        rows = c.route_gather(y, route)
        place = chosen.reshape(-1)[route.order.clamp(min=0).long()].clamp(min=0).long()
        scales = self.scales[place].to(self.dtype)
        answers = rows * scales
        out = c.route_combine(answers, route, share)
        if teacher is None:
            loss, lse = c.cross_entropy(out, self.table, targets)
            d_out, d_table = c.cross_entropy_backward(grad, out, self.table, targets, lse, dtype=torch.float32)
        else:
            loss, lse, picked = c.distill(out, self.table, targets, teacher, 2.0)
            d_out, d_table = c.distill_backward(grad, out, self.table, targets, teacher, lse, picked, 2.0, dtype=torch.float32)
        d_answers, d_share = c.route_combine_backward(d_out, answers, route, share)
        d_scales = c.embed_backward((d_answers * rows).float(), place.int(), experts)
        d_logits = c.gate_backward(d_share, logits, chosen, "sigmoid")
        d_y = c.route_gather_backward(d_answers * scales, route) + (d_logits @ self.gate).to(self.dtype)
        d_gate = d_logits.T @ y.float()
        d_x = c.layer_norm_backward(d_y, x, mean, rstd)[0]
        d_table = d_table + c.embed_backward(d_x, tokens, self.table.shape[0], scale=dim ** 0.5, dtype=torch.float32)
        return loss, chosen, d_table, d_gate, d_scales

    def plain(self, tokens, targets, grad, chosen, teacher=None):
        """The same through autograd in 64 bits, for the chosen experts."""
        torch = self.torch
        table, gate, scales = (p.double().requires_grad_() for p in (self.table, self.gate, self.scales))
        dim = table.shape[1]
        x = table[tokens.long()] * dim ** 0.5
        y = torch.nn.functional.layer_norm(x, (dim,), eps=1e-5)
        s = torch.sigmoid(y @ gate.T).gather(1, chosen.long())
        share = s / s.sum(1, keepdim=True)
        out = (share.unsqueeze(-1) * scales[chosen.long()] * y.unsqueeze(1)).sum(1)
        if teacher is None:
            loss = torch.nn.functional.cross_entropy(out @ table.T, targets.long(), reduction="none")
        else:
            q = torch.log_softmax(out @ table.T / 2, 1).gather(1, targets.long())
            p = torch.softmax(teacher.double() / 2, 1)
            loss = 4 * (p * (torch.log(p) - q)).sum(1)
        (loss * grad.double()).sum().backward()
        return loss.detach(), table.grad, gate.grad, scales.grad


@pytest.mark.parametrize("kind,far", [("f32", 2e-5), ("bf16", 0.03), ("f16", 0.004)])
@pytest.mark.parametrize("taught", [False, True])
def test_a_run_of_the_verbs_together(torch, ctx, kind, far, taught):
    """Tolerances of the whole run: about ten roundings of the type one after
    the other between a parameter and its gradient (2^-8 each for bf16, 2^-11
    for fp16), which add as independent errors do; in 32 bits sums of up to 700
    terms."""
    say("run", kind, taught)
    g = gen(torch, 12)
    n, vocab, dim, experts = 700, 900, 96, 12
    m = Model(torch, ctx, vocab, dim, experts, dt(torch, kind), 5)
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda").int()
    grad = (0.5 + torch.rand(n, generator=g, device="cuda")) * (4.0 / n ** 0.5)
    if taught:
        targets = torch.stack([(tokens + k * 7) % vocab for k in range(5)], 1).int().contiguous()
        teacher = randn(torch, g, n, 5)
    else:
        targets, teacher = ((tokens.long() * 31 + 7) % vocab).int(), None
    loss, chosen, *grads = m.loss(tokens, targets, grad, teacher)
    want, *exact = m.plain(tokens, targets, grad, chosen, teacher)
    for name, a, b in zip(("loss", "table", "gate", "scales"), (loss, *grads), (want, *exact)):
        off = float((a.double() - b).norm() / b.norm())
        say("  ", name, off)
        assert off < far, (name, off)
    ctx.sync()


def test_captured_and_replayed(torch, hgb):
    """A capture holds whole calls; every replay on new inputs gives what the
    same calls give eagerly, with eager work between the replays."""
    say("capture")
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = hgb.Context(0, stream)
        g = gen(torch, 3)
        n, vocab, dim = 300, 1500, 72
        x = randn(torch, g, n, dim, dtype=torch.bfloat16)
        table = randn(torch, g, vocab, dim, dtype=torch.bfloat16, scale=0.2)
        target = torch.randint(0, vocab, (n,), generator=g, device="cuda").int()
        tokens = torch.randint(-1, vocab, (n, 9), generator=g, device="cuda").int()
        teacher, grad = randn(torch, g, n, 9), randn(torch, g, n)
        logits, bias = randn(torch, g, n, 40), randn(torch, g, 40, scale=0.1)

        def calls():
            chosen, share = c.gate(logits, 4, "softmax", bias, groups=4, keep=2)
            d = c.gate_backward(share, logits, chosen)
            loss, lse = c.cross_entropy(x, table, target)
            dx, dw = c.cross_entropy_backward(grad, x, table, target, lse)
            l2, lse2, picked = c.distill(x, table, tokens, teacher, 1.5)
            dx2, dw2 = c.distill_backward(grad, x, table, tokens, teacher, lse2, picked, 1.5, dtype=torch.float32)
            return chosen, share, d, loss, lse, dx, dw, l2, lse2, picked, dx2, dw2

        calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            held = calls()
        for turn in range(4):
            for t, scale in ((x, 1), (logits, 1), (teacher, 1), (grad, 1)):
                t.copy_(randn(torch, g, *t.shape, scale=scale))
            target.copy_(torch.randint(0, vocab, (n,), generator=g, device="cuda").int())
            graph.replay()
            got = [t.clone() for t in held]
            want = calls()
            for k, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), (turn, k)
            torch.cuda.synchronize()
        c.sync()
        c.close()


def test_two_contexts_at_once(torch, hgb):
    """Two streams' calls, in flight together, with workspaces of their own."""
    say("two contexts")
    g = gen(torch, 8)
    n, vocab, dim = 2000, 6000, 128
    x = randn(torch, g, n, dim, dtype=torch.float16)
    table = randn(torch, g, vocab, dim, dtype=torch.float16, scale=0.2)
    target = torch.randint(0, vocab, (n,), generator=g, device="cuda").int()
    logits = randn(torch, g, n, 96, dtype=torch.float16)
    grad = randn(torch, g, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    contexts = [hgb.Context(0, s) for s in streams]
    results = [[], []]
    for _ in range(5):
        for s, c, r in zip(streams, contexts, results):
            with torch.cuda.stream(s):
                chosen, share = c.gate(logits, 6)
                loss, lse = c.cross_entropy(x, table, target)
                r.append((chosen, share, loss, *c.cross_entropy_backward(grad, x, table, target, lse)))
    torch.cuda.synchronize()
    for r in results:
        for other in r:
            for a, b in zip(results[0][0], other):
                assert torch.equal(a, b)
    for c in contexts:
        c.sync()
        c.close()


@pytest.mark.parametrize("kind,out_kind,last", [("bf16", "bf16", 0), ("bf16", "f32", 0), ("f32", "f32", 0), ("bf16", "bf16", 1), ("f32", "f32", 70)])
def test_several_pieces_of_the_vocabulary(torch, ctx, kind, out_kind, last):
    """More of the logits' gradient than is held at a time: sums over the pieces, and a target in each; a last piece of few tokens."""
    size = 4 if kind == "f32" else 2
    planes = 2 if out_kind != kind else 1
    n, dim = 5000, 24
    piece = (1 << 30) // (n * size * planes) // 256 * 256
    vocab = piece + last if last else piece * 5 // 2
    say("pieces", n, vocab, dim, kind, out_kind)
    g, x, table, target = problem(torch, n, vocab, dim, kind, 0, 0, 31)
    target = (torch.rand(n, generator=g, device="cuda").double() * vocab).int()
    loss, lse = ctx.cross_entropy(x, table, target)
    grad = randn(torch, g, n)
    dx, dw = ctx.cross_entropy_backward(grad, x, table, target, lse, dtype=dt(torch, out_kind))
    ctx.sync()
    rows = torch.arange(0, n, 97, device="cuda")   # dx by rows; dtable by tokens
    xd, wd = x.double(), table.double()
    z = xd[rows] @ wd.T
    q = torch.exp(z - lse[rows].double()[:, None])
    dz = q.clone()
    dz[torch.arange(len(rows), device="cuda"), target[rows].long()] -= 1
    dz *= grad[rows].double()[:, None]
    p = Plain(torch, x[rows], table, 1.0)
    check(torch, loss[rows], p.lse - p.z.gather(1, target[rows, None].long())[:, 0], p.lse_off + p.z_off + 4 * U * p.z.abs().amax(1), "loss")
    step = half_step(torch, dt(torch, kind))[0] if kind != "f32" else 0.0
    rel, tiny = half_step(torch, dt(torch, kind))
    err = q * p.q_off[:, None] * grad[rows].abs().double()[:, None] + dz.abs() * (step * 1.001 + 2 * U)
    want = dz @ wd
    check(torch, dx[rows], want, (err @ wd.abs() + (vocab + 300) * U * (dz.abs() @ wd.abs())) * (1 + rel) + want.abs() * rel * 1.001 + tiny, "dx")
    del z, q, dz, p
    some = torch.cat([target[:40].long(), torch.arange(0, vocab, vocab // 37, device="cuda"), torch.tensor([vocab - 1], device="cuda")]).unique()
    z = xd @ wd[some].T
    q = torch.exp(z - lse.double()[:, None])
    dz = (q - (target.long()[:, None] == some).double()) * grad.double()[:, None]
    off = ((dim + 2) * U * (xd.abs() @ wd[some].abs().T)).amax() + U * (8 * z.abs().amax() + 8 * lse.abs().max() + 8)
    step2 = step if out_kind == kind else step * step
    err = q * off * grad.double().abs()[:, None] + dz.abs() * (step2 * 1.001 + 2 * U)
    rel, tiny = half_step(torch, dt(torch, out_kind))
    want = dz.T @ xd
    check(torch, dw[some], want, (err.T @ xd.abs() + (2 * n + 300) * U * (dz.abs().T @ xd.abs())) * (1 + rel) + want.abs() * rel * 1.001 + tiny, "dtable")
    assert bool(dw.isfinite().all()) and bool(dx.isfinite().all())


def test_several_pieces_of_the_rows(torch, ctx):
    """More partial sums than are held at a time, in the forward pass."""
    n, vocab, dim = 17000, 262144, 8
    say("row pieces", n, vocab, dim)
    g, x, table, target = problem(torch, n, vocab, dim, "bf16", 0, 0, 41)
    loss, lse = ctx.cross_entropy(x, table, target)
    tokens = torch.stack([target, target], 1).contiguous()
    l2, lse2, picked = ctx.distill(x, table, tokens, torch.zeros(n, 2, device="cuda"))
    ctx.sync()
    rows = torch.cat([torch.arange(0, n, 331, device="cuda"), torch.arange(16300, 16460, device="cuda"), torch.arange(n - 40, n, device="cuda")])
    p = Plain(torch, x[rows], table, 1.0)
    check(torch, lse[rows], p.lse, p.lse_off, "lse")
    z = p.z.gather(1, target[rows, None].long())[:, 0]
    check(torch, loss[rows], p.lse - z, p.lse_off + p.z_off + 4 * U * p.z.abs().amax(1), "loss")
    check(torch, picked[rows, 1], z, p.z_off + 4 * U * p.z.abs().amax(1), "picked")
    assert torch.equal(lse2, lse) and bool(loss.isfinite().all())


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_into_a_buffer_beside_the_rows(torch, ctx, kind):
    """dx into other columns of the buffer that holds x; what lies between stays."""
    g, x, table, target = problem(torch, 270, 640, 40, kind, 0, 0, 6)
    lse = ctx.cross_entropy(x, table, target)[1]
    grad = randn(torch, g, 270)
    want, dw = ctx.cross_entropy_backward(grad, x, table, target, lse)
    for shift, extra in ((40, 8), (41, 3), (48, 0)):
        buf = torch.full((270, shift + 40 + extra), 5.0, dtype=x.dtype, device="cuda")
        buf[:, :40] = x
        out = buf[:, shift:shift + 40]
        got, dw2 = ctx.cross_entropy_backward(grad, buf[:, :40], table, target, lse, out=out)
        assert got.data_ptr() == out.data_ptr() and torch.equal(out, want) and torch.equal(dw2, dw)
        assert torch.equal(buf[:, :40], x) and bool((buf[:, 40:shift] == 5).all()) and bool((buf[:, shift + 40:] == 5).all())
    with pytest.raises(Exception, match="overlaps"):
        ctx.cross_entropy_backward(grad, x, table, target, lse, out=x)


def test_gate_of_the_largest_sizes(torch, ctx):
    """All 64 slots of 1,023 experts, and a million rows of few."""
    g = gen(torch, 2)
    z = randn(torch, g, 77, 1023)
    chosen, share = ctx.gate(z, 64, "softmax", renormalise=False)
    top = z.double().topk(64, 1)
    assert torch.equal(chosen.long(), top.indices)
    want = torch.softmax(z.double(), 1).gather(1, top.indices)
    check(torch, share, want, want * SHARE, "share")
    z = randn(torch, g, 1 << 20, 5, dtype=torch.bfloat16)
    chosen, share = ctx.gate(z, 2)
    key = z.double() * 1024 - torch.arange(5, device="cuda") * 1e-6   # bf16 values, ties to the lower
    top = key.topk(2, 1).indices
    assert torch.equal(chosen.long(), top)
    ctx.sync()


@pytest.mark.parametrize("n,vocab,dim,kind", [(5, 300, 32768, "bf16"), (40, 270, 32768, "f32"), (300, 70, 20001, "f16"), (33, 4, 9999, "bf16")])
def test_the_widest_rows(torch, ctx, n, vocab, dim, kind):
    """Many steps of the logits' sum, and many tiles of the gradients' columns."""
    say("wide", n, vocab, dim, kind)
    g, x, table, target = problem(torch, n, vocab, dim, kind, 0, 0, 51)
    p = Plain(torch, x, table, 1.0)
    loss, lse = ctx.cross_entropy(x, table, target)
    check(torch, lse, p.lse, p.lse_off, "lse")
    grad = randn(torch, g, n) * (64.0 if kind == "f16" else 1.0)
    got = ctx.cross_entropy_backward(grad, x, table, target, lse)
    q = torch.exp(p.z - lse.double()[:, None])
    dz = q.clone()
    dz[torch.arange(n, device="cuda"), target.long()] -= 1
    rate = grad.double()[:, None]
    check_grads(torch, got, x, table, dz * rate, q * p.q_off[:, None] * rate.abs() + 2 * U * dz.abs() * rate.abs(), kind, kind,
                rate.abs().max(), "wide")
    ctx.sync()


def test_many_rows_of_few_tokens(torch, ctx):
    """A sum over the rows in as many shares as fill the CUs, and partial sums of one tile."""
    n, vocab, dim = 300001, 3, 33
    g, x, table, target = problem(torch, n, vocab, dim, "f32", 0, 0, 61)
    target[::7] = -1
    loss, lse = ctx.cross_entropy(x, table, target)
    p = Plain(torch, x, table, 1.0)
    check(torch, lse, p.lse, p.lse_off, "lse")
    grad = randn(torch, g, n)
    dx, dw = ctx.cross_entropy_backward(grad, x, table, target, lse)
    live = (target >= 0).double()[:, None]
    q = torch.exp(p.z - lse.double()[:, None])
    dz = (q - torch.nn.functional.one_hot(target.clamp(min=0).long(), vocab)) * grad.double()[:, None] * live
    err = q * p.q_off[:, None] * grad.double().abs()[:, None] * live + 4 * U * dz.abs()
    check(torch, dx, dz @ table.double(), err @ table.double().abs() + 40 * U * (dz.abs() @ table.double().abs()), "dx")
    # of a share: steps of 32 rows, one after the other; then the shares
    terms = n // 100 + 600
    check(torch, dw, dz.T @ x.double(), err.T @ x.double().abs() + terms * U * (dz.abs().T @ x.double().abs()), "dtable")
    ctx.sync()


@pytest.mark.parametrize("n,vocab,dim,kind,out_kind", [(1 << 24, 40, 8, "bf16", "bf16"), (1 << 23, 7, 24, "f32", "f32"), (8, 1 << 24, 8, "bf16", "f32"),
                                                       (3, 1 << 24, 12, "f32", "f32"), (300, 1 << 24, 136, "bf16", "bf16")])
def test_the_most_rows_and_tokens(torch, ctx, n, vocab, dim, kind, out_kind):
    """Rows, table and logits' gradient beyond 4 GB, against 64 bits at some rows and some tokens."""
    say("most", n, vocab, dim, kind, out_kind)
    g, x, table, target = problem(torch, n, vocab, dim, kind, 0, 0, 83)
    loss, lse = ctx.cross_entropy(x, table, target)
    grad = randn(torch, g, n)
    dx, dw = ctx.cross_entropy_backward(grad, x, table, target, lse, dtype=dt(torch, out_kind))
    ctx.sync()
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())
    step, tiny = half_step(torch, dt(torch, kind)) if kind != "f32" else (0.0, 0.0)
    step2, tiny2 = half_step(torch, dt(torch, out_kind)) if out_kind != "f32" else (0.0, 0.0)
    parts = 4 * ((vocab + 255) // 256)

    def logits(rows, tokens):
        """z, and how far 32 bits may be off."""
        xd, wd = x[rows].double(), table[tokens].double()
        return xd @ wd.T, (dim + 2) * U * (xd.abs() @ wd.abs().T)

    def rates(rows, tokens):
        """dz, and how far it may be off before its rounding."""
        z, off = logits(rows, tokens)
        q = torch.exp(z - lse[rows].double()[:, None])
        rate = grad[rows].double()[:, None]
        dz = (q - (target[rows].long()[:, None] == tokens[None]).double()) * rate
        top = z.abs().amax() + lse[rows].double().abs().amax()
        return dz, q * rate.abs() * (off + 8 * U * (top + 1)) + 2 * U * dz.abs()

    some = torch.cat([torch.arange(min(n, 3), device="cuda"), torch.arange(max(0, n - 3), n, device="cuda"),
                      torch.randint(0, n, (4,), generator=g, device="cuda")])
    sums = torch.full((len(some),), -float("inf"), dtype=torch.float64, device="cuda")
    off, top = torch.zeros_like(sums), torch.zeros_like(sums)
    want, bound = torch.zeros(len(some), dim, dtype=torch.float64, device="cuda"), torch.zeros(len(some), dim, dtype=torch.float64, device="cuda")
    for tokens in torch.arange(vocab, device="cuda").split(1 << 20):
        z, far = logits(some, tokens)
        sums = torch.logaddexp(sums, torch.logsumexp(z, 1))
        off, top = torch.maximum(off, far.amax(1)), torch.maximum(top, z.abs().amax(1))
        dz, far = rates(some, tokens)
        wd = table[tokens].double()
        want += dz @ wd
        bound += (far + (step * 1.001 + (vocab + 300) * U) * dz.abs()) @ wd.abs()
    check(torch, lse[some], sums, off + U * (128 + parts + 8 * top + 4 * sums.abs() + 8), "lse")
    check(torch, dx[some], want, bound * (1 + step) + want.abs() * step * 1.001 + tiny, "dx")

    some = torch.cat([torch.arange(min(vocab, 3), device="cuda"), torch.arange(max(0, vocab - 3), vocab, device="cuda"),
                      torch.randint(0, vocab, (4,), generator=g, device="cuda")])
    want, bound = torch.zeros(len(some), dim, dtype=torch.float64, device="cuda"), torch.zeros(len(some), dim, dtype=torch.float64, device="cuda")
    held = step if out_kind == kind else step * step
    terms = n // 100 + 600 if n > 100000 else 2 * n + 300   # many rows: more than 100 shares, then the shares
    for rows in torch.arange(n, device="cuda").split(1 << 20):
        dz, far = rates(rows, some)
        xd = x[rows].double()
        want += dz.T @ xd
        bound += (far + (held * 1.001 + terms * U) * dz.abs()).T @ xd.abs()
    check(torch, dw[some], want, bound * (1 + step2) + want.abs() * step2 * 1.001 + tiny2, "dtable")
