"""The vector operators' cases, their plain forms and the calls of the framework's own.

Three operators over the rows and tokens of a binned matrix: the embedding of
tokens (bins, or tree leaves) and its gradient by token, the layer norm of the
embedded rows and its gradients, and the sorting of rows by expert (a tree's
leaf, say) and back with its gradients."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


def listed():
    return [
        # scoring a few rows: 28 binned features of 8 rows
        {"name": "embed 8 rows", "op": "embed", "kind": "bins", "rows": 8, "features": 28, "vocab": 7196, "dim": 64, "table": "f32", "type": "f32", "pad": False},
        # a batch of 131,072 rows of 28 features, 257 slots each, in 16 bits from the 32-bit table
        {"name": "embed 131072 rows", "op": "embed", "kind": "bins", "rows": 131072, "features": 28, "vocab": 7196, "dim": 64, "table": "f32", "type": "bf16", "pad": False},
        # its gradient: few tokens, each many times
        {"name": "embed grad 131072 rows", "op": "embed_grad", "kind": "bins", "rows": 131072, "features": 28, "vocab": 7196, "dim": 64, "table": "f32", "type": "bf16", "pad": False},
        # a large vocabulary (leaves of a whole forest), most of it absent from the batch, some tokens frequent
        {"name": "embed grad 262144 leaves", "op": "embed_grad", "kind": "ids", "rows": 16384, "features": 1, "vocab": 262144, "dim": 512, "table": "bf16", "type": "bf16", "pad": False},
        # an odd width and odd counts, with padding
        {"name": "embed grad odd", "op": "embed_grad", "kind": "ids", "rows": 5001, "features": 1, "vocab": 1023, "dim": 129, "table": "f16", "type": "f16", "pad": True},
        # a few rows of 28 features of 64 values
        {"name": "norm 8 rows", "op": "norm", "rows": 8, "dim": 1792, "type": "bf16", "weight": "f32"},
        # a batch of them
        {"name": "norm 32768 rows", "op": "norm", "rows": 32768, "dim": 1792, "type": "bf16", "weight": "f32"},
        # its backward pass
        {"name": "norm grad 32768 rows", "op": "norm_grad", "rows": 32768, "dim": 1792, "type": "bf16", "weight": "f32"},
        # an odd width in 32 bits
        {"name": "norm grad odd", "op": "norm_grad", "rows": 4099, "dim": 333, "type": "f32", "weight": "f32"},
        # a few rows to the experts of 64 leaves and back, as a server does
        {"name": "route 3 rows", "op": "route", "rows": 3, "top": 2, "experts": 64, "dim": 512, "type": "bf16", "drop": 0.0},
        # a training batch, 4 of 64 experts a row
        {"name": "route 32768 rows", "op": "route", "rows": 32768, "top": 4, "experts": 64, "dim": 1024, "type": "bf16", "drop": 0.0},
        # and its backward pass, with a tenth of the slots dropped
        {"name": "route grad 32768 rows", "op": "route_grad", "rows": 32768, "top": 4, "experts": 64, "dim": 1024, "type": "bf16", "drop": 0.1},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "route", "route_grad"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("embed", "embed_grad"):
        table = rng.choice(["f32", kind])
        bins = rng.random() < 0.5
        dim = _log(rng, 8, 1024)
        most = 234_000_000 // dim  # values of the largest listed case
        if bins:
            features = rng.randint(2, 64)
            vocab = features * rng.choice([16, 65, 255, 257])
            rows = _log(rng, 1, max(2, min(131072, most // features)))
        else:
            features = 1
            vocab = _log(rng, 2, min(262144, 134_000_000 // dim))
            rows = _log(rng, 1, min(1_000_000, most))
        return {"op": op, "kind": "bins" if bins else "ids", "rows": rows, "features": features, "vocab": vocab, "dim": dim, "table": table, "type": kind, "pad": rows > 15 and not bins and rng.random() < 0.3}
    if op in ("norm", "norm_grad"):
        dim = _log(rng, 16, 16384)
        return {"op": op, "rows": _log(rng, 1, min(131072, 58_000_000 // dim)), "dim": dim, "type": kind, "weight": rng.choice(["f32", kind])}
    dim, top = _log(rng, 16, 4096), rng.randint(1, 8)
    experts = max(top, _log(rng, 2, 512))
    rows = _log(rng, 1, min(65536, 134_000_000 // (dim * top)))
    return {"op": op, "rows": rows, "top": top, "experts": experts, "dim": dim, "type": kind, "drop": rng.choice([0.0, 0.1]) if rows > 15 else 0.0}


def _tokens(case, rand):
    n, f, v = case["rows"], case["features"], case["vocab"]
    if case["kind"] == "bins":  # token = the feature's first plus the bin; low bins are the likelier, as after binning a skewed value
        slots = v // f
        b = (rand(n, f) ** 1.5 * slots).long().clamp_(max=slots - 1)
        return (b + torch.arange(f, device=b.device) * slots).int()
    u = rand(n)  # frequent and rare tokens: the numbers' logarithm is even, so that a few make up most of a batch
    t = (torch.exp(u.double() * math.log(v + 1.0)) - 1).long().clamp_(max=v - 1)
    return ((t * 7919 + 13) % v).int() if v % 7919 else t.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    def randn(kind, *shape):
        return torch.randn(shape, generator=gen, device="cuda").to(TYPES[kind])

    op, d, s = case["op"], case["dim"], dict(case)
    if op in ("embed", "embed_grad"):
        s["tokens"] = _tokens(case, rand)
        s["scale"] = math.sqrt(d)
        s["padding"] = int(s["tokens"].reshape(-1)[0]) if case["pad"] else -1
        if op == "embed":
            s["weights"] = randn(case["table"], case["vocab"], d) * 0.02
        else:
            s["grad"] = randn(case["type"], *s["tokens"].shape, d)
    elif op in ("norm", "norm_grad"):
        n = case["rows"]
        s["x"] = (randn("f32", n, d) * (0.5 + rand(n, 1)) + randn("f32", n, 1)).to(TYPES[case["type"]])
        s["w"] = (1 + 0.1 * randn("f32", d)).to(TYPES[case["weight"]])
        s["b"] = (0.1 * randn("f32", d)).to(TYPES[case["weight"]])
        if op == "norm_grad":  # what the forward pass kept
            s["grad"] = randn(case["type"], n, d)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS).float()
    else:
        n, k, e = case["rows"], case["top"], case["experts"]
        score = rand(n, e) ** 2 + 0.5 * rand(e)  # some experts are asked for more than others
        best = score.topk(k, 1)
        s["chosen"] = best.indices.int()
        if case["drop"]:
            s["chosen"][rand(n, k) < case["drop"]] = -1
        s["share"] = torch.softmax(best.values.float() * 4, 1)
        s["answers"] = randn(case["type"], n * k, d)
        if op == "route":
            s["x"] = randn(case["type"], n, d)
        else:  # the sorted order, as the forward pass left it
            s["order"], s["position"], s["offsets"] = _sorted(s["chosen"], e)
            s["grad"] = randn(case["type"], n, d)
            s["grad_sorted"] = randn(case["type"], n * k, d)
    return s


def _sorted(chosen, experts):
    flat = chosen.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, device=flat.device))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=flat.device)
    place = torch.where(flat < 0, torch.full_like(place, -1), place)
    order = torch.where(torch.arange(order.numel(), device=flat.device) < offsets[-1], order, torch.full_like(order, -1))
    return order.int(), place.reshape(chosen.shape).int(), offsets.int()


_handle = []


def _context():
    if not _handle:
        from histogram_gradient_boosted_amd.binding import Context
        _handle.append(Context(0))
    return _handle[0]


def _run_own(s):
    c, op = _context(), s["op"]
    if op == "embed":
        return c.embed(s["weights"], s["tokens"], scale=s["scale"], pad=s["padding"], dtype=TYPES[s["type"]])
    if op == "embed_grad":
        return c.embed_backward(s["grad"], s["tokens"], s["vocab"], scale=s["scale"], pad=s["padding"], dtype=TYPES[s["table"]])
    if op == "norm":
        return c.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
    if op == "norm_grad":
        return c.layer_norm_backward(s["grad"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "route":
        r = c.route(s["chosen"], s["experts"])
        return r.order, r.position, r.offsets, c.route_gather(s["x"], r), c.route_combine(s["answers"], r, s["share"])
    from histogram_gradient_boosted_amd.binding import Route
    r = Route(s["order"], s["position"], s["offsets"])
    d_answers, d_share = c.route_combine_backward(s["grad"], s["answers"], r, s["share"])
    return d_answers, d_share, c.route_gather_backward(s["grad_sorted"], r)


def _slots(values, position):
    """Each slot's row of `values`, in 32 bits, zero where the slot is dropped."""
    live = (position >= 0).unsqueeze(-1)
    return values[position.clamp(min=0).long()].float() * live


def _spread(rows, order, top):
    """Row of slot order[j] for each place j; zero past the last."""
    live = (order >= 0).unsqueeze(-1)
    return torch.where(live, rows[order.clamp(min=0).long() // top], torch.zeros((), dtype=rows.dtype, device=rows.device))


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "embed":
        t = s["tokens"].long()
        out = s["weights"][t].float() * s["scale"]
        return torch.where((t == s["padding"]).unsqueeze(-1), torch.zeros_like(out), out).to(TYPES[s["type"]])
    if op == "embed_grad":  # long sums: 64 bits
        t, g = s["tokens"].reshape(-1).long(), s["grad"].reshape(-1, s["dim"])
        g = g.double() * (t != s["padding"]).unsqueeze(-1)
        out = torch.zeros(s["vocab"], s["dim"], dtype=torch.float64, device=g.device).index_add_(0, t, g)
        return (out * s["scale"]).to(TYPES[s["table"]])
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        c = x - mean
        rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
        return (c * rstd * s["w"].float() + s["b"].float()).to(s["x"].dtype), mean[:, 0], rstd[:, 0]
    if op == "norm_grad":
        g, h = s["grad"].float(), (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        a = g * s["w"].float()
        dx = s["rstd"][:, None] * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
        dw, db = (g * h).sum(0, dtype=torch.float64), g.sum(0, dtype=torch.float64)
        return dx.to(s["x"].dtype), dw.to(s["w"].dtype), db.to(s["w"].dtype)
    if op == "route":
        order, position, offsets = _sorted(s["chosen"], s["experts"])
        out = (_slots(s["answers"], position) * s["share"].unsqueeze(-1)).sum(1)
        return order, position, offsets, _spread(s["x"], order, s["top"]), out.to(s["x"].dtype)
    order, position, top = s["order"], s["position"], s["top"]
    g = s["grad"].float()
    share = s["share"].reshape(-1)[order.clamp(min=0).long()].unsqueeze(-1)
    d_answers = _spread(g, order, top) * share
    d_share = (_slots(s["answers"], position) * g.unsqueeze(1)).sum(-1)
    dx = _slots(s["grad_sorted"], position).sum(1)
    return d_answers.to(s["grad"].dtype), d_share, dx.to(s["grad"].dtype)


def work(case):
    op, d, n = case["op"], case["dim"], case["rows"]
    e = SIZE[case["type"]]
    if op in ("embed", "embed_grad"):
        n, v, t = n * case["features"], case["vocab"], SIZE[case["table"]]
        if op == "embed":
            return {"bytes": 4 * n + min(n, v) * d * t + n * d * e, "flops": n * d}
        return {"bytes": 4 * n + n * d * e + v * d * t, "flops": n * d}
    if op == "norm":
        return {"bytes": 2 * n * d * e + 2 * d * SIZE[case["weight"]] + 8 * n, "flops": 8 * n * d}
    if op == "norm_grad":
        return {"bytes": 3 * n * d * e + 3 * d * SIZE[case["weight"]] + 8 * n, "flops": 14 * n * d}
    k = case["top"]
    if op == "route":
        return {"bytes": 2 * n * d * e + 2 * n * k * d * e + 16 * n * k + 4 * case["experts"], "flops": 2 * n * k * d}
    return {"bytes": 2 * n * d * e + 3 * n * k * d * e + 12 * n * k, "flops": 4 * n * k * d}


def _exact_order(chosen, experts):
    """Places by counting: a slot's expert's first place, and how many slots of that expert come before it."""
    flat = chosen.reshape(-1).long()
    n = flat.numel()
    count = torch.bincount(flat + 1, minlength=experts + 1)[1:]
    first = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    first[1:] = count.cumsum(0)
    place = torch.full((n,), -1, dtype=torch.int64, device=flat.device)
    for e in range(experts):
        at = (flat == e).nonzero()[:, 0]
        place[at] = first[e] + torch.arange(at.numel(), device=flat.device)
    order = torch.full((n,), -1, dtype=torch.int64, device=flat.device)
    live = (place >= 0).nonzero()[:, 0]
    order[place[live]] = live
    return order.int(), place.reshape(chosen.shape).int(), first.int()


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["dim"]
    if op == "embed":
        t = s["tokens"].reshape(-1).long()
        out = torch.index_select(s["weights"], 0, t).double().mul_(s["scale"])
        out[t == s["padding"]] = 0
        return out.reshape(*s["tokens"].shape, d)
    if op == "embed_grad":  # running sums over the tokens in order; a token's sum is a difference of two of them
        t, g = s["tokens"].reshape(-1).long(), s["grad"].reshape(-1, d)
        keep = (t != s["padding"]).nonzero()[:, 0]
        t, g = t[keep], g[keep]
        order = torch.argsort(t)
        ends = torch.searchsorted(t[order], torch.arange(case["vocab"] + 1, device=t.device))
        out = torch.empty(case["vocab"], d, dtype=torch.float64, device=t.device)
        for c in range(0, d, 64):
            run_ = torch.zeros(t.numel() + 1, min(64, d - c), dtype=torch.float64, device=t.device)
            torch.cumsum(g[order, c:c + 64].double(), 0, out=run_[1:])
            out[:, c:c + 64] = (run_[ends[1:]] - run_[ends[:-1]]) * s["scale"]
        return out
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        return torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double()), mean, rstd
    if op == "norm_grad":  # through products with the centred rows
        g, w, r = s["grad"].double(), s["w"].double(), s["rstd"].double()[:, None]
        c = s["x"].double() - s["mean"].double()[:, None]
        along = torch.mv(g, w)[:, None] / d
        across = torch.mv(g * c, w)[:, None] * r * r / d
        return (g * w - along - c * across) * r, torch.mv((g * c).T.contiguous(), r[:, 0]), torch.mv(g.T.contiguous(), torch.ones_like(r[:, 0]))
    n, k = case["rows"], case["top"]
    if op == "route":
        order, position, offsets = _exact_order(s["chosen"], case["experts"])
        xs = torch.zeros(n * k, d, dtype=torch.float64, device=order.device)
        out = torch.zeros(n, d, dtype=torch.float64, device=order.device)
        for j in range(k):
            at = (position[:, j] >= 0).nonzero()[:, 0]
            to = position[at, j].long()
            xs[to] = s["x"][at].double()
            out[at] += s["answers"][to].double() * s["share"][at, j, None].double()
        return order, position, offsets, xs, out
    position, g = s["position"], s["grad"].double()
    d_answers = torch.zeros(n * k, d, dtype=torch.float64, device=g.device)
    d_share = torch.zeros(n, k, dtype=torch.float64, device=g.device)
    dx = torch.zeros(n, d, dtype=torch.float64, device=g.device)
    for j in range(k):
        at = (position[:, j] >= 0).nonzero()[:, 0]
        to = position[at, j].long()
        d_answers[to] = g[at] * s["share"][at, j, None].double()
        d_share[at, j] = (g[at] * s["answers"][to].double()).sum(1)
        dx[at] += s["grad_sorted"][to].double()
    return d_answers, d_share, dx
