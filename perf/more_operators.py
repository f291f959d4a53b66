"""Cases, plain forms and calls of the operators between the embedded rows and what a model answers.

Three operators, each with its gradient: the gate, which picks each row's
experts and their shares for the routing; the cross entropy of a row's next
token under a softmax over the whole vocabulary, straight from the rows and the
token table; and the distillation from a teacher's top logits over the same
vocabulary."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # a server's few rows to 2 of the 64 experts
        {"name": "gate 3 rows", "op": "gate", "rows": 3, "experts": 64, "top": 2, "score": "softmax", "bias": False, "groups": 1, "keep": 1, "renorm": True, "type": "bf16", "mask": 0.0},
        # a training batch: 8 of 256 experts out of 4 of 8 groups, with the bias that evens out their load
        {"name": "gate 32768 rows", "op": "gate", "rows": 32768, "experts": 256, "top": 8, "score": "sigmoid", "bias": True, "groups": 8, "keep": 4, "renorm": True, "type": "f32", "mask": 0.0},
        # the gradient of a gate whose shares are the softmax itself
        {"name": "gate grad 32768 rows", "op": "gate_grad", "rows": 32768, "experts": 64, "top": 4, "score": "softmax", "bias": False, "groups": 1, "keep": 1, "renorm": False, "type": "bf16", "mask": 0.0},
        # an odd number of experts, some masked out row by row
        {"name": "gate grad odd", "op": "gate_grad", "rows": 5001, "experts": 333, "top": 5, "score": "sigmoid", "bias": True, "groups": 3, "keep": 2, "renorm": True, "type": "f16", "mask": 0.2},
        # scoring a few rows against the bins of 28 features
        {"name": "entropy 8 rows", "op": "entropy", "rows": 8, "vocab": 7196, "dim": 64, "type": "f32", "pad": 0.0, "out": "f32"},
        # a batch's loss over a middling vocabulary
        {"name": "entropy 16384 rows", "op": "entropy", "rows": 16384, "vocab": 32768, "dim": 1024, "type": "bf16", "pad": 0.05, "out": "bf16"},
        # the gradients of a large vocabulary (leaves of a whole forest), the table's in 32 bits
        {"name": "entropy grad 262144 leaves", "op": "entropy_grad", "rows": 4096, "vocab": 262144, "dim": 512, "type": "bf16", "pad": 0.0, "out": "f32"},
        # odd counts and an odd width, with padding
        {"name": "entropy grad odd", "op": "entropy_grad", "rows": 5001, "vocab": 1023, "dim": 129, "type": "f16", "pad": 0.1, "out": "f16"},
        # a few rows against a teacher over the large vocabulary: the table is read once
        {"name": "distill 8 rows", "op": "distill", "rows": 8, "vocab": 262144, "dim": 512, "top": 20, "heat": 1.0, "type": "bf16", "pad": 0.0, "out": "bf16"},
        # a batch against a teacher's 64 best
        {"name": "distill 8192 rows", "op": "distill", "rows": 8192, "vocab": 32768, "dim": 1024, "top": 64, "heat": 2.0, "type": "bf16", "pad": 0.05, "out": "bf16"},
        # and its gradients
        {"name": "distill grad 8192 rows", "op": "distill_grad", "rows": 8192, "vocab": 32768, "dim": 1024, "top": 32, "heat": 2.0, "type": "bf16", "pad": 0.05, "out": "bf16"},
        # odd sizes in 32 bits
        {"name": "distill grad odd", "op": "distill_grad", "rows": 2047, "vocab": 7196, "dim": 257, "top": 7, "heat": 1.5, "type": "f32", "pad": 0.1, "out": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["gate", "gate_grad", "entropy", "entropy_grad", "distill", "distill_grad"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("gate", "gate_grad"):
        groups = rng.choice([1, 1, 2, 4, 7, 8])
        per = _log(rng, 2, 1023 // groups)
        keep = rng.randint(1, groups)
        return {"op": op, "rows": _log(rng, 1, 32768), "experts": groups * per, "top": rng.randint(1, min(16, keep * per)), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "keep": keep, "renorm": rng.random() < 0.6, "type": kind, "mask": rng.choice([0.0, 0.0, 0.2])}
    dim = _log(rng, 16, 2048)
    vocab = _log(rng, 2, 262144)
    rows = _log(rng, 1, max(2, min(32768, int(5.4e11 / vocab / dim), int(1.07e9 / vocab))))
    case = {"op": op, "rows": rows, "vocab": vocab, "dim": dim, "type": kind, "pad": rng.choice([0.0, 0.1]) if rows > 15 else 0.0, "out": rng.choice(["f32", kind])}
    if op in ("distill", "distill_grad"):
        case["top"], case["heat"] = rng.randint(1, min(64, vocab)), rng.choice([1.0, 2.0, 3.5])
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op, n, s, kind = case["op"], case["rows"], dict(case), TYPES[case["type"]]
    if op in ("gate", "gate_grad"):
        e, top = case["experts"], case["top"]
        s["logits"] = (1.5 * randn(n, e) + 0.7 * randn(e)).to(kind)  # some experts are liked by most rows
        if case["mask"]:
            s["logits"][rand(n, e) < case["mask"]] = float("-inf")
        s["balance"] = (0.1 if case["score"] == "sigmoid" else 0.3 / e) * randn(e) if case["bias"] else None
        if op == "gate_grad":  # what the forward pass gave
            s["chosen"] = _gate(s)[0]
            s["grad"] = randn(n, top)
        return s
    v, d = case["vocab"], case["dim"]
    s["table"] = (randn(v, d) * (2.0 / math.sqrt(d))).to(kind)
    tokens = (rand(n).double() ** 3 * v).long().clamp_(max=v - 1)  # low tokens are the likelier
    x = randn(n, d)
    x += s["table"][tokens].float() * (rand(n, 1) * 4)  # rows that have learned something of their token
    s["x"] = x.to(kind)
    s["grad"] = (0.5 + rand(n)) * ((256.0 if case["type"] == "f16" else 1.0) / n)  # a weighted mean's; 16 bits with few of them for the exponent, with the loss scaled up
    padded = rand(n) < case["pad"]
    if op in ("entropy", "entropy_grad"):
        s["tokens"] = torch.where(padded, torch.full_like(tokens, -1), tokens).int()
        if op == "entropy_grad":
            s["lse"] = _lse(_logits(s, 1.0))
        return s
    # the teacher's best tokens: the row's own and others, best first; padded rows have none, some rows fewer
    top = case["top"]
    step = max(1, v // (top + 1))
    ids = (tokens[:, None] + torch.arange(top, device="cuda") * step) % v  # distinct, as top <= vocab
    s["tokens"] = torch.where(padded[:, None] | ((torch.arange(top, device="cuda") >= top - top // 4) & (rand(n, 1) < 0.3)), torch.full_like(ids, -1), ids).int()
    s["teacher"] = (3 + 2 * randn(n, top)).sort(1, descending=True).values.to(kind)
    if op == "distill_grad":
        z = _logits(s, 1.0 / case["heat"])
        s["lse"] = _lse(z)
        s["picked"] = z.gather(1, s["tokens"].clamp(min=0).long())
    return s


_handle = []


def _context():
    if not _handle:
        from histogram_gradient_boosted_amd.binding import Context
        _handle.append(Context(0))
    return _handle[0]


def _run_own(s):
    c, op = _context(), s["op"]
    if op == "gate":
        return c.gate(s["logits"], s["top"], score=s["score"], bias=s["balance"], groups=s["groups"], keep=s["keep"], renormalise=s["renorm"], scale=1.5)
    if op == "gate_grad":
        return c.gate_backward(s["grad"], s["logits"], s["chosen"], score=s["score"], renormalise=s["renorm"], scale=1.5)
    if op == "entropy":
        return c.cross_entropy(s["x"], s["table"], s["tokens"])
    if op == "entropy_grad":
        return c.cross_entropy_backward(s["grad"], s["x"], s["table"], s["tokens"], s["lse"], dtype=TYPES[s["out"]])
    if op == "distill":
        return c.distill(s["x"], s["table"], s["tokens"], s["teacher"], temperature=s["heat"])
    return c.distill_backward(s["grad"], s["x"], s["table"], s["tokens"], s["teacher"], s["lse"], s["picked"], temperature=s["heat"], dtype=TYPES[s["out"]])


def _first(keys, count):
    """Indices of the largest along the last axis, ties to the lowest index."""
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices[..., :count]


def _scores(s):
    z = s["logits"].double()
    if s["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    m = z.max(1, keepdim=True).values
    e = torch.exp(z - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _gate(s):
    """Chosen experts and their shares. In 64 bits: which of two close keys is the larger decides."""
    n, e, groups = s["rows"], s["experts"], s["groups"]
    low = torch.full((), float("-inf"), dtype=torch.float64, device="cuda")
    score = _scores(s)
    key = score if s["balance"] is None else score + s["balance"].double()
    key = torch.where(s["logits"] == float("-inf"), low, key)  # a masked expert is never chosen
    if groups > 1:
        by = key.view(n, groups, -1)
        best = torch.sort(by, dim=-1, descending=True).values[..., :2].sum(-1)
        kept = torch.zeros(n, groups, dtype=torch.bool, device="cuda").scatter_(1, _first(best, s["keep"]), True)
        key = torch.where(kept.unsqueeze(-1), by, low).view(n, e)
    chosen = _first(key, s["top"])
    live = key.gather(1, chosen) > low
    share = score.gather(1, chosen) * live
    if s["renorm"]:
        share = share / share.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(live, chosen, torch.full_like(chosen, -1)).int(), (1.5 * share).float()


def _gate_grad(s):
    score, live = _scores(s), s["chosen"] >= 0
    at = s["chosen"].clamp(min=0).long()
    g, picked = s["grad"].double() * 1.5 * live, score.gather(1, at) * live
    if s["renorm"]:
        total = picked.sum(1, keepdim=True).clamp(min=1e-300)
        g = (g - (g * picked).sum(1, keepdim=True) / total) / total * live
    ds = torch.zeros_like(score).scatter_add_(1, at, g)
    if s["score"] == "sigmoid":
        return (ds * score * (1 - score)).to(s["logits"].dtype)
    return (score * (ds - (ds * score).sum(1, keepdim=True))).to(s["logits"].dtype)


def _logits(s, scale):
    return s["x"].float() @ s["table"].float().T * scale


def _lse(z):
    m = z.max(1, keepdim=True).values
    return m[:, 0] + torch.log(torch.exp(z - m).sum(1))


def _through(s, dz):
    """The gradients of the rows and of the table from the logits'."""
    return (dz @ s["table"].float()).to(s["x"].dtype), (dz.T @ s["x"].float()).to(TYPES[s["out"]])


def _teacher(s):
    """The teacher's probabilities at temperature `heat` over the tokens that it gives; zeros where there are none."""
    live = s["tokens"] >= 0
    t = s["teacher"].float() / s["heat"]
    t = torch.where(live, t, torch.full_like(t, float("-inf")))
    m = t.max(1, keepdim=True).values
    e = torch.exp(t - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    return live, e / e.sum(1, keepdim=True).clamp(min=1e-30)


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "gate":
        return _gate(s)
    if op == "gate_grad":
        return _gate_grad(s)
    at = s["tokens"].clamp(min=0).long()
    live = s["tokens"] >= 0
    if op == "entropy":
        z = _logits(s, 1.0)
        lse = _lse(z)
        loss = lse - z.gather(1, at[:, None])[:, 0]
        return torch.where(live, loss, torch.zeros_like(loss)), lse
    if op == "entropy_grad":
        dz = torch.exp(_logits(s, 1.0) - s["lse"][:, None])
        dz.scatter_add_(1, at[:, None], torch.full_like(dz[:, :1], -1.0))
        return _through(s, dz * torch.where(live, s["grad"], torch.zeros_like(s["grad"]))[:, None])
    heat = s["heat"]
    live, p = _teacher(s)
    some = live.any(1)
    if op == "distill":
        z = _logits(s, 1.0 / heat)
        lse, picked = _lse(z), z.gather(1, at) * live
        logp = torch.log(torch.where(p > 0, p, torch.ones_like(p)))
        loss = heat * heat * (p * (logp - picked)).sum(1) + heat * heat * lse
        return torch.where(some, loss, torch.zeros_like(loss)), lse, picked
    dz = torch.exp(_logits(s, 1.0 / heat) - s["lse"][:, None])
    dz.scatter_add_(1, at, -p)
    return _through(s, dz * torch.where(some, heat * s["grad"], torch.zeros_like(s["grad"]))[:, None])


def work(case):
    op, n, e = case["op"], case["rows"], SIZE[case["type"]]
    if op == "gate":
        return {"bytes": n * case["experts"] * e + 8 * n * case["top"], "flops": 8 * n * case["experts"]}
    if op == "gate_grad":
        return {"bytes": 2 * n * case["experts"] * e + 8 * n * case["top"], "flops": 8 * n * case["experts"]}
    v, d, k = case["vocab"], case["dim"], case.get("top", 1)
    given = (n + v) * d * e + n * k * (4 + (e if "top" in case else 0))
    if op in ("entropy", "distill"):
        return {"bytes": given + 8 * n + (4 * n * k if "top" in case else 0), "flops": 2 * n * v * d}
    return {"bytes": given + 8 * n + (4 * n * k if "top" in case else 0) + n * d * e + v * d * SIZE[case["out"]], "flops": 6 * n * v * d}


def _exact_gate(s):
    """Row by row of the keys' order: the place of each expert is the number of experts that come before it."""
    z, e, top, groups = s["logits"].double(), s["experts"], s["top"], s["groups"]
    none = torch.isinf(z)
    score = torch.sigmoid(z) if s["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
    key = score.clone()
    if s["balance"] is not None:
        key += s["balance"].double()
    key.masked_fill_(none, -math.inf)
    if groups > 1:
        size = e // groups
        worth = torch.stack([key[:, g * size:(g + 1) * size].topk(2, 1).values.sum(1) for g in range(groups)], 1)
        for g in range(groups):
            before = (worth > worth[:, g:g + 1]).sum(1) + (worth[:, :g] == worth[:, g:g + 1]).sum(1)
            key[before >= s["keep"], g * size:(g + 1) * size] = -math.inf
    chosen = torch.full((s["rows"], top), -1, dtype=torch.int64, device="cuda")
    share = torch.zeros(s["rows"], top, dtype=torch.float64, device="cuda")
    row = torch.arange(s["rows"], device="cuda")
    for k in range(top):
        best = key.amax(1)
        at = (key == best[:, None]).int().argmax(1)  # the first of the largest
        live = best > -math.inf
        chosen[:, k] = torch.where(live, at, chosen[:, k])
        share[:, k] = torch.where(live, score[row, at], share[:, k])
        key[row, at] = -math.inf
    if s["renorm"]:
        share /= share.sum(1, keepdim=True) + (share.sum(1, keepdim=True) == 0)
    return chosen.int(), 1.5 * share


def _exact_gate_grad(s):
    """Through the logarithms: d share_k = share_k (d log s_k - mean of d log s), and d log s from the logits."""
    z = s["logits"].double()
    out = torch.zeros_like(z)
    live = s["chosen"] >= 0
    at = s["chosen"].clamp(min=0).long()
    picked = torch.where(live, z.gather(1, at), torch.full((), -math.inf, dtype=z.dtype, device=z.device))
    log = torch.nn.functional.logsigmoid(picked) if s["score"] == "sigmoid" else torch.log_softmax(z, 1).gather(1, at).masked_fill(~live, -math.inf)
    w = torch.nan_to_num(torch.softmax(log, 1), nan=0.0) if s["renorm"] else torch.exp(log) * live
    a = 1.5 * s["grad"].double() * w
    if s["renorm"]:
        a = a - w * a.sum(1, keepdim=True)
    a = torch.where(live, a, torch.zeros_like(a))
    if s["score"] == "sigmoid":
        return out.scatter_add_(1, at, torch.where(live, a * torch.sigmoid(-picked), torch.zeros_like(a)))
    return out.scatter_add_(1, at, a) - torch.nan_to_num(torch.softmax(z, 1), nan=0.0) * a.sum(1, keepdim=True)


def _teacher_exact(s):
    t = torch.where(s["tokens"] < 0, torch.full((), -math.inf, dtype=torch.float64, device="cuda"), s["teacher"].double() / s["heat"])
    some = (s["tokens"] >= 0).any(1)
    log = torch.log_softmax(t, 1)
    return some, log, torch.nan_to_num(torch.exp(log), nan=0.0)


def exact(case, seed):
    s = prepare(case, seed)
    op, n = case["op"], case["rows"]
    if op == "gate":
        return _exact_gate(s)
    if op == "gate_grad":
        return _exact_gate_grad(s)
    w, x = s["table"].double(), s["x"].double()
    heat = case.get("heat", 1.0)
    forward = op in ("entropy", "distill")
    tokens = s["tokens"].long().view(n, -1)
    piece = max(1, 200_000_000 // case["vocab"])
    lse = torch.empty(n, dtype=torch.float64, device="cuda")
    picked = torch.zeros(tokens.shape, dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    if op == "distill_grad":
        some, _, p = _teacher_exact(s)
        rate = heat * s["grad"].double() * some
    elif op == "entropy_grad":
        p, rate = (tokens >= 0).double(), s["grad"].double() * (tokens[:, 0] >= 0)
    for a in range(0, n, piece):  # a piece of the rows at a time
        rows = slice(a, min(n, a + piece))
        z = torch.mm(x[rows], w.t()).div_(heat)
        if forward:
            lse[rows] = torch.logsumexp(z, 1)
            picked[rows] = torch.where(tokens[rows] >= 0, z.gather(1, tokens[rows].clamp(min=0)), picked[rows])
            continue
        q = z.sub_(s["lse"][rows].double()[:, None]).exp_()
        for k in range(tokens.shape[1]):
            q[torch.arange(q.shape[0], device="cuda"), tokens[rows, k].clamp(min=0)] -= p[rows, k]
        q *= rate[rows][:, None]
        dx[rows] = q @ w
        dw += q.t() @ x[rows]
    if op == "entropy":
        return torch.where(tokens[:, 0] >= 0, lse - picked[:, 0], torch.zeros_like(lse)), lse
    if op == "distill":
        some, log, p = _teacher_exact(s)
        terms = torch.where(p > 0, p * (log - (picked - lse[:, None])), torch.zeros_like(p))
        return torch.where(some, heat * heat * terms.sum(1), torch.zeros_like(lse)), lse, picked
    return dx, dw
