"""Cases of the grouped-product operators: rows of a dense matrix that a sparse choice sends to groups.

Four operators, each with a plain form in elementary torch operations (32 bits inside, one rounding
where an operator hands back 16-bit values) and the library's entry points:

  route     router scores -> the chosen experts of every token (ids ascending, -1 where nothing could
            be chosen), their weights, and the same choice transposed (offsets, order, position); with
            "grad" also the gradient of the logits for a given gradient of the weights
  experts   a gated expert layer for serving: up product, silu(gate) * up, down product, weighted sum
  product   one expert product in training: forward, weighted sum, and the gradients of both
  adapters  a shared projection with a low-rank adapter per request

`own` chooses the side: False the plain forms, True the calls of sparse_gemm_irregular_gb300.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NEG = float("-inf")


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of sixteen requests: a call whose latency is all that counts
        dict(name="route decode", kind="route", tokens=16, experts=64, top_k=6, score="softmax", groups=1, kept=1,
             bias=False, renormalise=True, dtype="f32", grad=False),
        # a prompt batch through a router with a balance bias and expert groups; a few padding tokens
        dict(name="route prompt groups", kind="route", tokens=16384, experts=256, top_k=8, score="sigmoid", groups=8,
             kept=4, bias=True, renormalise=True, dtype="f32", grad=False),
        # a training batch: choice and gradient, 16-bit logits, weights kept as plain softmax scores
        dict(name="route train", kind="route", tokens=65536, experts=64, top_k=6, score="softmax", groups=1, kept=1,
             bias=False, renormalise=False, dtype="bf16", grad=True),
        # decoding: one to a few tokens per expert, bound by reading the chosen experts' weights
        dict(name="experts decode", kind="experts", tokens=8, experts=64, top_k=6, dim=2048, hidden=1024, dtype="bf16"),
        # small odd sizes in half precision, experts with very different numbers of tokens
        dict(name="experts odd f16", kind="experts", tokens=1021, experts=10, top_k=3, dim=1000, hidden=712,
             dtype="f16"),
        # a prompt batch: bound by the matrix instructions
        dict(name="experts prompt", kind="experts", tokens=8192, experts=64, top_k=6, dim=2048, hidden=1024,
             dtype="bf16"),
        # a small training step on few tokens, odd counts
        dict(name="product train small", kind="product", tokens=509, experts=16, top_k=2, dim=1024, out=776,
             dtype="f16"),
        # a training step at full size: forward and both gradients
        dict(name="product train", kind="product", tokens=16384, experts=32, top_k=4, dim=2048, out=2048, dtype="bf16"),
        # decoding of 64 requests with 48 adapters between them, some requests without one
        dict(name="adapters decode", kind="adapters", tokens=64, requests=64, adapters=48, rank=16, dim=4096, out=4096,
             dtype="bf16"),
        # ragged prompts in half precision, odd sizes
        dict(name="adapters odd f16", kind="adapters", tokens=777, requests=9, adapters=5, rank=24, dim=1000, out=520,
             dtype="f16"),
        # prompts of 24 requests at once
        dict(name="adapters prompt", kind="adapters", tokens=8192, requests=24, adapters=16, rank=64, dim=4096, out=4096,
             dtype="bf16"),
    ]


def _spread(rng, lo, hi, multiple=1):
    """A size between lo and hi, even over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, max(1, round(v / multiple)) * multiple))


def draw(rng):
    biggest = {k: max(_cost(c) for c in listed() if c["kind"] == k) for k in ("route", "experts", "product", "adapters")}
    while True:
        c = _drawn(rng)
        sizes = [v for v in c.values() if isinstance(v, int)] + [2 * c.get("hidden", 0)]
        if _cost(c) <= biggest[c["kind"]] and 3072 not in sizes:
            return c


def _drawn(rng):
    kind = rng.choice(["route", "experts", "product", "adapters"])
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _spread(rng, max(2, 8 // groups), 256 // groups)
        sig = rng.random() < 0.5
        kept = rng.randint(1, groups)
        return dict(kind=kind, tokens=_spread(rng, 1, 65536), experts=experts,
                    top_k=rng.randint(1, min(8, experts * kept // groups)), score="sigmoid" if sig else "softmax",
                    groups=groups, kept=kept, bias=sig and rng.random() < 0.7, renormalise=rng.random() < 0.6,
                    dtype=rng.choice(["f32", "bf16", "f16"]), grad=rng.random() < 0.5)
    if kind == "experts":
        experts = _spread(rng, 4, 128)
        return dict(kind=kind, tokens=_spread(rng, 1, 8192), experts=experts, top_k=rng.randint(1, min(8, experts)),
                    dim=_spread(rng, 256, 4096, 8), hidden=_spread(rng, 128, 2048, 8), dtype=rng.choice(["bf16", "f16"]))
    if kind == "product":
        experts = _spread(rng, 4, 64)
        return dict(kind=kind, tokens=_spread(rng, 64, 16384), experts=experts, top_k=rng.randint(1, min(4, experts)),
                    dim=_spread(rng, 256, 4096, 8), out=_spread(rng, 256, 4096, 8), dtype=rng.choice(["bf16", "f16"]))
    tokens = _spread(rng, 1, 8192)
    return dict(kind=kind, tokens=tokens, requests=_spread(rng, 1, min(tokens, 128)), adapters=_spread(rng, 1, 64),
                rank=rng.choice([8, 16, 24, 32, 64, 128]), dim=_spread(rng, 256, 8192, 8), out=_spread(rng, 256, 8192, 8),
                dtype=rng.choice(["bf16", "f16"]))


def _touched(c):
    """Experts that at least one token is expected to choose."""
    p = torch.softmax(_popularity(c["experts"]).double(), 0)
    return float((1 - (1 - (p * c["top_k"]).clamp(max=1.0)) ** c["tokens"]).sum())


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    t, k = c["tokens"], c.get("top_k", 1)
    p = t * k
    if c["kind"] == "route":
        b = t * c["experts"] * size + p * 8 + p * 8 + 4 * (c["experts"] + 1) + (4 * c["experts"] if c["bias"] else 0)
        f = 6 * t * c["experts"]
        if c["grad"]:
            b += 2 * t * c["experts"] * size + p * 12
            f += 8 * t * c["experts"]
        return {"bytes": b, "flops": f}
    if c["kind"] == "experts":
        d, h = c["dim"], c["hidden"]
        return {"bytes": _touched(c) * 3 * h * d * size + 2 * t * d * size + 12 * p, "flops": 6 * p * d * h}
    if c["kind"] == "product":
        d, n, e = c["dim"], c["out"], c["experts"]
        # x, w, dout read; y, out, dy, dx, dw written
        b = size * (2 * t * d + 2 * e * n * d + 2 * t * n + 2 * p * n) + 24 * p
        return {"bytes": b, "flops": 6 * p * d * n + 6 * p * n}
    d, n, r = c["dim"], c["out"], c["rank"]
    g = c["adapters"] * (1 - (1 - 0.9 / c["adapters"]) ** c["requests"])  # adapters that some request uses
    return {"bytes": size * (t * d + t * n + n * d + g * r * (d + n)) + 4 * t,
            "flops": 2 * t * d * n + 1.8 * t * r * (d + n)}


def _cost(c):
    """Time that the plain form needs, roughly, in seconds."""
    w = work(c)
    return w["bytes"] / 2e12 + w["flops"] / 5e13


# ---- inputs ----------------------------------------------------------------------------------
def _popularity(experts):
    """Offsets of the router's logits: some experts are chosen several times as often as others."""
    e = torch.arange(experts, dtype=torch.float32)
    return 0.9 * torch.sin(1.7 * e + 0.3 * torch.sin(5.0 * e))


def _logits(c, g):
    t, e = c["tokens"], c["experts"]
    l = torch.randn(t, e, device="cuda", generator=g) + _popularity(e).cuda()
    if t >= 64:  # padding tokens at the end of the batch route nowhere; some tokens may not use some experts
        l[t - t // 50:] = NEG
        l[: t // 8].masked_fill_(torch.rand(t // 8, e, device="cuda", generator=g) < 0.05, NEG)
    return l


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dt)

    s = {"case": c}
    if c["kind"] == "route":
        s["logits"] = _logits(c, g).to(dt)
        # balance biases move in steps of a thousandth
        s["bias"] = torch.randint(-60, 61, (c["experts"],), device="cuda", generator=g) * 1e-3 if c["bias"] else None
        s["grad_weights"] = torch.randn(c["tokens"], c["top_k"], device="cuda", generator=g) if c["grad"] else None
        return s
    if c["kind"] == "adapters":
        t, d, n, r = c["tokens"], c["dim"], c["out"], c["rank"]
        cuts = torch.randint(0, t + 1, (c["requests"] - 1,), device="cuda", generator=g).sort().values
        if c["requests"] == t:  # decoding: a token each
            cuts = torch.arange(1, t, device="cuda")
        request = torch.searchsorted(cuts, torch.arange(t, device="cuda"), right=True)
        which = torch.randint(0, c["adapters"], (c["requests"],), device="cuda", generator=g)
        which[torch.rand(c["requests"], device="cuda", generator=g) < 0.1] = -1  # no adapter
        s["ids"] = which[request].int()
        s["x"], s["w"] = normal(t, d), normal(n, d, std=d ** -0.5)
        s["a"], s["b"] = normal(c["adapters"], r, d, std=d ** -0.5), normal(c["adapters"], n, r, std=0.1)
        s["scale"] = torch.rand(c["adapters"], device="cuda", generator=g) + 0.5
        return s
    rule = dict(top_k=c["top_k"], score="softmax", groups=1, kept=1, group_score="max", renormalise=True, scale=1.0)
    s["ids"], s["weights"] = _choose(_logits(c, g), None, rule)
    s["offsets"], s["order"], s["position"] = _transpose(s["ids"], c["experts"])
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # rows of the fullest expert
    t, d = c["tokens"], c["dim"]
    s["x"] = normal(t, d)
    if c["kind"] == "experts":
        h = c["hidden"]
        s["w_up"] = normal(c["experts"], 2 * h, d, std=d ** -0.5)
        s["w_down"] = normal(c["experts"], d, h, std=h ** -0.5)
    else:
        s["w"] = normal(c["experts"], c["out"], d, std=d ** -0.5)
        s["dout"] = normal(t, c["out"])
    return s


# ---- plain forms -----------------------------------------------------------------------------
def _scores(logits, score):
    """(usable logits, scores) in 32 bits: NaN counts as -inf, +inf as the largest finite value."""
    l = logits.float()
    l = torch.where(torch.isnan(l), NEG, l).clamp(max=torch.finfo(torch.float32).max)
    if score == "sigmoid":
        return l, 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.where(l > NEG, torch.exp(l - torch.where(top > NEG, top, 0.0)), 0.0)
    total = e.sum(1, keepdim=True)
    return l, torch.where(total > 0, e / total, 0.0)


def _choose(logits, bias, rule):
    """The chosen experts of each token (ascending, -1 where fewer can be chosen) and their weights."""
    t, experts = logits.shape
    l, s = _scores(logits, rule["score"])
    # without a bias the logits themselves are compared: both scores rise with them
    c = l if bias is None else torch.where(l > NEG, s + bias, NEG)
    if rule["kept"] < rule["groups"]:
        by = (s if bias is None and rule["group_score"] == "top2" else c).view(t, rule["groups"], -1)
        usable = (l > NEG).view(t, rule["groups"], -1)
        best = torch.where(usable, by, NEG).sort(dim=2, descending=True).values
        of = best[..., 0]
        if rule["group_score"] == "top2" and best.shape[2] > 1:
            of = of + torch.where(best[..., 1] > NEG, best[..., 1], 0.0)
        at = of.sort(dim=1, descending=True, stable=True).indices[:, : rule["kept"]]
        keep = torch.zeros(t, rule["groups"], dtype=torch.bool, device=l.device).scatter_(1, at, True)
        c = torch.where(keep[:, :, None].expand_as(by).reshape(t, experts), c, NEG)
    best, at = c.sort(dim=1, descending=True, stable=True)
    at = torch.where(best > NEG, at, experts)[:, : rule["top_k"]].sort(dim=1).values
    w = torch.where(at < experts, s.gather(1, at.clamp(max=experts - 1)), 0.0)
    if rule["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(at < experts, at, -1).int(), w * rule["scale"]


def _transpose(ids, experts):
    """Slots (token * top_k + j) in order of their expert, and where each slot went."""
    flat = ids.reshape(-1).long()
    key, order = torch.where(flat < 0, experts, flat).sort(stable=True)
    offsets = (key[None, :] < torch.arange(experts + 1, device=ids.device)[:, None]).sum(1)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=ids.device)
    return (offsets.int(), torch.where(key < experts, order, -1).int(),
            torch.where(flat < 0, -1, position).int().view(ids.shape))


def _route_grad(logits, ids, rule, grad):
    _, s = _scores(logits, rule["score"])
    at, there = ids.clamp(min=0).long(), ids >= 0
    ds = torch.where(there, grad * rule["scale"], 0.0)
    if rule["renormalise"]:
        chosen = torch.where(there, s.gather(1, at), 0.0)
        total = chosen.sum(1, keepdim=True)
        share = torch.where(total > 0, chosen / total, 0.0)
        ds = torch.where(there & (total > 0), (ds - (ds * share).sum(1, keepdim=True)) / total, 0.0)
    full = torch.zeros_like(s).scatter_add_(1, at, ds)
    if rule["score"] == "sigmoid":
        return (full * s * (1.0 - s)).to(logits.dtype)
    return (s * (full - (full * s).sum(1, keepdim=True))).to(logits.dtype)


def _padded(s):
    """(experts, most) row positions in expert order, and which of them are there."""
    first, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = first + torch.arange(max(1, s["most"]), device=first.device)
    return at, at < end


def _rows(v, at, there):
    return torch.where(there[..., None], v.float()[torch.where(there, at, 0)], 0.0)


def _unpad(v, at, there, rows):
    out = torch.zeros(rows + 1, v.shape[-1], device=v.device, dtype=torch.float32)
    out[torch.where(there, at, rows)] = v
    return out[:rows]


def _weighted(y, position, weights):
    there = position >= 0
    rows = y.float()[position.clamp(min=0).long()]
    return torch.where(there[..., None], rows * weights[..., None], 0.0).sum(1)


def _plain_experts(s):
    k, hidden = s["case"]["top_k"], s["case"]["hidden"]
    at, there = _padded(s)
    token = s["order"].long()[torch.where(there, at, 0)] // k
    up = torch.matmul(_rows(s["x"], token, there), s["w_up"].float().transpose(1, 2))
    gate, up = up[..., :hidden], up[..., hidden:]
    y = torch.matmul(gate / (1.0 + torch.exp(-gate)) * up, s["w_down"].float().transpose(1, 2))
    y = _unpad(y, at, there, s["order"].numel())
    return _weighted(y, s["position"], s["weights"]).to(s["x"].dtype)


def _plain_product(s):
    c, x, w = s["case"], s["x"], s["w"]
    k, rows = c["top_k"], s["order"].numel()
    at, there = _padded(s)
    token = s["order"].long()[torch.where(there, at, 0)] // k
    xp = _rows(x, token, there)
    y = _unpad(torch.matmul(xp, w.float().transpose(1, 2)), at, there, rows).to(x.dtype)
    out = _weighted(y, s["position"], s["weights"]).to(x.dtype)
    # gradients of the weighted sum
    slot, real = s["order"].clamp(min=0).long(), s["order"] >= 0
    dslot = s["dout"].float()[slot // k]
    dy = torch.where(real[:, None], dslot * s["weights"].reshape(-1)[slot][:, None], 0.0).to(x.dtype)
    dots = torch.where(real, (dslot * y.float()).sum(1), 0.0)
    dweights = torch.where(s["position"] >= 0, dots[s["position"].clamp(min=0).long()], 0.0)
    # gradients of the product
    dyp = _rows(dy, at, there)
    dw = torch.matmul(dyp.transpose(1, 2), xp).to(w.dtype)
    dx = _unpad(torch.matmul(dyp, w.float()), at, there, rows)
    dx = _weighted(dx, s["position"], torch.ones_like(s["weights"])).to(x.dtype)
    return {"y": y, "out": out, "dy": dy, "dweights": dweights, "dx": dx, "dw": dw}


def _plain_adapters(s):
    c, x = s["case"], s["x"].float()
    t, g, r = c["tokens"], c["adapters"], c["rank"]
    mine = (s["ids"][:, None] == torch.arange(g, device=x.device)).float() * s["scale"]
    v = torch.matmul(x, s["a"].float().view(g * r, -1).t()).view(t, g, r) * mine[:, :, None]
    y = torch.matmul(x, s["w"].float().t()) + torch.matmul(
        v.view(t, g * r), s["b"].float().transpose(1, 2).reshape(g * r, -1))
    return y.to(s["x"].dtype)


def _rule(c):
    return dict(top_k=c["top_k"], score=c["score"], groups=c["groups"], kept=c["kept"],
                group_score="top2" if c["bias"] else "max", renormalise=c["renormalise"],
                scale=2.5 if c["score"] == "sigmoid" else 1.0)


def _plain(s):
    c = s["case"]
    if c["kind"] == "route":
        rule = _rule(c)
        ids, weights = _choose(s["logits"], s["bias"], rule)
        offsets, order, position = _transpose(ids, c["experts"])
        out = {"ids": ids, "weights": weights, "offsets": offsets, "order": order, "position": position}
        if c["grad"]:
            out["dlogits"] = _route_grad(s["logits"], ids, rule, s["grad_weights"])
        return out
    return {"experts": _plain_experts, "product": _plain_product, "adapters": _plain_adapters}[c["kind"]](s)


# ---- the library's operators -----------------------------------------------------------------
def _library(s):
    import sparse_gemm_irregular_gb300 as sg
    c = s["case"]
    if c["kind"] == "route":
        rule = _rule(c)
        r = sg.route(s["logits"], rule["top_k"], bias=s["bias"], score=rule["score"], groups=rule["groups"],
                     groups_kept=rule["kept"], group_score=rule["group_score"], renormalise=rule["renormalise"],
                     scale=rule["scale"])
        out = {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order, "position": r.position}
        if c["grad"]:
            out["dlogits"] = sg.route_backward(s["logits"], r, s["grad_weights"])
        return out
    if c["kind"] == "adapters":
        return sg.adapted_product(s["x"], s["w"], s["a"], s["b"], s["ids"], s["scale"])
    r = sg.Routing(ids=s["ids"], weights=s["weights"], offsets=s["offsets"], order=s["order"], position=s["position"])
    if c["kind"] == "experts":
        return sg.experts(s["x"], s["w_up"], s["w_down"], r)
    y = sg.expert_product(s["x"], s["w"], r)
    out = sg.combine(y, r)
    dy, dweights = sg.combine_backward(s["dout"], y, r)
    dx, dw = sg.expert_product_backward(dy, s["x"], s["w"], r)
    return {"y": y, "out": out, "dy": dy, "dweights": dweights, "dx": dx, "dw": dw}


def run(state):
    return _library(state) if own else _plain(state)


# ---- the definitions in 64 bits --------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["kind"] == "route":
        return _exact_route(s)
    if c["kind"] == "adapters":
        x = s["x"].double()
        y = x @ s["w"].double().t()
        for i in range(c["adapters"]):
            mine = (s["ids"] == i).nonzero()[:, 0]
            v = x[mine] @ s["a"][i].double().t() * s["scale"][i].double()
            y[mine] += v @ s["b"][i].double().t()
        return y
    token_of = lambda e: (s["ids"] == e).nonzero()  # noqa: E731  rows (token, j) of one expert, by token
    x, weights, ids = s["x"].double(), s["weights"].double(), s["ids"]
    if c["kind"] == "experts":
        out, h = torch.zeros_like(x), c["hidden"]
        for e in range(c["experts"]):
            at = token_of(e)
            up = x[at[:, 0]] @ s["w_up"][e].double().t()
            mid = torch.nn.functional.silu(up[:, :h]) * up[:, h:]
            out.index_add_(0, at[:, 0], (mid @ s["w_down"][e].double().t()) * weights[at[:, 0], at[:, 1], None])
        return out
    dout, n, rows = s["dout"].double(), c["out"], ids.numel()
    y, dy = (torch.zeros(rows, n, dtype=torch.float64, device="cuda") for _ in range(2))
    out, dx = torch.zeros(c["tokens"], n, dtype=torch.float64, device="cuda"), torch.zeros_like(x)
    dw, dweights = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda"), torch.zeros_like(weights)
    begin = 0
    for e in range(c["experts"]):
        at = token_of(e)
        tok, j, w = at[:, 0], at[:, 1], s["w"][e].double()
        ye = x[tok] @ w.t()
        de = dout[tok] * weights[tok, j, None]
        y[begin: begin + len(at)], dy[begin: begin + len(at)] = ye, de
        out.index_add_(0, tok, ye * weights[tok, j, None])
        dweights[tok, j] = (dout[tok] * ye).sum(1)
        dx.index_add_(0, tok, de @ w)
        dw[e] = de.t() @ x[tok]
        begin += len(at)
    return {"y": y, "out": out, "dy": dy, "dweights": dweights, "dx": dx, "dw": dw}


def _exact_route(s):
    """Weights and gradient in 64 bits of the experts that the definition's 32-bit comparison chooses."""
    c, rule = s["case"], _rule(s["case"])
    ids = _choose(s["logits"], s["bias"], rule)[0].long()  # whole numbers: the choice itself is not rounded
    l = torch.nan_to_num(s["logits"].double(), nan=NEG, neginf=NEG).requires_grad_(c["grad"])
    none = (l == NEG).all(1, keepdim=True)
    safe = torch.where(none, 0.0, l)
    p = torch.sigmoid(safe) if c["score"] == "sigmoid" else torch.softmax(safe, 1)
    w = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
    if c["renormalise"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    w = w * rule["scale"]
    out = {"ids": None, "weights": w.detach(), "offsets": None, "order": None, "position": None}
    if c["grad"]:
        w.backward(s["grad_weights"].double())
        out["dlogits"] = torch.nan_to_num(l.grad, nan=0.0)
    return out
