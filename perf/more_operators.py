"""A router with biased choices among groups of experts, and the products of sorted rows with
their experts' matrices in the activation format, with gradients, as cases to be measured.

    route              router logits -> the top-k experts by softmax or sigmoid score plus a bias
                       for balance, from the best groups only, and their weights
    route_backward     the weights' gradient -> the logits' gradient
    product            sorted rows times their expert's matrix, with bias, activation and residual
                       in the epilogue (and the values before the activation, for training)
    activation_backward  the outputs' gradient -> the gradient before the activation, and the bias'
    product_backward   that gradient -> the rows' and the matrices' gradients

`run` computes them in their plain form, or, where `own` is true, through the library.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one decode step of four sequences: a router's latency
        dict(name="route_decode", op="route", tokens=4, experts=64, top_k=8, type="bf16", score="sigmoid", bias=True,
             groups=8, kept=4, group_top=2, renorm=True, scale=2.5, masked=0.0),
        # a long prompt over many experts
        dict(name="route_prefill", op="route", tokens=16384, experts=512, top_k=10, type="f32", score="sigmoid", bias=True,
             groups=8, kept=4, group_top=2, renorm=True, scale=1.0, masked=0.0),
        # a training step's tokens (an odd number of them), sigmoid scores
        dict(name="route_backward", op="route_backward", tokens=4099, experts=128, top_k=8, type="bf16", score="sigmoid",
             bias=True, groups=4, kept=2, group_top=2, renorm=True, scale=2.5, masked=0.0),
        # a long batch, softmax over all experts: every logit has a gradient
        dict(name="route_backward_softmax", op="route_backward", tokens=16384, experts=512, top_k=10, type="f32",
             score="softmax", bias=True, groups=8, kept=3, group_top=1, renorm=False, scale=16.0, masked=0.0),
        # one new token through the first matrices of its eight experts
        dict(name="product_decode", op="product", tokens=1, experts=64, top_k=8, n=2048, k=2048, type="bf16", out="bf16",
             act="swiglu", bias=False, resid=False, pre=False),
        # 64 sequences decoding at once: a few rows for each of 128 experts
        dict(name="product_batch", op="product", tokens=64, experts=128, top_k=8, n=4096, k=1536, type="bf16", out="bf16",
             act="none", bias=True, resid=False, pre=False),
        # one matrix for all rows in 32 bits, odd sizes, the whole epilogue
        dict(name="product_odd", op="product", tokens=333, experts=1, top_k=1, n=1000, k=1040, type="f32", out="f32",
             act="gelu", bias=True, resid=True, pre=False),
        # a training step's experts: the values before the activation are kept for the gradient
        dict(name="product_train", op="product", tokens=4096, experts=64, top_k=8, n=4096, k=4096, type="bf16", out="bf16",
             act="swiglu", bias=True, resid=False, pre=True),
        # its gradient before the activation
        dict(name="activation_backward", op="activation_backward", tokens=4096, experts=64, top_k=8, n=4096, type="bf16",
             out="bf16", act="swiglu", bias=True),
        # a small batch through one matrix in 32 bits
        dict(name="activation_backward_odd", op="activation_backward", tokens=333, experts=1, top_k=1, n=1000, type="f32",
             out="f32", act="gelu", bias=True),
        # the gradients of a prompt's rows and of all experts' matrices
        dict(name="product_backward", op="product_backward", tokens=2048, experts=64, top_k=8, n=2048, k=2048, type="bf16",
             grads="both", d_w="bf16"),
        # the gradient of a router's own matrix: many rows, few columns
        dict(name="product_backward_router", op="product_backward", tokens=16384, experts=1, top_k=1, n=64, k=2048,
             type="bf16", grads="both", d_w="f32"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over the logarithm."""
    return max(low, min(high, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "product", "product", "product", "activation_backward",
                     "product_backward", "product_backward"])
    kind = rng.choice(["f32", "bf16"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, _spread(rng, 2, 16)])
        each = _spread(rng, 2, 512 // groups)
        kept = rng.randint(1, groups)
        return dict(op=op, tokens=_spread(rng, 1, 16384), experts=groups * each, top_k=rng.randint(1, min(12, kept * each)),
                    type=kind, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.7, groups=groups, kept=kept,
                    group_top=rng.choice([1, 2]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    masked=rng.choice([0.0, 0.0, 0.1]))
    kind = rng.choice(["bf16", "bf16", kind])
    experts = _spread(rng, 1, 128)
    top_k = rng.randint(1, min(experts, 8))
    act = rng.choice(["none", "relu", "gelu", "silu", "swiglu", "swiglu"])
    out = rng.choice([kind, "f32"])
    n, k = 16 * _spread(rng, 1, 256), 8 * _spread(rng, 4, 512)
    case = dict(op=op, experts=experts, top_k=top_k, n=n, type=kind)
    if op == "activation_backward":
        most = max(1, 4096 * 8 * 4096 // 2 // (top_k * n))
        return dict(case, tokens=_spread(rng, 1, min(8192, most)), out=out, act=act, bias=act == "none" or rng.random() < 0.6)
    # a product in 32 bits costs about sixteen times as much, and two gradients twice
    largest = 32768 * 4096 * 4096 // (32 if kind == "f32" else 2)
    if op == "product":
        case.update(k=k, out=out, act=act, bias=rng.random() < 0.5, resid=rng.random() < 0.5,
                    pre=act != "none" and rng.random() < 0.4)
    else:
        case.update(k=k, grads=rng.choice(["both", "both", "rows", "matrices"]), d_w=rng.choice([kind, "f32"]))
        largest //= 2
    case["experts"] = experts = max(1, min(experts, 16 * 4096 * 4096 // (n * k)))
    case["top_k"] = top_k = min(top_k, experts)
    case["tokens"] = _spread(rng, 1, max(1, min(8192, largest // (top_k * n * k))))
    return case


# ---- inputs ---------------------------------------------------------------------------


def _router(case, gen):
    """Router logits [tokens, experts]: some experts are liked more than others, some are out of
    service."""
    liked = 0.7 * torch.randn(case["experts"], generator=gen, device=DEV)
    z = torch.randn(case["tokens"], case["experts"], generator=gen, device=DEV) + liked
    if case.get("masked"):
        z[:, torch.rand(case["experts"], generator=gen, device=DEV) < case["masked"]] = float("-inf")
    return z


def _hidden(rows, cols, gen, kind=torch.float32):
    """Hidden states: unit variance, a few channels far larger than the others."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x *= 1 + 15 * (torch.rand(cols, generator=gen, device=DEV) < 0.01)
    return x.to(kind)


def _offsets(case, gen):
    """The first row of each expert, of rows sorted by expert; None for one expert."""
    if case["experts"] == 1:
        return None
    ids = _router(case, gen).topk(case["top_k"], dim=1).indices
    counts = torch.bincount(ids.reshape(-1), minlength=case["experts"])
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _groups(state, rows, experts):
    """What the plain products keep: the experts that have rows, and for each the rows it has
    (padded to the largest count with the row behind the last)."""
    offsets = state["offsets"]
    if offsets is None:
        offsets = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    counts = (offsets[1:] - offsets[:-1]).long()
    active = counts.nonzero().squeeze(1)
    at = offsets[:-1].long()[active, None] + torch.arange(int(counts.max()), device=DEV)
    state["active"], state["at"] = active, torch.where(at < offsets[1:].long()[active, None], at, rows)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, state = case["op"], {"case": case}
    kind = TYPES[case["type"]]
    if op in ("route", "route_backward"):
        state["logits"] = _router(case, gen).to(kind)
        # a bias of the size that balances the experts that are liked more
        state["bias"] = 0.1 * torch.randn(case["experts"], generator=gen, device=DEV) if case["bias"] else None
        shape = (case["tokens"], case["top_k"])
        state["ids"] = torch.empty(shape, dtype=torch.int32, device=DEV)
        state["w"] = torch.empty(shape, device=DEV)
        if op == "route_backward":
            state["d_w"] = torch.randn(shape, generator=gen, device=DEV)
            ids, w = _plain_route(state)
            state["ids"].copy_(ids)
            state["w"].copy_(w)
            state["d_logits"] = torch.empty_like(state["logits"])
        return state
    rows, experts, n = case["tokens"] * case["top_k"], case["experts"], case["n"]
    state["offsets"] = _offsets(case, gen)
    _groups(state, rows, experts)
    if op == "activation_backward":
        cols = n // 2 if case["act"] == "swiglu" else n
        state["pre"] = _hidden(rows, n, gen, kind) if case["act"] != "none" else None
        state["d_out"] = torch.randn(rows, cols, generator=gen, device=DEV).to(TYPES[case["out"]])
        state["d_pre"] = torch.empty(rows, n, dtype=kind, device=DEV)
        state["d_bias"] = torch.empty(experts, n, device=DEV) if case["bias"] else None
        return state
    k = case["k"]
    state["x"] = _hidden(rows, k, gen, kind)
    state["w"] = torch.empty(experts, n, k, dtype=kind, device=DEV)
    for e in range(experts):
        state["w"][e] = 0.02 * torch.randn(n, k, generator=gen, device=DEV)
    if op == "product":
        cols = n // 2 if case["act"] == "swiglu" else n
        out = TYPES[case["out"]]
        state["bias"] = 0.1 * torch.randn(experts, n, generator=gen, device=DEV) if case["bias"] else None
        state["resid"] = _hidden(rows, cols, gen, out) if case["resid"] else None
        state["pre"] = torch.empty(rows, n, dtype=kind, device=DEV) if case["pre"] else None
        state["out"] = torch.empty(rows, cols, dtype=out, device=DEV)
        return state
    state["d_pre"] = torch.randn(rows, n, generator=gen, device=DEV).to(kind)
    state["d_x"] = torch.empty(rows, k, dtype=kind, device=DEV) if case["grads"] != "matrices" else None
    state["d_w"] = torch.empty(experts, n, k, dtype=TYPES[case["d_w"]], device=DEV) if case["grads"] != "rows" else None
    return state


# ---- the plain forms ------------------------------------------------------------------


def _scores(logits, score):
    """Scores in 64 bits: choices that lie next to each other have to be told apart."""
    z = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(s):
    case, logits = s["case"], s["logits"]
    t, e = logits.shape
    p = _scores(logits, case["score"])
    c = p if s["bias"] is None else p + s["bias"].double()
    c = torch.where(logits == float("-inf"), float("-inf"), c)
    if case["kept"] < case["groups"]:
        each = torch.sort(c.view(t, case["groups"], -1), dim=2, descending=True).values[:, :, :case["group_top"]]
        total = torch.where(each == float("-inf"), 0, each).sum(dim=2)
        total = torch.where(each[:, :, 0] == float("-inf"), float("-inf"), total)
        best = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros(t, case["groups"], dtype=torch.bool, device=c.device).scatter(1, best, True)
        # behind every expert of a kept group, the masked ones among them
        c = torch.where(c == float("-inf"), torch.finfo(torch.float64).min, c)
        c = torch.where(keep.repeat_interleave(e // case["groups"], dim=1), c, float("-inf"))
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
    w = p.gather(1, ids)
    if case["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0)
    return ids.to(torch.int32), (case["scale"] * w).float()


def _plain_route_backward(s):
    case, ids = s["case"], s["ids"].long()
    z, w, d_w, scale = s["logits"].float(), s["w"], s["d_w"], case["scale"]
    mean = (w * d_w).sum(dim=1, keepdim=True)
    if case["score"] == "softmax" and not case["renorm"]:
        e = torch.exp(z - z.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        g = torch.zeros_like(z).scatter(1, ids, scale * d_w)
        return (p * (g - mean)).to(s["logits"].dtype)
    d = w * (d_w - mean / scale) if case["renorm"] else w * d_w
    if case["score"] == "sigmoid":
        d = d / (1 + torch.exp(z.gather(1, ids)))
    return torch.zeros_like(z).scatter(1, ids, d).to(s["logits"].dtype)


def _padded(x, at):
    """The rows of each expert, padded to the same count with zeros."""
    return torch.nn.functional.pad(x.float(), (0, 0, 0, 1))[at]


def _unpadded(y, at, rows):
    out = torch.zeros(rows + 1, y.shape[2], device=y.device)
    out[at.reshape(-1)] = y.reshape(-1, y.shape[2])
    return out[:-1]


def _activation(h, act):
    if act == "relu":
        return torch.where(h > 0, h, 0)
    if act == "gelu":
        return 0.5 * h * (1 + torch.erf(h * 0.5 ** 0.5))
    if act == "silu":
        return h / (1 + torch.exp(-h))
    if act == "swiglu":
        gate, up = h.chunk(2, dim=1)
        return gate / (1 + torch.exp(-gate)) * up
    return h


def _plain_product(s):
    case, at = s["case"], s["at"]
    rows = s["x"].shape[0]
    y = torch.bmm(_padded(s["x"], at), s["w"][s["active"]].float().transpose(1, 2).contiguous())
    if s["bias"] is not None:
        y = y + s["bias"][s["active"]][:, None, :]
    h = _unpadded(y, at, rows)
    out = _activation(h, case["act"])
    if s["resid"] is not None:
        out = out + s["resid"].float()
    out = out.to(s["out"].dtype)
    return (out, h.to(s["pre"].dtype)) if s["pre"] is not None else out


def _plain_activation_backward(s):
    case, d = s["case"], s["d_out"].float()
    act = case["act"]
    if act != "none":
        h = s["pre"].float()
        gate = h.chunk(2, dim=1)[0] if act == "swiglu" else h
        sig = 1 / (1 + torch.exp(-gate))
        if act == "relu":
            d = torch.where(h > 0, d, 0)
        elif act == "gelu":
            d = d * (0.5 * (1 + torch.erf(h * 0.5 ** 0.5)) + h * torch.exp(-0.5 * h * h) * 0.3989422804014327)
        elif act == "silu":
            d = d * sig * (1 + h * (1 - sig))
        else:
            up = h.chunk(2, dim=1)[1]
            d = torch.cat([d * up * sig * (1 + gate * (1 - sig)), d * gate * sig], dim=1)
    d_pre = d.to(s["d_pre"].dtype)
    if s["d_bias"] is None:
        return d_pre
    d_bias = torch.zeros(s["d_bias"].shape, device=d.device)
    d_bias[s["active"]] = _padded(d, s["at"]).sum(dim=1, dtype=torch.float64).float()
    return d_pre, d_bias


def _plain_product_backward(s):
    case, at, rows = s["case"], s["at"], s["x"].shape[0]
    d = _padded(s["d_pre"], at)
    out = []
    if s["d_x"] is not None:
        out.append(_unpadded(torch.bmm(d, s["w"][s["active"]].float()), at, rows).to(s["d_x"].dtype))
    if s["d_w"] is not None:
        d_w = torch.zeros(s["d_w"].shape, dtype=s["d_w"].dtype, device=d.device)
        d_w[s["active"]] = torch.bmm(d.transpose(1, 2).contiguous(), _padded(s["x"], at)).to(d_w.dtype)
        out.append(d_w)
    return tuple(out)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        from expert_slot_cache_amd import binding
        if op == "route":
            binding.route_groups(s["logits"], s["ids"], s["w"], bias=s["bias"], score=case["score"], renorm=case["renorm"],
                                 n_groups=case["groups"], kept_groups=case["kept"], group_top=case["group_top"],
                                 scale=case["scale"])
            return s["ids"], s["w"]
        if op == "route_backward":
            binding.route_groups_backward(s["logits"], s["ids"], s["w"], s["d_w"], s["d_logits"], score=case["score"],
                                          renorm=case["renorm"], scale=case["scale"])
            return s["d_logits"]
        if op == "product":
            binding.expert_product(s["x"], s["w"], s["out"], bias=s["bias"], resid=s["resid"], pre=s["pre"],
                                   act=case["act"], offsets=s["offsets"])
            return (s["out"], s["pre"]) if s["pre"] is not None else s["out"]
        if op == "activation_backward":
            binding.activation_backward(s["d_out"], s["pre"], s["d_pre"], d_bias=s["d_bias"], act=case["act"],
                                        offsets=s["offsets"])
            return (s["d_pre"], s["d_bias"]) if s["d_bias"] is not None else s["d_pre"]
        binding.expert_product_backward(s["d_pre"], s["x"], s["w"], d_x=s["d_x"], d_w=s["d_w"], offsets=s["offsets"])
        return tuple(v for v in (s["d_x"], s["d_w"]) if v is not None)
    if op == "route":
        return _plain_route(s)
    if op == "route_backward":
        return _plain_route_backward(s)
    if op == "product":
        return _plain_product(s)
    if op == "activation_backward":
        return _plain_activation_backward(s)
    return _plain_product_backward(s)


def work(case):
    op, t, e, top_k = case["op"], case["tokens"], case["experts"], case["top_k"]
    b = SIZE[case["type"]]
    if op == "route":
        return {"bytes": t * (e * b + 8 * top_k) + 4 * e * case["bias"], "flops": 6 * t * e}
    if op == "route_backward":
        dense = case["score"] == "softmax" and not case["renorm"]
        read = 12 * top_k + (e * b if dense else 0 if case["score"] == "softmax" else top_k * b)
        return {"bytes": t * (read + e * b), "flops": 6 * t * (e if dense else top_k)}
    rows, n = t * top_k, case["n"]
    if op == "activation_backward":
        cols = n // 2 if case["act"] == "swiglu" else n
        read = cols * SIZE[case["out"]] + (n * b if case["act"] != "none" else 0)
        return {"bytes": rows * (read + n * b) + 4 * e * n * case["bias"], "flops": 8 * rows * n}
    k = case["k"]
    # the experts that any row goes to (all are taken as liked alike: an upper bound of what a step reads)
    used = e * (1 - (1 - top_k / e) ** t)
    if op == "product":
        cols = n // 2 if case["act"] == "swiglu" else n
        row = k * b + cols * SIZE[case["out"]] * (2 if case["resid"] else 1) + (n * b if case["pre"] else 0)
        return {"bytes": used * n * (k * b + (4 if case["bias"] else 0)) + rows * row, "flops": 2 * rows * n * k}
    total = {"bytes": rows * n * b, "flops": 0}
    if case["grads"] != "matrices":
        total["bytes"] += used * n * k * b + rows * k * b
        total["flops"] += 2 * rows * n * k
    if case["grads"] != "rows":
        total["bytes"] += rows * k * b + e * n * k * SIZE[case["d_w"]]
        total["flops"] += 2 * rows * n * k
    return total


# ---- the definitions in 64 bits --------------------------------------------------------


def _exact_route(s):
    """Taken out one after another: the groups, then the experts, each time the first of the
    largest that are left."""
    case, z = s["case"], s["logits"].double()
    t, e = z.shape
    p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)
    c = p + s["bias"].double() if s["bias"] is not None else p.clone()
    low = torch.tensor(-1e300, dtype=torch.float64, device=DEV)      # masked; -inf: taken, or no choice
    c[z == float("-inf")] = low
    size = e // case["groups"]
    if case["groups"] > 1:
        top = min(case["group_top"], size)
        best = c.view(t, case["groups"], size).topk(top, dim=2).values
        live = best > low
        score = torch.where(live.any(dim=2), (best * live).sum(dim=2), low)
        chosen = torch.zeros(t, case["groups"], dtype=torch.bool, device=DEV)
        for _ in range(case["kept"]):
            first = _first_largest(score)
            chosen.scatter_(1, first, True)
            score = score.scatter(1, first, float("-inf"))
        c = c.masked_fill(~chosen[:, torch.arange(e, device=DEV) // size], float("-inf"))
    ids = []
    for _ in range(case["top_k"]):
        ids.append(_first_largest(c))
        c = c.scatter(1, ids[-1], float("-inf"))
    ids = torch.cat(ids, dim=1)
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return ids.to(torch.int32), case["scale"] * w


def _first_largest(c):
    """The lowest index [t, 1] of each row's largest value."""
    index = torch.arange(c.shape[1], device=c.device)
    return torch.where(c == c.amax(dim=1, keepdim=True), index, c.shape[1]).amin(dim=1, keepdim=True)


def _exact_route_backward(s):
    """By the chain rule through the scores: d score, then the scores' own gradient."""
    case, z, ids = s["case"], s["logits"].double(), s["ids"].long()
    p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)
    # what the operator is given are its weights; d score of w = scale p / sum(p) follows from them
    w, g = s["w"].double(), case["scale"] * s["d_w"].double()
    if case["renorm"]:
        # over the sum of the chosen scores, in which p / sum(p) = w / scale
        total = p.gather(1, ids).sum(dim=1, keepdim=True)
        g = (g - (w * s["d_w"].double()).sum(dim=1, keepdim=True)) / total
        g = torch.where(total > 0, g, 0)
    d_p = torch.zeros_like(p).scatter_add(1, ids, g)
    if case["score"] == "sigmoid":
        return d_p * p * (1 - p)
    return p * (d_p - (d_p * p).sum(dim=1, keepdim=True))


def _runs(s, rows, experts):
    """(expert, first row, row behind its last) of the experts that have rows."""
    ends = [0, rows] if s["offsets"] is None else s["offsets"].tolist()
    return [(g, ends[g], ends[g + 1]) for g in range(experts) if ends[g + 1] > ends[g]]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "route_backward":
        return _exact_route_backward(s)
    rows, experts, n = case["tokens"] * case["top_k"], case["experts"], case["n"]
    fn = torch.nn.functional
    if op == "product":
        out = torch.empty(s["out"].shape, dtype=torch.float64, device=DEV)
        pre = torch.empty(rows, n, dtype=torch.float64, device=DEV)
        for g, a, b in _runs(s, rows, experts):
            h = s["x"][a:b].double() @ s["w"][g].double().t()
            if s["bias"] is not None:
                h += s["bias"][g].double()
            pre[a:b] = h
            act = case["act"]
            if act == "swiglu":
                h = fn.silu(h[:, :n // 2]) * h[:, n // 2:]
            elif act != "none":
                h = {"relu": fn.relu, "gelu": fn.gelu, "silu": fn.silu}[act](h)
            out[a:b] = h if s["resid"] is None else h + s["resid"][a:b].double()
        return (out, pre) if s["pre"] is not None else out
    if op == "activation_backward":
        d, act = s["d_out"].double(), case["act"]
        if act != "none":
            h = s["pre"].double()
            normal = torch.distributions.Normal(torch.zeros((), dtype=torch.float64, device=DEV), 1.0)
            if act == "relu":
                d = d * (h > 0)
            elif act == "gelu":
                d = d * (normal.cdf(h) + h * normal.log_prob(h).exp())
            else:
                gate = h[:, :n // 2] if act == "swiglu" else h
                sig = torch.sigmoid(gate)
                slope = sig + gate * sig * torch.sigmoid(-gate)
                d = torch.cat([d * h[:, n // 2:] * slope, d * gate * sig], dim=1) if act == "swiglu" else d * slope
        if s["d_bias"] is None:
            return d
        d_bias = torch.zeros(experts, n, dtype=torch.float64, device=DEV)
        for g, a, b in _runs(s, rows, experts):
            d_bias[g] = d[a:b].sum(dim=0)
        return d, d_bias
    out = []
    if s["d_x"] is not None:
        d_x = torch.empty(rows, case["k"], dtype=torch.float64, device=DEV)
        for g, a, b in _runs(s, rows, experts):
            d_x[a:b] = s["d_pre"][a:b].double() @ s["w"][g].double()
        out.append(d_x)
    if s["d_w"] is not None:
        d_w = torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV)
        for g, a, b in _runs(s, rows, experts):
            d_w[g] = s["d_pre"][a:b].double().t().contiguous() @ s["x"][a:b].double()
        out.append(d_w)
    return tuple(out)
