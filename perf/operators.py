"""The operators around the experts of a mixture-of-experts layer, as cases to be measured.

    route             router logits -> the top-k experts of each token and their weights
    route_backward    the weights' gradient -> the logits' gradient
    sort              tokens -> one row per (token, expert) pair, sorted by expert, as they are
                      or rounded to e4m3 with one power-of-two scale per 128 values
    combine           the rows back to their tokens, weighted and summed (without weights it is
                      the gradient of sort)
    combine_backward  the tokens' gradient -> the rows' gradient and the weights' gradient
    product           sorted e4m3 rows times their expert's e4m3 matrix, one scale per 128 values
                      of a row and per 128 x 128 values of a matrix
    experts           both products of the experts: the first with SwiGLU and the rounding of its
                      result to e4m3 in its epilogue, the second on that result

`run` computes them in their plain form, or, where `own` is true, through the library.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
BLOCK = 128
TOP = 448.0                                   # the largest e4m3 value


def listed():
    return [
        # one decode step of four sequences: a router's latency
        dict(name="route_decode", op="route", tokens=4, experts=64, top_k=8, type="bf16", renorm=True),
        # a long prompt over many experts
        dict(name="route_prefill", op="route", tokens=16384, experts=512, top_k=10, type="f32", renorm=False),
        # a training step's tokens (an odd number of them), softmax over all experts
        dict(name="route_backward", op="route_backward", tokens=4099, experts=128, top_k=8, type="bf16", renorm=False),
        # eight sequences decoding: the pairs of a small step
        dict(name="sort_decode", op="sort", tokens=8, experts=64, top_k=8, hidden=2048, type="bf16", fp8=False, padded=0.0),
        # a prompt's tokens for 8-bit experts, an eighth of the batch being padding
        dict(name="sort_prefill", op="sort", tokens=4096, experts=128, top_k=8, hidden=4096, type="bf16", fp8=True, padded=0.125),
        # the sum over a prompt's pairs with the residual
        dict(name="combine_prefill", op="combine", tokens=4001, experts=64, top_k=8, hidden=2048, type="bf16",
             weights=True, resid=True, padded=0.0),
        # its gradient in training, ten experts to a token
        dict(name="combine_backward", op="combine_backward", tokens=2048, experts=512, top_k=10, hidden=2560, type="bf16",
             padded=0.0),
        # one new token through its eight experts: the experts' bytes once
        dict(name="experts_decode", op="experts", tokens=1, experts=64, top_k=8, hidden=2048, inter=1024),
        # a prompt of 2048 tokens through all experts
        dict(name="experts_prefill", op="experts", tokens=2048, experts=64, top_k=8, hidden=2048, inter=1024),
        # 64 sequences decoding at once: a few rows for each of 128 experts
        dict(name="product_batch", op="product", tokens=64, experts=128, top_k=8, n=4096, k=1536, out="bf16"),
        # one matrix for all rows, odd sizes (a last block of 16 values, 104 columns)
        dict(name="product_odd", op="product", tokens=333, experts=1, top_k=1, n=1000, k=1040, out="f32"),
        # training-sized: 512 rows and more for each expert
        dict(name="product_large", op="product", tokens=4096, experts=64, top_k=8, n=4096, k=4096, out="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over the logarithm."""
    return max(low, min(high, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["route", "route_backward", "sort", "combine", "combine_backward", "product", "product", "experts"])
    kind = rng.choice(["f32", "bf16"])
    experts = _spread(rng, 4, 512)
    top_k = rng.randint(1, min(experts, 12))
    if op in ("route", "route_backward"):
        return dict(op=op, tokens=_spread(rng, 1, 16384), experts=experts, top_k=top_k, type=kind, renorm=rng.random() < 0.5)
    if op in ("sort", "combine", "combine_backward"):
        hidden = _spread(rng, 64, 8192)
        fp8 = op == "sort" and rng.random() < 0.5
        if fp8 or rng.random() < 0.6:
            hidden = (hidden + 15) // 16 * 16
        most = max(1, (4096 * 8 * 2560 // 2 if kind == "f32" else 4096 * 8 * 2560) // (top_k * hidden))
        case = dict(op=op, tokens=_spread(rng, 1, min(8192, most)), experts=experts, top_k=top_k, hidden=hidden, type=kind,
                    padded=rng.choice([0.0, 0.0, 0.2]))
        if op == "sort":
            return dict(case, fp8=fp8)
        if op == "combine":
            return dict(case, weights=rng.random() < 0.7, resid=rng.random() < 0.5)
        return case
    experts = _spread(rng, 1, 128)
    top_k = rng.randint(1, min(experts, 8))
    if op == "product":
        n, k = _spread(rng, 48, 4096), 16 * _spread(rng, 4, 256)
        case = dict(op=op, experts=experts, top_k=top_k, n=n, k=k, out=rng.choice(["f32", "bf16"]))
        size = n * k
    else:
        case = dict(op=op, experts=experts, top_k=top_k, hidden=16 * _spread(rng, 8, 256), inter=128 * _spread(rng, 1, 16))
        size = 3 * case["hidden"] * case["inter"]
    case["experts"] = experts = max(1, min(experts, 64 * 4096 * 4096 // size))
    case["top_k"] = top_k = min(top_k, experts)
    case["tokens"] = _spread(rng, 1, max(1, min(4096, 32768 * 4096 * 4096 // 2 // (top_k * size))))
    return case


# ---- inputs ---------------------------------------------------------------------------


def _router(case, gen):
    """Router logits [tokens, experts]: some experts are liked more than others."""
    liked = 0.7 * torch.randn(case["experts"], generator=gen, device=DEV)
    return torch.randn(case["tokens"], case["experts"], generator=gen, device=DEV) + liked


def _ids(case, gen):
    """Expert ids [tokens, top_k], distinct in a row; -1 in the rows of padding tokens."""
    ids = _router(case, gen).topk(case["top_k"], dim=1).indices.to(torch.int32)
    if case.get("padded"):
        ids[torch.rand(case["tokens"], generator=gen, device=DEV) < case["padded"]] = -1
    return ids


def _weights(case, gen):
    return torch.softmax(torch.randn(case["tokens"], case["top_k"], generator=gen, device=DEV), dim=1)


def _hidden(rows, cols, gen, kind=torch.float32):
    """Hidden states: unit variance, a few channels far larger than the others."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x *= 1 + 15 * (torch.rand(cols, generator=gen, device=DEV) < 0.01)
    return x.to(kind)


def _matrices(experts, n, k, gen):
    """e4m3 matrices [experts, n, k] and their scales [experts, blocks of n, blocks of k]: each
    block's largest value at 448."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    codes = torch.empty(experts, n, k, dtype=F8, device=DEV)
    scales = torch.empty(experts, nb, kb, device=DEV)
    for e in range(experts):
        w = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEV)
        w[:n, :k] = 0.02 * torch.randn(n, k, generator=gen, device=DEV)
        b = w.view(nb, BLOCK, kb, BLOCK)
        scales[e] = b.abs().amax(dim=(1, 3)) / TOP
        codes[e] = (b / scales[e][:, None, :, None]).reshape(nb * BLOCK, kb * BLOCK)[:n, :k].to(F8)
    return codes, scales


def _offsets(ids, experts):
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat[flat >= 0], minlength=experts)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def _rows_of(ids, experts):
    """Where each (token, k) pair stands among the pairs sorted by expert (-1: nowhere)."""
    flat = ids.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, experts, flat), stable=True).indices
    rows = torch.empty_like(flat)
    rows[order] = torch.arange(flat.numel(), device=DEV)
    return torch.where(flat < 0, -1, rows).to(torch.int32).view(ids.shape)


def _groups(state, offsets):
    """What the plain products keep: the experts that have rows, and for each the rows it has
    (padded to the largest count with the row behind the last)."""
    counts = (offsets[1:] - offsets[:-1]).long()
    active = counts.nonzero().squeeze(1)
    most = int(counts.max())
    at = offsets[:-1].long()[active, None] + torch.arange(most, device=DEV)
    last = state["codes"].shape[0]
    state["active"], state["at"] = active, torch.where(at < offsets[1:].long()[active, None], at, last)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, state = case["op"], {"case": case}
    if op in ("route", "route_backward"):
        state["logits"] = _router(case, gen).to(TYPES[case["type"]])
        shape = (case["tokens"], case["top_k"])
        state["ids"] = torch.empty(shape, dtype=torch.int32, device=DEV)
        state["w"] = torch.empty(shape, device=DEV)
        if op == "route_backward":
            state["d_w"] = torch.randn(shape, generator=gen, device=DEV)
            ids, w = _plain_route(state["logits"], case)
            state["ids"].copy_(ids)
            state["w"].copy_(w)
            state["d_logits"] = torch.empty_like(state["logits"])
        return state
    ids = state["ids"] = _ids(case, gen)
    pairs = ids.numel()
    if op == "sort":
        state["x"] = _hidden(case["tokens"], case["hidden"], gen, TYPES[case["type"]])
        state["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device=DEV)
        state["rows"] = torch.empty_like(ids)
        state["sorted"] = torch.zeros(pairs, case["hidden"], device=DEV).to(F8 if case["fp8"] else TYPES[case["type"]])
        state["scales"] = torch.zeros(pairs, -(-case["hidden"] // BLOCK), device=DEV) if case["fp8"] else None
        return state
    if op in ("combine", "combine_backward"):
        kind = TYPES[case["type"]]
        state["rows"] = _rows_of(ids, case["experts"])
        state["ys"] = _hidden(pairs, case["hidden"], gen, kind)
        state["w"] = _weights(case, gen) if case.get("weights", True) else None
        if op == "combine":
            state["resid"] = _hidden(case["tokens"], case["hidden"], gen, kind) if case["resid"] else None
            state["out"] = torch.empty(case["tokens"], case["hidden"], dtype=kind, device=DEV)
        else:
            state["d_out"] = _hidden(case["tokens"], case["hidden"], gen, kind)
            state["d_ys"] = torch.zeros(pairs, case["hidden"], dtype=kind, device=DEV)
            state["d_w"] = torch.empty(ids.shape, device=DEV)
        return state
    offsets = state["offsets"] = _offsets(ids, case["experts"])
    k = case["k"] if op == "product" else case["hidden"]
    x = _hidden(case["tokens"], k, gen, torch.bfloat16)
    codes, scales = _plain_round(x)
    order = torch.sort(ids.reshape(-1), stable=True).indices // case["top_k"]
    state["codes"] = codes.view(torch.uint8)[order].view(F8)      # uint8: indexing has no e4m3 form
    state["scales"] = scales[order]
    if op == "product":
        state["w"], state["w_scales"] = _matrices(case["experts"], case["n"], k, gen)
        state["out"] = torch.zeros(pairs, case["n"], dtype=TYPES[case["out"]], device=DEV)
    else:
        inter = case["inter"]
        state["w13"], state["w13_scales"] = _matrices(case["experts"], 2 * inter, k, gen)
        state["w2"], state["w2_scales"] = _matrices(case["experts"], k, inter, gen)
        state["act"] = torch.zeros(pairs, inter, device=DEV).to(F8)
        state["act_scales"] = torch.zeros(pairs, inter // BLOCK, device=DEV)
        state["out"] = torch.zeros(pairs, k, dtype=torch.bfloat16, device=DEV)
    _groups(state, offsets)
    return state


# ---- the plain forms ------------------------------------------------------------------


def _softmax(logits):
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(logits, case):
    logits = logits.float()
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
    if case["renorm"]:
        return ids.to(torch.int32), _softmax(logits.gather(1, ids))
    return ids.to(torch.int32), _softmax(logits).gather(1, ids)


def _plain_route_backward(s):
    case, ids = s["case"], s["ids"].long()
    logits = s["logits"].float()
    if case["renorm"]:
        p = torch.zeros_like(logits).scatter(1, ids, s["w"])
    else:
        p = _softmax(logits)
    g = torch.zeros_like(logits).scatter(1, ids, s["d_w"])
    return (p * (g - (p * g).sum(dim=1, keepdim=True))).to(s["logits"].dtype)


def _plain_round(x):
    """x's rows as e4m3 values and scales: per 128 values the smallest power of two that brings
    the largest under 448 (1 for a block of zeros)."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    b = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    m, e = torch.frexp(b.abs().amax(dim=2))              # 448 = 0.875 * 2^9
    e = torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-126)
    scale = torch.where(m == 0, torch.ones_like(m), torch.ldexp(torch.ones_like(m), e))
    return (b / scale[:, :, None]).view(rows, blocks * BLOCK)[:, :cols].to(F8), scale


def _plain_sort(s):
    case, ids = s["case"], s["ids"]
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, case["experts"], flat)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(flat < 0, -1, place).to(torch.int32).view(ids.shape)
    counts = torch.bincount(key, minlength=case["experts"] + 1)[:case["experts"]]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    there = torch.arange(flat.numel(), device=flat.device) < offsets[-1]
    token = order // case["top_k"]
    if not case["fp8"]:
        return torch.where(there[:, None], s["x"][token], 0), offsets, rows
    codes, scales = _plain_round(s["x"])
    codes = torch.where(there[:, None], codes.view(torch.uint8)[token], 0).view(F8)
    return codes, torch.where(there[:, None], scales[token], 0), offsets, rows


def _plain_combine(s):
    rows = s["rows"].long()
    y = torch.where((rows >= 0)[:, :, None], s["ys"][rows.clamp(min=0)].float(), 0)
    if s["w"] is not None:
        y = y * s["w"][:, :, None]
    out = y.sum(dim=1)
    if s["resid"] is not None:
        out = out + s["resid"].float()
    return out.to(s["ys"].dtype)


def _plain_combine_backward(s):
    rows = s["rows"].long()
    there = rows >= 0
    d = s["d_out"].float()
    y = s["ys"][rows.clamp(min=0)].float()
    d_w = torch.where(there, (y * d[:, None, :]).sum(dim=2), 0)
    d_ys = torch.zeros(s["ys"].shape[0] + 1, s["ys"].shape[1], dtype=s["ys"].dtype, device=d.device)
    at = torch.where(there, rows, s["ys"].shape[0]).reshape(-1)
    d_ys[at] = (s["w"][:, :, None] * d[:, None, :]).to(d_ys.dtype).view(-1, d.shape[1])
    return d_ys[:-1], d_w


def _widen(codes, scales):
    """The values of e4m3 rows [..., cols] with a scale per 128 of them."""
    return codes.float() * scales.repeat_interleave(BLOCK, dim=-1)[..., :codes.shape[-1]]


def _plain_product(s, codes, scales, w, w_scales):
    """[rows, n] in 32 bits: the rows of each expert, padded to the same count, times its matrix."""
    x = torch.nn.functional.pad(_widen(codes, scales), (0, 0, 0, 1))
    m = _widen(w.view(torch.uint8)[s["active"]].view(F8),
               w_scales[s["active"]].repeat_interleave(BLOCK, dim=1)[:, :w.shape[1]])
    y = torch.bmm(x[s["at"]], m.transpose(1, 2).contiguous())
    out = torch.zeros(codes.shape[0] + 1, w.shape[1], device=codes.device)
    out[s["at"].reshape(-1)] = y.view(-1, w.shape[1])
    return out[:-1]


def _plain_experts(s):
    h = _plain_product(s, s["codes"], s["scales"], s["w13"], s["w13_scales"])
    inter = s["case"]["inter"]
    gate, up = h[:, :inter], h[:, inter:]
    codes, scales = _plain_round(gate / (1 + torch.exp(-gate)) * up)
    return _plain_product(s, codes, scales, s["w2"], s["w2_scales"]).to(torch.bfloat16)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        from expert_slot_cache_amd import binding
        if op == "route":
            binding.route(s["logits"], s["ids"], s["w"], renorm=case["renorm"])
            return s["ids"], s["w"]
        if op == "route_backward":
            binding.route_backward(s["logits"], s["ids"], s["w"], s["d_w"], s["d_logits"], renorm=case["renorm"])
            return s["d_logits"]
        if op == "sort":
            binding.sort_tokens(s["x"], s["ids"], s["sorted"], s["offsets"], s["rows"], scales=s["scales"])
            if case["fp8"]:
                return s["sorted"], s["scales"], s["offsets"], s["rows"]
            return s["sorted"], s["offsets"], s["rows"]
        if op == "combine":
            binding.combine_rows(s["ys"], s["rows"], s["out"], topk_w=s["w"], resid=s["resid"])
            return s["out"]
        if op == "combine_backward":
            binding.combine_rows_backward(s["d_out"], s["ys"], s["rows"], s["w"], s["d_ys"], s["d_w"])
            return s["d_ys"], s["d_w"]
        if op == "product":
            binding.scaled_product(s["codes"], s["scales"], s["w"], s["w_scales"], s["out"], offsets=s["offsets"])
            return s["out"]
        binding.scaled_product(s["codes"], s["scales"], s["w13"], s["w13_scales"], s["act"], offsets=s["offsets"],
                               swiglu_scales=s["act_scales"])
        binding.scaled_product(s["act"], s["act_scales"], s["w2"], s["w2_scales"], s["out"], offsets=s["offsets"])
        return s["out"]
    if op == "route":
        return _plain_route(s["logits"], case)
    if op == "route_backward":
        return _plain_route_backward(s)
    if op == "sort":
        return _plain_sort(s)
    if op == "combine":
        return _plain_combine(s)
    if op == "combine_backward":
        return _plain_combine_backward(s)
    if op == "product":
        return _plain_product(s, s["codes"], s["scales"], s["w"], s["w_scales"]).to(s["out"].dtype)
    return _plain_experts(s)


def work(case):
    op, t, e, k = case["op"], case["tokens"], case["experts"], case["top_k"]
    size = {"f32": 4, "bf16": 2}
    if op in ("route", "route_backward"):
        b = size[case["type"]]
        if op == "route":
            return {"bytes": t * (e * b + 8 * k), "flops": 4 * t * e}
        read = 12 * k if case["renorm"] else e * b + 8 * k
        return {"bytes": t * (read + e * b), "flops": 6 * t * (k if case["renorm"] else e)}
    pairs = t * k
    if op in ("sort", "combine", "combine_backward"):
        b, h = size[case["type"]], case["hidden"]
        live = pairs * (1 - case["padded"])
        if op == "sort":
            row = h + 4 * -(-h // BLOCK) if case["fp8"] else h * b
            return {"bytes": t * (1 - case["padded"]) * h * b + live * row + 8 * pairs + 4 * e, "flops": 2 * t * h if case["fp8"] else 0}
        if op == "combine":
            return {"bytes": live * h * b + t * h * b * (2 if case["resid"] else 1) + 8 * pairs, "flops": 2 * live * h}
        return {"bytes": t * h * b + 2 * live * h * b + 12 * pairs, "flops": 3 * live * h}
    # the experts that any row goes to (all are taken as liked alike: an upper bound of what a step reads)
    used = e * (1 - (1 - k / e) ** t)

    def one(n, kk, out_bytes):
        weights = used * (n * kk + 4 * -(-n // BLOCK) * -(-kk // BLOCK))
        return weights + pairs * (kk + 4 * -(-kk // BLOCK)) + pairs * out_bytes, 2 * pairs * n * kk

    if op == "product":
        b, f = one(case["n"], case["k"], case["n"] * size[case["out"]])
        return {"bytes": b, "flops": f}
    h, i = case["hidden"], case["inter"]
    b1, f1 = one(2 * i, h, i + 4 * i // BLOCK)
    b2, f2 = one(h, i, 2 * h)
    return {"bytes": b1 + b2, "flops": f1 + f2}


# ---- the definitions in 64 bits --------------------------------------------------------


def _round64(v):
    """Rows in 64 bits, each 128 values rounded to the nearest e4m3 multiple of the block's scale:
    the values, and the scales."""
    rows, cols = v.shape
    out, scales = torch.empty_like(v), []
    for at in range(0, cols, BLOCK):
        b = v[:, at:at + BLOCK]
        big = b.abs().amax(dim=1, keepdim=True)
        scale = torch.exp2(torch.ceil(torch.log2(big / TOP)))
        scale = torch.where(big > TOP * scale, 2 * scale, scale)
        scale = torch.where(big <= TOP * scale / 2, scale / 2, scale)
        scale = torch.where(big == 0, torch.ones_like(scale), scale.clamp(min=2.0 ** -126))
        u = b / scale
        binade = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(binade - 3)
        out[:, at:at + BLOCK] = torch.round(u / step) * step
        scales.append(scale)
    return out, torch.cat(scales, dim=1)


def _values64(codes, scales):
    v = codes.double()
    for j in range(scales.shape[-1]):
        v[..., BLOCK * j:BLOCK * (j + 1)] *= scales[..., j:j + 1].double()
    return v


def _product64(x, w, w_scales, offsets):
    out = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    ends = offsets.tolist()
    for e in range(w.shape[0]):
        if ends[e + 1] > ends[e]:
            m = w[e].double()
            for i in range(w_scales.shape[1]):
                for j in range(w_scales.shape[2]):
                    m[BLOCK * i:BLOCK * (i + 1), BLOCK * j:BLOCK * (j + 1)] *= w_scales[e, i, j].double()
            out[ends[e]:ends[e + 1]] = x[ends[e]:ends[e + 1]] @ m.t()
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("route", "route_backward"):
        z = s["logits"].double()
        if op == "route":
            ids = torch.sort(-z, dim=1, stable=True).indices[:, :case["top_k"]]
            total = torch.logsumexp(z.gather(1, ids) if case["renorm"] else z, dim=1, keepdim=True)
            return ids.to(torch.int32), torch.exp(z.gather(1, ids) - total)
        ids, g = s["ids"].long(), s["d_w"].double()
        if case["renorm"]:
            w = torch.softmax(z.gather(1, ids), dim=1)
            return torch.zeros_like(z).scatter(1, ids, w * (g - (w * g).sum(1, keepdim=True)))
        p = torch.softmax(z, dim=1)
        mean = (p.gather(1, ids) * g).sum(1, keepdim=True)
        return (-p * mean).scatter_add(1, ids, p.gather(1, ids) * g)
    if op == "sort":
        ids, k = s["ids"], case["top_k"]
        lists = [(ids == e).reshape(-1).nonzero().squeeze(1) for e in range(case["experts"])]
        pairs = torch.cat(lists)
        rows = torch.full_like(ids, -1)
        rows.view(-1)[pairs] = torch.arange(pairs.numel(), dtype=torch.int32, device=ids.device)
        offsets = torch.tensor([0] + [len(v) for v in lists], device=ids.device).cumsum(0).to(torch.int32)
        x = s["x"].double()
        back = (0, 0, 0, ids.numel() - pairs.numel())
        pad = torch.nn.functional.pad
        if not case["fp8"]:
            return pad(x[pairs // k], back), offsets, rows
        v, scales = _round64(x)
        return pad(v[pairs // k], back), pad(scales[pairs // k], back), offsets, rows
    if op == "combine":
        out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=DEV)
        if s["resid"] is not None:
            out += s["resid"].double()
        for j in range(case["top_k"]):
            r = s["rows"][:, j].long()
            t = (r >= 0).nonzero().squeeze(1)
            y = s["ys"][r[t]].double()
            out[t] += y if s["w"] is None else s["w"][t, j, None].double() * y
        return out
    if op == "combine_backward":
        d = s["d_out"].double()
        d_ys, d_w = torch.zeros_like(s["ys"], dtype=torch.float64), torch.zeros_like(s["w"], dtype=torch.float64)
        for j in range(case["top_k"]):
            r = s["rows"][:, j].long()
            t = (r >= 0).nonzero().squeeze(1)
            d_ys[r[t]] = s["w"][t, j, None].double() * d[t]
            d_w[t, j] = torch.linalg.vecdot(s["ys"][r[t]].double(), d[t])
        return d_ys, d_w
    x = _values64(s["codes"], s["scales"])
    if op == "product":
        return _product64(x, s["w"], s["w_scales"], s["offsets"])
    h = _product64(x, s["w13"], s["w13_scales"], s["offsets"])
    i = case["inter"]
    v, scales = _round64(torch.nn.functional.silu(h[:, :i]) * h[:, i:])
    return _product64(_values64(v, scales), s["w2"], s["w2_scales"], s["offsets"])
