"""The mixture-of-experts operators and the products with few rows, as cases to run and to compare.

* route: a router's scores to each token's experts and their weights, and the gradient of the scores;
* dispatch: (token, expert) pairs sorted by expert, and the tokens' rows carried there, plain or packed in FP4;
* combine: the experts' rows back to their tokens, weighted and summed, and the gradients of rows and weights;
* matvec: products of a few rows in 16 or 32 bits with 4-bit weights, one matrix or each row's own experts.

``own`` chooses between the framework's kernels and a plain form of elementary torch operations, in 32 bits except for
the choice of experts, whose scores may lie next to one another, in 64.
"""
import math

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
FLT_MIN = 1.17549435e-38


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _route(name, tokens, experts, top_k, *, score="softmax", bias=False, groups=1, top_groups=1, best=1,
           renormalize=True, scale=1.0, dtype="bf16", backward=False):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "score": score,
            "bias": bias, "groups": groups, "top_groups": top_groups, "best": best, "renormalize": renormalize,
            "scale": scale, "dtype": dtype, "backward": backward}


def _dispatch(name, tokens, experts, top_k, width, *, rows="bf16", dropped=False):
    return {"name": name, "op": "dispatch", "tokens": tokens, "experts": experts, "top_k": top_k, "width": width,
            "rows": rows, "dropped": dropped}


def _combine(name, tokens, experts, top_k, width, *, dtype="bf16", grouped=True, dropped=False, backward=False):
    return {"name": name, "op": "combine", "tokens": tokens, "experts": experts, "top_k": top_k, "width": width,
            "dtype": dtype, "grouped": grouped, "dropped": dropped, "backward": backward}


def _matvec(name, fmt, tokens, n, k, *, experts=0, top_k=1, spread=True, dtype="bf16", dropped=False):
    """experts 0: one matrix. spread: a token's row goes to all its experts, else each pair has a row of its own."""
    return {"name": name, "op": "matvec", "fmt": fmt, "tokens": tokens, "n": n, "k": k, "experts": experts,
            "top_k": top_k, "spread": spread, "dtype": dtype, "dropped": dropped}


def listed():
    return [
        # one interactive user's next token: nothing but latency
        _route("route_1x32", 1, 32, 4),
        # a long prompt over many experts: sigmoid scores with a balancing bias, limited to four of eight groups
        _route("route_16384x256", 16384, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, best=2, scale=2.5,
               dtype="f32"),
        # the training step of a softmax router with plain weights
        _route("route_backward_16384x160", 16384, 160, 6, renormalize=False, dtype="f32", backward=True),
        # a serving batch's next tokens, quantized once and carried to their experts packed
        _dispatch("dispatch_32x4_packed", 32, 32, 4, 2880, rows="mxfp4"),
        # a prompt on a GPU that holds part of the experts: the others' pairs are left out
        _dispatch("dispatch_4096x4", 4096, 32, 4, 2880, dropped=True),
        # a serving batch's results, in the order of its pairs
        _combine("combine_32x4", 32, 32, 4, 2880, grouped=False),
        # a prompt's results from the grouped product
        _combine("combine_4096x4", 4096, 32, 4, 2880),
        # a training step in fp32, odd width
        _combine("combine_backward_2048x8_f32", 2048, 64, 8, 1001, dtype="f32", backward=True),
        # one token through a linear layer
        _matvec("matvec_1x4096x4096", "nvfp4", 1, 4096, 4096),
        # a small serving batch through a large one
        _matvec("matvec_16x8192x8192", "mxfp4", 16, 8192, 8192),
        # one token through the first product of its four experts
        _matvec("experts_1x4_5760x2880", "mxfp4", 1, 5760, 2880, experts=32, top_k=4),
        # a serving batch through the second product of its experts, fp32 rows of their own
        _matvec("experts_32x4_2880x2880_f32", "nvfp4", 32, 2880, 2880, experts=32, top_k=4, spread=False, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_route(rng):
    E = rng.choice((8, 16, 32, 60, 64, 96, 128, 160, 256, 384, 512))
    groups = rng.choice([g for g in (1, 1, 1, 2, 4, 8) if E % g == 0])
    top_groups = rng.randint(1, groups)
    score = rng.choice(("softmax", "sigmoid"))
    k = min(rng.choice((1, 2, 4, 6, 8, 8, 10)), E // groups * top_groups)
    case = _route("", _log(rng, 1, 16384), E, k, score=score, bias=rng.random() < 0.5, groups=groups,
                  top_groups=top_groups, best=rng.choice((1, 2)) if E // groups > 1 else 1,
                  renormalize=rng.random() < 0.6, scale=rng.choice((1.0, 1.0, 2.5)),
                  dtype=rng.choice(("bf16", "f32")), backward=rng.random() < 0.3)
    case["tokens"] = max(1, min(case["tokens"], 16384 * 256 // E))
    return case


def _draw_pairs(rng):
    E = rng.choice((4, 8, 16, 32, 60, 64, 128, 256))
    T, k = _log(rng, 1, 8192), rng.choice((1, 2, 3, 4, 6, 8))
    k = min(k, E)
    width = rng.choice((_log(rng, 1, 160) * 32, _log(rng, 32, 2880)))
    while T * k * width > 4096 * 4 * 2880:
        T = max(1, T // 2 + rng.randrange(3))
    return T, E, k, width


def _draw_matvec(rng):
    fmt, dtype = rng.choice(("mxfp4", "nvfp4")), "f32" if rng.random() < 0.2 else "bf16"
    blk = BLOCK[fmt]
    if rng.random() < 0.5:
        case = _matvec("", fmt, _log(rng, 1, 48), _log(rng, 16, 16384), blk * _log(rng, 1, 8192 // blk), dtype=dtype)
        while case["n"] * case["k"] * (2 if case["tokens"] > 16 else 1) > 8192 * 8192:
            case["n"] = case["n"] * 2 // 3
        return case
    E = rng.choice((4, 8, 16, 32, 64))
    T, k = _log(rng, 1, 48), min(rng.choice((1, 2, 4, 4, 8)), E)
    case = _matvec("", fmt, T, _log(rng, 64, 6000), blk * _log(rng, 1, 4096 // blk), experts=E, top_k=k,
                   spread=rng.random() < 0.5, dtype=dtype, dropped=rng.random() < 0.2)
    while E * case["n"] * case["k"] > 32 * 2880 * 2880:
        case["n"] = case["n"] * 2 // 3
    return case


def draw(rng):
    kind = rng.choice(("route", "dispatch", "combine", "matvec", "matvec"))
    if kind == "route":
        case = _draw_route(rng)
    elif kind == "matvec":
        case = _draw_matvec(rng)
    else:
        T, E, k, width = _draw_pairs(rng)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        if dtype == "f32":
            T = -(-T // 2)
        dropped = rng.random() < 0.3
        if kind == "combine":
            case = _combine("", T, E, k, width, dtype=dtype, grouped=dropped or rng.random() < 0.7, dropped=dropped,
                            backward=rng.random() < 0.4)
        else:
            rows = rng.choice(("plain", "mxfp4", "nvfp4"))
            if rows == "plain":
                rows = dtype
            else:
                T, width = -(-T // 2), max(32, width // 32 * 32)
            case = _dispatch("", T, E, k, width, rows=rows, dropped=dropped)
    del case["name"]
    return case


def work(case):
    T = case["tokens"]
    if case["op"] == "route":
        E, k, size = case["experts"], case["top_k"], SIZE[case["dtype"]]
        if case["backward"]:
            return {"bytes": 2 * T * E * size + 8 * T * k, "flops": 8 * T * E}
        return {"bytes": T * E * size + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
    if case["op"] == "dispatch":
        k, H = case["top_k"], case["width"]
        if case["rows"] in SIZE:
            moved = SIZE[case["rows"]] * T * H * (1 + k)
        else:  # packed rows in and out, read again, and their values in fp32
            moved = T * (H // 2 + H // BLOCK[case["rows"]]) * (1 + 2 * k) + 4 * T * k * H
        return {"bytes": moved + 12 * T * k + 4 * case["experts"], "flops": T * k * H}
    if case["op"] == "combine":
        k, H, size = case["top_k"], case["width"], SIZE[case["dtype"]]
        if case["backward"]:
            return {"bytes": T * H * size * (1 + 2 * k) + 12 * T * k, "flops": 3 * T * k * H}
        return {"bytes": T * H * size * (1 + k) + 8 * T * k, "flops": 2 * T * k * H}
    N, K, E, k = case["n"], case["k"], case["experts"], case["top_k"]
    matrices = E * (1.0 - (1.0 - k / E) ** T) if E else 1.0  # as many experts as T tokens meet
    pairs, size = T * k, SIZE[case["dtype"]]
    moved = matrices * N * (K // 2 + K // BLOCK[case["fmt"]]) + (T if case["spread"] else pairs) * K * size
    return {"bytes": int(moved + pairs * N * size), "flops": 2 * pairs * N * K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _logits(g, T, E, dt):
    """A router's outputs: some experts are liked better than others."""
    return (1.3 * torch.randn(T, E, generator=g, device="cuda")
            + 0.5 * torch.randn(E, generator=g, device="cuda")).to(dt)


def _ids(g, case):
    """Each token's experts, and -1 for those that another GPU holds."""
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    ids = _logits(g, T, E, torch.float32).argsort(-1, descending=True)[:, :k].to(torch.int32)
    if case["dropped"]:
        ids = torch.where(ids < E - E // 4, ids, torch.full_like(ids, -1))
    return ids.contiguous()


def _weights(g, T, k):
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05
    return w / w.sum(-1, keepdim=True)


def _nearest_code(q):
    """Nearest of {0, 0.5, 1, 1.5, 2, 3, 4, 6} to |q|, ties to the even code, with the sign in bit 3."""
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code | (torch.signbit(q).to(torch.uint8) << 3)


def _quantized(x, fmt):
    """x [R, C] fp32 -> packed codes, scale bytes and (NVFP4) the tensor scale, rows on whole lines."""
    blocks = x.unflatten(-1, (-1, BLOCK[fmt]))
    amax = blocks.abs().amax(-1)
    ts = None
    if fmt == "mxfp4":
        byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)  # 2^e with e = floor(log2 amax) - 2, held as e + 127
        q = torch.ldexp(blocks, (127 - byte)[..., None])
    else:
        ts = (x.abs().amax() / 2688.0).reshape(1)
        s = (amax * (1.0 / (6.0 * ts))).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte = s.view(torch.uint8)
        eff = s.float() * ts
        q = blocks * torch.where(eff >= FLT_MIN, 1.0 / eff, torch.zeros_like(eff))[..., None]
    code = _nearest_code(q).flatten(-2)
    rows, half, blocks_n = x.shape[0], x.shape[1] // 2, byte.shape[1]
    codes = torch.zeros(rows, -(-half // 128) * 128, dtype=torch.uint8, device="cuda")[:, :half]
    scales = torch.zeros(rows, -(-blocks_n // 16) * 16, dtype=torch.uint8, device="cuda")[:, :blocks_n]
    codes.copy_(code[:, 0::2] | (code[:, 1::2] << 4))
    scales.copy_(byte)
    return codes, scales, ts


def _prepare_matvec(case, seed):
    g = _generator(seed)
    T, N, K, E, k, fmt = (case[n] for n in ("tokens", "n", "k", "experts", "top_k", "fmt"))
    state = {"case": case, "ids": None}
    rows = T
    if E:
        state["ids"] = _ids(g, case)
        rows = T if case["spread"] else T * k
    x = torch.randn(rows, K, generator=g, device="cuda")
    x[:, torch.rand(K, generator=g, device="cuda") < 0.01] *= 20.0  # a few channels are large, as activations are
    state["x"] = x.to(DTYPE[case["dtype"]])
    count = max(E, 1)
    half, blocks = K // 2, K // BLOCK[fmt]
    codes = torch.zeros(count, N, -(-half // 128) * 128, dtype=torch.uint8, device="cuda")[:, :, :half]
    scales = torch.zeros(count, N, -(-blocks // 16) * 16, dtype=torch.uint8, device="cuda")[:, :, :blocks]
    ts = torch.ones(count, device="cuda") if fmt == "nvfp4" else None
    for e in range(count):
        c, s, t = _quantized(0.02 * torch.randn(N, K, generator=g, device="cuda"), fmt)
        codes[e].copy_(c)
        scales[e].copy_(s)
        if t is not None:
            ts[e:e + 1] = t
    if not E:
        codes, scales = codes[0], scales[0]
    return state | {"codes": codes, "scales": scales, "tensor_scale": ts}


def prepare(case, seed):
    if case["op"] == "matvec":
        return _prepare_matvec(case, seed)
    g = _generator(seed)
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    state = {"case": case}
    if case["op"] == "route":
        state["logits"] = _logits(g, T, E, DTYPE[case["dtype"]])
        state["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        if case["backward"]:
            state["ids"] = _plain_choice(state)[0].to(torch.int32)
            state["grad"] = torch.randn(T, k, generator=g, device="cuda")
        return state
    state["ids"] = _ids(g, case)
    if case["op"] == "dispatch":
        x = torch.randn(T, case["width"], generator=g, device="cuda")
        if case["rows"] in DTYPE:
            state["x"] = x.to(DTYPE[case["rows"]])
        else:
            state["codes"], state["scales"], state["tensor_scale"] = _quantized(x, case["rows"])
        return state
    dt = DTYPE[case["dtype"]]
    state["weights"] = _weights(g, T, k)
    state["rows"] = torch.randn(T * k, case["width"], generator=g, device="cuda").to(dt)
    if case["grouped"]:
        state["groups"] = _plain_groups(state["ids"], E)
        # rows behind the last expert's are whatever memory held
        state["rows"][torch.arange(T * k, device="cuda") >= state["groups"][0][-1]] = math.nan
    else:
        state["groups"] = None
    if case["backward"]:
        state["grad"] = torch.randn(T, case["width"], generator=g, device="cuda").to(dt)
    return state


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _plain_choice(s):
    """The chosen experts by their scores in 64 bits, best first, ties to the lowest index."""
    case = s["case"]
    x = s["logits"].double()
    if case["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        score = p / p.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score if s["bias"] is None else score + s["bias"].double()
    if case["top_groups"] < case["groups"]:
        parts = choice.unflatten(-1, (case["groups"], -1))
        rank = parts.sort(-1, descending=True).values[..., :case["best"]].sum(-1)
        order = rank.sort(dim=-1, descending=True, stable=True).indices
        kept = torch.zeros_like(rank, dtype=torch.bool).scatter_(-1, order[..., :case["top_groups"]], True)
        choice = parts.masked_fill(~kept[..., None], -math.inf).flatten(-2)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[..., :case["top_k"]]
    return ids, score


def _plain_scores(s):
    x = s["logits"].float()
    if s["case"]["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        return p / p.sum(-1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-x))


def _plain_route(s):
    case = s["case"]
    if not case["backward"]:
        ids = _plain_choice(s)[0]
        w = _plain_scores(s).gather(-1, ids)
        if case["renormalize"]:
            w = w / w.sum(-1, keepdim=True)
        return {"weights": w * case["scale"], "ids": ids.to(torch.int32)}
    ids, score = s["ids"].long(), _plain_scores(s)
    grad, chosen = s["grad"] * case["scale"], score.gather(-1, ids)
    if case["renormalize"]:
        total = chosen.sum(-1, keepdim=True)
        grad = (grad - (grad * chosen).sum(-1, keepdim=True) / total) / total
    full = torch.zeros_like(score).scatter_(-1, ids, grad)
    if case["score"] == "softmax":
        out = score * (full - (full * score).sum(-1, keepdim=True))
    else:
        out = full * score * (1.0 - score)
    return {"logits": out.to(s["logits"].dtype)}


def _plain_groups(ids, E):
    """offsets, order and place of the pairs sorted by expert; pairs of no expert come last."""
    flat = ids.flatten().long()
    flat = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = flat.sort(stable=True).indices
    place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    return offsets.to(torch.int32), order.to(torch.int32), place.view(ids.shape).to(torch.int32)


def _values(codes, scales, fmt, tensor_scale):
    """What packed codes [..., C / 2] under scale bytes [..., C / block] stand for, in fp32."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=codes.device)
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).flatten(-2)
    if fmt == "mxfp4":
        scale = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    else:
        scale = scales.contiguous().view(torch.float8_e4m3fn).float() * tensor_scale
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * scale[..., None]).flatten(-2)


def _plain_dispatch(s):
    case = s["case"]
    offsets, order, place = _plain_groups(s["ids"], case["experts"])
    token = order.long() // case["top_k"]
    if case["rows"] in DTYPE:
        rows = s["x"][token]
    else:
        rows = _values(s["codes"][token], s["scales"][token], case["rows"], s["tensor_scale"])
    inside = torch.arange(order.numel(), device=order.device) < offsets[-1]
    rows = torch.where(inside[:, None], rows, torch.zeros((), dtype=rows.dtype, device=rows.device))
    return {"offsets": offsets, "order": order, "place": place, "rows": rows}


def _plain_combine(s):
    case, w = s["case"], s["weights"]
    T, k = w.shape
    dt = s["rows"].dtype
    if s["groups"] is None:
        at = torch.arange(T * k, device=w.device).view(T, k)
        there = torch.ones_like(at, dtype=torch.bool)
    else:
        at = s["groups"][2].long()
        there = at < s["groups"][0][-1]
    rows = torch.where(there[..., None], s["rows"][at].float(), torch.zeros((), device=w.device))  # [T, k, H]
    if not case["backward"]:
        return {"out": (rows * w[..., None]).sum(1).to(dt)}
    grad = s["grad"].float()
    grad_w = (rows * grad[:, None]).sum(-1)
    grad_rows = torch.zeros_like(s["rows"])
    grad_rows[at] = torch.where(there[..., None], grad[:, None] * w[..., None], torch.zeros((), device=w.device)).to(dt)
    return {"rows": grad_rows, "weights": grad_w}


def _plain_matvec(s):
    case, x, ids = s["case"], s["x"].float(), s["ids"]
    fmt, ts = case["fmt"], s["tensor_scale"]
    if ids is None:
        return {"y": (x @ _values(s["codes"], s["scales"], fmt, ts).T).to(s["x"].dtype)}
    T, k = ids.shape
    if case["spread"]:
        x = x.repeat_interleave(k, 0)
    y = torch.zeros(T * k, case["n"], device=x.device)
    for e in range(case["experts"]):
        w = _values(s["codes"][e], s["scales"][e], fmt, None if ts is None else ts[e])
        y = torch.where(ids.view(-1, 1) == e, x @ w.T, y)
    return {"y": y.view(T, k, -1).to(s["x"].dtype)}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _handles(s):
    """What a program makes once beside its buffers: the weights as the framework holds them, the pairs' order."""
    if "F" not in s:
        import block_scaled_fp4_amax_amd as F
        s["F"] = F
        if "codes" in s:
            fmt = s["case"]["fmt" if s["case"]["op"] == "matvec" else "rows"]
            s["packed"] = F.Quantized({"mxfp4": F.FP4_MXFP4, "nvfp4": F.FP4_NVFP4}[fmt], s["codes"], s["scales"],
                                      s["tensor_scale"])
        if s.get("groups") is not None:
            s["made"] = F.MoeGroups(*s["groups"])
    return s["F"]


def _own(s):
    case, F = s["case"], _handles(s)
    if case["op"] == "matvec":
        return {"y": F.matvec(s["x"], s["packed"], s["ids"])}
    if case["op"] == "route":
        kind = {"score": case["score"], "renormalize": case["renormalize"], "scale": case["scale"]}
        if case["backward"]:
            return {"logits": F.moe_route_backward(s["grad"], s["logits"], s["ids"], **kind)}
        w, ids = F.moe_route(s["logits"], case["top_k"], bias=s["bias"], groups=case["groups"],
                             top_groups=case["top_groups"], group_best=case["best"], **kind)
        return {"weights": w, "ids": ids}
    if case["op"] == "dispatch":
        g = F.moe_group(s["ids"], case["experts"])
        if case["rows"] in DTYPE:
            rows = F.moe_dispatch(s["x"], g)
        else:
            rows = F.dequantize(F.moe_dispatch(s["packed"], g))
        return {"offsets": g.offsets, "order": g.order, "place": g.place, "rows": rows}
    groups = s.get("made")
    if case["backward"]:
        rows, w = F.moe_combine_backward(s["grad"], s["rows"], s["weights"], groups)
        return {"rows": rows, "weights": w}
    return {"out": F.moe_combine(s["rows"], s["weights"], groups)}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "route":
        return _plain_route(state)
    if op == "dispatch":
        return _plain_dispatch(state)
    return _plain_combine(state) if op == "combine" else _plain_matvec(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(case, s):
    z = s["logits"].double()
    T, E = z.shape
    soft = case["score"] == "softmax"
    # probability of each expert: log-sum-exp, or the logistic function by the sign that does not overflow
    if soft:
        p = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
    else:
        small = torch.exp(-z.abs())
        p = torch.where(z >= 0, 1 / (1 + small), small / (1 + small))
    at = torch.arange(E, device="cuda").expand(T, E)
    if case["backward"]:
        ids = s["ids"].long()
    else:
        left = p + (0 if s["bias"] is None else s["bias"].double())
        G, n = case["groups"], E // case["groups"]
        if case["top_groups"] < G:
            inner = left.reshape(T, G, n).clone()
            rank = inner.amax(-1)
            if case["best"] == 2:
                first = (inner == rank[..., None]).int().argmax(-1, keepdim=True)
                rank = rank + inner.scatter(-1, first, -math.inf).amax(-1)
            ahead = (rank[:, None, :] > rank[:, :, None]).sum(-1)
            lower = torch.ones(G, G, device="cuda").tril(-1).bool()
            ahead = ahead + ((rank[:, None, :] == rank[:, :, None]) & lower).sum(-1)
            left = torch.where((ahead < case["top_groups"]).repeat_interleave(n, 1), left,
                               torch.full_like(left, -math.inf))
        ids = torch.empty(T, case["top_k"], dtype=torch.int64, device="cuda")
        for j in range(case["top_k"]):
            top = left.amax(-1, keepdim=True)
            ids[:, j] = torch.where(left == top, at, E).amin(-1)
            left = left.scatter(-1, ids[:, j:j + 1], -math.inf)
    q = torch.gather(p, 1, ids)
    if not case["backward"]:
        w = case["scale"] * (q / q.sum(1, keepdim=True) if case["renormalize"] else q)
        return {"weights": w, "ids": ids.to(torch.int32)}
    d = s["grad"].double() * case["scale"]
    hit = torch.zeros_like(p)
    if case["renormalize"]:
        r = q / q.sum(1, keepdim=True)
        d = r * (d - (r * d).sum(1, keepdim=True))          # by log q
        return {"logits": hit.scatter(1, ids, d if soft else d * (1 - q))}
    if not soft:
        return {"logits": hit.scatter(1, ids, d * q * (1 - q))}
    hit.scatter_(1, ids, d * q)
    return {"logits": hit - p * (d * q).sum(1, keepdim=True)}


def _exact_groups(ids, E):
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(E + 1)]
    for p, e in enumerate(flat):
        lists[e if 0 <= e < E else E].append(p)
    order = [p for part in lists for p in part]
    place = [0] * len(order)
    for r, p in enumerate(order):
        place[p] = r
    offsets = [0]
    for part in lists[:E]:
        offsets.append(offsets[-1] + len(part))
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    return as_int(offsets), as_int(order), as_int(place).view(ids.shape)


def _exact_values(codes, scales, fmt, ts):
    """E2M1 by its fields: (-1)^s 2^(e - 1) (1 + m / 2), or m / 2 where e = 0; E8M0 and E4M3 scales by theirs."""
    n = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], -1).double()
    e, m = torch.floor(n % 8 / 2), n % 2
    v = (1 - 2 * torch.floor(n / 8)) * torch.where(e == 0, m / 2, 2.0 ** (e - 1) * (1 + m / 2))
    b = scales.double()
    if fmt == "mxfp4":
        sc = 2.0 ** (b - 127)
    else:
        e, m = torch.floor(b % 128 / 8), b % 8
        sc = torch.where(e == 0, 2.0 ** -6 * m / 8, 2.0 ** (e - 7) * (1 + m / 8)) * ts.double()
    return v * sc.repeat_interleave(BLOCK[fmt], -1)


def _exact_matvec(case, s):
    x, ids = s["x"].double(), s["ids"]
    ts = s["tensor_scale"]
    if ids is None:
        return {"y": x @ _exact_values(s["codes"], s["scales"], case["fmt"], ts).T}
    T, k = ids.shape
    y = torch.zeros(T * k, case["n"], dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.flatten().tolist())):
        if e < 0:
            continue
        pairs = (ids.flatten() == e).nonzero().flatten()
        w = _exact_values(s["codes"][e], s["scales"][e], case["fmt"], None if ts is None else ts[e])
        y[pairs] = x[pairs // k if case["spread"] else pairs] @ w.T
    return {"y": y.view(T, k, -1)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        return _exact_matvec(case, s)
    if case["op"] == "route":
        return _exact_route(case, s)
    T, k = case["tokens"], case["top_k"]
    if case["op"] == "dispatch":
        offsets, order, place = _exact_groups(s["ids"], case["experts"])
        x = (s["x"].double() if case["rows"] in DTYPE
             else _exact_values(s["codes"], s["scales"], case["rows"], s["tensor_scale"]))
        rows = torch.zeros(T * k, case["width"], dtype=torch.float64, device="cuda")
        n = int(offsets[-1])
        rows[:n] = x[order[:n].long() // k]
        return {"offsets": offsets, "order": order, "place": place, "rows": rows}
    if s["groups"] is None:
        place, n = torch.arange(T * k, device="cuda").view(T, k), T * k
    else:
        offsets, _, place = _exact_groups(s["ids"], case["experts"])
        place, n = place.long(), int(offsets[-1])
    rows, w = s["rows"].double(), s["weights"].double()
    rows[n:] = 0
    w = torch.where(place < n, w, torch.zeros_like(w))
    if not case["backward"]:
        out = torch.zeros(T, case["width"], dtype=torch.float64, device="cuda")
        for j in range(k):
            out += w[:, j:j + 1] * rows[place[:, j]]
        return {"out": out}
    grad = s["grad"].double()
    grad_rows, grad_w = torch.zeros_like(rows), torch.zeros_like(w)
    for j in range(k):
        grad_rows[place[:, j]] = w[:, j:j + 1] * grad
        grad_w[:, j] = (rows[place[:, j]] * grad).sum(-1)
    return {"rows": grad_rows, "weights": grad_w}
