"""The 4-bit key-value cache operators, as cases to run and to compare.

Three operators on a paged cache whose keys and values are held in MXFP4 or NVFP4:

* append: new keys and values are rotated to their positions (keys only), quantized and written to their slots; the
  step's queries are rotated in the same call;
* read: the rows of given slots as plain numbers again;
* attention: queries of one token or of many, packed over a ragged batch, against each sequence's cached rows.

``own`` chooses between the framework's kernels and a plain form of elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
FLT_MIN = 1.17549435e-38
POOL_ROWS = 1 << 15  # distinct cached rows per head; longer caches repeat them in random order


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attention(name, fmt, batch, q_len, kv_len, heads, kv_heads, dim, page, *, ragged=False, causal=True, window=0,
               softcap=0.0, dtype="bf16"):
    return {"name": name, "op": "attention", "fmt": fmt, "batch": batch, "q_len": q_len, "kv_len": kv_len,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": ragged, "causal": causal,
            "window": window, "softcap": softcap, "dtype": dtype}


def _append(name, fmt, tokens, heads, kv_heads, dim, page, *, rotary=None, interleaved=False, dtype="bf16"):
    return {"name": name, "op": "append", "fmt": fmt, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "rotary": dim if rotary is None else rotary, "interleaved": interleaved,
            "dtype": dtype}


def listed():
    return [
        # one interactive user's next token: nothing but latency
        _attention("decode_1x997", "mxfp4", 1, 1, 997, 32, 8, 128, 16),
        # an ordinary serving batch of unequal lengths, one token each
        _attention("decode_32x4096", "nvfp4", 32, 1, 4096, 32, 8, 128, 64, ragged=True),
        # a full serving batch with long contexts: the cache's bytes are everything
        _attention("decode_64x16384", "mxfp4", 64, 1, 16384, 64, 8, 128, 128, ragged=True),
        # one very long document: few rows, so the work is split along the keys
        _attention("decode_1x130001", "nvfp4", 1, 1, 130001, 16, 2, 128, 16),
        # a model with small heads, a sliding window and capped scores, in fp32
        _attention("decode_window_f32", "nvfp4", 16, 1, 2500, 16, 16, 64, 32, ragged=True, window=1024,
                   softcap=30.0, dtype="f32"),
        # a few drafted tokens per sequence, checked in one pass
        _attention("verify_24x5", "mxfp4", 24, 5, 3001, 32, 8, 128, 32, ragged=True),
        # chunks of prompts appended to what is cached already
        _attention("chunks_4x1024", "nvfp4", 4, 1024, 6000, 32, 4, 128, 64, ragged=True),
        # a whole long prompt
        _attention("prompt_8192", "mxfp4", 1, 8192, 8192, 32, 8, 128, 128),
        # a decoder's rows against an encoder's states of another length, no causal order
        _attention("cross_8x448x1500", "mxfp4", 8, 448, 1500, 20, 20, 64, 16, ragged=True, causal=False),
        # one decode step's rows of a serving batch
        _append("append_32", "mxfp4", 32, 32, 8, 128, 16),
        # odd head size, part of it rotated in adjacent pairs, fp32 activations
        _append("append_1001_f32", "nvfp4", 1001, 12, 4, 80, 64, rotary=48, interleaved=True, dtype="f32"),
        # a long prompt's rows
        _append("append_16384", "nvfp4", 16384, 32, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    fmt = rng.choice(("mxfp4", "nvfp4"))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    dim = rng.choice((64, 128, 128, 128, 96, 192, 256, 32) if fmt == "mxfp4" else (64, 128, 128, 128, 80, 112, 256, 16))
    kv_heads = rng.choice((1, 2, 3, 4, 8, 8, 16))
    heads = kv_heads * rng.choice((1, 2, 4, 4, 5, 8, 16))
    page = rng.choice((16, 32, 64, 128, 256))
    if rng.random() < 0.25:
        rotary = rng.choice((dim, dim, dim // 2))
        case = _append("", fmt, _log(rng, 1, 16384), heads, kv_heads, dim, page, rotary=rotary,
                       interleaved=rng.random() < 0.3, dtype=dtype)
        while case["tokens"] * case["dim"] * (heads + 2 * kv_heads) * (2 if dtype == "f32" else 1) > 16384 * 48 * 128:
            case["tokens"] = max(1, case["tokens"] // 2 + rng.randrange(8))
    else:
        kind = rng.choice(("decode", "decode", "few", "prompt"))
        q_len = 1 if kind == "decode" else rng.randint(2, 16) if kind == "few" else _log(rng, 17, 4096)
        kv_len = _log(rng, 1 if kind != "prompt" else 64, 131072 if kind == "decode" else 8192)
        causal = rng.random() < 0.8
        if causal:
            kv_len = max(kv_len, q_len)
        window = _log(rng, 16, 4096) if causal and rng.random() < 0.2 else 0
        case = _attention("", fmt, _log(rng, 1, 64), q_len, kv_len, heads, kv_heads, dim, page,
                          ragged=rng.random() < 0.7, causal=causal, window=window,
                          softcap=30.0 if rng.random() < 0.15 else 0.0, dtype=dtype)
        # the plain form holds the padded batch's cached rows and its scores in fp32
        while (case["batch"] * case["kv_len"] * kv_heads * dim > 64 * 16384 * 8 * 128
               or case["batch"] * case["q_len"] * case["kv_len"] * heads * max(dim, 64) > 8192 * 8192 * 16 * 128):
            if case["batch"] > 1:
                case["batch"] //= 2
            else:
                case["kv_len"] = max(case["kv_len"] * 2 // 3, 1)
                case["q_len"] = min(case["q_len"], case["kv_len"]) if causal else case["q_len"]
    del case["name"]
    return case


def _lengths(case):
    """Each sequence's number of queries and of cached rows (these queries' own among them where causal)."""
    n, ql, kl = case["batch"], case["q_len"], case["kv_len"]
    if not case["ragged"]:
        return [ql] * n, [kl] * n
    r = random.Random("%d %d %d" % (n, ql, kl))
    q = [ql] + [r.randint(max(1, ql // 4), ql) for _ in range(n - 1)]
    k = [kl] + [r.randint(max(1, kl // 4), kl) for _ in range(n - 1)]
    if case["causal"]:
        k = [max(a, b) for a, b in zip(q, k)]
    order = list(range(n))
    r.shuffle(order)
    return [q[i] for i in order], [k[i] for i in order]


def work(case):
    D, H, Hkv = case["dim"], case["heads"], case["kv_heads"]
    size = 4 if case["dtype"] == "f32" else 2
    row = D // 2 + D // BLOCK[case["fmt"]]  # one cached key or value of one head
    if case["op"] == "append":
        T = case["tokens"]
        moved = T * D * size * (2 * H + 2 * Hkv)       # queries in and out, keys and values in
        moved += T * Hkv * 2 * (2 * row + 2 * D)        # cache rows written, read again, and given out in bf16
        moved += T * (16 + 4 * case["rotary"])
        return {"bytes": moved, "flops": T * D * (3 * H + 12 * Hkv)}
    pairs = keys = 0
    qs, ks = _lengths(case)
    for q, k in zip(qs, ks):
        w = case["window"]
        if not case["causal"]:
            pairs += q * k
            keys += k
        else:
            low = k - q
            full = q * low + q * (q + 1) // 2            # sum over rows of (low + i + 1)
            if w:
                cut = [max(0, low + i + 1 - w) for i in range(q)]
                full -= sum(cut)
                keys += k - cut[0]
            else:
                keys += k
            pairs += full
    T = sum(qs)
    moved = 2 * T * H * D * size + 4 * T * H + keys * Hkv * 2 * row + 4 * len(qs) * -(-max(ks) // case["page"])
    return {"bytes": moved, "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _prepare_append(case, seed):
    g = _generator(seed)
    T, H, Hkv, D, page, fmt = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "page", "fmt"))
    dt = DTYPE[case["dtype"]]
    pages = -(-T // page) + 3
    # one fused projection's output: the three operands are strided views of it
    qkv = torch.randn(T, H + 2 * Hkv, D, generator=g, device="cuda")
    qkv[..., : max(1, D // 16)] *= 6.0  # a few channels carry the large values, as keys do
    qkv = qkv.to(dt)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    if T > 3:
        slots[torch.rand(T, generator=g, device="cuda") < 0.03] = -1  # padding rows of the step
    limit = 4 * T + 64
    positions = torch.randint(0, limit, (T,), generator=g, device="cuda")
    half = case["rotary"] // 2
    angle = torch.arange(limit, device="cuda")[:, None] * 10000.0 ** (-torch.arange(half, device="cuda") / max(half, 1))
    scale = torch.full((Hkv,), 30.0 / 2688.0, device="cuda")
    shape = (pages, Hkv, page)
    state = {"case": case, "q": qkv[:, :H], "k": qkv[:, H:H + Hkv], "v": qkv[:, H + Hkv:], "slots": slots,
             "positions": positions, "cos": angle.cos().contiguous(), "sin": angle.sin().contiguous(),
             "k_tensor_scale": scale, "v_tensor_scale": scale.clone()}
    for n in ("k", "v"):
        state[n + "_codes"] = torch.zeros(*shape, D // 2, dtype=torch.uint8, device="cuda")
        state[n + "_scales"] = torch.zeros(*shape, D // BLOCK[fmt], dtype=torch.uint8, device="cuda")
    return state


def _prepare_attention(case, seed):
    g = _generator(seed)
    H, Hkv, D, page, fmt = (case[k] for k in ("heads", "kv_heads", "dim", "page", "fmt"))
    qs, ks = _lengths(case)
    need = [-(-k // page) for k in ks]
    pages, width = sum(need) + 2, max(need)
    q = 1.5 * torch.randn(sum(qs), H, D, generator=g, device="cuda")
    ts = torch.full((Hkv,), 30.0 / 2688.0, device="cuda")
    state = {"case": case, "q": q.to(DTYPE[case["dtype"]]), "k_tensor_scale": ts, "v_tensor_scale": ts.clone()}
    # each sequence's pages lie anywhere in the cache; the table's unused entries hold nothing valid
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    need_t = torch.tensor(need, device="cuda")
    column = torch.arange(width, device="cuda")
    place = (need_t.cumsum(0) - need_t)[:, None] + column
    used = column < need_t[:, None]
    table = torch.where(used, order[place.clamp(max=pages - 1)], torch.full_like(order[:1], -1))
    kv = torch.tensor(ks, device="cuda", dtype=torch.int32)
    # positions at and past a sequence's end, and pages of no sequence, hold bytes that stand for no number
    held = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    held[table[used].long()] = (column[:, None] * page + torch.arange(page, device="cuda") < kv[:, None, None])[used]
    for n in ("k", "v"):
        rows = min(POOL_ROWS, max(64, pages * page))
        x = torch.randn(rows, D, generator=g, device="cuda")
        if n == "k":
            x[:, : max(1, D // 16)] *= 4.0
        codes, scales = _quantize_rows(x, fmt, ts[:1])
        pick = torch.randint(0, rows, (pages, Hkv, page), generator=g, device="cuda")
        keep = held[:, None, :, None]
        state[n + "_codes"] = torch.where(keep, codes[pick], torch.full_like(codes[:1, :1], 255))
        state[n + "_scales"] = torch.where(keep, scales[pick], torch.full_like(scales[:1, :1], 255))
    offsets = torch.tensor([0] + qs, device="cuda").cumsum(0).to(torch.int32)
    state |= {"table": table.contiguous(), "kv_lens": kv, "q_offsets": offsets, "q_lens": qs, "max_kv_len": max(ks)}
    return state


def prepare(case, seed):
    return _prepare_append(case, seed) if case["op"] == "append" else _prepare_attention(case, seed)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, rotary, interleaved):
    """x [T, H, D] fp32, cos and sin [T, 1, rotary / 2]: pairs (i, i + rotary / 2), or (2i, 2i + 1) if interleaved."""
    r, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., : rotary // 2], r[..., rotary // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _nearest_code(q):
    """Nearest of {0, 0.5, 1, 1.5, 2, 3, 4, 6} to |q|, ties to the even code, with the sign in bit 3."""
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code | (torch.signbit(q).to(torch.uint8) << 3)


def _quantize_rows(x, fmt, tensor_scale):
    """x [..., D] fp32 -> packed codes [..., D / 2], scale bytes [..., D / block]; tensor_scale broadcasts over
    [..., 1]."""
    blocks = x.unflatten(-1, (-1, BLOCK[fmt]))
    amax = blocks.abs().amax(-1)
    if fmt == "mxfp4":
        # 2^e with e = floor(log2 amax) - 2, held as e + 127
        byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)
        q = torch.ldexp(blocks, (127 - byte)[..., None])
    else:
        s = (amax * (1.0 / (6.0 * tensor_scale))).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte = s.view(torch.uint8)
        eff = s.float() * tensor_scale
        r = torch.where(eff >= FLT_MIN, 1.0 / eff, torch.zeros_like(eff))
        q = blocks * r[..., None]
    code = _nearest_code(q).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.to(torch.uint8)


def _values(codes, scales, fmt, tensor_scale):
    """What packed codes [..., D / 2] under scale bytes [..., D / block] stand for, in fp32."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=codes.device)
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).flatten(-2)
    if fmt == "mxfp4":
        scale = torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)
    else:
        scale = scales.view(torch.float8_e4m3fn).float() * tensor_scale
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * scale[..., None]).flatten(-2)


def _plain_append(s):
    case = s["case"]
    fmt, page = case["fmt"], case["page"]
    cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]
    turn = (cos, sin, case["rotary"], case["interleaved"])
    q = _rotate(s["q"].float(), *turn).to(s["q"].dtype)
    held = s["slots"] >= 0
    where = s["slots"][held]
    back = []
    for n, x in (("k", _rotate(s["k"].float(), *turn)), ("v", s["v"].float())):
        ts = s[n + "_tensor_scale"][:, None]
        codes, scales = _quantize_rows(x, fmt, ts)
        at = (where // page, slice(None), where % page)
        s[n + "_codes"][at] = codes[held]
        s[n + "_scales"][at] = scales[held]
        y = torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device)
        y[held] = _values(s[n + "_codes"][at], s[n + "_scales"][at], fmt, ts).to(torch.bfloat16)
        back.append(y)
    return {"q": q, "k": back[0], "v": back[1]}


def _plain_attention(s):
    case = s["case"]
    H, Hkv, D, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    B, G, L, Q = case["batch"], H // Hkv, s["max_kv_len"], max(s["q_lens"])
    dev = s["q"].device
    j = torch.arange(L, device=dev)
    lens = s["kv_lens"].long()
    inside = j < lens[:, None]                                             # [B, L]
    rows = s["table"].long().clamp(min=0)[:, j // page]                    # [B, L]
    kv = []
    for n in ("k", "v"):
        x = _values(s[n + "_codes"][rows, :, j % page], s[n + "_scales"][rows, :, j % page], case["fmt"],
                    s[n + "_tensor_scale"][:, None])                       # [B, L, Hkv, D]
        kv.append(torch.where(inside[..., None, None], x, torch.zeros((), device=dev)).transpose(1, 2).contiguous())
    starts = s["q_offsets"].long()
    q_lens = starts[1:] - starts[:-1]
    i = torch.arange(Q, device=dev)
    real = i < q_lens[:, None]                                             # [B, Q]
    q = s["q"].new_zeros(B, Q, H, D, dtype=torch.float32)
    q[real] = s["q"].float()
    q = q.view(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    score = torch.matmul(q, kv[0].transpose(-1, -2)) * D ** -0.5
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    seen = inside[:, None, :].expand(B, Q, L)
    if case["causal"]:
        at = (lens - q_lens)[:, None] + i                                  # position of each query
        seen = seen & (j <= at[..., None])
        if case["window"]:
            seen = seen & (j > at[..., None] - case["window"])
    score = score.view(B, Hkv, G, Q, L).masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, Hkv, G * Q, L), kv[1]).view(B, Hkv, G, Q, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, Q, H, D)[real]
    lse = lse.permute(0, 3, 1, 2).reshape(B, Q, H)[real]
    return {"out": out.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _handle(s):
    """The cache's handle, which a program makes once beside its buffers."""
    if "cache" not in s:
        import block_scaled_fp4_amax_amd as F
        s["F"] = F
        s["cache"] = F.KVCache(s["case"]["fmt"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                               s["k_tensor_scale"], s["v_tensor_scale"])
    return s["F"], s["cache"]


def run(state):
    case = state["case"]
    if not own:
        return _plain_append(state) if case["op"] == "append" else _plain_attention(state)
    F, cache = _handle(state)
    if case["op"] == "append":
        q = F.kv_append(cache, state["k"], state["v"], state["slots"], q=state["q"], positions=state["positions"],
                        cos=state["cos"], sin=state["sin"], interleaved=case["interleaved"])
        k, v = F.kv_read(cache, state["slots"], torch.bfloat16)
        return {"q": q, "k": k, "v": v}
    out, lse = F.kv_attention(state["q"], cache, state["table"], state["kv_lens"],
                              q_offsets=None if case["q_len"] == 1 else state["q_offsets"],
                              max_kv_len=state["max_kv_len"], causal=case["causal"], window=case["window"],
                              softcap=case["softcap"], return_lse=True)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_elements(codes):
    """E2M1 by its fields: (-1)^s * 2^(e - 1) * (1 + m / 2), or m / 2 where e = 0; two elements a byte, low first."""
    n = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], -1).double()
    sign = 1 - 2 * torch.floor(n / 8)
    e, m = torch.floor(n % 8 / 2), n % 2
    return sign * torch.where(e == 0, m / 2, 2.0 ** (e - 1) * (1 + m / 2))


def _exact_scales(b, fmt):
    b = b.double()
    if fmt == "mxfp4":
        return 2.0 ** (b - 127)
    e, m = torch.floor(b % 128 / 8), b % 8
    return torch.where(e == 0, 2.0 ** -6 * m / 8, 2.0 ** (e - 7) * (1 + m / 8))


def _exact_rows(s, n, page, offset, head):
    """The rows of one head at (page, offset), [rows, D]."""
    fmt = s["case"]["fmt"]
    el = _exact_elements(s[n + "_codes"][page, head, offset])
    sc = _exact_scales(s[n + "_scales"][page, head, offset], fmt)
    if fmt == "nvfp4":
        sc = sc * s[n + "_tensor_scale"][head].double()
    return el * sc.repeat_interleave(BLOCK[fmt], -1)


def _exact_round(x, step_of):
    """x to the nearest multiple of its own step, ties to even (torch.round's)."""
    step = step_of(x.abs())
    return torch.round(x / step) * step


def _exact_quantized(x, fmt, ts):
    """What x [..., D] becomes in the cache: each block by its scale, each element to the E2M1 grid."""
    blocks = x.reshape(*x.shape[:-1], -1, BLOCK[fmt])
    top = blocks.abs().amax(-1, keepdim=True)
    one = torch.ones((), dtype=torch.float64, device=x.device)
    if fmt == "mxfp4":
        scale = 2.0 ** torch.where(top > 0, torch.floor(torch.log2(top)) - 2, -127 * one).clamp(-127, 127)
    else:
        s = (top / (6 * ts[..., None])).clamp(max=448)
        scale = _exact_round(s, lambda a: 2.0 ** (torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)) * ts[..., None]
    z = torch.where(scale > 0, blocks / torch.where(scale > 0, scale, one), 0 * one).clamp(-6, 6)
    z = _exact_round(z, lambda a: torch.where(a < 2, 0.5 * one, torch.where(a < 4, one, 2 * one)))
    return (z * scale).reshape(x.shape)


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    half = case["rotary"] // 2
    c, sn = s["cos"].double()[s["positions"]][:, None], s["sin"].double()[s["positions"]][:, None]
    at = torch.arange(half, device="cuda")
    first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)

    def turned(x):
        x = x.double()
        y = x.clone()
        y[..., first] = x[..., first] * c - x[..., second] * sn
        y[..., second] = x[..., second] * c + x[..., first] * sn
        return y

    there = (s["slots"] >= 0)[:, None, None].double()
    ts = [s[n + "_tensor_scale"].double()[:, None] for n in ("k", "v")]
    return {"q": turned(s["q"]), "k": _exact_quantized(turned(s["k"]), case["fmt"], ts[0]) * there,
            "v": _exact_quantized(s["v"].double(), case["fmt"], ts[1]) * there}


def _exact_attention(case, seed):
    s = _prepare_attention(case, seed)
    H, Hkv, D, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    G = H // Hkv
    out = torch.zeros(sum(s["q_lens"]), H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(s["q_lens"]), H), -math.inf, dtype=torch.float64, device="cuda")
    start = 0
    for b, (n, length) in enumerate(zip(s["q_lens"], s["kv_lens"].tolist())):
        j = torch.arange(length, device="cuda")
        where, offset = s["table"][b].long()[j // page], j % page
        for h in range(Hkv):
            k, v = (_exact_rows(s, name, where, offset, h) for name in ("k", "v"))
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                q = s["q"][start + lo:start + hi, h * G:(h + 1) * G].double()       # [rows, G, D]
                z = (q.reshape(-1, D) @ k.T).reshape(hi - lo, G, length) / math.sqrt(D)
                if case["softcap"]:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                if case["causal"]:
                    back = (length - n + torch.arange(lo, hi, device="cuda"))[:, None] - j
                    hidden = (back < 0) | (back >= case["window"]) if case["window"] else back < 0
                    z.masked_fill_(hidden[:, None], -math.inf)
                total = torch.logsumexp(z, -1)
                w = torch.exp(z - total[..., None]).nan_to_num_(0.0)
                out[start + lo:start + hi, h * G:(h + 1) * G] = (w.reshape(-1, length) @ v).reshape(hi - lo, G, D)
                lse[start + lo:start + hi, h * G:(h + 1) * G] = total
        start += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "append":
        return _exact_append(case, seed)
    if work(case)["flops"] > 2e12:  # would take too long in 64 bits
        return None
    return _exact_attention(case, seed)
