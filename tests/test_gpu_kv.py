"""The 4-bit key-value cache on the GPU: append and read bit for bit against
the CPU oracle's quantizer on rows rotated in fp32, attention against its
definition in 64 bits over the values the cache stands for."""
import numpy as np
import pytest
import torch

from gpu_util import assert_codes_equal, oracle_input
from kv_util import (K_AMAX, V_AMAX, attention_bounds, attention_f64, check_attention, lay_out, random_cache,
                     rotate_f32, spoil)

pytestmark = pytest.mark.gpu

MX, NV = 0, 1
BF, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
def append_case(F, O, fmt, dtype, T, heads, kv_heads, dim, page, rotary, interleaved, fos, seed=0, fused=True,
                in_place=False):
    rng = np.random.RandomState(seed)
    pages = -(-T // page) + 2
    nv = fmt == NV
    cache = F.KVCache.empty("nvfp4" if nv else "mxfp4", pages, page, kv_heads, dim, k_amax=K_AMAX, v_amax=V_AMAX,
                            four_over_six=fos)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(0xEE)
    n = heads + 2 * kv_heads
    x = torch.from_numpy(rng.standard_normal((T, n, dim)).astype(np.float32))
    x[..., : max(1, dim // 16)] *= 5
    if T > 2:
        x[1] = 0
        x[2] *= 1e-30
    x = x.to(dtype).cuda()
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    if not fused:
        q, k, v = (t.contiguous() for t in (q, k, v))
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1
        slots[4] = pages * page
    limit = 3 * T + 7
    pos = rng.randint(0, limit, T).astype(np.int64)
    half = rotary // 2
    ang = rng.uniform(-np.pi, np.pi, (limit, max(half, 1)))[:, :half]
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    kw = dict(positions=torch.from_numpy(pos).cuda(), cos=torch.from_numpy(cos).cuda(),
              sin=torch.from_numpy(sin).cuda(), interleaved=interleaved) if rotary else {}
    ref = {}
    for name, t in (("q", q), ("k", k), ("v", v)):
        f = t.float().cpu().numpy()
        ref[name] = rotate_f32(f, cos[pos], sin[pos], interleaved) if rotary and name != "v" else f
    if heads:
        out = F.kv_append(cache, k, v, torch.from_numpy(slots).cuda(), q=q, four_over_six=fos,
                          q_out=q if in_place else None, **kw)
    else:
        out = F.kv_append(cache, k, v, torch.from_numpy(slots).cuda(), four_over_six=fos, **kw)
        assert out is None
    torch.cuda.synchronize()
    if heads:
        want = torch.from_numpy(ref["q"]).to(dtype)
        assert torch.equal(out.cpu(), want), "rotated queries differ"
    there = (slots >= 0) & (slots < pages * page)
    back = F.kv_read(cache, torch.from_numpy(slots).cuda(), F32)
    back16 = F.kv_read(cache, torch.from_numpy(slots).cuda())
    for name, amax, codes, scales, y, y16 in (("k", K_AMAX, cache.k_codes, cache.k_scales, back[0], back16[0]),
                                              ("v", V_AMAX, cache.v_codes, cache.v_scales, back[1], back16[1])):
        r = O.quantize(np.ascontiguousarray(ref[name].reshape(T * kv_heads, dim)), fmt,
                       flags=O.FOUR_OVER_SIX if fos else 0, amax=amax if nv else None)
        want_c = np.full(tuple(codes.shape), 0xEE, np.uint8)
        want_s = np.full(tuple(scales.shape), 0xEE, np.uint8)
        pg, at = slots[there] // page, slots[there] % page
        want_c[pg, :, at] = r["codes"].reshape(T, kv_heads, -1)[there]
        want_s[pg, :, at] = r["scales"].reshape(T, kv_heads, -1)[there]
        assert_codes_equal(codes.cpu().numpy(), want_c, f"{name} codes")
        assert_codes_equal(scales.cpu().numpy(), want_s, f"{name} scales")
        val = O.dequantize(fmt, r["codes"], r["scales"], r["tensor_scale"]).reshape(T, kv_heads, dim)
        val = np.where(there[:, None, None], val, np.float32(0)).astype(np.float32)
        assert np.array_equal(y.cpu().numpy(), val), f"{name} read back differs"
        assert torch.equal(y16.cpu(), torch.from_numpy(val).to(BF)), f"{name} read back in bf16 differs"


APPEND = [
    # (fmt, dtype, T, heads, kv_heads, dim, page, rotary, interleaved, fos)
    (MX, BF, 1, 8, 2, 128, 16, 128, False, False),
    (NV, BF, 1, 8, 2, 128, 16, 128, False, False),
    (MX, BF, 37, 12, 3, 64, 16, 64, False, True),
    (NV, BF, 37, 12, 3, 64, 32, 64, True, True),
    (NV, F32, 50, 4, 4, 80, 64, 40, False, False),    # rotary / 2 = 20: partners one by one
    (NV, F32, 50, 4, 4, 80, 64, 80, False, True),
    (MX, F32, 21, 5, 1, 96, 16, 96, True, False),
    (MX, BF, 21, 5, 1, 96, 16, 48, False, False),     # a unit across the end of the rotary part
    (NV, BF, 19, 3, 3, 16, 16, 8, False, False),
    (NV, BF, 19, 3, 3, 16, 16, 2, True, False),
    (MX, F32, 9, 2, 2, 32, 128, 32, False, False),
    (NV, BF, 33, 7, 1, 240, 16, 240, False, False),
    (MX, BF, 130, 32, 8, 256, 64, 256, False, False),
    (NV, BF, 1500, 16, 8, 128, 64, 128, False, False),  # a wave takes a whole token
    (MX, F32, 1500, 16, 8, 128, 64, 64, True, True),
    (NV, BF, 40, 0, 4, 112, 16, 112, False, False),   # no queries
    (MX, BF, 40, 6, 2, 64, 16, 0, False, False),      # no rotation
    (NV, F32, 40, 0, 2, 64, 16, 0, False, True),
]


@pytest.mark.parametrize("case", APPEND, ids=["-".join(str(x).replace("torch.", "") for x in c) for c in APPEND])
def test_append_and_read_match_the_oracle(fp4, oracle, case):
    print(f"[append] {case}", flush=True)
    append_case(fp4, oracle, *case, seed=len(str(case)))


def test_append_of_dense_operands_and_in_place_queries(fp4, oracle):
    append_case(fp4, oracle, NV, BF, 65, 8, 2, 128, 16, 128, False, False, seed=5, fused=False)
    append_case(fp4, oracle, MX, BF, 65, 8, 2, 128, 16, 64, False, False, seed=6, in_place=True)
    append_case(fp4, oracle, MX, F32, 2100, 8, 2, 96, 16, 40, False, False, seed=7, in_place=True)


def test_append_skips_positions_outside_the_tables(fp4):
    cache = fp4.KVCache.empty("mxfp4", 2, 16, 2, 64)
    x = torch.randn(3, 4, 64, device="cuda")
    cos, sin = torch.ones(5, 32, device="cuda"), torch.zeros(5, 32, device="cuda")
    out = fp4.kv_append(cache, x[:, :2], x[:, 2:], torch.tensor([3, 4, 5], device="cuda"), q=x,
                        positions=torch.tensor([5, -1, 4], device="cuda"), cos=cos, sin=sin)
    assert torch.isnan(out[:2]).all() and torch.equal(out[2], x[2])
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        assert not t[0, :, 3:5].any() and t[0, :, 5].any()


def test_append_without_tokens_and_read_without_slots(fp4):
    cache = fp4.KVCache.empty("mxfp4", 2, 16, 2, 64)
    x = torch.randn(0, 2, 64, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert fp4.kv_append(cache, x, x, none, q=x).shape == (0, 2, 64)
    k, v = fp4.kv_read(cache, none)
    assert k.shape == v.shape == (0, 2, 64)


def test_append_passes_infinities_past_the_rotary_part(fp4):
    """Elements that are not rotated come through as they are, with no
    product in between."""
    cache = fp4.KVCache.empty("mxfp4", 1, 16, 1, 64)
    q = torch.full((1, 1, 64), float("inf"), device="cuda")
    kv = torch.zeros(1, 1, 64, device="cuda")
    t = torch.ones(1, 8, device="cuda")
    out = fp4.kv_append(cache, kv, kv, torch.zeros(1, dtype=torch.int64, device="cuda"), q=q,
                        positions=torch.zeros(1, dtype=torch.int64, device="cuda"), cos=t, sin=torch.zeros_like(t))
    assert torch.isposinf(out[..., 16:]).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attention_case(F, O, fmt, dtype, lens, q_lens, heads, kv_heads, dim, page, causal=True, window=0, softcap=0.0,
                   scale=None, seed=0, q_scale=1.5, max_kv_len=None, ref_of=attention_f64):
    need = sum(-(-n // page) for n in lens)
    cache, k, v = random_cache(F, O, fmt, need + 2, page, kv_heads, dim, seed)
    table = lay_out(cache, lens, seed)
    spoil(cache, table, lens)
    T = sum(q_lens)
    g = torch.Generator().manual_seed(seed + 1)
    q = (q_scale * torch.randn(T, heads, dim, generator=g)).to(dtype)
    decode = all(n == 1 for n in q_lens)
    offs = None if decode else torch.tensor(np.cumsum([0] + list(q_lens)), dtype=torch.int32, device="cuda")
    kw = dict(q_offsets=offs, causal=causal, window=window, softcap=softcap, scale=scale, return_lse=True,
              max_kv_len=max(lens) if max_kv_len is None else max_kv_len)
    td, ld = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = F.kv_attention(q.cuda(), cache, td, ld, **kw)
    torch.cuda.synchronize()
    sc = dim ** -0.5 if scale is None else scale
    ref = ref_of(q.double().numpy(), k, v, table, page, lens, q_lens, causal, window, softcap, sc)
    tol, tol_lse = attention_bounds(ref, fmt == NV, dtype == BF, dim, max(lens + [1]), softcap)
    check_attention(out, lse, ref, tol, tol_lse, f"fmt {fmt} {dtype} lens {lens[:4]} q {list(q_lens)[:4]}")
    again, lse2 = F.kv_attention(q.cuda(), cache, td, ld, **kw)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "two calls differ"


BOTH = [MX, NV]
FD = [(f, d) for f in BOTH for d in (BF, F32)]
FD_IDS = ["mx-bf16", "mx-f32", "nv-bf16", "nv-f32"]


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 2), (64, 6, 6), (32, 4, 1), (96, 10, 2), (256, 4, 1),
                                                (192, 24, 1), (128, 34, 2)])
def test_decode_lengths(fp4, oracle, fmt, dtype, dim, heads, kv_heads):
    """One query per sequence over lengths from none to several tiles, ending
    inside tiles and pages; fewer and more than 16 heads per kv head."""
    print(f"[decode] {fmt} {dtype} {dim} {heads} {kv_heads}", flush=True)
    attention_case(fp4, oracle, fmt, dtype, [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 127, 129, 300], [1] * 13, heads,
                   kv_heads, dim, 16, seed=dim + heads)


@pytest.mark.parametrize("dim", [16, 48, 80, 112, 240])
def test_decode_head_sizes_of_nvfp4(fp4, oracle, dim):
    attention_case(fp4, oracle, NV, BF, [1, 77, 200], [1] * 3, 6, 3, dim, 32, seed=dim)
    attention_case(fp4, oracle, NV, F32, [1, 77, 200], [1] * 3, 6, 3, dim, 32, seed=dim)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_long_sequences_cut_into_chunks(fp4, oracle, fmt, dtype, page):
    print(f"[long] {fmt} {dtype} {page}", flush=True)
    attention_case(fp4, oracle, fmt, dtype, [5003], [1], 4, 1, 128, page, seed=3)
    attention_case(fp4, oracle, fmt, dtype, [2049, 7, 4000], [1] * 3, 4, 2, 64, page, seed=4)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
def test_uneven_batches(fp4, oracle, fmt, dtype):
    """Batches whose key tiles are cut into equal runs: items that end, begin
    and lie within runs, more than 64 sequences, sequences without rows or
    queries between them, heads past 128."""
    print(f"[uneven] {fmt} {dtype}", flush=True)
    rng = np.random.RandomState(40)
    lens = [int(x) for x in rng.randint(0, 60, 90)]
    lens[3], lens[40], lens[77] = 12000, 9000, 7001
    attention_case(fp4, oracle, fmt, dtype, lens, [1] * 90, 4, 2, 64, 16, seed=41)
    q_lens = [int(x) for x in rng.randint(0, 4, 90)]
    attention_case(fp4, oracle, fmt, dtype, lens, q_lens, 4, 1, 64, 64, seed=42)
    attention_case(fp4, oracle, fmt, dtype, [7000, 0, 100, 4000], [1] * 4, 6, 2, 256, 32, seed=43)
    attention_case(fp4, oracle, fmt, dtype, [9000, 30, 6000], [1] * 3, 20, 1, 96, 32, seed=44, window=5000)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_queries(fp4, oracle, fmt, dtype, causal):
    """Sequences without queries, without rows, with more queries than rows
    (causal: the first ones see nothing), and ordinary ones."""
    print(f"[ragged] {fmt} {dtype} {causal}", flush=True)
    attention_case(fp4, oracle, fmt, dtype, [40, 0, 130, 9, 1, 300, 64], [5, 3, 0, 20, 1, 33, 64], 6, 2, 64, 16,
                   causal=causal, seed=8)
    attention_case(fp4, oracle, fmt, dtype, [515, 200], [130, 70], 8, 2, 128, 32, causal=causal, seed=9)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
def test_many_queries(fp4, oracle, fmt, dtype):
    """Prompts: more rows than any tile, a history before them or none."""
    print(f"[prompt] {fmt} {dtype}", flush=True)
    attention_case(fp4, oracle, fmt, dtype, [700, 450], [260, 450], 8, 2, 128, 64, seed=10)
    attention_case(fp4, oracle, fmt, dtype, [390], [333], 5, 5, 64, 16, seed=11)
    attention_case(fp4, oracle, fmt, dtype, [300], [290], 2, 1, 256, 32, seed=12)
    attention_case(fp4, oracle, fmt, dtype, [300], [140], 3, 1, 96, 32, seed=13, causal=False)


def prompt_f64(q, k, v, table, page, lens, q_lens, causal, window, softcap, scale):
    """attention_f64's results for large cases: float64 on the GPU, a kv head
    and sequence at a time."""
    T, H, D = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    q, k, v = (torch.from_numpy(x).cuda() for x in (q, k, v))
    out, absv = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    lse, mag = torch.full((T, H), -np.inf, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    vmax = torch.zeros(T, H, 1, dtype=torch.float64)
    start = 0
    for b, n in enumerate(q_lens):
        L = int(lens[b])
        j = np.arange(L)
        at = (torch.from_numpy(table[b][j // page]).long(), torch.from_numpy(j % page))
        back = (L - n + torch.arange(n, device="cuda"))[:, None] - torch.arange(L, device="cuda")
        hidden = torch.zeros_like(back, dtype=torch.bool) if not causal else (back < 0) | (window > 0) & (back >= window)
        for h in range(Hkv if L else 0):
            kk, vv = k[at[0].cuda(), h, at[1].cuda()], v[at[0].cuda(), h, at[1].cuda()]
            for head in range(h * G, h * G + G):
                qq = q[start:start + n, head]
                s = qq @ kk.T * scale
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                s = s.masked_fill(hidden, -np.inf)
                l = torch.logsumexp(s, 1)
                w = torch.exp(s - l[:, None]).nan_to_num(0.0)
                sl = slice(start, start + n)
                out[sl, head], absv[sl, head] = (w @ vv).cpu(), (w @ vv.abs()).cpu()
                lse[sl, head] = l.cpu()
                mag[sl, head] = ((qq.abs() @ kk.abs().T).amax(1) * abs(scale)).cpu()
                vmax[sl, head, 0] = vv.abs().max().cpu()
        start += n
    return tuple(x.numpy() for x in (out, lse, absv, mag, vmax))


LARGE = [
    # (heads, kv_heads, dim, page, lens, q_lens, causal, window, softcap)
    (16, 16, 128, 64, [900, 1500, 70], [900, 700, 70], True, 0, 0.0),
    (12, 12, 128, 16, [1100, 640], [500, 640], True, 0, 0.0),
    (40, 20, 64, 16, [1000, 750, 0, 33], [1000, 500, 5, 33], True, 0, 0.0),
    (20, 20, 64, 32, [640, 400], [600, 400], True, 90, 20.0),
    (16, 8, 96, 32, [777, 1300], [777, 1031], True, 0, 0.0),
    (32, 4, 128, 128, [700, 900], [500, 800], False, 0, 0.0),
    (24, 24, 256, 32, [500, 700], [500, 650], True, 0, 0.0),
    (24, 12, 192, 64, [500, 700], [500, 650], True, 333, 0.0),
]


@pytest.mark.parametrize("fmt", BOTH)
@pytest.mark.parametrize("case", LARGE, ids=[f"{c[0]}x{c[2]}-{len(c[4])}" for c in LARGE])
def test_prompts_of_many_rows(fp4, oracle, fmt, case):
    """Prompts of some hundred rows a sequence, at every size of head."""
    heads, kv_heads, dim, page, lens, q_lens, causal, window, softcap = case
    print(f"[large] {fmt} {case}", flush=True)
    attention_case(fp4, oracle, fmt, BF, lens, q_lens, heads, kv_heads, dim, page, causal=causal, window=window,
                   softcap=softcap, seed=30, ref_of=prompt_f64)


FILLING = [
    # rows and heads enough for the form for many rows: two workgroups of 128 rows a CU (heads of 64, long keys: three)
    (64, 64, 128, 64, [300, 760], [300, 720], True, 0, 0.0),
    (96, 16, 128, 32, [700, 90], [650, 90], True, 0, 0.0),
    (64, 32, 96, 16, [500, 640, 0, 40], [480, 640, 3, 45], True, 90, 20.0),
    (128, 64, 64, 32, [500, 300, 33], [470, 300, 33], True, 0, 0.0),
    (128, 64, 64, 16, [560, 420], [560, 420], False, 0, 0.0),
    (128, 64, 32, 16, [400, 260], [400, 260], True, 0, 0.0),
    (64, 64, 256, 32, [300, 760], [300, 740], True, 0, 0.0),
    (64, 64, 192, 64, [300, 760], [280, 740], True, 333, 0.0),
]


@pytest.mark.parametrize("fmt", BOTH)
@pytest.mark.parametrize("case", FILLING, ids=[f"{c[0]}x{c[2]}-{c[4][0]}" for c in FILLING])
def test_prompts_that_fill_the_gpu(fp4, oracle, fmt, case):
    heads, kv_heads, dim, page, lens, q_lens, causal, window, softcap = case
    print(f"[filling] {fmt} {case}", flush=True)
    attention_case(fp4, oracle, fmt, BF, lens, q_lens, heads, kv_heads, dim, page, causal=causal, window=window,
                   softcap=softcap, seed=32, ref_of=prompt_f64)


MIDDLE = [
    # some queries of each sequence: two row tiles in each of the launches for few rows
    (128, 16, 128, 64, [300, 77, 901, 0, 120], [7, 9, 5, 2, 12], True, 0, 0.0),           # one round, wide workgroups
    (128, 16, 96, 16, [300, 77, 901, 33, 120], [7, 0, 11, 2, 12], False, 0, 15.0),
    (128, 16, 128, 32, [500, 700, 450, 300, 120], [9, 7, 8, 9, 6], True, 61, 0.0),
    (64, 16, 64, 16, [100, 130, 31, 64] * 4, [30, 34, 31, 40] * 4, True, 0, 0.0),          # many workgroups
    (64, 16, 96, 16, [100, 130, 31, 64] * 4, [30, 33, 31, 40] * 4, False, 0, 0.0),
    (64, 8, 128, 64, [6700, 300, 41], [10, 12, 3], True, 0, 0.0),                         # runs of long keys
    (64, 8, 32, 16, [6311, 6550], [11, 10], False, 0, 0.0),
]


@pytest.mark.parametrize("fmt", BOTH)
@pytest.mark.parametrize("case", MIDDLE, ids=[f"{c[0]}x{c[2]}-{c[4][0]}" for c in MIDDLE])
def test_some_queries_of_each_sequence(fp4, oracle, fmt, case):
    heads, kv_heads, dim, page, lens, q_lens, causal, window, softcap = case
    print(f"[middle] {fmt} {case}", flush=True)
    attention_case(fp4, oracle, fmt, BF, lens, q_lens, heads, kv_heads, dim, page, causal=causal, window=window,
                   softcap=softcap, seed=31)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("window", [1, 17, 100])
def test_window(fp4, oracle, fmt, dtype, window):
    print(f"[window] {fmt} {dtype} {window}", flush=True)
    attention_case(fp4, oracle, fmt, dtype, [1, 50, 300, 777], [1] * 4, 4, 2, 64, 16, window=window, seed=14)
    attention_case(fp4, oracle, fmt, dtype, [400, 90], [150, 95], 4, 2, 128, 16, window=window, seed=15)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
def test_softcap_and_scale(fp4, oracle, fmt, dtype):
    attention_case(fp4, oracle, fmt, dtype, [333, 20], [1, 1], 8, 2, 128, 16, softcap=5.0, seed=16, q_scale=4.0)
    attention_case(fp4, oracle, fmt, dtype, [150], [140], 4, 2, 64, 16, softcap=30.0, scale=0.3, seed=17)
    attention_case(fp4, oracle, fmt, dtype, [200], [1], 4, 2, 64, 16, scale=0.0, seed=18)
    attention_case(fp4, oracle, fmt, dtype, [200, 160], [1, 150], 4, 2, 64, 16, scale=-0.2, seed=19)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
def test_peaked_and_tiny_scores(fp4, oracle, fmt, dtype):
    """Queries that leave one key almost all the weight (the running maximum
    rises many times), and queries far below and above fp16's range."""
    attention_case(fp4, oracle, fmt, dtype, [600, 64], [1, 1], 4, 2, 128, 16, seed=20, q_scale=60.0)
    attention_case(fp4, oracle, fmt, dtype, [600, 64], [1, 40], 4, 2, 128, 16, seed=21, q_scale=1e-12)
    attention_case(fp4, oracle, fmt, dtype, [130], [130], 4, 2, 128, 16, seed=22, q_scale=3e6, scale=2e-7)


def test_lengths_are_cut_to_max_kv_len(fp4, oracle):
    """kv_lens beyond max_kv_len, and below zero, count as the bound and 0."""
    cache, k, v = random_cache(fp4, oracle, MX, 8, 16, 2, 64, 1)
    table = np.arange(8, dtype=np.int32).reshape(2, 4)
    q = torch.randn(2, 4, 64).to(BF)
    out, lse = fp4.kv_attention(q.cuda(), cache, torch.from_numpy(table).cuda(),
                                torch.tensor([1000, -5], dtype=torch.int32, device="cuda"), max_kv_len=50,
                                causal=False, return_lse=True)
    ref = attention_f64(q.double().numpy(), k, v, table, 16, [50, 0], [1, 1], False, 0, 0.0, 64 ** -0.5)
    check_attention(out, lse, ref, *attention_bounds(ref, False, True, 64, 50, 0.0), "cut")


def test_wild_page_numbers_and_offsets_stay_in_bounds(fp4, oracle):
    """Page numbers outside the cache are clamped, offsets outside the tokens
    too: the call ends, and the sequences with proper values are right."""
    cache, k, v = random_cache(fp4, oracle, NV, 6, 16, 2, 64, 2)
    table = np.array([[0, 1], [2 ** 31 - 1, -2 ** 31], [4, 5]], np.int32)
    q = torch.randn(3, 4, 64).to(BF)
    lens = torch.tensor([20, 32, 17], dtype=torch.int32, device="cuda")
    out, lse = fp4.kv_attention(q.cuda(), cache, torch.from_numpy(table).cuda(), lens, return_lse=True)
    ref = attention_f64(q.double().numpy(), k, v, np.clip(table, 0, 5), 16, [20, 32, 17], [1, 1, 1], True, 0, 0.0,
                        64 ** -0.5)
    check_attention(out, lse, ref, *attention_bounds(ref, True, True, 64, 32, 0.0), "wild pages")
    offs = torch.tensor([-7, 2, 1, 99], dtype=torch.int32, device="cuda")
    fp4.kv_attention(q.cuda(), cache, torch.from_numpy(table).cuda(), lens, q_offsets=offs)
    torch.cuda.synchronize()


def test_rows_outside_every_sequence_are_not_written(fp4, oracle):
    cache, _, _ = random_cache(fp4, oracle, MX, 4, 16, 1, 64, 3)
    q = torch.randn(10, 2, 64, device="cuda").to(BF)
    out = torch.full_like(q, 7.0)
    offs = torch.tensor([2, 5, 8], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    fp4.kv_attention(q, cache, table, torch.tensor([20, 30], dtype=torch.int32, device="cuda"), q_offsets=offs, out=out)
    assert (out[:2] == 7).all() and (out[8:] == 7).all() and not (out[2:8] == 7).all(-1).any()


@pytest.mark.parametrize("fmt", BOTH)
def test_offsets_past_32_bits(fp4, oracle, fmt):
    """Pages that lie more than 2^32 bytes into the buffers."""
    page, heads, dim = 16, 2, 64
    blk = 16 if fmt == NV else 32
    small, k, v = random_cache(fp4, oracle, fmt, 3, page, heads, dim, 4)
    bufs = []
    for src in (small.k_codes, small.k_scales, small.v_codes, small.v_scales):
        step = 2300 * 1000 * 1000 // 16 * 16
        flat = torch.empty(2 * step + 4096, dtype=torch.uint8, device="cuda")
        w = src.shape[3]
        t = flat.as_strided((3, heads, page, w), (step, page * w, w, 1))
        t.copy_(src)
        bufs.append(t)
    cache = fp4.KVCache("nvfp4" if fmt == NV else "mxfp4", *bufs, small.k_tensor_scale, small.v_tensor_scale)
    table = np.array([[2, 0, 1]], np.int32)
    q = torch.randn(1, 4, dim).to(BF)
    out, lse = fp4.kv_attention(q.cuda(), cache, torch.from_numpy(table).cuda(),
                                torch.tensor([45], dtype=torch.int32, device="cuda"), return_lse=True)
    ref = attention_f64(q.double().numpy(), k, v, table, page, [45], [1], True, 0, 0.0, dim ** -0.5)
    check_attention(out, lse, ref, *attention_bounds(ref, fmt == NV, True, dim, 45, 0.0), "far pages")
    slots = torch.tensor([2 * page + 3, page], device="cuda")
    got = fp4.kv_read(cache, slots, F32)
    assert np.array_equal(got[0].double().cpu().numpy(), k[[2, 1], :, [3, 0]])
    assert np.array_equal(got[1].double().cpu().numpy(), v[[2, 1], :, [3, 0]])
    x = torch.randn(1, heads, dim, device="cuda")
    fp4.kv_append(cache, x, x, slots[:1])
    fp4.kv_append(small, x, x, slots[:1])
    assert torch.equal(cache.k_codes[2], small.k_codes[2]) and torch.equal(cache.v_scales[2], small.v_scales[2])


def test_strided_queries_and_outputs(fp4, oracle):
    """Queries and outputs as views with heads outermost, or inside a wider
    row; keys and values in one interleaved buffer."""
    cache, k, v = random_cache(fp4, oracle, NV, 6, 16, 2, 64, 6)
    both = torch.empty(6, 2, 2, 16, 32, dtype=torch.uint8, device="cuda")
    both[:, 0], both[:, 1] = cache.k_codes, cache.v_codes
    sc = torch.empty(6, 2, 2, 16, 4, dtype=torch.uint8, device="cuda")
    sc[:, 0], sc[:, 1] = cache.k_scales, cache.v_scales
    mixed = fp4.KVCache("nvfp4", both[:, 0], sc[:, 0], both[:, 1], sc[:, 1], cache.k_tensor_scale,
                        cache.v_tensor_scale)
    q = torch.randn(3, 8, 64).to(BF)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    wide = torch.zeros(3, 5, dtype=torch.int32, device="cuda")
    wide[:, :2] = table
    lens = torch.tensor([32, 5, 20], dtype=torch.int32, device="cuda")
    want = fp4.kv_attention(q.cuda(), cache, table, lens)
    qh = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros(8, 3, 64, dtype=BF, device="cuda").transpose(0, 1)
    assert torch.equal(fp4.kv_attention(qh, mixed, wide[:, :2], lens, out=out), want)
    pad = torch.zeros(3, 12, 96, dtype=BF, device="cuda")
    pad[:, 2:10, 16:80] = q.cuda()
    assert torch.equal(fp4.kv_attention(pad[:, 2:10, 16:80], mixed, wide[:, :2], lens), want)


def test_on_another_stream(fp4, oracle):
    cache, _, _ = random_cache(fp4, oracle, MX, 200, 16, 2, 128, 7)
    q = torch.randn(1, 8, 128, device="cuda").to(BF)
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(1, 200)
    lens = torch.tensor([3111], dtype=torch.int32, device="cuda")
    want = fp4.kv_attention(q, cache, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(4):
        got.append(fp4.kv_attention(q, cache, table, lens, stream=side.cuda_stream))
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    side.synchronize()
    for y in got:
        assert torch.equal(y, want)


def test_decode_steps_in_a_graph(fp4, oracle):
    """append + attention captured once and replayed: new tokens, slots and
    lengths come through the same buffers."""
    heads, kv_heads, dim, page, pages = 8, 2, 128, 16, 40
    cache = fp4.KVCache.empty("nvfp4", pages, page, kv_heads, dim, k_amax=K_AMAX, v_amax=V_AMAX)
    other = fp4.KVCache.empty("nvfp4", pages, page, kv_heads, dim, k_amax=K_AMAX, v_amax=V_AMAX)
    half = dim // 2
    ang = torch.arange(600, device="cuda")[:, None] * 10000.0 ** (-torch.arange(half, device="cuda") / half)
    cos, sin = ang.cos().contiguous(), ang.sin().contiguous()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    x = torch.zeros(1, heads + 2 * kv_heads, dim, dtype=BF, device="cuda")
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(c, x, pos, lens):
        q = fp4.kv_append(c, x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], pos, q=x[:, :heads],
                          positions=pos, cos=cos, sin=sin)
        return fp4.kv_attention(q, c, table, lens)

    step(other, x, pos, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(cache, x, pos, lens)
    for t in range(0, 35):
        x.copy_(torch.randn_like(x, dtype=F32))
        pos.fill_(t)
        lens.fill_(t + 1)
        graph.replay()
        want = step(other, x, pos, lens)
        torch.cuda.synchronize()
        assert torch.equal(y, want), f"replay {t}"
        assert torch.equal(cache.k_codes, other.k_codes) and torch.equal(cache.v_scales, other.v_scales)
