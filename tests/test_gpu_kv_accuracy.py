"""Attention over the 4-bit cache where its arithmetic is strained: softcaps of
every size, weights far below the largest, scores far from 0."""
import numpy as np
import pytest
import torch

from kv_util import attention_bounds, attention_f64, check_attention, lay_out, random_cache

pytestmark = pytest.mark.gpu

MX, NV = 0, 1
BF, F32 = torch.bfloat16, torch.float32
FD = [(f, d) for f in (MX, NV) for d in (BF, F32)]
FD_IDS = ["mx-bf16", "mx-f32", "nv-bf16", "nv-f32"]


def attend(F, cache, q, table, lens, q_lens, **kw):
    """out, lse of one call over sequences of `lens` rows."""
    offs = torch.tensor(np.cumsum([0] + list(q_lens)), dtype=torch.int32, device="cuda")
    out, lse = F.kv_attention(q.cuda(), cache, torch.from_numpy(table).cuda(),
                              torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              q_offsets=None if all(n == 1 for n in q_lens) else offs, max_kv_len=max(lens),
                              return_lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


# ---------------------------------------------------------------------------
# softcap
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("softcap", [1e-45, 1e-38, 1e-3, 0.5, 30.0, 1e3, 1e6, 1e9, 3e38])
@pytest.mark.parametrize("q_scale", [0.05, 2.0])
def test_softcap_of_any_size(fp4, oracle, fmt, dtype, softcap, q_scale):
    """The capped score is as exact as the score itself, whatever the cap:
    16 roundings more (products with the cap and its inverse, and tanh within
    10 units of 2^-24 of its own size), as if 16 elements of a head more were
    summed. A cap below the normal numbers leaves scores of 0."""
    print(f"[softcap] {fmt} {dtype} {softcap} {q_scale}", flush=True)
    lens, q_lens, heads, kv_heads, dim, page = [90, 33, 161], [1, 20, 7], 4, 2, 32, 16
    cache, k, v = random_cache(fp4, oracle, fmt, 23, page, kv_heads, dim, 50)
    table = lay_out(cache, lens, 51)
    g = torch.Generator().manual_seed(52)
    q = (q_scale * torch.randn(sum(q_lens), heads, dim, generator=g)).to(dtype)
    out, lse = attend(fp4, cache, q, table, lens, q_lens, softcap=softcap)
    cap = float(np.float32(softcap))
    ref = attention_f64(q.double().numpy(), k, v, table, page, lens, q_lens, True, 0, cap, float(np.float32(dim ** -0.5)))
    tol, tol_lse = attention_bounds(ref, fmt == NV, dtype == BF, dim + 16, max(lens), 0.0)
    check_attention(out, lse, ref, tol, tol_lse, f"softcap {softcap}")


# ---------------------------------------------------------------------------
# weights far below the largest
# ---------------------------------------------------------------------------
def cache_of(F, O, fmt, x, page):
    """A cache of one kv head whose rows are x = (k, v), each [rows, dim] fp32
    (whole pages), quantized by the oracle; and their values."""
    out, vals = [], []
    for t in x:
        r = O.quantize(np.ascontiguousarray(t, np.float32), fmt, amax=float(np.abs(t).max()) if fmt == NV else None)
        vals.append(np.asarray(O.dequantize(fmt, r["codes"], r["scales"], r["tensor_scale"]), np.float64)
                    .reshape(-1, 1, page, t.shape[1]))
        out += [torch.from_numpy(r[n].reshape(-1, 1, page, r[n].shape[-1]).copy()).cuda() for n in ("codes", "scales")]
        out.append(torch.full((1,), float(r["tensor_scale"])).cuda() if fmt == NV else None)
    kc, ks, kt, vc, vs, vt = out
    return F.KVCache("nvfp4" if fmt == NV else "mxfp4", kc, ks, vc, vs, kt, vt), *vals


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("queries", [1, 3])
@pytest.mark.parametrize("keys,bits", [(41, 20.0), (900, 26.0), (130001, 31.5), (4000, 45.0), (60, 80.0)])
def test_small_weights_of_fp32_calls(fp4, oracle, fmt, queries, keys, bits):
    """One key takes nearly all the weight and has values of 0; the result is
    what the others, each 2^-bits of it, leave: fp32 calls keep them all."""
    print(f"[sink] {fmt} {queries} {keys} {bits}", flush=True)
    dim, page = 32, 16
    rows = -(-keys // page) * page
    rng = np.random.RandomState(60)
    k = np.zeros((rows, dim), np.float32)
    sink = keys // 2
    k[sink] = rng.uniform(1, 4, dim)
    v = rng.uniform(0.5, 6.0, (rows, dim)).astype(np.float32)
    v[sink] = 0
    cache, kv, vv = cache_of(fp4, oracle, fmt, (k, v), page)
    q = torch.from_numpy(rng.uniform(0.5, 1.5, (queries, 1, dim)).astype(np.float32))
    dots = q.double().numpy()[:, 0] @ kv[sink // page, 0, sink % page]
    scale = float(np.float32(bits * np.log(2) / dots.max()))
    table = np.arange(rows // page, dtype=np.int32)[None]
    out, lse = attend(fp4, cache, q, table, [keys], [queries], scale=scale, causal=False)
    ref = attention_f64(q.double().numpy(), kv, vv, table, page, [keys], [queries], False, 0, 0.0, scale)
    # every term of attention_bounds but NVFP4's loss of small weights
    tol, tol_lse = attention_bounds(ref, False, False, dim, keys, 0.0)
    check_attention(out, lse, ref, tol, tol_lse, f"sink {keys} {bits}")


# ---------------------------------------------------------------------------
# scores of any finite size
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("scale", [3e5, 7e8, 1.1e20, -9e7])
def test_large_scores(fp4, oracle, fmt, dtype, queries, scale):
    """Scores so large that the largest of a row takes all the weight, and
    equal ones share it: k has one element that counts, -6 to 6 in exact
    values, and the query is a one there."""
    print(f"[large scores] {fmt} {dtype} {queries} {scale}", flush=True)
    dim, page, keys = 32, 16, 200
    rng = np.random.RandomState(61)
    k, v = np.zeros((208, dim), np.float32), rng.choice([-4, -3, -2, 1, 2, 3, 6], (208, dim)).astype(np.float32)
    k[:, 0] = rng.choice([-4, -3, -2, -1, 0, 1, 2, 3], 208)
    k[:, 16] = v[:, 31] = 6                # one scale for all blocks of a row
    best = 6 if scale > 0 else -6
    k[[70, 130, 131, 150], 0] = best       # four rows with the largest score
    cache, kv, vv = cache_of(fp4, oracle, fmt, (k, v), page)
    assert np.array_equal(kv.reshape(208, dim)[:, 0], k[:, 0]) or fmt == NV
    q = torch.zeros(queries, 1, dim, dtype=dtype)
    q[..., 0] = 1
    table = np.arange(13, dtype=np.int32)[None]
    out, lse = attend(fp4, cache, q, table, [keys], [queries], scale=scale, causal=False)
    vals, keyv = vv.reshape(208, dim), kv.reshape(208, dim)[:keys, 0]
    top = np.flatnonzero(keyv * np.sign(scale) == (keyv * np.sign(scale)).max())
    assert list(top) == [70, 130, 131, 150]
    want = vals[top].mean(0)
    got = out.double().cpu().numpy()[:, 0]
    # equal weights: a quarter of an exact sum, and one rounding
    assert (np.abs(got - want) <= np.abs(vals[top]).mean(0) * 2.0 ** (-8 if dtype == BF else -22)).all()
    score = keyv[top[0]] * float(np.float32(scale))
    assert np.allclose(lse.double().cpu().numpy(), score + np.log(4), rtol=2.0 ** -21)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("queries,keys", [(1, 200), (40, 200), (1, 9000)])
@pytest.mark.parametrize("scale", [-2e29, -1e37])
def test_scores_far_below_zero(fp4, oracle, fmt, dtype, queries, keys, scale):
    """Scores of -6e29 and less are scores still: a row whose keys all have
    them is their mean, not a row that sees nothing."""
    print(f"[low scores] {fmt} {dtype} {queries} {keys} {scale}", flush=True)
    dim, page = 32, 16
    rows = -(-keys // page) * page
    k = np.full((rows, dim), 6, np.float32)
    v = np.random.RandomState(62).choice([1, 2, 3, 4, 6], (rows, dim)).astype(np.float32)
    v[:, 31] = 6
    v[:, 15] = 6
    cache, kv, vv = cache_of(fp4, oracle, fmt, (k, v), page)
    q = torch.zeros(queries, 1, dim, dtype=dtype)
    q[..., 0] = 1
    table = np.arange(rows // page, dtype=np.int32)[None]
    out, lse = attend(fp4, cache, q, table, [keys], [queries], scale=scale, causal=False)
    want = vv.reshape(rows, dim)[:keys].mean(0)
    got = out.double().cpu().numpy()[:, 0]
    # equal weights: fp32 sums of `keys` terms, and one rounding
    assert (np.abs(got - want) <= want * (2.0 ** (-8 if dtype == BF else -23) + (keys + 64) * 2.0 ** -23)).all()
    assert np.allclose(lse.double().cpu().numpy(), kv.reshape(-1)[0] * float(np.float32(scale)), rtol=2.0 ** -21)
