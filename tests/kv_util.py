"""Helpers of the key-value cache tests: random caches, and the operators'
definitions in 64 bits on the CPU."""
import numpy as np
import torch

K_AMAX, V_AMAX = 40.0, 30.0


def rotate_f32(x, cos, sin, interleaved):
    """x [T, H, D] fp32 (numpy), cos and sin [T, R / 2]: each product and sum
    rounded once to fp32."""
    y = x.copy()
    half = cos.shape[1]
    c, s = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ya, yb = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ya, yb
    else:
        y[..., :half], y[..., half:2 * half] = ya, yb
    return y


def random_cache(F, O, fmt, pages, page, heads, dim, seed, fos=False, garbage=True):
    """A cache whose every row is a quantized random vector (by the oracle):
    (KVCache, k [pages, heads, page, dim], v) with the values as float64."""
    g = torch.Generator().manual_seed(seed)
    nv = fmt == O.NVFP4
    out, vals = [], []
    div = np.float32(1792.0 if fos else 2688.0)
    for amax in (K_AMAX, V_AMAX):
        x = torch.randn(pages * heads * page, dim, generator=g)
        x[:, : max(1, dim // 16)] *= 4
        r = O.quantize(x.numpy(), fmt, flags=O.FOUR_OVER_SIX if fos else 0, amax=amax if nv else None)
        v = O.dequantize(fmt, r["codes"], r["scales"], r["tensor_scale"])
        vals.append(np.asarray(v, np.float64).reshape(pages, heads, page, dim))
        for n in ("codes", "scales"):
            out.append(torch.from_numpy(r[n].reshape(pages, heads, page, -1).copy()))
        if nv:
            assert np.float32(r["tensor_scale"]) == np.float32(amax) / div
    ts = [torch.full((heads,), float(np.float32(a) / div)).cuda() if nv else None for a in (K_AMAX, V_AMAX)]
    cache = F.KVCache("nvfp4" if nv else "mxfp4", *(t.cuda() for t in out), *ts)
    return cache, vals[0], vals[1]


def lay_out(cache, lens, seed, width=None, spare=1):
    """A block table [batch, width] over random distinct pages for sequences of
    `lens` rows; entries past a sequence's pages are -1."""
    page = cache.page_size
    need = [-(-n // page) for n in lens]
    width = max(need + [1]) if width is None else width
    order = np.random.RandomState(seed).permutation(cache.num_pages)
    assert sum(need) + spare <= cache.num_pages
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def spoil(cache, table, lens):
    """Bytes that stand for no number (0xFF: NaN scales) wherever no sequence
    has a row."""
    page = cache.page_size
    held = np.zeros((cache.num_pages, page), bool)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            held[table[b, j], : min(page, n - j * page)] = True
    m = torch.from_numpy(~held).cuda()[:, None, :, None]
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.masked_fill_(m, 255)


def attention_f64(q, k, v, table, page, lens, q_lens, causal, window, softcap, scale):
    """q [tokens, H, D] float64; k, v [pages, Hkv, page, D]. Returns out, lse,
    the weighted sum of |v| and the largest score magnitudes that the
    tolerances are made of: sum_d |q k| * scale per row (its maximum over the
    keys seen), and the number of keys."""
    T, H, D = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    out, absv = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, mag = np.full((T, H), -np.inf), np.zeros((T, H))
    vmax = np.zeros((T, H, 1))
    start = 0
    for b, n in enumerate(q_lens):
        L = int(lens[b])
        j = np.arange(L)
        rows = (table[b][j // page], j % page) if L else None
        for h in range(Hkv):
            if not L:
                continue
            kk, vv = k[rows[0], h, rows[1]], v[rows[0], h, rows[1]]
            for i in range(n):
                last = L - n + i if causal else L - 1
                first = max(0, last - window + 1) if window else 0
                if last < first:
                    continue
                sl = slice(first, last + 1)
                qq = q[start + i, h * G:(h + 1) * G]
                s = qq @ kk[sl].T * scale
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                top = s.max(1, keepdims=True)
                e = np.exp(s - top)
                z = e.sum(1, keepdims=True)
                hs = slice(h * G, (h + 1) * G)
                out[start + i, hs] = e / z @ vv[sl]
                absv[start + i, hs] = e / z @ np.abs(vv[sl])
                lse[start + i, hs] = (top + np.log(z))[:, 0]
                mag[start + i, hs] = (np.abs(qq) @ np.abs(kk[sl]).T).max(1) * abs(scale)
                vmax[start + i, hs, 0] = np.abs(vv[sl]).max()
        start += n
    return out, lse, absv, mag, vmax


def attention_bounds(ref, fmt_nv, bf16, D, max_len, softcap):
    """Element bounds of the kernel's result, from its arithmetic.
    Scores: fp32 accumulation over D, a few roundings and the hardware's exp2;
    fp32 queries are held to 2^-22 (NVFP4: two fp16 terms) or 2^-24. A score
    off by e scales its weight by 1 + e, in the numerator and the sum alike.
    Weights: 16-bit rounding (bf16 2^-8, fp16 2^-11), to the third power and
    squared where three and two terms are kept; fp16 loses at most 2^-25 of the lifted scale 2^-6 per key.
    Sums: fp32 over max_len keys. Result: one rounding."""
    out, lse, absv, mag, vmax = ref
    e = (D + 8) * 2.0 ** -24 * mag + 2.0 ** -20
    if not bf16:
        e = e + 2.0 ** -21 * mag
    if softcap:
        e = e + softcap * 2.0 ** -20
    u_p = (2.0 ** -11 if fmt_nv else 2.0 ** -8) if bf16 else (2.0 ** -22 if fmt_nv else 2.0 ** -24)
    sums = (max_len + 64) * 2.0 ** -24
    tol = (u_p + 2 * e[..., None] + 2 * sums) * absv + (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(out)
    if fmt_nv:
        tol = tol + max_len * 2.0 ** -31 * vmax
    tol_lse = e + sums + 2.0 ** -20 + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0)
    return tol + 1e-30, tol_lse


def check_attention(got, got_lse, ref, tol, tol_lse, what):
    out, lse = ref[0], ref[1]
    g, gl = got.double().cpu().numpy(), got_lse.double().cpu().numpy()
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty), f"{what}: rows without keys differ"
    assert (g[empty] == 0).all(), f"{what}: a row without keys is not zero"
    err = np.abs(g - out)
    assert np.isfinite(g).all(), f"{what}: {np.count_nonzero(~np.isfinite(g))} values are not finite"
    bad = err > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} beyond the bound, worst {np.max(err / tol):.3g} of it at "
                           f"{np.unravel_index(np.argmax(err / tol), err.shape)}")
    el = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, lse))
    assert (el <= tol_lse).all(), f"{what}: lse beyond the bound, worst {np.max(el / tol_lse):.3g} of it"
