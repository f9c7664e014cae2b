"""Definitions in 64 bits of the mixture-of-experts operators (host, numpy)."""
import numpy as np

INF = np.inf


def scores(z, score):
    """z [T, E] float64 -> the scores; -inf counts as score 0, a row of -inf as zeros."""
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            small = np.exp(-np.abs(z))
            return np.where(z >= 0, 1.0, small) / (1.0 + small)
        top = z.max(1, keepdims=True)
        p = np.exp(z - np.where(np.isfinite(top), top, 0.0))
        total = p.sum(1, keepdims=True)
        return p / np.where(total > 0, total, 1.0)


def route(z, k, score="softmax", bias=None, groups=1, top_groups=None, best=1, renormalize=True, scale=1.0):
    """(weights, ids) of logits z [T, E] float64 by the definition."""
    T, E = z.shape
    top_groups = groups if top_groups is None else top_groups
    s = scores(z, score)
    banned = ~(z > -INF)
    c = s.copy()
    if bias is not None:
        b = bias.astype(np.float64)
        banned = banned | ~(b > -INF)
        c = s + np.where(b > -INF, b, 0.0)
    c = np.where(banned, -INF, c)
    if top_groups < groups:
        parts = np.sort(c.reshape(T, groups, -1), -1)[..., ::-1]
        rank = parts[..., 0].copy()
        if best == 2 and parts.shape[-1] > 1:
            rank = rank + np.where(parts[..., 1] > -INF, parts[..., 1], 0.0)
        order = np.argsort(-rank, 1, kind="stable")[:, :top_groups]
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, order, True, 1)
        c = np.where(np.repeat(kept, E // groups, 1), c, -INF)
    by = c if bias is not None else np.where(c > -INF, z, -INF)  # (scores may round to one number)
    ids = np.argsort(-by, 1, kind="stable")[:, :k]
    there = np.take_along_axis(c, ids, 1) > -INF
    return weights(z, np.where(there, ids, -1), score, renormalize, scale), np.where(there, ids, -1).astype(np.int32)


def weights(z, ids, score, renormalize, scale):
    there = ids >= 0
    at = np.where(there, ids, 0)
    zj = np.where(there, np.take_along_axis(z, at, 1), -INF)
    if renormalize:
        with np.errstate(invalid="ignore"):
            lw = zj if score == "softmax" else np.minimum(zj, 0) - np.log1p(np.exp(-np.abs(zj)))
            top = lw.max(1, keepdims=True)
            w = np.where(there, np.exp(lw - np.where(np.isfinite(top), top, 0)), 0.0)
        total = w.sum(1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    else:
        w = np.where(there, np.take_along_axis(scores(z, score), at, 1), 0.0)
    return w * scale


def route_gradient(grad, z, ids, score, renormalize, scale):
    """d sum(grad * weights) / dz by the chain rule, score by score."""
    T, E = z.shape
    out = np.zeros((T, E))
    s = scores(z, score)
    w = weights(z, ids, score, renormalize, 1.0)
    for j in range(ids.shape[1]):
        e = ids[:, j]
        rows = np.nonzero((e >= 0) & (e < E))[0]
        e = e[rows]
        g = grad[rows, j] * scale
        if renormalize:  # w_j = exp(lw_j) / sum: d by each chosen lw
            for i in range(ids.shape[1]):
                f = ids[rows, i]
                ok = f >= 0
                d = g * w[rows, j] * ((i == j) - w[rows, i])
                slope = (1 - s[rows, f]) if score == "sigmoid" else 1.0
                np.add.at(out, (rows[ok], f[ok]), (d * slope)[ok])
        elif score == "sigmoid":
            np.add.at(out, (rows, e), g * s[rows, e] * scores(-z, score)[rows, e])
        else:
            out[rows] -= (g * s[rows, e])[:, None] * s[rows]
            np.add.at(out, (rows, e), g * s[rows, e])
    return out


def group(ids, experts):
    """(offsets, order, place) of the stable sort; pairs without an expert last."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable").astype(np.int32)
    place = np.empty_like(order)
    place[order] = np.arange(order.size, dtype=np.int32)
    offsets = np.concatenate(([0], np.cumsum(np.bincount(key, minlength=experts + 1)[:experts]))).astype(np.int32)
    return offsets, order, place.reshape(ids.shape)


def values(q):
    """What a Quantized tensor (device) stands for, float64 on the host: E2M1 by its fields, scales by theirs."""
    codes, scales_ = q.codes.cpu().numpy().astype(np.int64), q.scales.cpu().numpy().astype(np.int64)
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    e, m = (n & 7) >> 1, n & 1
    v = np.where(n & 8, -1.0, 1.0) * np.where(e == 0, m * 0.5, 2.0 ** (e - 1.0) * (1 + m * 0.5))
    if q.fmt == 0:
        sc = 2.0 ** (scales_ - 127.0)
    else:
        e, m = (scales_ & 127) >> 3, scales_ & 7
        sc = np.where(e == 0, 2.0 ** -6 * m / 8.0, 2.0 ** (e - 7.0) * (1 + m / 8.0))
        ts = q.tensor_scale.double().cpu().numpy()
        sc = sc * ts.reshape(ts.shape + (1,) * (sc.ndim - 1)) if sc.ndim == 3 else sc * ts[0]
    return v * np.repeat(sc, 32 if q.fmt == 0 else 16, -1)
