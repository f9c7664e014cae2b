"""A router's choice, its weights and their gradient against the definition in
64 bits (moe_util): the ids have to be equal, ties and near ties included.

Weights: a score is exp of a difference rounded once (an error of |d| 2^-24),
times what the hardware's exponential, a correction, a division and a product
round (below 8 * 2^-24), over a sum of positive terms, each with its own such
error and at most 16 + 6 + 2 additions: 48 + 2 |d| units of 2^-24 with room,
d the distance from the row's largest logit. Below 1e-30 only the size counts."""
import numpy as np
import pytest
import torch

import moe_util as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def logits(T, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)).to(DT[dtype])


def check(fp4, z, k, bias=None, **kw):
    """Runs the router on host logits z; ids equal, weights within their bound. Returns the device's."""
    dev = z.cuda()
    b = None if bias is None else bias.cuda()
    opts = {("group_best" if n == "best" else n): v for n, v in kw.items()}
    w, ids = fp4.moe_route(dev, k, bias=b, **opts)
    z64 = z.double().numpy()
    want, want_ids = M.route(z64, k, bias=None if bias is None else bias.numpy(), **kw)
    got = ids.cpu().numpy()
    bad = np.nonzero((got != want_ids).any(1))[0]
    assert bad.size == 0, f"{bad.size} rows differ, first {bad[0]}: {got[bad[0]]}, not {want_ids[bad[0]]}"
    w = w.double().cpu().numpy()
    top = np.where(np.isfinite(z64), z64, -np.inf).max(1, keepdims=True)
    d = np.where(want_ids >= 0, top - np.take_along_axis(z64, np.maximum(want_ids, 0), 1), 0)
    with np.errstate(invalid="ignore"):
        tol = (48 + 2 * np.abs(d)) * U * np.abs(want) + 1e-30
    assert (np.abs(w - want) <= tol).all(), np.nanmax(np.abs(w - want) / tol)
    return ids


CASES = [
    # T, E, k, options
    (1, 32, 4, dict()),
    (1, 1, 1, dict()),
    (3, 7, 7, dict(renormalize=False)),
    (33, 17, 3, dict(score="sigmoid")),
    (64, 60, 4, dict(score="sigmoid", renormalize=False, scale=2.5)),
    (65, 64, 6, dict(renormalize=False, scale=16.0)),
    (7, 128, 8, dict(groups=8, top_groups=3)),
    (129, 256, 8, dict(score="sigmoid", groups=8, top_groups=4, best=2, scale=2.5)),
    (40, 160, 6, dict(groups=8, top_groups=3, renormalize=False)),
    (50, 60, 5, dict(groups=4, top_groups=2, best=2)),
    (20, 96, 20, dict(groups=32, top_groups=11, best=2)),
    (20, 64, 8, dict(groups=64, top_groups=9, best=2)),
    (9, 1024, 32, dict(score="sigmoid")),
    (9, 1000, 10, dict(groups=10, top_groups=4, best=2, renormalize=False)),
    (9, 257, 9, dict(score="sigmoid", groups=1)),
    (31, 240, 6, dict(groups=24, top_groups=7, best=2)),
    (31, 200, 15, dict(score="sigmoid", groups=40, top_groups=17)),
    (600, 190, 13, dict(score="sigmoid")),
    (601, 192, 8, dict(score="sigmoid", groups=8, top_groups=4, best=2, scale=2.5)),
    (37, 144, 6, dict(groups=9, top_groups=4, best=2)),
    # more tokens
    (1500, 8, 2, dict()),
    (1501, 16, 16, dict(score="sigmoid")),
    (2000, 32, 4, dict(scale=0.5)),
    (1999, 33, 20, dict(renormalize=False)),
    (1700, 128, 32, dict(score="sigmoid", groups=16, top_groups=5, best=2)),
    (1600, 256, 8, dict(groups=8, top_groups=4, best=2)),
    (1600, 252, 17, dict(groups=12, top_groups=7, renormalize=False)),
    (1300, 300, 8, dict(groups=20, top_groups=6, best=2)),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,kw", CASES, ids=[f"{c[0]}x{c[1]}k{c[2]}-{i}" for i, c in enumerate(CASES)])
def test_route(fp4, T, E, k, kw, with_bias, dtype):
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(T)) if with_bias else None
    check(fp4, logits(T, E, dtype, 100 + E), k, bias, **kw)


@pytest.mark.parametrize("T", [5, 1500])
@pytest.mark.parametrize("kw", [dict(), dict(score="sigmoid", groups=4, top_groups=2, best=2)],
                         ids=["softmax", "sigmoid-groups"])
def test_equal_values_go_to_the_lowest_index(fp4, T, kw):
    z = torch.zeros(T, 32)
    ids = check(fp4, z, 6, **kw)
    assert (ids.cpu() == torch.arange(6)).all()
    check(fp4, z, 6, torch.zeros(32), **kw)
    z = (logits(T, 32, "bf16", 3).float() * 4).round() / 4  # many equal logits
    z[:, 5] = -0.0
    z[:, 9] = 0.0
    check(fp4, z, 6, **kw)
    check(fp4, z.bfloat16(), 6, torch.zeros(32), **kw)
    check(fp4, z, 6, 0.25 * torch.arange(32).fmod(3), **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(200, 64), (1500, 64), (1500, 256)])
def test_choice_is_that_of_the_exact_scores(fp4, score, T, E):
    """Pairs of experts whose biased scores differ by less than fp32 rounds."""
    z = logits(T, E, "f32", 11).double().numpy()
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(4))).numpy()
    s = M.scores(z, score)
    rng = np.random.default_rng(5)
    for t in range(T):  # move one of the best experts' logits next to another's choice value
        best = np.argsort(-(s[t] + bias))[:4]
        a, b = rng.permutation(best)[:2]
        want = s[t, a] + float(bias[a]) - float(bias[b])
        if 1e-6 < want < 1 - 1e-6 and score == "sigmoid":
            z[t, b] = np.log(want / (1 - want))
        elif score == "softmax" and 0 < want < 1:
            for _ in range(60):  # its own score moves the sum
                rest = np.exp(z[t]).sum() - np.exp(z[t, b])
                want = np.exp(z[t, a]) / (rest + np.exp(z[t, b])) + float(bias[a]) - float(bias[b])
                if not 0 < want < 1:
                    break
                z[t, b] = np.log(rest * want / (1 - want))
    z = torch.from_numpy(z).float()
    c = M.scores(z.double().numpy(), score) + bias.astype(np.float64)
    near = np.sort(c, 1)[:, ::-1][:, :5]
    assert (near[:, :-1] - near[:, 1:] < 1e-7).any(1).mean() > 0.3  # (the rows are what they are meant to be)
    check(fp4, z, 4, torch.from_numpy(bias), score=score)
    check(fp4, z, 4, torch.from_numpy(bias), score=score, groups=8, top_groups=3, best=2)
    check(fp4, z, 4, score=score, groups=8, top_groups=3, best=2)


def near_ranks(T, E, score, bias, groups, top_groups, best):
    """Logits whose last group kept and first left out have ranks that differ by less than fp32 resolves."""
    z = logits(T, E, "f32", 21).double().numpy()
    b = 0.0 if bias is None else bias.double().numpy()
    rows = np.arange(T)

    def ranks():
        parts = np.sort((M.scores(z, score) + b).reshape(T, groups, -1), -1)
        return parts[..., -best:].sum(-1)

    order = np.argsort(-ranks(), 1)
    a, f = order[:, top_groups - 1], order[:, top_groups]
    e = f * (E // groups) + np.argmax((M.scores(z, score) + b).reshape(T, groups, -1)[rows, f], -1)
    for _ in range(60):  # the best score of the one left out moves to where the ranks meet
        r, s = ranks(), M.scores(z, score)[rows, e]
        want = np.clip(s + r[rows, a] - r[rows, f], 0.5 * s, 1 - 1e-6)
        z[rows, e] += np.log(want / s) + (np.log((1 - s) / (1 - want)) if score == "sigmoid" else 0)
    z = z.astype(np.float32).astype(np.float64)
    gap = np.abs(ranks()[rows, a] - ranks()[rows, f])
    assert ((gap > 1e-13) & (gap < 2e-7)).mean() > 0.3  # (the rows are what they are meant to be)
    z[gap < 1e-13] = np.arange(E) / E                   # (nearer than 64 bits tell: another row)
    return torch.from_numpy(z).float()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,best", [(256, 8, 4, 2), (64, 8, 3, 2), (160, 10, 4, 2), (192, 8, 4, 2),
                                                      (96, 3, 1, 2), (32, 16, 5, 2), (40, 5, 2, 2), (640, 20, 6, 2)])
def test_groups_are_those_of_the_exact_ranks(fp4, E, groups, top_groups, best, with_bias, score):
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(8)) if with_bias else None
    z = near_ranks(300, E, score, bias, groups, top_groups, best)
    check(fp4, z, 4, bias, score=score, groups=groups, top_groups=top_groups, best=best)


@pytest.mark.parametrize("T", [6, 1500])
def test_saturated_scores_and_large_biases(fp4, T):
    z = logits(T, 48, "f32", 6, 12.0)
    bias = 0.01 * torch.randn(48, generator=torch.Generator().manual_seed(1))
    check(fp4, z + 20, 5, bias, score="sigmoid")       # scores next to 1
    check(fp4, z + 20, 5, score="sigmoid")
    check(fp4, z - 150, 5, bias, score="sigmoid")      # scores below fp32's range
    check(fp4, z - 150, 5, score="sigmoid")
    check(fp4, 20 * z, 5, score="softmax", renormalize=True)
    bias[7::5] = -1e30                                 # left out by a number
    check(fp4, z, 5, bias)
    check(fp4, z, 5, bias, score="sigmoid", groups=6, top_groups=2, best=2)
    bias[8::5] = 1e6
    check(fp4, z, 5, bias, score="sigmoid")


@pytest.mark.parametrize("T", [8, 1500])
@pytest.mark.parametrize("kw", [dict(), dict(renormalize=False), dict(score="sigmoid"),
                                dict(groups=4, top_groups=2, best=2),
                                dict(score="sigmoid", groups=4, top_groups=2, best=1, renormalize=False)],
                         ids=["softmax", "plain", "sigmoid", "groups", "sigmoid-groups"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(fp4, T, kw, with_bias):
    z = logits(T, 40, "f32", 21)
    hide = torch.rand(T, 40, generator=torch.Generator().manual_seed(2))
    z[hide < 0.3] = -torch.inf
    z[0] = -torch.inf                    # nothing is left
    z[1, :] = -torch.inf
    z[1, 13] = -3.0                      # one expert is left
    z[2, 4:] = -torch.inf                # fewer than top_k
    z[3, :10] = -torch.inf               # a whole group
    z[4] = torch.finfo(torch.float32).min  # the lowest number is no mask
    bias = None
    if with_bias:
        bias = 0.1 * torch.randn(40, generator=torch.Generator().manual_seed(3))
        bias[[3, 17]] = -torch.inf
    ids = check(fp4, z, 6, bias, **kw).cpu()
    assert (ids[0] == -1).all() and ids[1, 0] == 13 and (ids[1, 1:] == -1).all()


def test_nan_is_never_chosen_and_ids_stay_in_bounds(fp4):
    for T in (30, 1500):
        z = logits(T, 24, "f32", 8)
        z[::3, 5] = torch.nan
        z[1::3, 6] = torch.inf
        bias = torch.zeros(24)
        for kw in (dict(), dict(score="sigmoid"), dict(bias=bias.cuda()), dict(groups=4, top_groups=1, group_best=2)):
            w, ids = fp4.moe_route(z.cuda(), 5, **kw)
            ids = ids.cpu()
            assert ((ids >= -1) & (ids < 24)).all() and not (ids[::3] == 5).any()
            for row in ids.tolist():
                real = [e for e in row if e >= 0]
                assert len(set(real)) == len(real)
        # sigmoid scores have no part in one another: other experts of such a row are unharmed
        w, ids = fp4.moe_route(z.cuda(), 5, score="sigmoid", renormalize=False)
        z2 = torch.where(z.isnan(), -torch.inf, z)
        want, want_ids = M.route(z2.double().numpy()[::3], 5, score="sigmoid", renormalize=False)
        assert (ids.cpu().numpy()[::3] == want_ids).all()


def test_row_pitch_and_empty(fp4):
    wide = logits(70, 90, "bf16", 31).cuda()
    part = wide[:, 7:41]
    w, ids = fp4.moe_route(part, 4)
    w2, ids2 = fp4.moe_route(part.contiguous(), 4)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    g = torch.randn(70, 4).cuda()
    assert torch.equal(fp4.moe_route_backward(g, part, ids), fp4.moe_route_backward(g, part.contiguous(), ids))
    w, ids = fp4.moe_route(wide[:0], 4)
    assert w.shape == ids.shape == (0, 4)
    assert fp4.moe_route_backward(g[:0], wide[:0], ids).shape == (0, 90)


BACKWARD = [(1, 32, 4), (5, 1, 1), (37, 60, 6), (33, 1024, 32), (1500, 16, 16), (1501, 160, 6), (1400, 256, 20),
            (4400, 160, 6), (4500, 100, 7)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k", BACKWARD)
def test_backward(fp4, T, E, k, renormalize, score, dtype):
    """Against the formula in 64 bits. A gradient is a product of at most three
    such scores with a difference of dw and a sum of k products: the error is
    within (64 + 2 |d|) 2^-24 of the sum of what enters it in magnitude, and bf16 rounds it once."""
    z = logits(T, E, dtype, 40 + E)
    ids = torch.from_numpy(M.route(z.double().numpy(), k, score=score)[1])
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    if k > 2:
        ids[T // 2, 1] = -1
    out = fp4.moe_route_backward(g.cuda(), z.cuda(), ids.cuda(), score=score, renormalize=renormalize, scale=1.5)
    assert out.dtype == z.dtype and out.shape == z.shape
    z64, i64 = z.double().numpy(), ids.numpy()
    want = M.route_gradient(g.double().numpy(), z64, i64, score, renormalize, 1.5)
    w = M.weights(z64, i64, score, renormalize, 1.5)
    size = (np.abs(g.double().numpy()) * w).sum(1, keepdims=True)
    mass = np.zeros_like(want)
    np.put_along_axis(mass, np.maximum(i64, 0), np.abs(w) * (np.abs(g.double().numpy()) * 1.5 + size), 1)
    if score == "softmax" and not renormalize:
        mass = mass + M.scores(z64, score) * size
    spread = 2 * np.abs(z64.max(1, keepdims=True) - z64)
    tol = (64 + spread) * U * mass + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_backward_against_differences(fp4, score, renormalize):
    T, E, k, h = 12, 20, 4, 1e-6
    z = logits(T, E, "f32", 77)
    z64 = z.double().numpy()
    ids = M.route(z64, k, score=score)[1]
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
    out = fp4.moe_route_backward(g.cuda(), z.cuda(), torch.from_numpy(ids).cuda(), score=score,
                                 renormalize=renormalize).double().cpu().numpy()
    loss = lambda y: (M.weights(y, ids, score, renormalize, 1.0) * g.double().numpy()).sum(1)
    for e in range(E):
        step = np.zeros((1, E))
        step[0, e] = h
        diff = (loss(z64 + step) - loss(z64 - step)) / (2 * h)
        # the difference: h^2 times a third derivative below 8, and 1e-16 / h of cancellation
        assert np.abs(out[:, e] - diff).max() <= 1e-9 + 1e-6 * np.abs(g.numpy()).max() * 4


def test_backward_counts_an_id_twice_and_skips_strangers(fp4):
    z = logits(4, 10, "f32", 5)
    g = torch.randn(4, 3, generator=torch.Generator().manual_seed(3))
    ids = torch.tensor([[2, 2, 7], [-1, 10, 3], [-1, -1, -1], [9, 0, 1 << 30]], dtype=torch.int32)
    for score in ("softmax", "sigmoid"):
        out = fp4.moe_route_backward(g.cuda(), z.cuda(), ids.cuda(), score=score, renormalize=False).cpu().double().numpy()
        known = np.where((ids.numpy() < 0) | (ids.numpy() >= 10), -1, ids.numpy())
        want = M.route_gradient(g.double().numpy(), z.double().numpy(), known, score, False, 1.0)
        assert np.abs(out - want).max() <= 80 * U * np.abs(g.numpy()).sum(1).max()
        assert (out[2] == 0).all()


def test_backward_of_masked_rows(fp4):
    z = logits(6, 12, "f32", 5)
    z[:, 3:6] = -torch.inf
    z[0] = -torch.inf
    for score in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            w, ids = fp4.moe_route(z.cuda(), 4, score=score, renormalize=renormalize)
            out = fp4.moe_route_backward(torch.ones_like(w), z.cuda(), ids, score=score, renormalize=renormalize).cpu()
            assert out.isfinite().all() and (out[0] == 0).all() and (out[:, 3:6] == 0).all()
