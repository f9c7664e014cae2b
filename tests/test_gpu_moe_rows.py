"""Sorting of pairs, dispatch and combine against the definitions (moe_util).
Sort and dispatch are exact. Combine sums k products in fp32, fused, in order:
an error of at most k 2^-24 of the sum of magnitudes, and one rounding of the
result; grad_rows one or two roundings (of the product, and to bf16);
grad_weights a sum of `width` products in fp32."""
import numpy as np
import pytest
import torch

import moe_util as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make_ids(T, k, E, seed, dropped=0.0):
    r = np.random.default_rng(seed)
    ids = np.argsort(r.random((T, E)), 1)[:, :k] if k <= E else r.integers(0, E, (T, k))
    ids = np.where(r.random(ids.shape) < dropped, r.choice([-1, E, 1 << 30, -(1 << 31)], ids.shape), ids)
    return torch.from_numpy(ids.astype(np.int32))


GROUPS = [(1, 1, 1, 0.0), (1, 4, 32, 0.0), (7, 3, 5, 0.3), (63, 1, 2, 0.0), (64, 1, 64, 0.0), (65, 1, 256, 0.1),
          (32, 4, 32, 0.0), (500, 8, 256, 0.0), (1024, 8, 1024, 0.2), (4095, 2, 17, 0.0), (8193, 1, 60, 0.0),
          (8192, 2, 128, 0.5), (50000, 2, 7, 0.01), (20011, 8, 1000, 0.0), (300, 4, 16, 1.0), (1000, 40, 8, 0.0)]


@pytest.mark.parametrize("T,k,E,dropped", GROUPS)
def test_group(fp4, T, k, E, dropped):
    ids = make_ids(T, k, E, T + E, dropped)
    g = fp4.moe_group(ids.cuda(), E)
    for name, got, want in zip(("offsets", "order", "place"), (g.offsets, g.order, g.place), M.group(ids.numpy(), E)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want), name


def test_group_of_one_expert_and_of_nothing(fp4):
    for n in (5000, 20000):
        ids = torch.full((n,), 3, dtype=torch.int32).cuda()
        g = fp4.moe_group(ids, 8)
        assert torch.equal(g.order.cpu(), torch.arange(n, dtype=torch.int32)) and torch.equal(g.place, g.order)
        assert g.offsets.tolist() == [0, 0, 0, 0] + [n] * 5
    g = fp4.moe_group(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 6)
    assert g.offsets.tolist() == [0] * 7 and g.order.numel() == 0 and g.place.shape == (0, 4)


ROWS = [(1, 1, 8, 1), (3, 4, 8, 5), (32, 4, 32, 2880), (17, 3, 60, 1001), (100, 8, 64, 4096), (9, 2, 4, 7), (50, 6, 16, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_dispatch(fp4, T, k, E, H, dropped, dtype):
    ids = make_ids(T, k, E, T * H, dropped)
    x = torch.randn(T, H + 3, generator=torch.Generator().manual_seed(H)).to(DT[dtype])
    for view in (x[:, :H].contiguous(), x[:, 2:2 + H]):
        dev = view.cuda() if view.is_contiguous() else x.cuda()[:, 2:2 + H]
        rows = fp4.moe_dispatch(dev, fp4.moe_group(ids.cuda(), E)).cpu()
        offsets, order, _ = M.group(ids.numpy(), E)
        want = torch.zeros(T * k, H, dtype=DT[dtype])
        n = offsets[-1]
        want[:n] = view[torch.from_numpy(order[:n].astype(np.int64)) // k]
        assert torch.equal(rows, want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,k,E,H,dropped", [(1, 4, 32, 32, 0.0), (33, 4, 8, 2880, 0.3), (5, 2, 4, 96, 0.0), (64, 8, 64, 4096, 0.1)])
def test_dispatch_of_packed_rows(fp4, fmt, T, k, E, H, dropped):
    """Quantizing, then carrying, is carrying, then quantizing."""
    ids = make_ids(T, k, E, H, dropped)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(H)).bfloat16().cuda()
    q = fp4.quantize(x, fmt, four_over_six=True)
    g = fp4.moe_group(ids.cuda(), E)
    rows = fp4.moe_dispatch(q, g)
    assert rows.fmt == q.fmt and rows.codes.shape == (T * k, H // 2) and rows.codes.stride(0) % 128 == 0
    offsets, order, _ = M.group(ids.numpy(), E)
    n, tok = offsets[-1], torch.from_numpy(order.astype(np.int64)) // k
    assert torch.equal(rows.codes[:n].cpu(), q.codes.cpu()[tok[:n]]) and (rows.codes[n:] == 0).all()
    assert torch.equal(rows.scales[:n].cpu(), q.scales.cpu()[tok[:n]]) and (rows.scales[n:] == 0).all()
    if n == T * k:
        again = fp4.quantize(fp4.moe_dispatch(x, g), fmt, four_over_six=True)
        assert torch.equal(again.codes, rows.codes) and torch.equal(again.scales, rows.scales)


def combine_ref(rows, w, at, there):
    """[T, H] and the sum of magnitudes, float64."""
    x = np.where(there[..., None], rows[at], 0.0) * w[..., None]
    return x.sum(1), np.abs(x).sum(1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("grouped", [True, False])
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_combine(fp4, T, k, E, H, grouped, dtype):
    ids = make_ids(T, k, E, T * H, 0.3 if grouped else 0.0)
    gen = torch.Generator().manual_seed(H)
    rows = torch.randn(T * k, H, generator=gen).to(DT[dtype])
    w = torch.rand(T, k, generator=gen)
    offsets, _, place = M.group(ids.numpy(), E)
    at = place if grouped else np.arange(T * k).reshape(T, k)
    there = at < (offsets[-1] if grouped else T * k)
    if grouped:
        rows[offsets[-1]:] = torch.nan  # rows of no expert may hold anything
    g = fp4.moe_group(ids.cuda(), E) if grouped else None
    r64 = np.nan_to_num(rows.double().numpy())
    step = 2.0 ** -8 if dtype == "bf16" else U
    for weights in (w, None):
        if weights is None and not grouped:
            rows = rows.view(T, k, H)
        w64 = np.ones((T, k)) if weights is None else w.double().numpy()
        want, size = combine_ref(r64, w64, at, there)
        out = fp4.moe_combine(rows.cuda(), None if weights is None else w.cuda(), g)
        assert out.dtype == DT[dtype] and out.shape == (T, H)
        err = np.abs(out.double().cpu().numpy() - want)
        assert (err <= (k + 1) * U * size + step * np.abs(want) + 1e-38).all()


def test_combine_into_a_part_of_a_matrix(fp4):
    T, k, H = 20, 3, 64
    rows = torch.randn(T * k, 100, device="cuda")[:, 5:5 + H]
    w = torch.rand(T, k, device="cuda")
    wide = torch.full((T, 80), 7.0, device="cuda")
    got = fp4.moe_combine(rows, w, out=wide[:, 9:9 + H])
    assert got.data_ptr() == wide[:, 9:].data_ptr()
    assert torch.equal(got.contiguous(), fp4.moe_combine(rows.contiguous(), w))
    assert (wide[:, :9] == 7).all() and (wide[:, 9 + H:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("grouped", [True, False])
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_combine_backward(fp4, T, k, E, H, grouped, dtype):
    ids = make_ids(T, k, E, T * H, 0.3 if grouped else 0.0)
    gen = torch.Generator().manual_seed(H)
    rows = torch.randn(T * k, H, generator=gen).to(DT[dtype])
    w = torch.rand(T, k, generator=gen)
    grad = torch.randn(T, H + 5, generator=gen).to(DT[dtype])
    offsets, _, place = M.group(ids.numpy(), E)
    at = place if grouped else np.arange(T * k).reshape(T, k)
    there = at < (offsets[-1] if grouped else T * k)
    if grouped:
        rows[offsets[-1]:] = torch.nan
    g = fp4.moe_group(ids.cuda(), E) if grouped else None
    gr, gw = fp4.moe_combine_backward(grad.cuda()[:, 2:2 + H], rows.cuda(), w.cuda(), g)
    g64 = grad[:, 2:2 + H].double().numpy()
    r64 = np.nan_to_num(rows.double().numpy())
    x = np.where(there[..., None], g64[:, None] * w.double().numpy()[..., None], 0.0)
    want = np.zeros((T * k, H))
    want[at] = x
    step = U if dtype == "f32" else U + 2.0 ** -8
    assert (np.abs(gr.double().cpu().numpy() - want) <= step * np.abs(want) + 1e-38).all()
    prod = np.where(there[..., None], g64[:, None] * r64[at], 0.0)
    assert gw.dtype == torch.float32
    assert (np.abs(gw.double().cpu().numpy() - prod.sum(-1)) <= (H + 1) * U * np.abs(prod).sum(-1) + 1e-38).all()
    # without weights: dispatch of the gradient; and its own backward is combine
    gr, none = fp4.moe_combine_backward(grad.cuda()[:, 2:2 + H], rows.cuda(), None, g)
    assert none is None
    want[at] = np.where(there[..., None], g64[:, None], 0.0)
    assert np.array_equal(gr.double().cpu().numpy(), want)
    if grouped:
        assert torch.equal(gr, fp4.moe_dispatch(grad.cuda()[:, 2:2 + H], g))


def test_gradient_of_combine_against_differences(fp4):
    """sum(out * grad) is linear in rows and in weights: a difference over any
    step is the gradient, but for the roundings of the two sums."""
    T, k, E, H = 6, 3, 8, 33
    ids = make_ids(T, k, E, 1, 0.2).cuda()
    g = fp4.moe_group(ids, E)
    gen = torch.Generator().manual_seed(1)
    rows, w, grad = (torch.randn(*s, generator=gen).cuda() for s in ((T * k, H), (T, k), (T, H)))
    gr, gw = fp4.moe_combine_backward(grad, rows, w, g)
    loss = lambda r, v: (fp4.moe_combine(r, v, g).double() * grad.double()).sum().item()
    base = loss(rows, w)
    tol = 8 * (k + 1) * H * U * float(grad.abs().max())* float(rows.abs().max()) * float(w.abs().max())
    n = int(g.offsets[-1])
    for r, c in ((0, 0), (n - 1, H - 1), (n // 2, 7)):
        moved = rows.clone()
        moved[r, c] += 1.0
        assert abs(loss(moved, w) - base - gr[r, c].item()) <= tol
    for t, j in ((0, 0), (3, 2), (5, 1)):
        moved = w.clone()
        moved[t, j] += 1.0
        assert abs(loss(rows, moved) - base - gw[t, j].item()) <= tol


def test_places_outside_the_rows_are_passed_over(fp4):
    """In bounds whatever the places say (they are checked on the device)."""
    T, k, H = 4, 2, 16
    bad = torch.tensor([[0, 1], [2, 1 << 30], [-5, 3], [7, 8]], dtype=torch.int32).cuda()
    g = fp4.MoeGroups(torch.tensor([0, 6], dtype=torch.int32).cuda(), torch.zeros(8, dtype=torch.int32).cuda(), bad)
    x = torch.randn(T, H).cuda()
    rows = fp4.moe_dispatch(x, g)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[3], x[2]) and (rows[7] == 0).all()
    out = fp4.moe_combine(torch.ones(8, H).cuda(), torch.ones(T, k).cuda(), g)
    assert out[:, 0].tolist() == [2, 1, 1, 0]
    gr, gw = fp4.moe_combine_backward(x, torch.ones(8, H).cuda(), torch.ones(T, k).cuda(), g)
    assert gw[1, 1] == gw[2, 0] == gw[3, 0] == gw[3, 1] == 0 and torch.equal(gr[3], x[2])


def test_no_slots_and_no_columns(fp4):
    """Tokens without a slot get zeros, weights of rows without columns a gradient of zero."""
    ids = torch.empty(5, 0, dtype=torch.int32, device="cuda")
    g = fp4.moe_group(ids, 4)
    assert g.offsets.tolist() == [0] * 5 and g.place.shape == (5, 0)
    x = torch.randn(5, 24, device="cuda")
    assert fp4.moe_dispatch(x, g).shape == (0, 24)
    none = torch.empty(5, 0, device="cuda")
    for rows in (torch.empty(0, 24, device="cuda"), torch.ones(3, 24, device="cuda")):
        out = torch.full((5, 24), 7.0, device="cuda")
        assert (fp4.moe_combine(rows, none, g, out=out) == 0).all()
    gr, gw = fp4.moe_combine_backward(x, torch.empty(0, 24, device="cuda"), none, g)
    assert gr.shape == (0, 24) and gw.shape == (5, 0)
    torch.full((10,), 7.0, device="cuda")  # (what an uninitialised result would show)
    gr, gw = fp4.moe_combine_backward(torch.empty(5, 0, device="cuda"), torch.empty(10, 0, device="cuda"),
                                      torch.ones(5, 2, device="cuda"))
    assert gr.shape == (10, 0) and (gw == 0).all()
