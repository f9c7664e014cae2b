"""Products of a few rows with 4-bit weights against the definition in 64 bits
(moe_util.values). Weights are exact in bf16 and activations whole (fp32 as
three terms), so the only error is that of fp32 sums over K: within
(2 K + 4) 2^-24 of the sum of magnitudes, as for the products of two 4-bit
operands; and one rounding of y."""
import numpy as np
import pytest
import torch

import moe_util as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def weights(fp4, fmt, N, K, seed, experts=0, **kw):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(*((experts,) if experts else ()), N, K, generator=g) * 0.05
    if K > 40:
        w[..., 33] *= 30
    return fp4.quantize(w.cuda(), fmt, **kw)


def check(y, x, W, out_dtype):
    """y [.., N] against x [.., K] times W [N, K] (or [.., N, K])."""
    x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
    want = np.einsum("...k,...nk->...n", x, W)
    size = np.einsum("...k,...nk->...n", np.abs(x), np.abs(W))
    tol = (2 * x.shape[-1] + 4) * U * size + (2.0 ** -8 if out_dtype is torch.bfloat16 else U) * np.abs(want) + 1e-38
    err = np.abs(y - want)
    assert (err <= tol).all(), f"worst {np.nanmax(err / tol):.3g} of the bound, {np.isnan(y).sum()} NaN"


SIZES = [(1, 16, 32), (1, 1, 64), (1, 4096, 4096), (2, 17, 96), (3, 100, 2880), (4, 33, 160), (5, 64, 544), (8, 1000, 1024),
         (9, 48, 8192), (16, 256, 2880), (17, 31, 320), (33, 130, 512), (64, 512, 1440), (70, 20, 16384)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M_,N,K", SIZES)
def test_one_matrix(fp4, fmt, dtype, M_, N, K):
    q = weights(fp4, fmt, N, K, N + K)
    x = torch.randn(M_, K, generator=torch.Generator().manual_seed(K)).to(DT[dtype]).cuda()
    W = M.values(q)
    y = fp4.matvec(x, q)
    assert y.dtype == DT[dtype] and y.shape == (M_, N)
    check(y, x, W, DT[dtype])
    other = torch.float32 if dtype == "bf16" else torch.bfloat16
    y2 = fp4.matvec(x, q, out_dtype=other)
    check(y2, x, W, other)
    one = fp4.matvec(x[0], q)
    assert one.shape == (N,)
    check(one[None], x[:1], W, DT[dtype])


@pytest.mark.parametrize("K", [16, 48, 112, 144, 528, 1040])
@pytest.mark.parametrize("M_", [1, 5, 20])
def test_odd_blocks_of_nvfp4(fp4, K, M_):
    """K an odd number of blocks: the last 16 bytes of a row are half a row's."""
    q = weights(fp4, "nvfp4", 70, K, K)
    x = torch.randn(M_, K, generator=torch.Generator().manual_seed(K)).cuda()
    check(fp4.matvec(x, q), x, M.values(q), torch.float32)
    # what lies behind a row's codes and scales has no part, NaN scales included
    q.codes.as_strided((70, q.codes.stride(0)), (q.codes.stride(0), 1))[:, K // 2:] = 255
    q.scales.as_strided((70, q.scales.stride(0)), (q.scales.stride(0), 1))[:, K // 16:] = 255
    check(fp4.matvec(x, q), x, M.values(q), torch.float32)
    xb = x.bfloat16()
    check(fp4.matvec(xb, q), xb, M.values(q), torch.bfloat16)


EXPERTS = [(1, 4, 32, 64, 96), (1, 1, 1, 16, 64), (7, 3, 5, 100, 320), (32, 4, 32, 144, 288), (16, 8, 256, 40, 64),
           (65, 2, 4, 48, 1024), (200, 4, 8, 33, 160), (64, 8, 16, 32, 96), (512, 8, 64, 17, 32)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,N,K", EXPERTS)
def test_by_experts(fp4, fmt, dtype, T, k, E, N, K):
    r = np.random.default_rng(T)
    ids = r.integers(0, E, (T, k))
    ids[r.random(ids.shape) < 0.1] = -1
    ids[r.random(ids.shape) < 0.05] = E
    q = weights(fp4, fmt, N, K, N + K, E)
    W = np.concatenate((M.values(q), np.zeros((1, N, K))))[np.where((ids < 0) | (ids >= E), E, ids)]
    dev = torch.from_numpy(ids.astype(np.int32)).cuda()
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(K)).to(DT[dtype]).cuda()
    y = fp4.matvec(x, q, dev)
    assert y.shape == (T, k, N)
    check(y, x[:, None].expand(T, k, K), W, DT[dtype])
    own = torch.randn(T, k, K, generator=torch.Generator().manual_seed(K)).to(DT[dtype]).cuda()
    y = fp4.matvec(own, q, dev)
    check(y, own, W, DT[dtype])
    assert torch.equal(fp4.matvec(own.flatten(0, 1), q, dev), y)
    flat = fp4.matvec(own.flatten(0, 1), q, dev.flatten())
    assert torch.equal(flat, y.flatten(0, 1))


def test_experts_without_a_row(fp4):
    q = weights(fp4, "mxfp4", 40, 64, 1, 4)
    x = torch.randn(3, 64).cuda()
    y = fp4.matvec(x, q, torch.full((3, 2), -1, dtype=torch.int32, device="cuda"))
    assert (y == 0).all()
    y = fp4.matvec(x, q, torch.tensor([[7, -3], [1 << 30, 4], [3, 3]], dtype=torch.int32, device="cuda"))
    assert (y[:2] == 0).all() and torch.equal(y[2, 0], y[2, 1])
    check(y[2, :1], x[2:], M.values(q)[3], torch.float32)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_wide_range_of_activations(fp4, fmt):
    """Large activations that meet weights of zero leave small ones their bits:
    one column in 32 holds 2^60, its weights are 0."""
    N, K = 50, 512
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(3)) * 0.05
    w[:, 7::32] = 0
    q = fp4.quantize(w.cuda(), fmt)
    W = M.values(q)
    for dtype in (torch.bfloat16, torch.float32):
        for rows in (1, 6):
            x = torch.randn(rows, K, generator=torch.Generator().manual_seed(4)) * 1e-3
            x[:, 7::32] = 2.0 ** 60
            x = x.to(dtype).cuda()
            check(fp4.matvec(x, q, out_dtype=torch.float32), x, W, torch.float32)


def test_fp32_activations_keep_all_their_bits(fp4):
    """One activation alone: y is its product with a weight, rounded once."""
    q = weights(fp4, "nvfp4", 64, 32, 5, tensor_scale=True)
    W = M.values(q)
    g = torch.Generator().manual_seed(8)
    for size in (1.0, 1e-20, 1e20, 1e37):
        x = torch.zeros(20, 32)
        x[:, 11] = torch.randn(20, generator=g) * size
        y = fp4.matvec(x.cuda(), q).double().cpu().numpy()
        want = x[:, 11:12].double().numpy() * W[None, :, 11]
        ok = np.abs(want) < 3.4e38
        # (the tensor scale is a second product: two roundings)
        assert (np.abs(y - want)[ok] <= (2 * U + 2 * U * U) * np.abs(want[ok])).all()


def test_scales_at_the_ends_of_their_range(fp4):
    N, K = 32, 64
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=torch.Generator().manual_seed(2)).cuda()
    x = torch.randn(2, K, generator=torch.Generator().manual_seed(3)).cuda()
    for byte in (3, 20, 127, 220, 245):
        s = torch.full((N, 16), byte, dtype=torch.uint8).cuda()[:, :K // 32]
        q = fp4.Quantized(fp4.FP4_MXFP4, codes, s, None)
        check(fp4.matvec(x, q), x, M.values(q), torch.float32)
    every = torch.arange(N * 4, dtype=torch.uint8).view(N, 4) % 127  # each E4M3 number
    s = torch.zeros(N, 16, dtype=torch.uint8)
    s[:, :4] = every
    q = fp4.Quantized(fp4.FP4_NVFP4, codes, s.cuda()[:, :4], torch.tensor([0.37]).cuda())
    check(fp4.matvec(x, q), x, M.values(q), torch.float32)
    check(fp4.matvec(x.repeat(5, 1), q), x.repeat(5, 1), M.values(q), torch.float32)


def test_strides(fp4):
    q = weights(fp4, "mxfp4", 48, 256, 2, 3)
    W = M.values(q)
    ids = torch.tensor([[0, 2], [1, 1], [2, 0]], dtype=torch.int32).cuda()
    wide = torch.randn(3, 300).bfloat16().cuda()
    for x in (wide[:, 8:264], wide[:, 3:259], torch.randn(256, 3).bfloat16().cuda().T):  # aligned, not, columns
        out = torch.zeros(3, 2, 60).cuda().bfloat16()
        y = fp4.matvec(x, q, ids, out=out[:, :, :48]) if False else fp4.matvec(x, q, ids)
        check(y, x[:, None].expand(3, 2, 256), W[ids.cpu().numpy()], torch.bfloat16)
    part = fp4.Quantized(q.fmt, q.codes[1:, 8:40], q.scales[1:, 8:40], None)  # some rows of some experts
    y = fp4.matvec(wide[:, 8:264], part, torch.tensor([[1], [0], [1]], dtype=torch.int32).cuda())
    check(y[:, 0], wide[:, 8:264], W[1:, 8:40][[1, 0, 1]], torch.bfloat16)
    big = torch.full((3, 100), 5.0).cuda()
    one = fp4.Quantized(q.fmt, q.codes[0], q.scales[0], None)
    got = fp4.matvec(wide[:, 8:264], one, out=big[:, 20:68])
    check(got, wide[:, 8:264], W[0], torch.float32)
    assert (big[:, :20] == 5).all() and (big[:, 68:] == 5).all()


def test_infinities_and_nan_stay_in_their_rows(fp4):
    q = weights(fp4, "nvfp4", 40, 128, 3)
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(6, 128).to(dtype).cuda()
        clean = fp4.matvec(x, q)
        x[1, 5], x[3, 70] = torch.inf, torch.nan
        y = fp4.matvec(x, q)
        assert not y[1].isfinite().any() and not y[3].isfinite().any()
        assert torch.equal(y[[0, 2, 4, 5]], clean[[0, 2, 4, 5]])


def test_empty(fp4):
    q = weights(fp4, "mxfp4", 40, 64, 3)
    assert fp4.matvec(torch.empty(0, 64).cuda(), q).shape == (0, 40)
    none = fp4.Quantized(q.fmt, q.codes[:0], q.scales[:0], None)
    assert fp4.matvec(torch.randn(3, 64).cuda(), none).shape == (3, 0)
    q3 = weights(fp4, "mxfp4", 40, 64, 3, 2)
    assert fp4.matvec(torch.empty(0, 64).cuda(), q3, torch.empty(0, 4, dtype=torch.int32).cuda()).shape == (0, 4, 40)


def test_no_columns(fp4):
    """K = 0: a sum of nothing."""
    q = fp4.Quantized(fp4.FP4_MXFP4, torch.empty(2, 40, 0, dtype=torch.uint8).cuda(), torch.empty(2, 40, 0, dtype=torch.uint8).cuda(), None)
    ids = torch.tensor([[0], [1], [5]], dtype=torch.int32).cuda()
    for x in (torch.empty(3, 0).cuda(), torch.empty(3, 0).cuda().bfloat16()):
        assert fp4.matvec(x, q, ids).abs().sum() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M_,N,K", [(1, 70000, 96), (3, 33000, 544), (7, 20001, 1504), (2, 9000, 5120), (6, 17000, 5152)])
def test_many_rows_of_weights(fp4, fmt, dtype, M_, N, K):
    """Several tiles of W a wave, and x in LDS by parts."""
    q = weights(fp4, fmt, N, K, 5)
    x = torch.randn(M_, K, generator=torch.Generator().manual_seed(K)).to(DT[dtype]).cuda()
    y = fp4.matvec(x, q)
    cut = torch.cat((torch.arange(0, 200), torch.arange(N // 2, N // 2 + 100), torch.arange(N - 200, N)))
    part = fp4.Quantized(q.fmt, q.codes.cpu()[cut], q.scales.cpu()[cut], q.tensor_scale)
    check(y[:, cut.cuda()], x, M.values(part), DT[dtype])
    same = fp4.matvec(x, fp4.Quantized(q.fmt, q.codes[100:300], q.scales[100:300], q.tensor_scale))
    # (the waves that share a sum may differ with N: within two such bounds)
    assert (y[:, 100:300].float() - same.float()).abs().max() <= 2.0 ** -6 * y.float().abs().max()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tiles_of_many_experts(fp4, fmt, dtype):
    T, k, E, N, K = 40, 2, 48, 1900, 1088
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    q = weights(fp4, fmt, N, K, 6, E)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(K)).to(DT[dtype]).cuda()
    y = fp4.matvec(x, q, ids.cuda())
    W = M.values(q)
    for t in range(T):
        check(y[t], x[t][None].expand(k, K), W[ids[t].numpy()], DT[dtype])


def test_same_bits_twice_and_whatever_lies_beside(fp4):
    """The order of sums depends on K alone: a row's result does not change
    with the rows beside it, nor from call to call, within one form."""
    for fmt in ("mxfp4", "nvfp4"):
        q = weights(fp4, fmt, 300, 2880, 9)
        x = torch.randn(3, 2880).bfloat16().cuda()
        y = fp4.matvec(x, q)
        assert torch.equal(y, fp4.matvec(x, q))
        assert torch.equal(y[:2], fp4.matvec(x[:2], q))
