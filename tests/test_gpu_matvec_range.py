"""Products of a few rows at the ends of fp32's range. Sums are fp32 and hold
no more than the products they stand for: where the sum of magnitudes is finite,
y is, within the bound of test_gpu_matvec.py ((2 K + 4) 2^-24 of that sum, one
rounding of y), and at the lower end within K 2^-139 besides."""
import numpy as np
import pytest
import torch

import moe_util as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROWS = (1, 6, 12)  # passes of 4, 8 and 16 rows


def check(y, x, W):
    """y fp32. Elements whose magnitudes sum up to more than fp32 holds are passed over; returns how many are left."""
    x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
    want, size = x @ W.T, np.abs(x) @ np.abs(W).T
    fits = size * (1 + (2 * x.shape[1] + 4) * U) < 2.0 ** 128 * (1 - U)
    tol = (2 * x.shape[1] + 4) * U * size + U * np.abs(want) + x.shape[1] * 2.0 ** -139
    err = np.abs(y - want)
    assert (err <= tol)[fits].all(), f"worst {np.nanmax((err / tol)[fits]):.3g} of the bound, {np.isnan(y[fits]).sum()} NaN"
    return fits.sum()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("weight", [1e-3, 0.1, 20.0])
def test_nvfp4_holds_no_more_than_its_products(fp4, rows, weight, dtype):
    """Activations up to fp32's largest against weights far below 2688 times the tensor scale's reciprocal."""
    N, K = 40, 96
    g = torch.Generator().manual_seed(rows)
    q = fp4.quantize((weight * torch.randn(N, K, generator=g)).cuda(), "nvfp4")
    W = M.values(q)
    for size in (1e35, 1e36, 1e37):
        x = torch.randn(rows, K, generator=g).clamp(-3, 3) * size
        x[:, 5::7] = 3.3e38 / max(1.0, 200 * weight)
        x = x.to(DT[dtype]).cuda()
        many = check(fp4.matvec(x, q, out_dtype=torch.float32), x, W)
        assert many == rows * N or weight > 1
        one = torch.zeros(rows, K)
        one[:, 11] = torch.linspace(0.3, 1.0, rows) * 3.3e38 / max(1.0, weight)
        one = one.to(DT[dtype]).cuda()
        assert check(fp4.matvec(one, q, out_dtype=torch.float32), one, W) > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
def test_nvfp4_tensor_scales_of_every_size(fp4, rows, dtype):
    """Blocks with every E4M3 scale under tensor scales over fp32's whole range, activations as large as leave y finite."""
    N, K = 32, 128
    g = torch.Generator().manual_seed(7)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g).cuda()
    s = torch.zeros(N, 16, dtype=torch.uint8)
    s[:, :K // 16] = torch.arange(N * K // 16).view(N, -1) % 127
    x = torch.randn(rows, K, generator=g)
    for e in (-149, -130, -120, -100, -60, -42, -41, -40, -39, -38, -20, -9, -8, -7, -6, -5, 0, 20, 90, 116, 120, 121, 126):
        ts = torch.tensor([2.0 ** e * (1.0 if e < -126 else 1.37)], dtype=torch.float64).float().cuda()
        q = fp4.Quantized(fp4.FP4_NVFP4, codes, s.cuda()[:, :K // 16], ts)
        W = M.values(q)
        largest = min(2.0 ** 126, 2.0 ** 127 / np.abs(W).sum(1).max()) / 4
        for size in (largest, 1.0 if largest > 1 else largest * 2.0 ** -10):
            z = (x * size).to(DT[dtype]).cuda()
            assert check(fp4.matvec(z, q, out_dtype=torch.float32), z, W) == rows * N, e
    q = fp4.Quantized(fp4.FP4_NVFP4, codes, s.cuda()[:, :K // 16], torch.zeros(1).cuda())
    assert (fp4.matvec(x.to(DT[dtype]).cuda(), q) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nvfp4_by_experts_of_different_tensor_scales(fp4, dtype):
    """Each expert's power of two is its own."""
    E, N, K, T, k = 5, 48, 64, 6, 3
    g = torch.Generator().manual_seed(3)
    size = torch.tensor([1e-20, 1e-3, 0.5, 300.0, 1e20])[:, None, None]
    q = fp4.quantize((size * torch.randn(E, N, K, generator=g)).cuda(), "nvfp4")
    W = M.values(q)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=g)
    x = (torch.randn(T, K, generator=g) * 1e16).to(DT[dtype]).cuda()
    y = fp4.matvec(x, q, ids.cuda(), out_dtype=torch.float32)
    for t in range(T):
        for j in range(k):
            check(y[t, j][None], x[t][None], W[ids[t, j]])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows", ROWS)
def test_any_nan_is_a_nan(fp4, fmt, rows):
    """Also one that only the lower 16 bits tell from an infinity."""
    q = fp4.quantize(torch.randn(40, 128, generator=torch.Generator().manual_seed(2)).cuda(), fmt)
    for bits in (0x7f800001, 0xff800001, 0x7f80ffff, 0xff808000, 0x7f810000, 0x7fc00000, 0xffffffff):
        x = torch.ones(rows, 128)
        x[rows - 1, 77] = torch.tensor(bits - (1 << 32) if bits >> 31 else bits, dtype=torch.int32).view(torch.float32)
        y = fp4.matvec(x.cuda(), q)
        assert y[rows - 1].isnan().all() and y[:rows - 1].isfinite().all(), hex(bits)
    for inf in (torch.inf, -torch.inf):
        x = torch.zeros(rows, 128)
        x[rows - 1, 77] = inf
        y = fp4.matvec(x.cuda(), q)[rows - 1].cpu()
        w = torch.from_numpy(M.values(q)[:, 77])
        assert torch.equal(y.nan_to_num(nan=7.0, posinf=1.0, neginf=-1.0), torch.where(w == 0, 7.0, torch.sign(w * inf)).float())


def large_weights(fp4, N, K, byte, seed=5):
    """MXFP4 weights with the scale 2^(byte - 127) everywhere."""
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=torch.Generator().manual_seed(seed)).cuda()
    return fp4.Quantized(fp4.FP4_MXFP4, codes, torch.full((N, 16), byte, dtype=torch.uint8).cuda()[:, :K // 32], None)


@pytest.mark.parametrize("rows", ROWS)
def test_small_fp32_activations_keep_their_bits(fp4, rows):
    """Down to 2^-148: one activation alone is its product with a weight, rounded
    in sums of three terms (exact products, two additions); the bit of 2^-149 may be cut off."""
    N, K = 48, 64
    g = torch.Generator().manual_seed(rows)
    q = large_weights(fp4, N, K, 230)  # 2^103
    W = M.values(q)
    for e in (-100, -108, -110, -112, -116, -120, -124, -125, -126, -130, -140, -148, -149):
        x = torch.zeros(rows, K)
        x[:, 11] = ((1 + torch.rand(rows, generator=g).double()) * 2.0 ** e).float()
        y = fp4.matvec(x.cuda(), q).double().cpu().numpy()
        want = x[:, 11:12].double().numpy() * W[None, :, 11]
        assert (np.abs(y - want) <= 2 * U * np.abs(want) + 2.0 ** -149 * np.abs(W[None, :, 11])).all(), e
        full = (torch.randn(rows, K, generator=g).double() * 2.0 ** e).float()
        y = fp4.matvec(full.cuda(), q).double().cpu().numpy()
        want, size = full.double().numpy() @ W.T, full.abs().double().numpy() @ np.abs(W).T
        assert (np.abs(y - want) <= (2 * K + 4) * U * size + 2.0 ** -149 * np.abs(W).sum(1)).all(), e


@pytest.mark.parametrize("rows", ROWS)
def test_small_bf16_activations(fp4, rows):
    """bf16 rows are operands as they are, subnormal numbers too."""
    N, K = 48, 64
    g = torch.Generator().manual_seed(rows)
    for q in (large_weights(fp4, N, K, 230), fp4.quantize((1e30 * torch.randn(N, K, generator=g)).cuda(), "nvfp4")):
        W = M.values(q)
        for e in (-110, -126, -128, -131):
            x = (torch.randn(rows, K, generator=g).double() * 2.0 ** e).bfloat16()
            want, size = x.double().numpy() @ W.T, x.abs().double().numpy() @ np.abs(W).T
            y = fp4.matvec(x.cuda(), q, out_dtype=torch.float32).double().cpu().numpy()
            lost = 2.0 ** -132 * K * (float(q.tensor_scale) if q.tensor_scale is not None else 0.0)
            assert (np.abs(y - want) <= (2 * K + 4) * U * size + lost).all(), e


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("byte", [0, 1, 2, 3, 5])
def test_smallest_scales_of_mxfp4(fp4, byte, rows, dtype):
    """Weights that are subnormal in bf16."""
    N, K = 48, 64
    q = large_weights(fp4, N, K, byte)
    x = (torch.randn(rows, K, generator=torch.Generator().manual_seed(rows)) * 1e30).to(DT[dtype])
    W = M.values(q)
    want, size = x.double().numpy() @ W.T, x.abs().double().numpy() @ np.abs(W).T
    y = fp4.matvec(x.cuda(), q, out_dtype=torch.float32).double().cpu().numpy()
    assert (np.abs(y - want) <= (2 * K + 4) * U * size).all()
