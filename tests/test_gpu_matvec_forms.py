"""Forms of matvec's operands: sums of nothing and results without columns in
every shape that has them, and results by experts inside a wider tensor."""
import numpy as np
import pytest
import torch

import moe_util as M

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def without_columns(fp4, fmt, *lead):
    none = torch.empty(*lead, 0, dtype=torch.uint8).cuda()
    return fp4.Quantized(fp4.FP4_MXFP4, none, none, None) if fmt == "mxfp4" else \
        fp4.Quantized(fp4.FP4_NVFP4, none, none, torch.ones(lead[0] if len(lead) == 2 else 1).cuda())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sums_of_nothing(fp4, fmt, dtype):
    """K = 0 gives zeros."""
    q3, q = without_columns(fp4, fmt, 2, 40), without_columns(fp4, fmt, 40)
    ids = torch.tensor([[0, 1], [1, 5], [-1, 0]], dtype=torch.int32).cuda()
    for shape in ((3, 2, 0), (3, 0), (6, 0)):
        out = torch.full((3, 2, 40), 7.0, dtype=dtype, device="cuda")
        assert fp4.matvec(torch.empty(shape, dtype=dtype, device="cuda"), q3, ids, out=out) is out and (out == 0).all()
    for shape in ((5, 0), (1, 0), (0,)):
        y = fp4.matvec(torch.empty(shape, dtype=dtype, device="cuda"), q)
        assert y.shape == (*shape[:-1], 40) and (y == 0).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_results_without_columns(fp4, fmt):
    """N = 0, with the result given and not."""
    w = fp4.quantize(torch.randn(2, 32, 64).cuda(), fmt)
    q3 = fp4.Quantized(w.fmt, w.codes[:, :0], w.scales[:, :0], w.tensor_scale)
    q = fp4.Quantized(w.fmt, w.codes[0, :0], w.scales[0, :0], None if w.tensor_scale is None else w.tensor_scale[:1])
    ids = torch.zeros(3, 2, dtype=torch.int32).cuda()
    x = torch.randn(3, 64).cuda()
    for out in (torch.empty(3, 2, 0).cuda(), None):
        assert fp4.matvec(x, q3, ids, out=out).shape == (3, 2, 0)
    for rows, shape in ((x, (3, 0)), (x[0], (0,))):
        assert fp4.matvec(rows, q, out=torch.empty(shape).cuda()).shape == shape
    assert fp4.matvec(x[:0], q3, ids[:0], out=torch.empty(0, 2, 0).cuda()).shape == (0, 2, 0)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_results_of_experts_in_a_wider_tensor(fp4, fmt, dtype):
    """[tokens, top_k, N] with a pitch: the columns beside it stay as they were."""
    N, K = 48, 256
    q = fp4.quantize((0.1 * torch.randn(3, N, K, generator=torch.Generator().manual_seed(2))).cuda(), fmt)
    W = M.values(q)
    ids = torch.tensor([[0, 2], [1, 1], [2, -1]], dtype=torch.int32)
    x = torch.randn(3, K, generator=torch.Generator().manual_seed(3)).to(dtype)
    for first in (0, 5):
        wide = torch.full((3, 2, 60), 7.0, dtype=dtype, device="cuda")
        part = wide[:, :, first:first + N]
        assert fp4.matvec(x.cuda(), q, ids.cuda(), out=part) is part
        got = part.double().cpu().numpy()
        for t in range(3):
            for j in range(2):
                w = W[ids[t, j]] if ids[t, j] >= 0 else np.zeros((N, K))
                want, size = w @ x[t].double().numpy(), np.abs(w) @ np.abs(x[t].double().numpy())
                step = 2.0 ** -8 if dtype is torch.bfloat16 else U
                assert (np.abs(got[t, j] - want) <= (2 * K + 4) * U * size + step * np.abs(want)).all()
        assert (wide[:, :, :first] == 7).all() and (wide[:, :, first + N:] == 7).all()
