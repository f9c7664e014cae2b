"""A router's groups where the roundings of their ranks come together: the ids
are those of the exact numbers (moe_util, in 64 bits)."""
import numpy as np
import pytest
import torch

import moe_util as M

pytestmark = pytest.mark.gpu


def check(fp4, z, k, bias, **kw):
    opts = {("group_best" if n == "best" else n): v for n, v in kw.items()}
    _, ids = fp4.moe_route(z.cuda(), k, bias=bias.cuda(), **opts)
    _, want = M.route(z.double().numpy(), k, bias=bias.numpy(), **kw)
    bad = np.nonzero((ids.cpu().numpy() != want).any(1))[0]
    assert bad.size == 0, f"{bad.size} of {len(z)} rows differ, first {bad[0]}: {ids[bad[0]].tolist()}, not {want[bad[0]]}"


def meeting_roundings(T, E, groups, size, seed):
    """Sigmoid logits and a bias `size`, a power of two, for the two experts of
    each of two groups. Each biased score lies between two numbers of fp32, up to
    the resolution of its logit; the two ranks are equal but for that, and the
    sums of the scores rounded up, and of those rounded down, two steps apart."""
    r = np.random.default_rng(seed)
    step = size * 2.0 ** -23  # of a biased score
    low, high = int(0.5 / step), int(0.9 / step)
    n = r.integers(low + 2000, high - 2000, (T, 4))
    n[:, 1] += (1 - n[:, 0] - n[:, 1]) % 4
    n[:, 3] = n[:, 0] + n[:, 1] - n[:, 2]
    n = n[(n[:, 3] > low) & (n[:, 3] < high)]
    s = (n + 0.5) * step
    z = np.log(s / (1 - s)).astype(np.float32)
    z = (z.view(np.int32) + r.integers(-1, 2, z.shape)).astype(np.int32).view(np.float32)
    at = [0, 1, E // groups, E // groups + 1]
    full, bias = np.full((len(z), E), -3.0, np.float32), np.zeros(E, np.float32)
    full[:, at] = z
    bias[at] = size
    return torch.from_numpy(full), torch.from_numpy(bias)


@pytest.mark.parametrize("size", [16.0, 64.0, 256.0])
@pytest.mark.parametrize("E,groups,T", [(8, 4, 100000), (12, 4, 50000), (256, 8, 30000), (640, 20, 10000)])
def test_roundings_of_two_ranks_that_meet(fp4, E, groups, T, size):
    z, bias = meeting_roundings(T, E, groups, size, 1)
    check(fp4, z, 2, bias, score="sigmoid", groups=groups, top_groups=1, best=2)


@pytest.mark.parametrize("size", [16.0, 300.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_biases_of_either_sign(fp4, score, size):
    g = torch.Generator().manual_seed(5)
    z = torch.randn(3000, 64, generator=g)
    bias = size * torch.randn(64, generator=g).round() + 1e-6 * torch.randn(64, generator=g)
    for best in (1, 2):
        check(fp4, z, 6, bias, score=score, groups=8, top_groups=3, best=best)
        check(fp4, z, 6, bias, score=score, groups=16, top_groups=5, best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(32, 4), (24, 3), (60, 5), (256, 8), (640, 20)])
def test_ranks_beyond_fp32(fp4, score, E, groups):
    """A bias of the type's lowest number is no mask: its experts fill the slots
    that others leave, though the sum of two lies beyond fp32. So at the other end."""
    gs, low = E // groups, torch.finfo(torch.float32).min
    z = torch.randn(200, E, generator=torch.Generator().manual_seed(E))
    bias = torch.zeros(E)
    bias[gs:] = low
    check(fp4, z, min(gs + 2, 32), bias, score=score, groups=groups, top_groups=2, best=2)
    check(fp4, z, 4, bias, score=score, groups=groups, top_groups=1, best=2)
    bias[:] = low
    check(fp4, z, 4, bias, score=score, groups=groups, top_groups=2, best=2)
    bias[gs:2 * gs] = -torch.inf                       # and one group that is masked
    check(fp4, z, 4, bias, score=score, groups=groups, top_groups=2, best=2)
    bias = torch.zeros(E)
    bias[:gs], bias[gs:2 * gs] = 2e38, 3e38            # 4e38 and 6e38
    bias[2 * gs], bias[2 * gs + 1] = 3.3e38, 1e38      # 4.3e38
    for top in (1, 2):
        check(fp4, z, 4, bias, score=score, groups=groups, top_groups=top, best=2)
    check(fp4, z, 4, -bias, score=score, groups=groups, top_groups=groups - 1, best=2)
