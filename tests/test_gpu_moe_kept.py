"""Rows kept (the last of a sort's offsets) that no sort makes: below zero or
beyond the rows. They are read on the device, and count as 0 and as all rows."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kept", [-1, -5, -(1 << 31), 0])
def test_no_row_kept(fp4, kept, dtype):
    T, k, H = 5, 3, 40
    place = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).int().view(T, k)
    place[2, 1], place[4, 0] = -3, 1 << 30  # places outside the rows, too
    g = fp4.MoeGroups(torch.tensor([0, kept], dtype=torch.int32).cuda(), torch.zeros(T * k, dtype=torch.int32).cuda(),
                      place.cuda())
    x = torch.randn(T, H).to(dtype).cuda()
    rows = torch.full((T * k, H), torch.nan, dtype=dtype, device="cuda")
    w = torch.rand(T, k).cuda()
    for weights in (w, None):
        assert (fp4.moe_combine(rows, weights, g) == 0).all()
    gr, gw = fp4.moe_combine_backward(x, rows, w, g)
    there = place.flatten()[(place.flatten() >= 0) & (place.flatten() < T * k)].long().cuda()
    assert (gr[there] == 0).all() and (gw == 0).all()
    assert (fp4.moe_dispatch(x, g)[there] == 0).all()


def test_more_rows_kept_than_there_are(fp4):
    T, k, H = 5, 3, 40
    place = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).int().view(T, k).cuda()
    rows, w = torch.randn(T * k, H).cuda(), torch.rand(T, k).cuda()
    x = torch.randn(T, H).cuda()
    some = lambda n: fp4.MoeGroups(torch.tensor([n], dtype=torch.int32).cuda(), place, place)
    for many in (some(T * k + 1), some((1 << 31) - 1)):
        assert torch.equal(fp4.moe_combine(rows, w, many), fp4.moe_combine(rows, w, some(T * k)))
        for a, b in zip(fp4.moe_combine_backward(x, rows, w, many), fp4.moe_combine_backward(x, rows, w, some(T * k))):
            assert torch.equal(a, b)
        assert torch.equal(fp4.moe_dispatch(x, many), fp4.moe_dispatch(x, some(T * k)))
