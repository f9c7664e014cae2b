"""Cache buffers as views whose rows are where they belong, whatever the strides
of dimensions of one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dim", [("mxfp4", 32), ("mxfp4", 64), ("nvfp4", 16), ("nvfp4", 128)])
def test_a_single_head_with_rows_outermost(fp4, fmt, dim):
    """[pages, page_size, 1, bytes] buffers seen as [pages, 1, page_size, bytes]."""
    pages, page, blk = 5, 16, 16 if fmt == "nvfp4" else 32
    ts = [torch.full((1,), 0.01, device="cuda")] * 2 if fmt == "nvfp4" else [None, None]
    flat = [torch.zeros(pages, page, 1, w, dtype=torch.uint8, device="cuda") for w in (dim // 2, dim // blk) * 2]
    cache = fp4.KVCache(fmt, *(t.transpose(1, 2) for t in flat), *ts)
    same = fp4.KVCache(fmt, *(torch.zeros_like(t).view(pages, 1, page, -1) for t in flat), *ts)
    x = torch.randn(20, 2, dim, device="cuda").bfloat16()
    slots = torch.randperm(pages * page, device="cuda")[:20]
    for c in (cache, same):
        fp4.kv_append(c, x[:, :1], x[:, 1:], slots)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(cache, n), getattr(same, n)) and getattr(same, n).any()
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    lens = torch.tensor([pages * page], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, dim, device="cuda").bfloat16()
    assert torch.equal(fp4.kv_attention(q, cache, table, lens), fp4.kv_attention(q, same, table, lens))


def test_rows_apart_are_refused(fp4):
    flat = [torch.zeros(5, 16, 2, w, dtype=torch.uint8, device="cuda") for w in (32, 2) * 2]
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp4", *(t.transpose(1, 2) for t in flat))
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp4", *(t[:, :, :1, ::2].transpose(1, 2) for t in flat))
