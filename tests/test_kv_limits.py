"""Key-value cache calls at the limits of a launch and of their arguments:
refused with the documented status on the host, or answered."""
import pytest
import torch

from test_kv_boundary import FAKE, append_args, attend, attention_args, cache, cpu_only


def test_more_work_items_than_a_launch_has(fp4):
    """2^32 work items along x and more, which HIP refuses."""
    c = cache(fp4)
    assert fp4.fp4_kv_append(c, append_args(fp4, c, tokens=2 ** 26), None) == fp4.FP4_ERR_UNSUPPORTED
    assert fp4.fp4_kv_read(c, 2 ** 27, FAKE, FAKE, FAKE, 1, None) == fp4.FP4_ERR_UNSUPPORTED
    for n in (2 ** 23, 2 ** 24):
        assert attend(fp4, c, attention_args(fp4, c, batch=n, tokens=n)) == fp4.FP4_ERR_UNSUPPORTED
    # rows of one head each, in the form for prompts too
    c = cache(fp4, heads=2048)
    a = attention_args(fp4, c, batch=1, tokens=2 ** 20, q_heads=2048, q_offsets=FAKE)
    assert attend(fp4, c, a) == fp4.FP4_ERR_UNSUPPORTED


@cpu_only
def test_as_many_work_items_as_a_launch_has(fp4):
    """One workgroup less gets as far as the device check."""
    c = cache(fp4)
    assert fp4.fp4_kv_append(c, append_args(fp4, c, tokens=2 ** 26 - 4), None) == fp4.FP4_ERR_DEVICE
    assert fp4.fp4_kv_read(c, 2 ** 27 - 8, FAKE, FAKE, FAKE, 1, None) == fp4.FP4_ERR_DEVICE
    n = 2 ** 23 - 1
    assert attend(fp4, c, attention_args(fp4, c, batch=n, tokens=n)) == fp4.FP4_ERR_DEVICE


def test_windows_that_hide_nothing(fp4):
    """A window of max_kv_len rows or more plans the same work as none."""
    c = cache(fp4, pages=1 << 16)
    kw = dict(batch=1, tokens=1, table_width=8192, table_stride=8192, max_kv_len=131072)
    need = fp4.fp4_kv_attention_workspace(c, attention_args(fp4, c, **kw))
    assert need > 0
    for window in (131072, 2 ** 31, 2 ** 63 - 1):
        assert fp4.fp4_kv_attention_workspace(c, attention_args(fp4, c, window=window, **kw)) == need


@pytest.mark.gpu
def test_a_window_without_end(fp4):
    c = fp4.KVCache.empty("mxfp4", 600, 16, 2, 64)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, device="cuda"))
    for t in (c.k_scales, c.v_scales):
        t.fill_(126)
    table = torch.arange(600, dtype=torch.int32, device="cuda").view(1, 600)
    for n, length in ((1, 9000), (40, 300)):
        q = torch.randn(n, 4, 64, device="cuda").bfloat16()
        kw = dict(q_offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_kv_len=length)
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        want = fp4.kv_attention(q, c, table, lens, **kw)
        for window in (length, 2 ** 40, 2 ** 63 - 1):
            assert torch.equal(fp4.kv_attention(q, c, table, lens, window=window, **kw), want)


@pytest.mark.gpu
def test_append_of_as_many_heads_as_there_may_be(fp4):
    """Heads of which one token fills more than 65535 waves, against the same
    in four calls."""
    heads, dim, part = 65535, 256, 16384
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1, heads, dim, generator=g, device="cuda").bfloat16() for _ in range(3))
    slot = torch.tensor([5], device="cuda")
    ang = torch.rand(1, dim // 2, generator=g, device="cuda")
    kw = dict(positions=torch.zeros(1, dtype=torch.int64, device="cuda"), cos=ang.cos(), sin=ang.sin())
    whole = fp4.KVCache.empty("mxfp4", 1, 16, heads, dim)
    got = fp4.kv_append(whole, k, v, slot, q=q, **kw)
    for h in range(0, heads, part):
        s = slice(h, min(h + part, heads))
        some = fp4.KVCache.empty("mxfp4", 1, 16, s.stop - h, dim)
        assert torch.equal(got[:, s], fp4.kv_append(some, k[:, s], v[:, s], slot, q=q[:, s], **kw))
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(whole, n)[:, s], getattr(some, n))
