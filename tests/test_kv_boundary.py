"""Refusals of the key-value cache entry points, on the host: each wrong
argument gives its documented status before any HIP call. Device pointers are
fake; calls that would pass every check run only on a machine without a GPU."""
import ctypes

import pytest
import torch

FAKE = 0x7F0000000000
NO_GPU = not torch.cuda.is_available()
cpu_only = pytest.mark.skipif(not NO_GPU, reason="would launch on fake pointers: host-only check")


def cache(F, fmt=1, pages=10, page=16, heads=2, dim=128, size=None, cps=None, sps=None, **kw):
    blk = 16 if fmt == 1 else 32
    c = F.fp4_kv_cache(ctypes.sizeof(F.fp4_kv_cache) if size is None else size, fmt, pages, page, heads, dim, 0, FAKE,
                       FAKE, FAKE, FAKE, heads * page * dim // 2 if cps is None else cps,
                       heads * page * dim // blk if sps is None else sps, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append_args(F, c, dtype=1, tokens=5, q_heads=8, **kw):
    D, H = c.head_dim, c.kv_heads
    a = F.fp4_kv_append_args(ctypes.sizeof(F.fp4_kv_append_args), dtype, 0, q_heads, tokens, FAKE, FAKE, FAKE, FAKE,
                             H * D, D, H * D, D, q_heads * D, D, q_heads * D, D, FAKE, FAKE, FAKE, FAKE, 100, D, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention_args(F, c, dtype=1, batch=3, tokens=3, q_heads=8, **kw):
    D = c.head_dim
    a = F.fp4_kv_attention_args(ctypes.sizeof(F.fp4_kv_attention_args), dtype, 1, q_heads, batch, tokens, None, FAKE,
                                FAKE, 4, 4, 64, FAKE, FAKE, FAKE, q_heads * D, D, q_heads * D, D, 0.1, 0.0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attend(F, c, a, ws=FAKE, ws_bytes=1 << 40):
    return F.fp4_kv_attention(c, a, ws, ws_bytes, None)


def every_call(F, c):
    """The status each entry point gives for a cache handle."""
    return {F.fp4_kv_append(c, append_args(F, c), None), F.fp4_kv_read(c, 3, FAKE, FAKE, FAKE, 1, None),
            attend(F, c, attention_args(F, c))}


INVALID_CACHE = [dict(size=8), dict(fmt=3), dict(pages=-1), dict(heads=0), dict(dim=0), dict(dim=8), dict(dim=272),
                 dict(dim=100), dict(fmt=0, dim=48), dict(page=8), dict(page=24), dict(page=65536), dict(reserved=1),
                 dict(cps=16), dict(sps=16), dict(k_codes=None), dict(v_scales=None), dict(k_tensor_scale=None),
                 dict(v_tensor_scale=None), dict(pages=2 ** 30, cps=2 ** 40)]


@pytest.mark.parametrize("kw", INVALID_CACHE, ids=[str(k) for k in INVALID_CACHE])
def test_invalid_cache(fp4, kw):
    assert every_call(fp4, cache(fp4, **kw)) == {fp4.FP4_ERR_INVALID}


def test_misaligned_and_oversized_cache(fp4):
    for kw in (dict(k_codes=FAKE + 8), dict(v_scales=FAKE + 4), dict(k_tensor_scale=FAKE + 2), dict(cps=4096 + 8),
               dict(sps=4096 + 4)):
        assert every_call(fp4, cache(fp4, **kw)) == {fp4.FP4_ERR_ALIGN}, kw
    for kw in (dict(heads=65536), dict(heads=1024, page=32768, dim=256), dict(pages=2 ** 31)):
        assert every_call(fp4, cache(fp4, **kw)) == {fp4.FP4_ERR_UNSUPPORTED}, kw


def test_null_structs(fp4):
    L = fp4.lib()
    c = cache(fp4)
    assert L.fp4_kv_append(None, ctypes.byref(append_args(fp4, c)), None) == fp4.FP4_ERR_INVALID
    assert L.fp4_kv_append(ctypes.byref(c), None, None) == fp4.FP4_ERR_INVALID
    assert L.fp4_kv_read(None, 1, FAKE, FAKE, FAKE, 0, None) == fp4.FP4_ERR_INVALID
    assert L.fp4_kv_attention(ctypes.byref(c), None, None, 0, None) == fp4.FP4_ERR_INVALID
    assert L.fp4_kv_attention_workspace(ctypes.byref(c), None) == 0
    assert L.fp4_kv_attention_workspace(None, ctypes.byref(attention_args(fp4, c))) == 0


APPEND = [
    (dict(size=4), "INVALID"), (dict(dtype=2), "INVALID"), (dict(flags=2), "INVALID"), (dict(flags=512), "INVALID"),
    (dict(tokens=-1), "INVALID"), (dict(q_heads=-1), "INVALID"), (dict(rotary=-2), "INVALID"),
    (dict(rotary=130), "INVALID"), (dict(rotary=7), "INVALID"), (dict(max_position=-1), "INVALID"),
    (dict(reserved=1), "INVALID"), (dict(slots=None), "INVALID"), (dict(positions=None), "INVALID"),
    (dict(cos_table=None), "INVALID"), (dict(sin_table=None), "INVALID"), (dict(k=None), "INVALID"),
    (dict(v=None), "INVALID"), (dict(q=None), "INVALID"), (dict(q_out=None), "INVALID"),
    (dict(k_token_stride=-256), "INVALID"), (dict(q_out_head_stride=64), "INVALID"),
    (dict(q_out_token_stride=128), "INVALID"), (dict(k=FAKE + 8), "ALIGN"), (dict(q_out=FAKE + 2), "ALIGN"),
    (dict(v_head_stride=132), "ALIGN"), (dict(q_token_stride=1028), "ALIGN"), (dict(slots=FAKE + 4), "ALIGN"),
    (dict(positions=FAKE + 4), "ALIGN"), (dict(cos_table=FAKE + 2), "ALIGN"), (dict(tokens=2 ** 31), "UNSUPPORTED"),
    (dict(q_heads=70000), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,want", APPEND, ids=[str(k) for k, _ in APPEND])
def test_append_refusals(fp4, kw, want):
    c = cache(fp4)
    assert fp4.fp4_kv_append(c, append_args(fp4, c, **kw), None) == getattr(fp4, "FP4_ERR_" + want)


def test_append_empty_call(fp4):
    c = cache(fp4)
    assert fp4.fp4_kv_append(c, append_args(fp4, c, tokens=0, k=None, slots=None), None) == fp4.FP4_OK


def test_read_refusals(fp4):
    c = cache(fp4)
    read = fp4.fp4_kv_read
    assert read(c, 3, FAKE, FAKE, FAKE, 2, None) == fp4.FP4_ERR_INVALID
    assert read(c, -1, FAKE, FAKE, FAKE, 1, None) == fp4.FP4_ERR_INVALID
    assert read(c, 3, None, FAKE, FAKE, 1, None) == fp4.FP4_ERR_INVALID
    assert read(c, 3, FAKE, None, FAKE, 1, None) == fp4.FP4_ERR_INVALID
    assert read(c, 3, FAKE, FAKE, FAKE + 8, 1, None) == fp4.FP4_ERR_ALIGN
    assert read(c, 3, FAKE + 4, FAKE, FAKE, 1, None) == fp4.FP4_ERR_ALIGN
    assert read(c, 2 ** 31, FAKE, FAKE, FAKE, 1, None) == fp4.FP4_ERR_UNSUPPORTED
    assert read(c, 0, None, None, None, 1, None) == fp4.FP4_OK


ATTENTION = [
    (dict(size=4), "INVALID"), (dict(dtype=2), "INVALID"), (dict(flags=2), "INVALID"), (dict(batch=-1), "INVALID"),
    (dict(tokens=-1), "INVALID"), (dict(q_heads=0), "INVALID"), (dict(q_heads=7), "INVALID"),
    (dict(tokens=4), "INVALID"), (dict(table_width=-1), "INVALID"), (dict(table_stride=3), "INVALID"),
    (dict(max_kv_len=65), "INVALID"), (dict(max_kv_len=-1), "INVALID"), (dict(window=-1), "INVALID"),
    (dict(window=5, flags=0), "INVALID"), (dict(scale=float("nan")), "INVALID"), (dict(scale=float("inf")), "INVALID"),
    (dict(softcap=-1.0), "INVALID"), (dict(softcap=float("inf")), "INVALID"), (dict(kv_lens=None), "INVALID"),
    (dict(block_table=None), "INVALID"), (dict(q=None), "INVALID"), (dict(out=None), "INVALID"),
    (dict(q_token_stride=-8), "INVALID"), (dict(out_head_stride=64), "INVALID"), (dict(q=FAKE + 8), "ALIGN"),
    (dict(out=FAKE + 8), "ALIGN"), (dict(q_head_stride=132), "ALIGN"), (dict(out_token_stride=1028), "ALIGN"),
    (dict(kv_lens=FAKE + 2), "ALIGN"), (dict(q_offsets=FAKE + 2), "ALIGN"), (dict(block_table=FAKE + 2), "ALIGN"),
    (dict(lse=FAKE + 2), "ALIGN"), (dict(tokens=2 ** 25, batch=2 ** 25), "UNSUPPORTED"),
    (dict(table_width=2 ** 31, table_stride=2 ** 31), "UNSUPPORTED"), (dict(q_heads=65536), "UNSUPPORTED"),
]


@pytest.mark.parametrize("kw,want", ATTENTION, ids=[str(k) for k, _ in ATTENTION])
def test_attention_refusals(fp4, kw, want):
    c = cache(fp4)
    assert attend(fp4, c, attention_args(fp4, c, **kw)) == getattr(fp4, "FP4_ERR_" + want)


def test_attention_over_no_pages(fp4):
    c = cache(fp4, pages=0)
    assert attend(fp4, c, attention_args(fp4, c)) == fp4.FP4_ERR_INVALID


def test_attention_empty_call(fp4):
    c = cache(fp4)
    assert attend(fp4, c, attention_args(fp4, c, batch=0, tokens=0), None, 0) == fp4.FP4_OK
    offs = attention_args(fp4, c, tokens=0, q_offsets=FAKE)
    assert attend(fp4, c, offs, None, 0) == fp4.FP4_OK


def test_attention_workspace(fp4):
    """A long sequence is cut into chunks whose results need a workspace;
    many sequences, or short ones, need none."""
    c = cache(fp4, pages=1 << 16)
    big = attention_args(fp4, c, batch=1, tokens=1, table_width=8192, table_stride=8192, max_kv_len=131072)
    need = fp4.fp4_kv_attention_workspace(c, big)
    assert need > 0 and need % 4 == 0
    assert attend(fp4, c, big, None, 0) == fp4.FP4_ERR_WORKSPACE
    assert attend(fp4, c, big, FAKE, need - 1) == fp4.FP4_ERR_WORKSPACE
    assert attend(fp4, c, big, FAKE + 4, need) == fp4.FP4_ERR_ALIGN
    short = attention_args(fp4, c, max_kv_len=20)
    assert fp4.fp4_kv_attention_workspace(c, short) == 0
    bad = attention_args(fp4, c, q_heads=7)
    assert fp4.fp4_kv_attention_workspace(c, bad) == 0


@cpu_only
def test_calls_without_a_gpu(fp4):
    """Valid calls get as far as the device check."""
    c = cache(fp4)
    assert every_call(fp4, c) == {fp4.FP4_ERR_DEVICE}
    z = append_args(fp4, c, q_heads=0, q=None, q_out=None, rotary=0, positions=None, cos_table=None, sin_table=None)
    assert fp4.fp4_kv_append(c, z, None) == fp4.FP4_ERR_DEVICE
    assert attend(fp4, c, attention_args(fp4, c, lse=None, max_kv_len=0, block_table=None)) == fp4.FP4_ERR_DEVICE


def test_python_refusals(fp4):
    """Operands that are not device tensors of the right kind are refused in
    Python, with ValueError."""
    u8 = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp4", u8, u8[..., :4], u8, u8[..., :4])
    with pytest.raises(ValueError):
        fp4.KVCache("mxfp4", u8[0], u8, u8, u8)
    with pytest.raises(ValueError):
        fp4.KVCache.empty("nvfp4", 2, 16, 2, 64, device="cpu")


@pytest.mark.gpu
def test_python_refusals_of_device_tensors(fp4):
    c = fp4.KVCache.empty("mxfp4", 4, 16, 2, 64)
    x = torch.zeros(3, 2, 64, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    tab = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    cos = torch.zeros(5, 32, device="cuda")
    bad = [lambda: fp4.kv_append(c, x[:2], x, slots), lambda: fp4.kv_append(c, x.cpu(), x, slots),
           lambda: fp4.kv_append(c, x.half(), x.half(), slots), lambda: fp4.kv_append(c, x, x.bfloat16(), slots),
           lambda: fp4.kv_append(c, x, x, slots.int()), lambda: fp4.kv_append(c, x, x, slots, cos=cos),
           lambda: fp4.kv_append(c, x, x, slots, cos=cos, sin=cos.double(), positions=slots),
           lambda: fp4.kv_append(c, x, x, slots, q=x[..., :32]), lambda: fp4.kv_append(c, x, x, slots, q_out=x),
           lambda: fp4.kv_append(c, x[:, :1], x[:, :1], slots), lambda: fp4.kv_append(c, x, x, slots, q=x.bfloat16()),
           lambda: fp4.kv_append(c, x.transpose(1, 2).contiguous().transpose(1, 2), x, slots),
           lambda: fp4.kv_read(c, slots.cpu()), lambda: fp4.kv_read(c, slots, torch.float16),
           lambda: fp4.kv_attention(x, c, tab.long(), lens), lambda: fp4.kv_attention(x, c, tab, lens.long()),
           lambda: fp4.kv_attention(x, c, tab, lens[:2]), lambda: fp4.kv_attention(x.half(), c, tab, lens),
           lambda: fp4.kv_attention(x, c, tab, lens, q_offsets=lens), lambda: fp4.kv_attention(x[0], c, tab, lens),
           lambda: fp4.kv_attention(x, c, tab, lens, out=x.bfloat16()),
           lambda: fp4.KVCache.empty("nvfp4", 2, 16, 2, 64)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            print("refusal", i, flush=True)
            f()
    for f in (lambda: fp4.kv_attention(x[:2], c, tab, lens), lambda: fp4.kv_attention(x, c, tab, lens, causal=False, window=3),
              lambda: fp4.kv_attention(torch.zeros(3, 3, 64, device="cuda"), c, tab, lens)):
        with pytest.raises(fp4.Fp4Error):
            f()
