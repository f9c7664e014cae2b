"""Calls that name a stream: what they allocate belongs to that stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def late_writes(nbytes):
    """Queues, on the current stream, about 50 ms of waiting and then a write
    of 0xFF over memory that the allocator holds free afterwards: whoever is
    given it for another stream, without waiting for this one, is written over.
    (The wait is bounded: a number of clock cycles.)"""
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in nbytes for _ in range(4)]
    torch.cuda._sleep(100_000_000)
    for t in junk:
        t.fill_(255)


def ordered(side, call):
    """call(stream) on `side` while the current stream still has to write over
    freed memory of the sizes of the call's tensors; its results, on the host,
    when all is done."""
    got = call(side.cuda_stream)
    side.synchronize()      # the results are there, the late writes are not
    torch.cuda.synchronize()
    return [t.cpu() for t in (got if isinstance(got, tuple) else (got,))]


def make(fp4):
    cache = fp4.KVCache.empty("mxfp4", 300, 16, 2, 128)
    for t in (cache.k_codes, cache.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, device="cuda"))
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(126)
    return cache


def test_kv_attention_on_another_stream(fp4):
    cache = make(fp4)
    q = torch.randn(1, 8, 128, device="cuda").to(BF)
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300)
    lens = torch.tensor([4700], dtype=torch.int32, device="cuda")
    call = lambda s: fp4.kv_attention(q, cache, table, lens, return_lse=True, stream=s)
    want = [t.cpu() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late_writes([q.numel() * 2, 8 * 4, 1 << 20, 8 << 20])
    for y, w in zip(ordered(side, call), want):
        assert torch.equal(y, w)
    out = torch.empty_like(q)
    late_writes([1 << 20, 8 << 20])
    got = ordered(side, lambda s: fp4.kv_attention(q, cache, table, lens, out=out, stream=s))
    assert torch.equal(got[0], want[0]) and torch.equal(out.cpu(), want[0])


def test_kv_append_and_read_on_another_stream(fp4):
    cache, other = make(fp4), make(fp4)
    x = torch.randn(64, 8, 128, device="cuda").to(BF)
    slots = torch.arange(64, device="cuda") * 3
    ang = torch.rand(64, 64, device="cuda")
    pos = torch.arange(64, device="cuda")
    kw = dict(positions=pos, cos=ang.cos(), sin=ang.sin())
    want = fp4.kv_append(other, x[:, 4:6], x[:, 6:], slots, q=x[:, :4], **kw).cpu()
    want_kv = [t.cpu() for t in fp4.kv_read(other, slots)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late_writes([64 * 4 * 128 * 2])
    got = ordered(side, lambda s: fp4.kv_append(cache, x[:, 4:6], x[:, 6:], slots, q=x[:, :4], stream=s, **kw))
    assert torch.equal(got[0], want)
    late_writes([64 * 2 * 128 * 2])
    for y, w in zip(ordered(side, lambda s: fp4.kv_read(cache, slots, stream=s)), want_kv):
        assert torch.equal(y, w)


def test_results_outlive_reuse_on_the_callers_stream(fp4):
    """A result read late on the caller's stream and freed is not given to the
    next call on the other stream before it has been read."""
    cache = make(fp4)
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300).expand(64, 300).contiguous()
    lens = torch.full((64,), 300, dtype=torch.int32, device="cuda")
    q = torch.randn(64, 8, 128, device="cuda").to(BF)
    want = fp4.kv_attention(q, cache, table, lens).cpu()
    other = -q
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = fp4.kv_attention(q, cache, table, lens, stream=side.cuda_stream)
    side.synchronize()
    torch.cuda._sleep(100_000_000)
    copy = y.clone()
    del y
    for _ in range(4):
        fp4.kv_attention(other, cache, table, lens, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(copy.cpu(), want)


def test_the_default_stream_from_another(fp4):
    cache = make(fp4)
    q = torch.randn(1, 8, 128, device="cuda").to(BF)
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300)
    lens = torch.tensor([4700], dtype=torch.int32, device="cuda")
    want = fp4.kv_attention(q, cache, table, lens)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = fp4.kv_attention(q, cache, table, lens, stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_quantize_and_gemm_on_another_stream(fp4):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(256, 512, generator=g, device="cuda").to(BF).t()  # copied by the call
    w = torch.randn(512, 256, generator=g, device="cuda").to(BF)
    offsets = torch.tensor([0, 200, 512], dtype=torch.int32, device="cuda")
    qx, qw = fp4.quantize(x), fp4.quantize(w)
    pair = fp4.quantize(w.view(2, 256, 256), "mxfp4")
    qm = fp4.quantize(x, "mxfp4")
    calls = {
        "quantize": lambda s: fp4.quantize(x, four_over_six=True, stream=s),
        "dequantize": lambda s: fp4.dequantize(qx, stream=s),
        "gemm": lambda s: fp4.gemm(qx, qw, stream=s),
        "gemm_quantize_output": lambda s: fp4.gemm_quantize_output(qx, qw, amax=300.0, stream=s),
        "gemm_grouped": lambda s: fp4.gemm_grouped(qm, pair, offsets, stream=s),
    }
    parts = lambda y: (y.codes, y.scales, y.tensor_scale) if isinstance(y, fp4.Quantized) else (y,)
    side = torch.cuda.Stream()
    for name, call in calls.items():
        print(f"[streams] {name}", flush=True)
        want = [t.cpu() for t in parts(call(None))]
        torch.cuda.synchronize()
        late_writes([4, 512, 512 * 16, 512 * 128, 512 * 256 * 2, 512 * 512 * 2, 512 * 256 * 4, 512 * 512 * 4])
        got = ordered(side, lambda s: parts(call(s)))
        for y, z in zip(got, want):
            assert torch.equal(y, z), name
