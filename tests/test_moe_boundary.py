"""Refusals of the mixture-of-experts entry points and of the products of few
rows, on the host: each wrong argument gives its documented status before any
HIP call. Device pointers are fake; calls that would pass every check run only
on a machine without a GPU, where the last check refuses them."""
import ctypes

import pytest
import torch

FAKE = 0x7F0000000000
NO_GPU = not torch.cuda.is_available()
cpu_only = pytest.mark.skipif(not NO_GPU, reason="would launch on fake pointers: host-only check")


def route_args(F, dtype=0, tokens=10, experts=32, top_k=4, **kw):
    a = F.fp4_moe_route_args(ctypes.sizeof(F.fp4_moe_route_args), dtype, 0, experts, top_k, 1, 1, 1, tokens, FAKE,
                             experts, FAKE, FAKE, FAKE, 1.0, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INVALID_ROUTE = [dict(size=8), dict(dtype=2), dict(dtype=-1), dict(flags=4), dict(experts=0), dict(top_k=0),
                 dict(top_k=33, experts=32), dict(groups=0), dict(groups=5), dict(groups=4, top_groups=0),
                 dict(groups=4, top_groups=5), dict(group_best=0), dict(group_best=3), dict(tokens=-1),
                 dict(logits=None), dict(ld_logits=31), dict(ids=None), dict(scale=float("inf")),
                 dict(scale=float("nan")), dict(reserved=1)]


@pytest.mark.parametrize("kw", INVALID_ROUTE, ids=[str(k) for k in INVALID_ROUTE])
def test_invalid_route(fp4, kw):
    assert fp4.fp4_moe_route(route_args(fp4, **kw), None) == fp4.FP4_ERR_INVALID
    assert fp4.fp4_moe_route_backward(route_args(fp4, **kw), FAKE, FAKE, 32, None) == fp4.FP4_ERR_INVALID


def test_route_refusals(fp4):
    F = fp4
    assert F.fp4_moe_route(route_args(F, weights=None), None) == F.FP4_ERR_INVALID
    unsupported = [dict(experts=1025, ld_logits=1025), dict(top_k=33, experts=64, ld_logits=64), dict(tokens=1 << 26),
                   dict(experts=128, groups=128, top_groups=1, ld_logits=128)]
    for kw in unsupported:
        assert F.fp4_moe_route(route_args(F, **kw), None) == F.FP4_ERR_UNSUPPORTED, kw
    for kw in (dict(logits=FAKE + 2), dict(ids=FAKE + 1), dict(bias=FAKE + 2), dict(weights=FAKE + 2),
               dict(dtype=1, logits=FAKE + 1)):
        assert F.fp4_moe_route(route_args(F, **kw), None) == F.FP4_ERR_ALIGN, kw
    back = lambda g=FAKE, o=FAKE, ld=32, **kw: F.fp4_moe_route_backward(route_args(F, **kw), g, o, ld, None)
    assert back(g=None) == back(o=None) == back(ld=31) == F.FP4_ERR_INVALID
    assert back(g=FAKE + 2) == back(o=FAKE + 2) == back(o=FAKE + 1, dtype=1) == F.FP4_ERR_ALIGN
    assert F.fp4_moe_route(route_args(F, tokens=0, logits=None, ids=None, weights=None), None) == F.FP4_OK
    assert back(tokens=0, logits=None, ids=None) == F.FP4_OK


def test_route_tokens_past_the_grid(fp4):
    """Four tokens a workgroup of 256, and 2^32 - 1 work items in all."""
    F = fp4
    for call in (lambda n: F.fp4_moe_route(route_args(F, tokens=n), None),
                 lambda n: F.fp4_moe_route_backward(route_args(F, tokens=n), FAKE, FAKE, 32, None)):
        assert call((1 << 26) - 3) == F.FP4_ERR_UNSUPPORTED
        if NO_GPU:
            assert call((1 << 26) - 4) == F.FP4_ERR_DEVICE


def test_group_refusals(fp4):
    F = fp4
    ws = F.fp4_moe_group_workspace(100000, 64)
    assert ws > 0 and F.fp4_moe_group_workspace(100, 64) == 0
    assert F.fp4_moe_group_workspace(-1, 64) == F.fp4_moe_group_workspace(10, 0) == 0
    assert F.fp4_moe_group_workspace(10, 1025) == F.fp4_moe_group_workspace((1 << 24) + 1, 8) == 0
    call = lambda pairs=100, ids=FAKE, experts=64, offsets=FAKE, order=FAKE, place=FAKE, w=FAKE, n=1 << 30: \
        F.fp4_moe_group(pairs, ids, experts, offsets, order, place, w, n, None)
    for kw in (dict(pairs=-1), dict(experts=0), dict(ids=None), dict(offsets=None), dict(order=None), dict(place=None),
               dict(pairs=0, offsets=None)):
        assert call(**kw) == F.FP4_ERR_INVALID, kw
    assert call(experts=1025) == call(pairs=(1 << 24) + 1) == F.FP4_ERR_UNSUPPORTED
    for kw in (dict(ids=FAKE + 2), dict(offsets=FAKE + 2), dict(order=FAKE + 1), dict(place=FAKE + 2),
               dict(pairs=100000, w=FAKE + 8)):
        assert call(**kw) == F.FP4_ERR_ALIGN, kw
    assert call(pairs=100000, w=None) == call(pairs=100000, n=ws - 1) == F.FP4_ERR_WORKSPACE


def test_dispatch_refusals(fp4):
    F = fp4
    call = lambda tokens=10, k=2, place=FAKE, kept=FAKE, nb=64, x=FAKE, ldx=64, r=FAKE, ldr=64, nb2=0, x2=None, ldx2=0, \
        r2=None, ldr2=0: F.fp4_moe_dispatch(tokens, k, place, kept, nb, x, ldx, r, ldr, nb2, x2, ldx2, r2, ldr2, None)
    for kw in (dict(tokens=-1), dict(k=0), dict(nb=-1), dict(nb2=-1), dict(place=None), dict(x=None), dict(r=None),
               dict(ldx=63), dict(ldr=63), dict(nb2=8), dict(nb2=8, x2=FAKE, r2=FAKE, ldx2=7, ldr2=8),
               dict(nb2=8, x2=FAKE, r2=FAKE, ldx2=8, ldr2=7)):
        assert call(**kw) == F.FP4_ERR_INVALID, kw
    assert call(k=1025) == call(tokens=1 << 24) == F.FP4_ERR_UNSUPPORTED
    assert call(place=FAKE + 2) == call(kept=FAKE + 1) == F.FP4_ERR_ALIGN
    assert call(tokens=0) == call(nb=0) == F.FP4_OK


def test_combine_refusals(fp4):
    F = fp4
    call = lambda dtype=0, tokens=10, k=2, width=64, rows=FAKE, ldr=64, n=20, place=FAKE, kept=FAKE, w=FAKE, out=FAKE, \
        ldo=64: F.fp4_moe_combine(dtype, tokens, k, width, rows, ldr, n, place, kept, w, out, ldo, None)
    back = lambda dtype=0, tokens=10, k=2, width=64, g=FAKE, ldg=64, rows=FAKE, ldr=64, n=20, place=FAKE, kept=FAKE, \
        w=FAKE, gr=FAKE, ldgr=64, gw=FAKE: F.fp4_moe_combine_backward(dtype, tokens, k, width, g, ldg, rows, ldr, n, place,
                                                                     kept, w, gr, ldgr, gw, None)
    for kw in (dict(dtype=2), dict(tokens=-1), dict(k=0), dict(width=-1), dict(n=-1), dict(ldr=63)):
        assert call(**kw) == back(**kw) == F.FP4_ERR_INVALID, kw
    for kw in (dict(k=1025), dict(tokens=1 << 24), dict(width=(1 << 24) + 1, ldr=1 << 25)):
        assert call(**kw) == back(**kw) == F.FP4_ERR_UNSUPPORTED, kw
    for kw in (dict(rows=FAKE + 2), dict(place=FAKE + 2), dict(kept=FAKE + 2), dict(w=FAKE + 2),
               dict(dtype=1, rows=FAKE + 1)):
        assert call(**kw) == back(**kw) == F.FP4_ERR_ALIGN, kw
    assert call(rows=None) == call(out=None) == call(ldo=63) == F.FP4_ERR_INVALID
    assert call(out=FAKE + 2) == F.FP4_ERR_ALIGN
    for kw in (dict(g=None), dict(ldg=63), dict(gr=None), dict(ldgr=63), dict(rows=None)):
        assert back(**kw) == F.FP4_ERR_INVALID, kw
    assert back(tokens=1 << 22, k=4) == F.FP4_ERR_UNSUPPORTED
    assert back(g=FAKE + 2) == back(gr=FAKE + 1) == back(gw=FAKE + 2) == F.FP4_ERR_ALIGN
    assert call(tokens=0) == call(width=0) == back(tokens=0) == back(width=0) == F.FP4_OK


def matvec_args(F, fmt=1, x_dtype=1, pairs=3, N=64, K=256, **kw):
    blk = 16 if fmt == 1 else 32
    a = F.fp4_matvec_args(ctypes.sizeof(F.fp4_matvec_args), fmt, x_dtype, 1, pairs, 1, N, K, FAKE, K, FAKE, K // 2,
                          N * K // 2, FAKE, (K // blk + 15) // 16 * 16, N * ((K // blk + 15) // 16 * 16), FAKE, 1, None,
                          FAKE, N)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INVALID_MATVEC = [dict(size=8), dict(format=2), dict(x_dtype=2), dict(y_dtype=-1), dict(pairs=-1), dict(repeat=0),
                  dict(N=-1), dict(K=-16), dict(K=24), dict(format=0, K=48), dict(experts=0), dict(x=None), dict(ld_x=255),
                  dict(codes=None), dict(ld_codes=127), dict(scales=None), dict(ld_scales=15, K=512, ld_x=512, ld_codes=256),
                  dict(tensor_scale=None), dict(y=None), dict(ld_y=63), dict(experts=2, codes_expert_stride=-16),
                  dict(experts=2, scales_expert_stride=-16)]


@pytest.mark.parametrize("kw", INVALID_MATVEC, ids=[str(k) for k in INVALID_MATVEC])
def test_invalid_matvec(fp4, kw):
    assert fp4.fp4_matvec(matvec_args(fp4, **kw), None) == fp4.FP4_ERR_INVALID


def test_matvec_refusals(fp4):
    F = fp4
    for kw in (dict(experts=4097), dict(K=(1 << 24) + 16), dict(N=1 << 31), dict(N=1 << 27), dict(pairs=1 << 20),
               dict(pairs=4097, ids=FAKE), dict(ld_codes=1 << 23), dict(ld_scales=1 << 23)):
        assert F.fp4_matvec(matvec_args(F, **kw), None) == F.FP4_ERR_UNSUPPORTED, kw
    for kw in (dict(x=FAKE + 8), dict(ld_x=257), dict(codes=FAKE + 8), dict(ld_codes=136), dict(scales=FAKE + 8),
               dict(ld_scales=24), dict(experts=2, codes_expert_stride=8), dict(experts=2, scales_expert_stride=8),
               dict(tensor_scale=FAKE + 2), dict(ids=FAKE + 2), dict(y=FAKE + 1), dict(y_dtype=0, y=FAKE + 2)):
        assert F.fp4_matvec(matvec_args(F, **kw), None) == F.FP4_ERR_ALIGN, kw
    for kw in (dict(pairs=0, y=None, x=None), dict(N=0, codes=None)):
        assert F.fp4_matvec(matvec_args(F, **kw), None) == F.FP4_OK, kw


def test_fp32_rows_of_matvec_past_the_grid(fp4):
    """fp32 rows go eight a pass: 65535 passes are 2^19 - 8 rows."""
    F = fp4
    assert F.fp4_matvec(matvec_args(F, x_dtype=0, pairs=(1 << 19) - 7, ld_x=256), None) == F.FP4_ERR_UNSUPPORTED
    if NO_GPU:
        assert F.fp4_matvec(matvec_args(F, x_dtype=0, pairs=(1 << 19) - 8, ld_x=256), None) == F.FP4_ERR_DEVICE


@cpu_only
def test_good_calls_reach_the_device_check(fp4):
    F = fp4
    assert F.fp4_moe_route(route_args(F), None) == F.FP4_ERR_DEVICE
    assert F.fp4_moe_route(route_args(F, bias=None, experts=256, groups=8, top_groups=4, group_best=2, flags=3,
                                      ld_logits=256), None) == F.FP4_ERR_DEVICE
    assert F.fp4_moe_route_backward(route_args(F, weights=None, bias=None), FAKE, FAKE, 32, None) == F.FP4_ERR_DEVICE
    assert F.fp4_moe_group(0, None, 4, FAKE, None, None, None, 0, None) == F.FP4_ERR_DEVICE
    assert F.fp4_moe_dispatch(1, 1, FAKE, None, 3, FAKE + 1, 5, FAKE + 3, 7, 0, None, 0, None, 0, None) == F.FP4_ERR_DEVICE
    assert F.fp4_moe_combine(1, 1, 1, 3, FAKE + 2, 5, 9, None, None, None, FAKE + 6, 3, None) == F.FP4_ERR_DEVICE
    assert F.fp4_moe_combine_backward(0, 1, 1, 3, FAKE, 3, None, 0, 9, None, None, None, FAKE, 3, None,
                                      None) == F.FP4_ERR_DEVICE
    for kw in (dict(), dict(format=0), dict(ids=FAKE, experts=8), dict(K=0, x=None, codes=None, scales=None),
               dict(repeat=1 << 40), dict(pairs=(1 << 20) - 16)):
        assert F.fp4_matvec(matvec_args(F, **kw), None) == F.FP4_ERR_DEVICE, kw


def test_python_checks(fp4):
    """What the conveniences refuse by themselves, on tensors of the CPU."""
    z = torch.zeros(4, 8)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    q = fp4.Quantized(fp4.FP4_MXFP4, torch.zeros(16, 32, dtype=torch.uint8), torch.zeros(16, 2, dtype=torch.uint8), None)
    g = fp4.MoeGroups(torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    for call in (lambda: fp4.moe_route(z, 2), lambda: fp4.moe_route_backward(z, z, ids), lambda: fp4.moe_group(ids, 2),
                 lambda: fp4.moe_dispatch(z, g), lambda: fp4.moe_combine(z, z, g),
                 lambda: fp4.moe_combine_backward(z, z, z, g), lambda: fp4.matvec(torch.zeros(1, 64), q)):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()
