"""Products of a few rows where the passes over them are more than the
workgroups that fit at once, so that one workgroup takes many tiles of its
pass. Values against 64 bits, within the bound of test_gpu_matvec.py:
(2 K + 4) 2^-24 of the sum of magnitudes, and one rounding of y. (The
definition is evaluated on the GPU, in float64, expert by expert.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def random_weights(fp4, fmt, N, K, experts, seed):
    """Any codes; scales of a few powers of two (MXFP4), or any finite E4M3 (NVFP4)."""
    g = torch.Generator("cuda").manual_seed(seed)
    lead = (experts,) if experts else ()
    blk = 32 if fmt == "mxfp4" else 16
    pitch = -(-(K // blk) // 16) * 16
    codes = torch.randint(0, 256, (*lead, N, K // 2), dtype=torch.uint8, generator=g, device="cuda")
    low, high = (118, 126) if fmt == "mxfp4" else (1, 127)
    scales = torch.randint(low, high, (*lead, N, pitch), dtype=torch.uint8, generator=g, device="cuda")[..., :K // blk]
    if fmt == "mxfp4":
        return fp4.Quantized(fp4.FP4_MXFP4, codes, scales, None)
    ts = 0.001 * (1 + torch.rand(experts or 1, generator=g, device="cuda"))
    return fp4.Quantized(fp4.FP4_NVFP4, codes, scales, ts)


def values(codes, scales, fmt, ts):
    """float64 [N, K] of one matrix."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()]
    s = scales.double()
    if fmt == "mxfp4":
        s = torch.exp2(s - 127)
    else:
        e, m = torch.div(s, 8, rounding_mode="floor"), s % 8
        s = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e - 7) * (1 + m / 8)) * ts.double()
    return v * s.repeat_interleave(32 if fmt == "mxfp4" else 16, 1)


def check(y, x, W, dtype):
    want = x.double() @ W.T
    size = x.double().abs() @ W.abs().T
    tol = (2 * x.shape[1] + 4) * U * size + (2.0 ** -8 if dtype == "bf16" else U) * want.abs() + 1e-38
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {(err / tol).max().item():.3g} of the bound"


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype,M_,N,K", [("bf16", 8208, 300, 4096), ("bf16", 20000, 70, 96), ("bf16", 8192, 300, 512),
                                          ("f32", 4112, 300, 2880), ("f32", 8208, 150, 64), ("f32", 4096, 300, 5152)])
def test_many_passes_over_one_matrix(fp4, fmt, dtype, M_, N, K):
    q = random_weights(fp4, fmt, N, K, 0, M_ + K)
    x = torch.randn(M_, K, generator=torch.Generator("cuda").manual_seed(K), device="cuda").to(DT[dtype])
    y = fp4.matvec(x, q)
    check(y, x, values(q.codes, q.scales, fmt, q.tensor_scale), dtype)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype,T,k,E,N,K", [("bf16", 130, 8, 384, 300, 7168), ("bf16", 512, 8, 1024, 150, 2048),
                                             ("bf16", 1024, 4, 2048, 80, 64), ("f32", 512, 8, 256, 300, 2880),
                                             ("f32", 258, 8, 256, 150, 2048), ("f32", 964, 4, 32, 300, 2880)])
def test_many_passes_by_experts(fp4, fmt, dtype, T, k, E, N, K):
    q = random_weights(fp4, fmt, N, K, E, T + K)
    g = torch.Generator("cuda").manual_seed(K)
    ids = torch.randint(-1, E + 1, (T, k), dtype=torch.int32, generator=g, device="cuda")
    ids[: T // 3, 0] = E // 2  # one expert of many passes
    x = torch.randn(T, K, generator=g, device="cuda").to(DT[dtype])
    y = torch.full((T, k, N), torch.nan, dtype=DT[dtype], device="cuda")
    fp4.matvec(x, q, ids, out=y)
    rows, flat = y.flatten(0, 1), ids.flatten()
    tokens = torch.arange(T * k, device="cuda") // k
    assert (rows[(flat < 0) | (flat >= E)] == 0).all()
    for e in range(E):
        at = (flat == e).nonzero()[:, 0]
        if at.numel():
            ts = None if q.tensor_scale is None else q.tensor_scale[e]
            check(rows[at], x[tokens[at]], values(q.codes[e], q.scales[e], fmt, ts), dtype)


def test_all_pairs_of_many_without_an_expert(fp4):
    q = random_weights(fp4, "mxfp4", 300, 64, 2048, 1)
    ids = torch.full((4096,), -1, dtype=torch.int32, device="cuda")
    y = torch.full((4096, 300), 7.0, device="cuda")
    fp4.matvec(torch.ones(4096, 64, device="cuda"), q, ids, out=y)
    assert (y == 0).all()
