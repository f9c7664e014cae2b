"""Attention over the 4-bit cache where rows that a query does not see hold
infinities, NaN and pages of no one."""
import numpy as np
import pytest
import torch

from kv_util import attention_bounds, attention_f64, check_attention, lay_out, random_cache, spoil
from test_gpu_kv import prompt_f64

pytestmark = pytest.mark.gpu

MX, NV = 0, 1
BF, F32 = torch.bfloat16, torch.float32
FD = [(f, d) for f in (MX, NV) for d in (BF, F32)]
FD_IDS = ["mx-bf16", "mx-f32", "nv-bf16", "nv-f32"]


def masked_case(F, O, fmt, dtype, lens, q_lens, heads, kv_heads, dim, page, window=0, bad=(), poison="nan", seed=70,
                ref_of=attention_f64):
    """A causal call whose cached rows `bad` (sequence, row) are NaN, or of
    infinite values (MXFP4), beside the rows before each sequence's first
    window, which are NaN and whose whole pages the table does not name.
    Queries that see a bad row are not finite; the others are as if it were
    not there."""
    need = sum(-(-n // page) for n in lens)
    cache, k, v = random_cache(F, O, fmt, need + 2, page, kv_heads, dim, seed)
    table = lay_out(cache, lens, seed)
    spoil(cache, table, lens)
    given = table.copy()
    hidden = {(b, j) for b, (n, ql) in enumerate(zip(lens, q_lens)) if window and ql
              for j in range(max(0, n - ql + 1 - window))}
    for b, j in [*bad, *hidden]:
        pg, r = table[b, j // page], j % page
        if poison == "nan" or (b, j) in hidden:
            for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
                t[pg, :, r] = 255
        elif poison == "nan scales":
            cache.k_codes[pg, :, r] = cache.v_codes[pg, :, r] = 0
            cache.v_scales[pg, :, r] = 255
        else:  # 6 * 2^127
            cache.v_codes[pg, :, r] = 0x77
            cache.v_scales[pg, :, r] = 254
        k[pg, :, r] = 0
        v[pg, :, r] = 0
        if (b, j) in hidden and (j + 1) % page == 0:  # the whole page is
            given[b, j // page] = -1
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(sum(q_lens), heads, dim, generator=g).to(dtype)
    decode = all(n == 1 for n in q_lens)
    offs = None if decode else torch.tensor(np.cumsum([0] + list(q_lens)), dtype=torch.int32, device="cuda")
    out, lse = F.kv_attention(q.cuda(), cache, torch.from_numpy(given).cuda(),
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), q_offsets=offs, window=window,
                              return_lse=True, max_kv_len=max(lens))
    torch.cuda.synchronize()
    ref = ref_of(q.double().numpy(), k, v, table, page, lens, q_lens, True, window, 0.0, dim ** -0.5)
    tol, tol_lse = attention_bounds(ref, fmt == NV, dtype == BF, dim, max(lens), 0.0)
    starts = np.cumsum([0] + list(q_lens))
    sees = np.zeros(sum(q_lens), bool)
    for b, j in bad:
        for i in range(q_lens[b]):
            last = lens[b] - q_lens[b] + i
            sees[starts[b] + i] |= j <= last and (not window or j > last - window)
    clean = ~sees
    check_attention(out[torch.from_numpy(clean).cuda()], lse[torch.from_numpy(clean).cuda()],
                    tuple(x[clean] for x in ref), tol[clean], tol_lse[clean], f"fmt {fmt} {dtype} lens {lens[:4]}")
    if sees.any():
        assert not out[torch.from_numpy(sees).cuda()].isfinite().any(), "a row that sees a bad value is finite"


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
def test_rows_before_the_window(fp4, oracle, fmt, dtype, dim):
    """Rows and whole pages before every query's window: NaN, and pages given
    back (their table entries -1)."""
    print(f"[before] {fmt} {dtype} {dim}", flush=True)
    for window in (1, 20, 45):
        masked_case(fp4, oracle, fmt, dtype, [1, 47, 130, 301], [1] * 4, 4, 2, dim, 16, window=window)
    masked_case(fp4, oracle, fmt, dtype, [90, 200], [7, 40], 8, 2, dim, 16, window=21)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
def test_rows_before_the_window_of_long_sequences(fp4, oracle, fmt, dtype):
    print(f"[before, long] {fmt} {dtype}", flush=True)
    masked_case(fp4, oracle, fmt, dtype, [9000, 30, 6000], [1] * 3, 20, 1, 96, 32, window=5000)


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
@pytest.mark.parametrize("dim,heads,kv_heads", [(32, 4, 2), (64, 4, 4), (128, 8, 1), (256, 2, 1)])
def test_rows_hidden_by_the_order(fp4, oracle, fmt, dtype, dim, heads, kv_heads):
    """Rows of later tokens: NaN, which later queries see and earlier ones do
    not."""
    print(f"[hidden] {fmt} {dtype} {dim}", flush=True)
    masked_case(fp4, oracle, fmt, dtype, [130, 40, 64], [70, 9, 64], heads, kv_heads, dim, 16,
                bad=[(0, 100), (0, 129), (1, 35), (2, 0), (2, 63)])
    masked_case(fp4, oracle, fmt, dtype, [130], [70], heads, kv_heads, dim, 16, window=33, bad=[(0, 90), (0, 91)])


@pytest.mark.parametrize("fmt,dtype", FD, ids=FD_IDS)
def test_nan_scales_of_zeros_hidden_by_the_order(fp4, oracle, fmt, dtype):
    """Values of NaN scale alone, beside keys of 0."""
    print(f"[hidden, scales] {fmt} {dtype}", flush=True)
    masked_case(fp4, oracle, fmt, dtype, [130, 40], [70, 9], 8, 2, 128, 16, bad=[(0, 100), (0, 129), (1, 35)],
                poison="nan scales")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_infinite_values_hidden_by_the_order(fp4, oracle, dtype):
    print(f"[hidden, inf] {dtype}", flush=True)
    masked_case(fp4, oracle, MX, dtype, [130, 40], [70, 9], 8, 2, 128, 16, bad=[(0, 100), (0, 129), (1, 35)],
                poison="inf")


FILLING = [
    (64, 64, 128, 64, [300, 760], [300, 720], 0),
    (64, 32, 96, 16, [500, 640, 0, 40], [480, 640, 3, 45], 90),
    (128, 64, 64, 32, [500, 300, 33], [470, 300, 33], 0),
    (128, 64, 32, 16, [400, 260], [400, 260], 50),
    (64, 64, 256, 32, [300, 760], [300, 740], 0),
]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("case", FILLING, ids=[f"{c[0]}x{c[2]}" for c in FILLING])
def test_hidden_rows_in_prompts_that_fill_the_gpu(fp4, oracle, fmt, case):
    heads, kv_heads, dim, page, lens, q_lens, window = case
    print(f"[hidden, filling] {fmt} {case}", flush=True)
    masked_case(fp4, oracle, fmt, BF, lens, q_lens, heads, kv_heads, dim, page, window=window,
                bad=[(0, lens[0] - 70), (1, lens[1] - 1), (1, lens[1] - 40), (1, lens[1] - 211)], ref_of=prompt_f64)
