"""The attention block of examples/attention_block.py: prompts, then tokens,
then a sequence that ends and gives its pages to another, checked against
attention in 64 bits over what kv_read finds in the cache."""
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from kv_util import attention_bounds, attention_f64

sys.path.insert(0, str(Path(__file__).resolve().parents[1] / "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_block(fp4, fmt):
    import attention_block as ex
    heads, kv_heads, dim, hidden, page = 8, 2, 64, 256, 16
    prompts = [70, 1, 33]
    pages = 12
    cache = fp4.KVCache.empty(fmt, pages, page, kv_heads, dim, k_amax=16.0, v_amax=16.0, four_over_six=True)
    seqs = ex.Sequences(pages, page, len(prompts), 96)
    block = ex.AttentionBlock(hidden, heads, kv_heads, dim, cache, 96)
    g = torch.Generator().manual_seed(5)

    def step(counts):
        at = seqs.step(counts)
        x = torch.randn(sum(counts), hidden, generator=g).bfloat16().cuda()
        q, out = block.attend(x, at)
        slots = torch.arange(pages * page).cuda()
        k, v = (t.double().cpu().numpy().reshape(pages, page, kv_heads, dim).transpose(0, 2, 1, 3)
                for t in fp4.kv_read(cache, slots, torch.float32))
        ref = attention_f64(q.double().cpu().numpy(), k, v, seqs.table.numpy(), page, seqs.lens, counts, True, 0, 0.0,
                            dim ** -0.5)
        tol, _ = attention_bounds(ref, fmt == "nvfp4", True, dim, 96, 0.0)
        err = np.abs(out.double().cpu().numpy() - ref[0])
        assert (err <= tol).all(), f"{counts}: worst {np.max(err / tol):.3g} of the bound"
        y = block.linear(out.flatten(1), block.w_o)
        assert y.shape == x.shape and y.isfinite().all()

    step(prompts)
    for _ in range(3):
        step([1] * 3)
    seqs.end(0)
    step([40, 1, 1])        # another sequence in the first one's pages
    step([1, 0, 5])         # one pauses, one is given several tokens
    assert sorted(seqs.free + sum(seqs.pages, [])) == list(range(pages))


def test_example_runs(fp4, capsys):
    import attention_block as ex
    ex.main("mxfp4", hidden=512, heads=8, kv_heads=2, head_dim=64, prompts=(100, 7), tokens=3)
    assert "us a step" in capsys.readouterr().out
