"""The launches of products of a few rows, planned on the host for sizes up to
the documented limits: every plan ends, fits the GPU's limits and covers its
tiles and rows. (matvec_plan.h has no HIP in it and is compiled here alone.)"""
import ctypes
import itertools
import shutil
import subprocess
from pathlib import Path
from types import SimpleNamespace

import pytest

ROOT = Path(__file__).resolve().parents[1]
FIELDS = ("rg", "waves", "units", "part_shift", "seg_units", "rounds", "at_once", "tiles", "grid_x", "slots", "lds")
CUS = 256
LIMIT = {True: (1 << 20) - 16, False: (1 << 19) - 8}  # rows of one matrix: bf16, fp32


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    lib = tmp_path_factory.mktemp("plan") / "plan.so"
    subprocess.run([cxx, "-O1", "-std=c++17", "-ftrapv", "-shared", "-fPIC", "-I",
                    str(ROOT / "block_scaled_fp4_amax_amd" / "csrc"), str(ROOT / "tests" / "matvec_plan.cpp"), "-o", str(lib)],
                   check=True, capture_output=True)
    L = ctypes.CDLL(str(lib))

    def run(nv, bf16, ids, pairs, N, K, experts=1, cus=CUS):
        sizes = (ctypes.c_int64 * 8)(nv, bf16, ids, pairs, N, K, experts, cus)
        out = (ctypes.c_int64 * len(FIELDS))()
        L.plan(sizes, out)
        return SimpleNamespace(**dict(zip(FIELDS, out)))
    return run


def check(p, nv, bf16, ids, pairs, N, K, experts, cus=CUS):
    rows, per = 4 * p.rg, (p.waves >> p.part_shift) * p.rounds
    assert (p.rg, p.waves) in {(1, 4), (1, 8), (1, 16), (2, 8), (2, 16), (4, 16)} and (bf16 or p.rg < 4)
    assert p.tiles == -(-N // 16) and p.units == -(-K // 512)
    # the tiles: all of them, and no workgroup without one
    assert p.rounds >= 1 and p.grid_x >= 1 and p.grid_x * per >= p.tiles and (p.grid_x - 1) * per < p.tiles
    # the rows: as many slots as any way of the pairs over the experts needs
    if ids:
        met = min(pairs, experts)
        worst = met + (pairs - met) // rows  # one pair of each expert, the others full slots
        assert worst <= p.slots <= pairs
    else:
        assert p.slots == -(-pairs // rows)
    # the GPU: work items along x, workgroups along y, LDS (4 KB for what is not x)
    assert p.grid_x * 64 * p.waves < 1 << 32 and p.slots <= 65535
    assert 0 <= p.lds <= 160 * 1024 * p.waves // 16 - 1024
    # x: all of it, or turns of all waves of a tile
    assert p.seg_units == p.units or (p.seg_units > 0 and p.seg_units % (1 << p.part_shift) == 0)
    assert (1 << p.part_shift) <= p.waves and (p.part_shift == 0 or p.rounds == 1)
    if p.at_once:
        assert bf16 and p.rounds == 1 and 0 < p.units <= (2 if nv else 3) << p.part_shift
    # several rounds only from more workgroups than twice what fits at once, and no more than it takes
    most = 2 * (16 // p.waves) * cus
    if p.rounds > 1:
        assert p.seg_units == p.units
        fewer = (p.waves >> p.part_shift) * (p.rounds - 1)
        assert -(-p.tiles // fewer) * p.slots > most
        assert p.grid_x == 1 or p.grid_x * p.slots <= most


SIZES_N = [1, 16, 17, 300, 1536, 4096, 7168, 28672, 1 << 20, (1 << 26) - 64]
SIZES_K = [0, 32, 512, 544, 1024, 2048, 2880, 4096, 7168, 16384, 1 << 20, (1 << 24) - 512]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("nv", [True, False])
def test_one_matrix(plan, nv, bf16):
    top = LIMIT[bf16]
    rows = [1, 2, 4, 5, 8, 9, 16, 17, 70, 1000, 4096, 4097, 4112, 8192, 8193, 8200, 8208, 16384, 20000, 1 << 18, top - 1, top]
    for pairs, N, K in itertools.product(rows, SIZES_N, SIZES_K):
        check(plan(nv, bf16, False, pairs, N, K), nv, bf16, False, pairs, N, K, 1)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("nv", [True, False])
def test_by_experts(plan, nv, bf16):
    pairs_ = [1, 4, 63, 64, 65, 128, 500, 1024, 1040, 2048, 2064, 3088, 3856, 4095, 4096]
    experts_ = [1, 2, 8, 31, 32, 128, 160, 256, 384, 512, 1024, 2048, 4095, 4096]
    for pairs, experts, N, K in itertools.product(pairs_, experts_, SIZES_N, SIZES_K):
        check(plan(nv, bf16, True, pairs, N, K, experts), nv, bf16, True, pairs, N, K, experts)


@pytest.mark.parametrize("cus", [1, 32, 64, 304])
def test_other_numbers_of_compute_units(plan, cus):
    for nv, bf16, pairs, N, K in itertools.product([0, 1], [0, 1], [1, 9, 4096], [16, 300, 1 << 20], [0, 512, 4096, 1 << 20]):
        for ids, experts in ((False, 1), (True, 64), (True, 4096)):
            check(plan(nv, bf16, ids, pairs, N, K, experts, cus), nv, bf16, ids, pairs, N, K, experts, cus)


@pytest.mark.parametrize("bf16,N,K,experts,pairs", [
    (True, 4096, 7168, 384, 1040), (True, 7168, 2048, 384, 3088), (False, 4096, 2048, 256, 2064),
    (False, 1536, 2048, 128, 3088), (False, 5760, 2880, 32, 3856), (True, 4096, 4096, 0, 8208),
    (False, 4096, 2880, 0, 4112)])
def test_more_slots_than_workgroups_at_once(plan, bf16, N, K, experts, pairs):
    """One workgroup then has all tiles of its slot."""
    for nv in (False, True):
        p = plan(nv, bf16, experts > 0, pairs, N, K, max(experts, 1))
        check(p, nv, bf16, experts > 0, pairs, N, K, max(experts, 1))
        assert p.slots > 2 * (16 // p.waves) * CUS and p.grid_x == 1 and p.rounds == -(-p.tiles // p.waves)
