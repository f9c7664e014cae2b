// matvec_plan.h -- how a product of a few rows is cut into workgroups, waves
// and rounds, from sizes alone. Plain C++ without HIP: any size up to the limits
// can be planned, and checked, on a machine without a GPU.
#pragma once

#include <stdint.h>

namespace fp4impl {

constexpr int kMatvecUnit = 512;  // K of a wave's unit: four pieces of 128, 256 bytes of each row's codes

// What a form (NVFP4 or not, bf16 or fp32 rows, 4 rg rows of x a pass) needs.
// Operand rows of x in LDS: one for each of its rows, for each of three terms of fp32.
constexpr int matvec_op_rows(bool xbf, int rg) { return (xbf ? 1 : 3) * 4 * rg; }
// Scales on the sums instead of the weights (matvec.hip, Product).
constexpr bool matvec_diagonal(bool nv, bool xbf, int rg) { return nv && xbf && rg <= 2; }
// Units of bf16 calls that a wave loads before its first product, if it has no
// more (fp32 rows need the registers for themselves).
constexpr int matvec_at_once(bool nv) { return nv ? 2 : 3; }
// Bytes of LDS for seg_units units of x, and zeros where an operand needs them.
constexpr int kMatvecZeros = kMatvecUnit * 2;
constexpr int matvec_x_bytes(bool nv, bool xbf, int rg, int seg_units) {
  return matvec_op_rows(xbf, rg) * (seg_units * (kMatvecUnit * 2) + 16) + (matvec_diagonal(nv, xbf, rg) ? kMatvecZeros : 0);
}
// Bytes of LDS in which `waves` waves add up their sums.
constexpr int matvec_red_bytes(int rg, int waves) { return waves * rg * 256; }

struct MatvecSizes {
  bool nvfp4, x_bf16, ids;  // ids: each row has its own expert
  int64_t pairs, N, K;      // all at least 1, K also 0
  int experts, cus;         // cus: compute units of the GPU
};

struct MatvecPlan {
  int rg, waves;   // rows of x a pass, in fours; waves of a workgroup
  int units;       // of K
  int part_shift;  // 2^part_shift waves share a tile of 16 rows of W
  int seg_units;   // units of x in LDS at once
  int rounds;      // tiles of W a wave takes one after another
  bool at_once;    // a wave's weights are all loaded before the first product
  int tiles;       // of W
  int64_t grid_x;  // workgroups along the tiles
  int64_t slots;   // and along the rows of x: passes of 4 rg pairs
  int lds;         // bytes a workgroup
};

constexpr int kMatvecLds = 160 * 1024, kMatvecLdsApart = 4 * 1024;  // of a CU; kept for what is not x

// The plan for workgroups of W waves and passes of 4 rg rows.
inline MatvecPlan plan_matvec_waves(const MatvecSizes& m, int rg, int W, int64_t slots) {
  MatvecPlan p{};
  p.rg = rg;
  p.waves = W;
  p.units = (int)((m.K + kMatvecUnit - 1) / kMatvecUnit);
  p.tiles = (int)((m.N + 15) / 16);
  p.slots = slots;
  const int red = matvec_red_bytes(rg, W), all = 16 / W;  // (workgroups a CU)
  const int room = (kMatvecLds / all - kMatvecLdsApart / (W < 8 ? 2 : 1) - red) /
                   (matvec_op_rows(m.x_bf16, rg) * kMatvecUnit * 2);
  auto units_of = [&](int shift) { return (p.units + (1 << shift) - 1) >> shift; };  // a wave's
  auto at_once = [&](int shift) { return m.x_bf16 && units_of(shift) <= matvec_at_once(m.nvfp4); };
  // Waves for a tile: as many as leave the workgroups room on the GPU at once
  // (one a tile: 1 x 4096x4096 13.6 us for 5.4, 16 x 8192x8192 48 for 15; as
  // many as W has: 8 x 4 of 32 experts 54.6 for 42), or twice that where a wave
  // then has all its weights on the way at once (1 x 28672x4096 14.3 us for
  // 16.9). No more than x in LDS has units for.
  for (; (2 << p.part_shift) <= (W < room ? W : room) && (1 << p.part_shift) < p.units; p.part_shift++) {
    const int64_t blocks = (p.tiles * slots * (2 << p.part_shift) + W - 1) / W;
    const bool more = at_once(p.part_shift + 1) && !at_once(p.part_shift);
    if (blocks > (int64_t)(more ? 2 : 1) * all * m.cus) break;
  }
  // (all of x, or else whole turns of the waves)
  p.seg_units = p.units < room ? p.units : room >> p.part_shift << p.part_shift;
  // Tiles one after another, once there are more workgroups than twice what
  // fits at once: each would bring x anew (32 x 4 of 32 experts 5760x2880 MXFP4
  // 60 us, else 63; fp32 rows of 2880x2880 51, else 54; 8 x 4 NVFP4 42 and 39).
  // As few as leave no more workgroups than that, or all tiles to one workgroup
  // where the slots alone are more.
  // Not where x does not fit: every tile would bring all of it again.
  p.rounds = 1;
  if (p.part_shift == 0 && p.seg_units == p.units) {
    const int64_t most = 2 * (int64_t)all * m.cus / slots, along_x = W * (most > 1 ? most : 1);
    p.rounds = (int)((p.tiles + along_x - 1) / along_x);
  }
  const int per = (W >> p.part_shift) * p.rounds;  // tiles a workgroup
  p.grid_x = (p.tiles + (int64_t)per - 1) / per;
  // (1 x 4096x4096 5.4 us for 6.0, 4 x 1024x4096 5.6 for 6.4, 32 x 4096x4096 8.1 for 9.4)
  p.at_once = at_once(p.part_shift) && p.rounds == 1 && p.units > 0 &&
              (p.units <= p.seg_units || (p.seg_units & ((1 << p.part_shift) - 1)) == 0);
  p.lds = matvec_x_bytes(m.nvfp4, m.x_bf16, rg, p.seg_units) + (p.part_shift > 0 ? red : 0);
  if (m.ids && p.lds < 2 * m.experts + 2) p.lds = 2 * m.experts + 2;  // (16 bits an expert, before x comes)
  return p;
}

// Waves of a workgroup: 16 share one copy of x, but wait for all of it and for
// each other. Eight where two such workgroups have room on a CU with all of x
// (1 x 4096x4096 5.4 us, 16 waves 6.9; 32 x 4 of 32 experts 5760x2880 60 and 99).
// Four where that leaves room too and there are tiles for half the GPU's eight
// waves a CU (1 x 4 of 32 experts 5760x2880 9.5 us, 8 waves 11.6; 2 x 8 of 128
// experts 1536x4096 14.0 and 15.8).
inline MatvecPlan plan_matvec_rows(const MatvecSizes& m, int rg, int64_t slots) {
  const int units = (int)((m.K + kMatvecUnit - 1) / kMatvecUnit), x = matvec_x_bytes(m.nvfp4, m.x_bf16, rg, units);
  const int64_t tiles = (m.N + 15) / 16;
  if (rg == 1 && tiles * slots * 2 >= 8 * (int64_t)m.cus &&
      x + matvec_red_bytes(rg, 4) <= kMatvecLds / 4 - kMatvecLdsApart / 2)
    return plan_matvec_waves(m, rg, 4, slots);
  if (rg < 4 && x + matvec_red_bytes(rg, 8) <= kMatvecLds / 2 - kMatvecLdsApart) return plan_matvec_waves(m, rg, 8, slots);
  return plan_matvec_waves(m, rg, 16, slots);
}

inline MatvecPlan plan_matvec(const MatvecSizes& m) {
  // experts that may have pairs, and how many slots of `rows` pairs there are at most
  const int64_t met = m.ids ? (m.pairs < m.experts ? m.pairs : m.experts) : 1;
  auto slots = [&](int rows) {
    if (!m.ids) return (m.pairs + rows - 1) / rows;
    return met + m.pairs / rows < m.pairs ? met + m.pairs / rows : m.pairs;
  };
  // Rows a pass, by how many an expert has on average (some have twice that):
  // 4 cost least where they suffice (16 rows four at a time: the weights four
  // times); of 32 experts with 4 pairs each, slots of 8 take 60 us and of 4 77,
  // with fp32 rows 51 and 57. 16 x 5760x2880 as 16 rows 9.1 us, 8 and 8 11.0;
  // 32 x 4096x4096 8.1 and 10.1. fp32 rows come no more than 8 at a time: 16
  // are 48 operand rows, and LDS then holds 1024 of K (16 x 4096x4096 27 us for
  // 13, 12 x 8192x8192 59 for 28).
  if (m.pairs <= (m.ids ? 2 : 4) * met) return plan_matvec_rows(m, 1, slots(4));
  if (m.x_bf16 && m.pairs > 8 * met) return plan_matvec_rows(m, 4, slots(16));
  return plan_matvec_rows(m, 2, slots(8));
}

}  // namespace fp4impl
