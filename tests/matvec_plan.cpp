// The plan of a product of a few rows, for tests/test_matvec_plan.py.
#include "matvec_plan.h"

extern "C" void plan(const int64_t* in, int64_t* out) {
  const fp4impl::MatvecSizes m{in[0] != 0, in[1] != 0, in[2] != 0, in[3], in[4], in[5], (int)in[6], (int)in[7]};
  const fp4impl::MatvecPlan p = fp4impl::plan_matvec(m);
  const int64_t o[] = {p.rg, p.waves, p.units, p.part_shift, p.seg_units, p.rounds, p.at_once, p.tiles, p.grid_x, p.slots, p.lds};
  for (int i = 0; i < 11; i++) out[i] = o[i];
}
