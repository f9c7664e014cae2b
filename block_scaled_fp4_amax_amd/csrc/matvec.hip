// matvec.hip -- products of a few rows in 16 or 32 bits with 4-bit weights:
//   y[p, n] = sum_k deq(W_e)[n, k] x[p / repeat, k], e = ids[p] (or 0),
// accumulated in fp32. Activations are not rounded: bf16 ones are operands as
// they are, fp32 ones three bf16 terms. Weights times their block's scale are
// exact in bf16, so the matrix cores add exact products.
//
// A wave takes tiles of 16 rows of W and reads their bytes straight into
// registers, 16 a lane, once for up to 16 rows of x (8 of fp32); the rows of x
// lie in LDS for the whole workgroup. Where tiles are few, several waves share
// one along K and their sums are added up in LDS, always in one order.
//
// What bounds it (MI355X; bytes at the 5.08 TB/s of a large copy):
//   1 x 4096x4096 NVFP4, bf16        5.4 us  floor 1.9: launch, x to LDS, one trip to memory
//   1 x 28672x4096 NVFP4, bf16      14.2 us        13.0: memory
//   16 x 8192x8192 MXFP4, bf16      15.6 us         7.1: x to LDS (256 KB in two parts), then weights
//   16 x 4096x4096 NVFP4, fp32      15.1 us         2.0: each workgroup (128 in all) brings x,
//     in two parts, and cuts it into terms; the weights are read for each pass of 8 rows
//   12 x 8192x8192 NVFP4, fp32      27.0 us         7.6: the same, in four parts; vector
//     instructions 62 % of the cycles
//   1 x 4 of 32 experts 5760x2880    9.7 us         6.9: memory and one trip to it
//   8 x 4 of 32 experts 5760x2880   43   us        38.7: memory
//   32 x 4 of 32 experts 2880x2880, fp32 rows, NVFP4  51 us  29.6: vector instructions 59 % of
//     the cycles (every weight scaled and rounded), matrix ones 20 %; experts of over 8 pairs read again
#include "fp4_device.h"
#include "launch.h"
#include "matvec_plan.h"

namespace fp4impl {
using namespace fp4dev;

namespace {

constexpr int kUnit = kMatvecUnit;

// What the kernels take: sizes in 32 bits, and what only sizes decide.
struct Call {
  const void* x;
  const uint8_t *codes, *scales;
  const float* ts;
  const int32_t* ids;
  void* y;
  int64_t ld_x, c_es, s_es, ld_y;  // elements, bytes, bytes, elements
  uint32_t ld_c, ld_s;
  int pairs, repeat, N, K, experts;
  int units;                        // of K
  uint32_t last_code, last_scale;   // where a row's last 16 bytes start
  int y_bf16;
  int part_shift, seg_units, at_once, rounds;  // as in MatvecPlan
};

// NVFP4's tensor scale in two: a power of two that multiplies the codes, as the
// scale operand of their conversion, and the rest, which multiplies the sums.
// The power is below the scale, so that no sum is larger than the terms it
// stands for (without, it holds up to 2688 / max |W| times as much), and at most
// 2^-7, so that a block's sum without its scale (16 codes of 6) stays finite
// for every finite x. For scales below 2^-39 it is 2^-40, which no sum of 2^24
// weights of 2688 overflows either, and small products keep their bits.
struct TensorScale {
  float unit;
  float rest, wide;  // (wide: 2^7 where `rest` times that could overflow)
  __device__ __forceinline__ TensorScale(float ts) {
    const int e = (int)((__builtin_bit_cast(uint32_t, ts) >> 23) & 255u) - 128;  // 2^e is up to half of |ts|
    const int p = e < -40 ? -40 : e > -7 ? -7 : e;
    unit = power(p);
    rest = e > -7 ? ts : ts * power(-p);
    wide = e > -7 ? power(-p) : 1.0f;
  }
  static __device__ __forceinline__ float power(int p) { return __builtin_bit_cast(float, (uint32_t)(p + 127) << 23); }
};

// The eight values of a word of codes, times their block's scale: exact in
// bf16 (E2M1 has 2 significant bits, E4M3 4). unit: of NVFP4, above.
template <bool NV>
__device__ __forceinline__ bf16x8 weights8(uint32_t w, float scale, float unit) {
  uint32_t o[4];
  if constexpr (!NV) {
    o[0] = e2m1_unpack2_bf16<0>(w, scale);
    o[1] = e2m1_unpack2_bf16<1>(w, scale);
    o[2] = e2m1_unpack2_bf16<2>(w, scale);
    o[3] = e2m1_unpack2_bf16<3>(w, scale);
  } else {
    const f32x2 v[4] = {e2m1_unpack2<0>(w, unit), e2m1_unpack2<1>(w, unit), e2m1_unpack2<2>(w, unit),
                        e2m1_unpack2<3>(w, unit)};
#pragma unroll
    for (int i = 0; i < 4; i++)
      o[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(v[i].x * scale), (__bf16)(v[i].y * scale)});
  }
  return __builtin_bit_cast(bf16x8, u32x4{o[0], o[1], o[2], o[3]});
}

// Eight fp32 numbers as three bf16 terms that hold all their bits from 2^-148
// on: each the leading 8 bits of what is left, cut off, so that nothing
// overflows, and what is left times a power of two (kLeft: 2^7 and 2^8, 2^15 in
// all), no larger than the number itself. Without it, terms of numbers below
// 2^-110 would lie under bf16's smallest number.
constexpr float kLeft[2] = {0x1p7f, 0x1p8f};
__device__ __forceinline__ void split3(const u32x4 lo, const u32x4 hi, u32x4 (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    uint32_t part[3][2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int e = 2 * i + h;
      const uint32_t b0 = e < 4 ? lo[e] : hi[e - 4];
      const float v = __builtin_bit_cast(float, b0);
      // (an infinity is its first term alone; a NaN whose first term is an
      // infinity, since only its low bits say so, is one in the second)
      const float r1 = __builtin_fabsf(v) != __builtin_inff() ? (v - __builtin_bit_cast(float, b0 & 0xffff0000u)) * kLeft[0] : 0.0f;
      const uint32_t b1 = __builtin_bit_cast(uint32_t, r1);
      const float r2 = (r1 - __builtin_bit_cast(float, b1 & 0xffff0000u)) * kLeft[1];
      part[0][h] = b0;
      part[1][h] = b1;
      part[2][h] = __builtin_bit_cast(uint32_t, r2);
    }
#pragma unroll
    for (int q = 0; q < 3; q++) t[q][i] = (part[q][0] >> 16) | (part[q][1] & 0xffff0000u);
  }
}

__device__ __forceinline__ f32x4 mfma(u32x4 x, bf16x8 w, f32x4 acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), w, acc, 0, 0, 0);
}

// Where a tile of 16 rows of W lies: bases of the first (the same for all
// lanes), and the lane's row, lane % 16, from there.
struct Place {
  const uint8_t *codes, *scales;
  uint32_t code_row, scale_row;
  __device__ __forceinline__ Place(const Call& a, int expert, int n0) {
    const int c16 = threadIdx.x & 15;
    n0 = n0 < a.N ? n0 : a.N - 1;
    codes = a.codes + expert * a.c_es + (int64_t)n0 * a.ld_c;
    scales = a.scales + expert * a.s_es + (int64_t)n0 * a.ld_s;
    const int rows = a.N - 1 - n0;
    const uint32_t row = c16 < rows ? c16 : rows;
    code_row = row * a.ld_c;
    scale_row = row * a.ld_s;
  }
};

// One unit of a tile in a wave's registers: a lane has 32 consecutive values of
// row lane % 16 in each of four pieces of 128 (blocks lie within lanes, and its
// four words are operands of four v_mfma_f32_16x16x32_bf16, whose k are then
// 32 g + 8 j, g = lane / 16, j the word), and the row's scales of all four.
template <bool NV>
struct Weights {
  u32x4 w[4], s[NV ? 2 : 1];
  // (past the end: the row's last bytes, for which scale() gives zeros)
  __device__ __forceinline__ void load(const Call& a, const Place& p, int k0, int g) {
    const uint32_t last_code = a.last_code, last_scale = a.last_scale;
    const uint32_t at = (uint32_t)k0 / 2 + g * 16, sat = (uint32_t)k0 / (NV ? 16 : 32);
#pragma unroll
    for (int i = 0; i < (NV ? 2 : 1); i++) {
      const uint32_t o = sat + i * 16 < last_scale ? sat + i * 16 : last_scale;
      s[i] = *reinterpret_cast<const u32x4*>(p.scales + (p.scale_row + o));
    }
#pragma unroll
    for (int u = 0; u < 4; u++) {
      const uint32_t o = at + u * 64 < last_code ? at + u * 64 : last_code;
      w[u] = *reinterpret_cast<const u32x4*>(p.codes + (p.code_row + o));
    }
  }
  // The scales of the lane's first and second 16 values of piece u, which
  // starts at k.
  __device__ __forceinline__ f32x2 scale(int u, int k, int K, int g) const {
    const bool first = k + g * 32 < K, second = k + g * 32 + 16 < K;
    if constexpr (NV) {
      const uint32_t pair = (g & 2 ? s[u >> 1][(2 * u + 1) & 3] : s[u >> 1][(2 * u) & 3]) >> (16 * (g & 1));
      const f32x2 f = __builtin_amdgcn_cvt_pk_f32_fp8(pair, false);
      return f32x2{first ? f.x : 0.0f, second ? f.y : 0.0f};
    } else {
      const float f = e8m0_scale_operand(first ? (s[0][u] >> (8 * g)) & 0xffu : 0u);
      return f32x2{f, f};
    }
  }
};

// The words from here on are not known to be the ones loaded: their conversion
// stays behind this point (else it is moved ahead for a whole unit, before the
// next unit's loads are issued, and takes 64 registers).
__device__ __forceinline__ u32x4 pinned(u32x4 v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ u32x4 at16(const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// ---------------------------------------------------------------------------
// 4 RG rows of x, which the workgroup shares in LDS
// ---------------------------------------------------------------------------
// x lies in LDS as bf16 operand rows, one for each activation row and term,
// each 16 bytes longer than its values so that the rows' reads meet different
// banks. Terms of fp32 are rows like others: one matrix instruction multiplies
// all three, and their sums are added at the end. Behind the rows: zeros, as
// many as a unit of a row has bytes.
constexpr int kZeros = kMatvecZeros;
template <bool XBF, int RG>
constexpr int kOpRows = matvec_op_rows(XBF, RG);

// fp32 rows on their way to LDS: a lane's eight numbers at k of two rows, of
// which `live` are there (what the others hold meets only results that nobody
// reads), cut into three terms.
constexpr int kStageRows = 2;  // (12 x 8192x8192 NVFP4: 27.9 us; 1 row 28.3, 4 rows 32.9 with registers spilt)
struct StageX {
  u32x4 v[kStageRows][2];
  __device__ __forceinline__ void load(const Call& a, const int64_t (&xo)[kStageRows], int live, int k) {
#pragma unroll
    for (int r = 0; r < kStageRows; r++) {
      if (r < live) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(a.x) + (xo[r] + (k < a.K ? k : 0)) * 4;
        v[r][0] = at16(src);
        v[r][1] = at16(src + 16);
      }
    }
  }
  // to: row 0's place; plane: bytes from one term's rows to the next's
  __device__ __forceinline__ void put(const Call& a, int live, int k, uint8_t* to, int pitch, int plane) {
#pragma unroll
    for (int r = 0; r < kStageRows; r++) {
      if (r < live) {
        if (k >= a.K) v[r][0] = v[r][1] = u32x4{0, 0, 0, 0};
        u32x4 t[3];
        split3(v[r][0], v[r][1], t);
#pragma unroll
        for (int q = 0; q < 3; q++) *reinterpret_cast<u32x4*>(to + q * plane + r * pitch) = t[q];
      }
    }
  }
};

// bf16 rows need no work on their way to LDS and are copied there directly: a
// wave copies units of the rows, 1 KB each, lane i the 16 bytes 16 i of it. (No
// lane waits, and no register is taken.) Past K: zeros.
template <int W>
__device__ __forceinline__ void copy_x(const Call& a, int64_t xo, int row, int u0, int here, int wave, uint8_t* lds,
                                       int pitch) {
  const int lane = threadIdx.x & 63;
  for (int u = (wave - row) & (W - 1); u < here; u += W) {
    const int k = (u0 + u) * kUnit + lane * 8;
    uint8_t* to = lds + row * pitch + u * (kUnit * 2);
    if (k < a.K) {
      const uint8_t* from = reinterpret_cast<const uint8_t*>(a.x) + (xo + k) * 2;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint8_t*)from,
                                       (__attribute__((address_space(3))) uint8_t*)to, 16, 0, 0);
    } else {
      *reinterpret_cast<u32x4*>(to + lane * 16) = u32x4{0, 0, 0, 0};
    }
  }
}

// 4 RG rows of x, in LDS, times a wave's tile of 16 rows of W.
//
// NVFP4 with bf16 rows: instead of scaling every weight, an operand of x
// holds four rows in operand rows 4 g to 4 g + 3 of lane group g only, zeros in
// its other rows. Rows 4 g + r of the product, which is what lane group g
// receives, are then x[r] times this group's own 32 values: a lane has its own
// partial sums, and its block's scale multiplies four of them instead of
// sixteen weights.
// (With 16 rows that would take four such products, and scaling the weights
// costs no more.)
template <bool NV, bool XBF, int RG>
constexpr bool diagonal = matvec_diagonal(NV, XBF, RG);

template <bool NV, bool XBF, int RG>
struct Product {
  static_assert(XBF || RG <= 2);
  static constexpr bool DIAG = diagonal<NV, XBF, RG>;
  static constexpr int ROWS = kOpRows<XBF, RG>, OT = DIAG ? RG : (ROWS + 15) / 16;
  int from[OT], step[OT];  // of the lane's operands: where those of a segment's first unit lie, and from unit to unit
  f32x4 acc[OT];

  __device__ __forceinline__ Product(int pitch) {
    const int lane = threadIdx.x & 63, c16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int o = 0; o < OT; o++) {
      const int row = DIAG ? o * 4 + (c16 & 3) : (o * 16 + c16) % ROWS;
      const bool there = !DIAG || (c16 >> 2) == g;
      from[o] = there ? row * pitch + g * 64 : ROWS * pitch;
      step[o] = there ? kUnit * 2 : 0;
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int o = 0; o < OT; o++) acc[o] = f32x4{0, 0, 0, 0};
  }
  // One unit, which starts at k0 and is unit `at` of x in LDS.
  __device__ __forceinline__ void multiply(const Weights<NV>& o, int k0, int K, int at, const uint8_t* lds, float unit) {
    const int g = (threadIdx.x & 63) >> 4;
    const uint8_t* x[OT];
#pragma unroll
    for (int i = 0; i < OT; i++) x[i] = lds + (from[i] + at * step[i]);
#pragma unroll
    for (int u = 0; u < 4; u++) {
      __builtin_amdgcn_sched_barrier(0);  // (else the operands of all four pieces are read at once)
      const u32x4 codes = pinned(o.w[u]);
      const f32x2 sc = o.scale(u, k0 + u * 128, K, g);
      if constexpr (DIAG) {
        bf16x8 w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] = weights8<false>(codes[j], unit, 1.0f);
#pragma unroll
        for (int i = 0; i < OT; i++) {
          f32x4 d0 = {0, 0, 0, 0}, d1 = {0, 0, 0, 0};
          d0 = mfma(at16(x[i] + u * 256), w[0], d0);
          d1 = mfma(at16(x[i] + u * 256 + 32), w[2], d1);
          d0 = mfma(at16(x[i] + u * 256 + 16), w[1], d0);
          d1 = mfma(at16(x[i] + u * 256 + 48), w[3], d1);
#pragma unroll
          for (int r = 0; r < 4; r++) acc[i][r] = __builtin_fmaf(sc.y, d1[r], __builtin_fmaf(sc.x, d0[r], acc[i][r]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const bf16x8 w = weights8<NV>(codes[j], j < 2 ? sc.x : sc.y, unit);
#pragma unroll
          for (int i = 0; i < OT; i++) acc[i] = mfma(at16(x[i] + u * 256 + j * 16), w, acc[i]);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // In lanes of group g < RG: rows 4 g to 4 g + 3 of column lane % 16.
  __device__ __forceinline__ f32x4 result() {
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (DIAG) {
#pragma unroll
      for (int o = 0; o < OT; o++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          float v = acc[o][r];
          v += xor_shfl<16>(v);
          v += xor_shfl<32>(v);
          acc[o][r] = v;
        }
      if constexpr (RG == 2) acc[0] = g == 1 ? acc[1] : acc[0];
    } else if constexpr (!XBF) {
      // operand row term * 4 RG + m: group o * 4 + g is term (o * 4 + g) / RG
      constexpr float second = 1.0f / kLeft[0], third = second / kLeft[1];
#pragma unroll
      for (int r = 0; r < 4; r++) {
        float v = acc[0][r];
        if constexpr (RG == 1) {
          v = g == 0 ? v : g == 1 ? v * second : g == 2 ? v * third : 0.0f;
          v += xor_shfl<16>(v);
        } else {
          v = g < 2 ? v + acc[1][r] * third : v * second;
        }
        v += xor_shfl<32>(v);
        acc[0][r] = v;
      }
    }
    return acc[0];
  }
};

// ---------------------------------------------------------------------------
// the pairs of one expert
// ---------------------------------------------------------------------------
// What one workgroup does: `count` of an expert's pairs, in order, whose
// numbers are in its list. expert = -1: there are not so many slots.
struct Found {
  int expert, count;
};

// The pairs are cut into slots: of each expert that has any, as many as its
// pairs need at `rows` a slot. This finds the blockIdx.y-th of them. counts:
// LDS for 16 bits an expert (from 65 pairs on), list: for `rows` numbers.
__device__ __forceinline__ void find_slot(const Call& a, int rows, Found* s, uint32_t* counts, uint16_t* list) {
  const int lane = threadIdx.x & 63;
  if (a.pairs <= 64) {
    // one load, and an expert's lanes are found by comparison, experts in order of appearance
    if (threadIdx.x < 64) {
      const int id = lane < a.pairs ? a.ids[lane] : -1;
      uint64_t left = __builtin_amdgcn_ballot_w64((unsigned)id < (unsigned)a.experts), same = 0;
      int slot = blockIdx.y, expert = -1, count = 0;
      while (left != 0) {
        expert = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        same = __builtin_amdgcn_ballot_w64(id == expert);
        count = __builtin_popcountll(same) - slot * rows;
        if (count > 0) break;
        slot -= (__builtin_popcountll(same) + rows - 1) / rows;
        left &= ~same;
        expert = -1;
      }
      const int at = __builtin_popcountll(same & ((1ull << lane) - 1)) - slot * rows;
      if (expert >= 0 && id == expert && at >= 0 && at < rows) list[at] = lane;
      if (lane == 0) *s = Found{expert, count < rows ? count : rows};
    }
    __syncthreads();
    return;
  }
  for (int i = threadIdx.x; i < (a.experts + 1) / 2; i += blockDim.x) counts[i] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) {
    const int e = a.ids[p];
    if ((unsigned)e < (unsigned)a.experts) atomicAdd(&counts[e >> 1], e & 1 ? 1u << 16 : 1u);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    // the lane whose experts hold the slot, then the expert
    auto pairs_of = [&](int e) { return (int)((counts[e >> 1] >> (e & 1 ? 16 : 0)) & 0xffffu); };
    const int per = (a.experts + 63) / 64, first = lane * per, end = first + per < a.experts ? first + per : a.experts;
    int own = 0;
    for (int e = first; e < end; e++) own += (pairs_of(e) + rows - 1) / rows;
    int sum = own;
    for (int step = 1; step < 64; step <<= 1) {
      const int o = __shfl_up(sum, step, 64);
      sum += lane >= step ? o : 0;
    }
    int expert = -1, count = 0, slot = (int)blockIdx.y - (sum - own);
    if (slot >= 0 && slot < own) {
      for (int e = first; e < end; e++) {
        count = pairs_of(e);
        expert = e;
        const int n = (count + rows - 1) / rows;
        if (slot < n) break;
        slot -= n;
      }
    }
    const uint64_t has = __builtin_amdgcn_ballot_w64(expert >= 0);
    if (has != 0) {
      const int src = __builtin_ctzll(has);
      expert = __builtin_amdgcn_readlane(expert, src);
      count = __builtin_amdgcn_readlane(count, src);
      slot = __builtin_amdgcn_readlane(slot, src);
      int at = -slot * rows;
      for (int p0 = 0; p0 < a.pairs && at < rows; p0 += 64) {
        const bool mine = p0 + lane < a.pairs && a.ids[p0 + lane] == expert;
        const uint64_t m = __builtin_amdgcn_ballot_w64(mine);
        const int i = at + __builtin_popcountll(m & ((1ull << lane) - 1));
        if (mine && i >= 0 && i < rows) list[i] = p0 + lane;
        at += __builtin_popcountll(m);
      }
      count -= slot * rows;
    }
    if (lane == 0) *s = Found{expert, count < rows ? count : rows};
  }
  __syncthreads();
}

__device__ __forceinline__ void store_y(const Call& a, int p, int n, float v) {
  if (a.y_bf16) reinterpret_cast<__bf16*>(a.y)[p * a.ld_y + n] = (__bf16)v;
  else reinterpret_cast<float*>(a.y)[p * a.ld_y + n] = v;
}

// Rows of zeros for pairs without an expert, columns n0 to n0 + cols - 1.
__device__ __forceinline__ void zero_rows(const Call& a, int n0, int cols) {
  for (int p = threadIdx.x / 16; p < a.pairs; p += blockDim.x / 16) {
    if ((unsigned)a.ids[p] < (unsigned)a.experts) continue;
    for (int n = n0 + (threadIdx.x & 15); n < n0 + cols && n < a.N; n += 16) store_y(a, p, n, 0.0f);
  }
}

__device__ __forceinline__ int64_t x_offset(const Call& a, int pair) {
  const int row = a.repeat == 1 ? pair : (int)((unsigned)pair / (unsigned)a.repeat);
  return row * a.ld_x;
}

// Up to 4 RG pairs of one expert (its list, or else pairs `first` on) against
// the workgroup's tiles of W: `rounds` times W >> part_shift, one after another,
// each wave with the next unit's weights on their way while it multiplies, over
// the ends of tiles too.
template <bool NV, bool XBF, int RG, int W, bool LIST>
__device__ __forceinline__ void tiles_of(const Call& a, int expert, const uint16_t* list, int first, int live,
                                          uint8_t* lds) {
  constexpr int MR = 4 * RG, ROWS = kOpRows<XBF, RG>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  const int per = W >> a.part_shift, parts = 1 << a.part_shift, part = wave & (parts - 1);
  const int units = a.units, pitch = a.seg_units * (kUnit * 2) + 16;
  float* red = reinterpret_cast<float*>(lds + matvec_x_bytes(NV, XBF, RG, a.seg_units));  // [W][MR][16], if parts > 1
  int n0 = (blockIdx.x * a.rounds * per + (wave >> a.part_shift)) * 16;
  auto offset_of = [&](int row) {
    const int pair = LIST ? (int)list[row] : first + row;
    return x_offset(a, pair);
  };
  // x for a segment: bf16 rows straight to LDS; fp32 as items i of n * GROUPS
  // in registers, octet i % n of rows kStageRows * (i / n) on
  constexpr int GROUPS = MR / kStageRows;
  StageX x;
  int group = 0, oct = 0;
  auto load_x = [&](int i, int n, int k0) {
    group = 0;
    oct = i;
#pragma unroll
    for (int h = 1; h < GROUPS; h++) {
      group += i >= h * n ? 1 : 0;
      oct -= i >= h * n ? n : 0;
    }
    group *= kStageRows;
    int64_t xo[kStageRows];
#pragma unroll
    for (int r = 0; r < kStageRows; r++) xo[r] = offset_of(group + r < live ? group + r : live - 1);
    x.load(a, xo, live - group, k0 + oct * 8);
  };
  auto copy_all = [&](int u0, int here) {
    for (int row = 0; row < live; row++)
      copy_x<W>(a, offset_of(__builtin_amdgcn_readfirstlane(row)), row, u0, here, wave, lds, pitch);
  };
  // (before the weights, so as not to arrive behind them)
  const int in_lds = units < a.seg_units ? units : a.seg_units, n1 = in_lds * 64;
  if constexpr (XBF) copy_all(0, in_lds);
  else if (threadIdx.x < n1 * GROUPS) load_x(threadIdx.x, n1, 0);
  Place at(a, expert, n0);
  Product<NV, XBF, RG> rows(pitch);
  rows.clear();
  // (by a scalar load, which is waited for where `stage` says so: the compiler
  // would load it as a vector and wait for that, and all of x before it, ahead
  // of the weights: 1 x 28672x4096 16.9 us for 15.4)
  float ts = 1.0f, power = 1.0f;
  if constexpr (NV) ts = reinterpret_cast<const __attribute__((address_space(4))) float*>((uintptr_t)a.ts)[expert];
  auto stage = [&](int u0, bool loaded) {
    const int here = units - u0 < a.seg_units ? units - u0 : a.seg_units;
    if (!loaded) __syncthreads();
    if (Product<NV, XBF, RG>::DIAG && threadIdx.x < kZeros / 16)
      *reinterpret_cast<u32x4*>(lds + ROWS * pitch + threadIdx.x * 16) = u32x4{0, 0, 0, 0};
    if constexpr (XBF) {
      if (!loaded) copy_all(u0, here);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (the copies to LDS are counted there)
    } else {
      for (int i = threadIdx.x; i < here * 64 * GROUPS; i += 64 * W) {
        if (!loaded || i >= 64 * W) load_x(i, here * 64, u0 * kUnit);
        x.put(a, live - group, u0 * kUnit + oct * 8, lds + group * pitch + oct * 16, pitch, MR * pitch);
      }
    }
    __syncthreads();
    if (NV && loaded) {
      asm volatile("" : "+s"(ts));
      power = TensorScale(ts).unit;
    }
  };
  // the sums of a tile, over its waves, to y
  auto finish = [&]() {
    f32x4 acc = rows.result();
    if (parts > 1) {  // (one tile a wave)
      if (g < RG) {
#pragma unroll
        for (int r = 0; r < 4; r++) red[(wave * MR + 4 * g + r) * 16 + c16] = acc[r];
      }
      __syncthreads();
      if (part == 0 && g < RG) {
        for (int w = 1; w < parts; w++) {
#pragma unroll
          for (int r = 0; r < 4; r++) acc[r] += red[((wave + w) * MR + 4 * g + r) * 16 + c16];
        }
      }
    }
    const TensorScale scale(ts);
    if (part == 0 && g < RG && n0 + c16 < a.N) {
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int row = 4 * g + r;
        if (row < live) store_y(a, LIST ? list[row] : first + row, n0 + c16, NV ? acc[r] * scale.rest * scale.wide : acc[r]);
      }
    }
  };
  // A wave of few units has all their weights on the way at once.
  if constexpr (XBF) if (a.at_once) {
    constexpr int AT_ONCE = matvec_at_once(NV);
    Weights<NV> w[AT_ONCE];
#pragma unroll
    for (int d = 0; d < AT_ONCE; d++) {
      if (d * parts < units) w[d].load(a, at, (part + d * parts) * kUnit, g);
    }
#pragma unroll
    for (int d = 0; d < AT_ONCE; d++) {
      const int u = d * parts;
      if (u >= units) break;
      const int u0 = u < a.seg_units ? 0 : u / a.seg_units * a.seg_units;
      if (u == u0) stage(u0, d == 0);
      if (u + part < units) rows.multiply(w[d], (u + part) * kUnit, a.K, u + part - u0, lds, power);
    }
    finish();
    return;
  }
  Weights<NV> now;
  if (units > 0) now.load(a, at, part * kUnit, g);
  for (int round = 0; round < a.rounds; round++) {
    const bool last_tile = round + 1 == a.rounds;
    const Place after(a, expert, last_tile ? n0 : n0 + per * 16);
    int unit = part;
    for (int u0 = 0; u0 < units; u0 += a.seg_units) {
      const int here = units - u0 < a.seg_units ? units - u0 : a.seg_units;
      if (round == 0 || units > a.seg_units) stage(u0, round == 0 && u0 == 0);
      for (; unit < u0 + here; unit += parts) {
        Weights<NV> next;
        const bool over = unit + parts >= units;  // (of the last tile: bytes that nobody uses)
        next.load(a, over ? after : at, over && !last_tile ? part * kUnit : (unit + parts) * kUnit, g);
        rows.multiply(now, unit * kUnit, a.K, unit - u0, lds, power);
        now = next;
      }
    }
    finish();
    rows.clear();
    at = after;
    n0 += per * 16;
  }
}

}  // namespace

template <bool NV, bool XBF, int RG, int W>
__global__ __launch_bounds__(64 * W, 4) void matvec_kernel(Call a) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int first = blockIdx.y * (4 * RG), left = a.pairs - first;
  tiles_of<NV, XBF, RG, W, false>(a, 0, nullptr, first, left < 4 * RG ? left : 4 * RG, lds);
}

template <bool NV, bool XBF, int RG, int W>
__global__ __launch_bounds__(64 * W, 4) void matvec_experts_kernel(Call a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ Found found;
  __shared__ uint16_t list[4 * RG];
  const int cols = (W >> a.part_shift) * a.rounds * 16;
  if (blockIdx.y == 0) zero_rows(a, blockIdx.x * cols, cols);
  find_slot(a, 4 * RG, &found, reinterpret_cast<uint32_t*>(lds), list);  // (x comes there later)
  if (found.expert < 0) return;
  tiles_of<NV, XBF, RG, W, true>(a, __builtin_amdgcn_readfirstlane(found.expert), list, 0,
                                  __builtin_amdgcn_readfirstlane(found.count), lds);
}

namespace {

template <bool NV, bool XBF, int RG, int W>
hipError_t launch_form(const Call& c, const MatvecPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)p.grid_x, (unsigned)p.slots), block(64 * W);
  if (c.ids) hipLaunchKernelGGL((matvec_experts_kernel<NV, XBF, RG, W>), grid, block, p.lds, s, c);
  else hipLaunchKernelGGL((matvec_kernel<NV, XBF, RG, W>), grid, block, p.lds, s, c);
  return hipGetLastError();
}

template <bool NV, bool XBF>
hipError_t launch(const MatvecArgs& a, hipStream_t s) {
  const int64_t blk = NV ? 16 : 32;
  auto last16 = [](int64_t bytes) { return (uint32_t)(bytes > 16 ? (bytes + 15) / 16 * 16 - 16 : 0); };
  Call c{};
  c.x = a.x;
  c.codes = a.codes;
  c.scales = a.scales;
  c.ts = a.ts;
  c.ids = a.ids;
  c.y = a.y;
  c.ld_x = a.ld_x;
  c.c_es = a.c_es;
  c.s_es = a.s_es;
  c.ld_y = a.ld_y;
  c.ld_c = (uint32_t)a.ld_c;
  c.ld_s = (uint32_t)a.ld_s;
  c.pairs = (int)a.pairs;
  c.repeat = (int)a.repeat;
  c.N = (int)a.N;
  c.K = (int)a.K;
  c.experts = a.experts;
  c.last_code = last16(a.K / 2);
  c.last_scale = last16(a.K / blk);
  c.y_bf16 = a.y_bf16;
  const MatvecPlan p =
      plan_matvec(MatvecSizes{NV, XBF, a.ids != nullptr, a.pairs, a.N, a.K, a.experts, device_cu_count()});
  c.units = p.units;
  c.part_shift = p.part_shift;
  c.seg_units = p.seg_units;
  c.at_once = p.at_once;
  c.rounds = p.rounds;
  if (p.rg == 1) {
    if (p.waves == 4) return launch_form<NV, XBF, 1, 4>(c, p, s);
    if (p.waves == 8) return launch_form<NV, XBF, 1, 8>(c, p, s);
    return launch_form<NV, XBF, 1, 16>(c, p, s);
  }
  if constexpr (XBF) {
    if (p.rg == 4) return launch_form<NV, XBF, 4, 16>(c, p, s);
  }
  return p.waves == 8 ? launch_form<NV, XBF, 2, 8>(c, p, s) : launch_form<NV, XBF, 2, 16>(c, p, s);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t s) {
  if (a.nvfp4) return a.x_bf16 ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return a.x_bf16 ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace fp4impl
