// kv_attention.hip -- softmax attention over the paged 4-bit key-value cache.
//
//   s = scale (q . k), p = exp(s - max), out = sum(p v) / sum(p)
//
// in one pass over the keys with a running maximum and sum. A workgroup takes
// 16 rows (row = (query, head of the kv head's group)) of one sequence and kv
// head and a chunk of their visible keys; each of its waves takes every n-th
// 32-key tile of the chunk on its own, with no barrier until the waves'
// results are joined through LDS. Long key ranges are cut into chunks
// whose partial results (fp32 sum, maximum, denominator) go to the workspace
// and are joined by a second kernel.
//
// One wave, one tile of 32 keys, on v_mfma_f32_16x16x32 (lane l: c = l % 16,
// g = l / 16):
//   S^T = K Q^T: the A operand's rows are 16 keys, lane (c, g) holding of key
//     c the head's elements g * D/4 .. g * D/4 + D/4 - 1, so one row's codes
//     are read by four lanes, D/8 bytes each, and converted in registers. The
//     result has a query per column: lane (c, g) holds row c's scores of keys
//     4g .. 4g + 3 of both 16-key halves.
//   O^T += V^T P^T: those eight scores are exactly the lane's part of the B
//     operand if the contraction runs over the keys in that order, so the
//     weights never leave their lane. The A operand needs, for one element d
//     per lane, the same eight keys: the lane reads D/32 bytes of each of
//     them (elements c * D/16 ..) and transposes pairs of keys in registers.
// MXFP4 elements times their power-of-two scale are exact in bf16, NVFP4
// elements times their E4M3 scale in fp16; the NVFP4 tensor scales multiply
// the scores and the result. fp16 queries are brought to a common power of
// two per row first, so that no bf16 or fp32 query leaves fp16's range.
// fp32 calls split the queries (3 bf16 or 2 fp16 terms) and the weights (2
// terms) and multiply every term.
// (The block-scaled matrix instruction could take MXFP4 codes as they are,
// against queries split into two E4M3 terms. It was tried and left: it sums
// products of an 8-bit operand in groups of eight with about 16 bits, and
// scores came out up to 2^-16 of sum |q k| off, 300 times fp32's error.)
#include "fp4_device.h"
#include "launch.h"

namespace fp4impl {
using namespace fp4dev;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileKeys = 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum starts below every score that is not -inf; a masked
// score (-inf) then weighs exp2(-inf) = 0 also before the first visible key.
constexpr float kNoMax = -1e30f;
// A row's maximum is only raised when a score passes it by more than 2^8
// (weights may grow to that without harm in fp32), so that most tiles need
// neither the exchange across lanes nor the rescaling.
constexpr float kSlack = 8.0f;
// fp16 weights are held times 2^6, so that small ones stay clear of fp16's
// smallest number; the factor cancels in the division by their sum.
constexpr float kF16Lift = 6.0f;

// What one row tile of one kv head has to do.
struct RowTile {
  int b;        // sequence
  int q0, n;    // its first query and their number
  int row0;     // first row of the tile (row = query in sequence * group + head in group)
  int len;      // cached rows
  int lo, hi;   // keys that any row of the tile may see; lo is a multiple of kTileKeys
};

template <int ROWS>
__device__ __forceinline__ bool find_tile(const KvAttnArgs& a, int tile, RowTile& r) {
  const int G = a.group;
  if (!a.offs) {
    const int per = (G + ROWS - 1) / ROWS;
    r.b = tile / per;
    r.row0 = (tile - r.b * per) * ROWS;
    r.q0 = r.b;
    r.n = 1;
    if (r.b >= a.batch) return false;
  } else {
    const int lane = threadIdx.x & 63;
    const int T = (int)a.tokens, B = (int)a.batch;
    int before = 0;
    bool found = false;
    for (int b0 = 0; b0 < B; b0 += 64) {
      const int b = b0 + lane;
      int s = 0, e = 0;
      if (b < B) {
        s = min(max(a.offs[b], 0), T);
        e = max(min(max(a.offs[b + 1], 0), T), s);
      }
      const int mine = (int)(((int64_t)(e - s) * G + ROWS - 1) / ROWS);
      int upto = mine;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(upto, d, 64);
        if (lane >= d) upto += x;
      }
      const uint64_t hit = __ballot(before + upto > tile);
      if (hit) {
        const int src = __builtin_ctzll(hit);
        r.b = b0 + src;
        r.q0 = __builtin_amdgcn_readlane(s, src);
        r.n = __builtin_amdgcn_readlane(e, src) - r.q0;
        r.row0 = (tile - before - __builtin_amdgcn_readlane(upto - mine, src)) * ROWS;
        found = true;
        break;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (!found) return false;
  }
  r.len = min(max(a.lens[r.b], 0), (int)a.max_len);
  // the last visible key grows with the query, and so does the first
  const int t0 = r.row0 / G, t1 = min((r.row0 + ROWS - 1) / G, r.n - 1);
  r.hi = a.causal ? min(max(r.len - r.n + t1 + 1, 0), r.len) : r.len;
  r.lo = 0;
  if (a.window > 0) {
    const int64_t first = (int64_t)r.len - r.n + t0 + 1 - a.window;
    r.lo = first > 0 ? (int)first & ~(kTileKeys - 1) : 0;
  }
  if (r.lo > r.hi) r.lo = r.hi & ~(kTileKeys - 1);
  return true;
}

// Chunks that the tile's keys make (at least one: a tile without keys still
// writes its empty result).
__device__ __forceinline__ int tile_chunks(const RowTile& r, int64_t chunk) {
  const int64_t n = r.hi - r.lo;
  return n <= chunk ? 1 : (int)((n + chunk - 1) / chunk);
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  const bf16x2 p = {(__bf16)x, (__bf16)y};
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  const f16x2 p = {(_Float16)x, (_Float16)y};
  return __builtin_bit_cast(uint32_t, p);
}
template <bool NV>
__device__ __forceinline__ uint32_t pack16bit(float x, float y) {
  return NV ? pack_f16(x, y) : pack_bf16(x, y);
}
// x and y rounded to 16 bits, and what the rounding left.
template <bool NV>
__device__ __forceinline__ uint32_t split16bit(float& x, float& y) {
  const uint32_t w = pack16bit<NV>(x, y);
  if constexpr (NV) {
    const f16x2 p = __builtin_bit_cast(f16x2, w);
    x -= (float)p.x;
    y -= (float)p.y;
  } else {
    x -= bf16_lo(w);
    y -= bf16_hi(w);
  }
  return w;
}

template <bool NV>
__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 acc) {
  if constexpr (NV)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), acc, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc, 0, 0, 0);
}

__device__ __forceinline__ uint32_t e2m1_pair_f16(uint32_t w, int sel) {
  const f16x2 p = sel == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0)
                  : sel == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1)
                  : sel == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2)
                             : __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ uint32_t e2m1_pair_bf16(uint32_t w, float scale, int sel) {
  return sel == 0   ? e2m1_unpack2_bf16<0>(w, scale)
         : sel == 1 ? e2m1_unpack2_bf16<1>(w, scale)
         : sel == 2 ? e2m1_unpack2_bf16<2>(w, scale)
                    : e2m1_unpack2_bf16<3>(w, scale);
}
// The E4M3 values of the two low bytes of w in fp16 (exact).
__device__ __forceinline__ f16x2 e4m3_pair_f16(uint32_t w) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, f16x2 y) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x) * y);
}

// Eight consecutive codes under one scale byte as an MFMA operand.
template <bool NV>
__device__ __forceinline__ u32x4 convert8(uint32_t w, uint32_t scale_byte) {
  if constexpr (NV) {
    const f16x2 s = e4m3_pair_f16(scale_byte | (scale_byte << 8));
    return u32x4{mul_f16x2(e2m1_pair_f16(w, 0), s), mul_f16x2(e2m1_pair_f16(w, 1), s),
                 mul_f16x2(e2m1_pair_f16(w, 2), s), mul_f16x2(e2m1_pair_f16(w, 3), s)};
  } else {
    const float s = e8m0_scale_operand(scale_byte);
    return u32x4{e2m1_unpack2_bf16<0>(w, s), e2m1_unpack2_bf16<1>(w, s), e2m1_unpack2_bf16<2>(w, s),
                 e2m1_unpack2_bf16<3>(w, s)};
  }
}

// The codes x and y of two keys (eight elements d each, under scale bytes sx
// and sy), transposed: out[d] = (key x, key y) of element d, in 16 bits each.
// PAIRS: how many pairs of elements the words hold.
template <bool NV, int PAIRS>
__device__ __forceinline__ void convert_key_pair(uint32_t x, uint32_t y, uint32_t sx, uint32_t sy, uint32_t* out) {
  if constexpr (NV) {
    // the two keys' nibbles of one element side by side in a byte
    const uint32_t even = (x & 0x0f0f0f0fu) | ((y & 0x0f0f0f0fu) << 4);
    const uint32_t odd = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
    const f16x2 s = e4m3_pair_f16(sx | (sy << 8));
#pragma unroll
    for (int i = 0; i < PAIRS; i++) {
      out[2 * i] = mul_f16x2(e2m1_pair_f16(even, i), s);
      out[2 * i + 1] = mul_f16x2(e2m1_pair_f16(odd, i), s);
    }
  } else {
    const float fx = e8m0_scale_operand(sx), fy = e8m0_scale_operand(sy);
#pragma unroll
    for (int i = 0; i < PAIRS; i++) {
      const uint32_t p = e2m1_pair_bf16(x, fx, i), q = e2m1_pair_bf16(y, fy, i);
      out[2 * i] = __builtin_amdgcn_perm(q, p, 0x05040100u);
      out[2 * i + 1] = __builtin_amdgcn_perm(q, p, 0x07060302u);
    }
  }
}

// tanh by one exponential; 1 and -1 where it over- and underflows.
__device__ __forceinline__ float tanh_exp(float x) {
  return 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * (2.0f * kLog2e)));
}

__device__ __forceinline__ float tensor_scale_of(const float* ts, int h) {
  const float s = ts[h];
  return s >= kFltMin && s <= 3.40282347e38f ? s : 1.0f;
}

// N consecutive elements of a result row.
template <bool BF16, int N>
__device__ __forceinline__ void store_row(const KvAttnArgs& a, int token, int head, int d, const float* v) {
  typedef uint32_t words __attribute__((ext_vector_type(N / 2 > 4 ? 4 : N / 2)));
  typedef float floats __attribute__((ext_vector_type(N > 4 ? 4 : N)));
  if constexpr (BF16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + token * a.o_ts_ + head * a.o_hs + d;
    constexpr int W = N / 2 > 4 ? 4 : N / 2;
#pragma unroll
    for (int i = 0; i < N; i += 2 * W) {
      words w;
#pragma unroll
      for (int j = 0; j < W; j++) w[j] = pack_bf16(v[i + 2 * j], v[i + 2 * j + 1]);
      *reinterpret_cast<words*>(o + i) = w;
    }
  } else {
    float* o = static_cast<float*>(a.out) + token * a.o_ts_ + head * a.o_hs + d;
    constexpr int W = N > 4 ? 4 : N;
#pragma unroll
    for (int i = 0; i < N; i += W) {
      floats w;
#pragma unroll
      for (int j = 0; j < W; j++) w[j] = v[i + j];
      *reinterpret_cast<floats*>(o + i) = w;
    }
  }
}

// The result of a row: its weighted sum by its denominator, and lse.
template <bool NV>
__device__ __forceinline__ float row_factor(const KvAttnArgs& a, int h, float sum) {
  return sum == 0.0f ? 0.0f : (NV ? tensor_scale_of(a.c.v_ts, h) : 1.0f) / sum;
}
template <bool NV>
__device__ __forceinline__ float row_lse(float top, float sum) {
  return sum == 0.0f ? -__builtin_huge_valf() : kLn2 * ((NV ? top - kF16Lift : top) + __builtin_amdgcn_logf(sum));
}

// How one lane holds a 32-key tile's codes and scale bytes.
template <int DP, bool NV, bool BF16>
struct Tile {
  static constexpr int kBlk = NV ? 16 : 32;
  // K: words of 8 codes of one key per lane, elements g * DP/4 on, and the
  // scale bytes over them
  static constexpr int kKWords = DP / 32;
  static constexpr int kKScales = DP / 4 > kBlk ? DP / 4 / kBlk : 1;
  static constexpr int kVWords = DP > 128 ? 2 : 1;
  uint32_t k[2][kKWords];
  uint32_t ks[2][kKScales];
  uint32_t v[8][kVWords];
  uint32_t vs[8];
};

// Where a tile's rows lie: the pages of its two 16-key halves.
struct TilePages {
  int p[2];
};

// NW waves; FULL: the head size is DP itself.
template <int DP, bool NV, bool BF16, bool FULL, int NW>
__global__ __launch_bounds__(64 * NW, DP == 256 ? 1 : DP == 128 ? 2 : 3) void kv_attn_kernel(KvAttnArgs a, int splits, int64_t chunk) {
  using Regs = Tile<DP, NV, BF16>;
  constexpr int kRows = 16;
  constexpr int kBlk = Regs::kBlk;
  constexpr int kChunkV = DP / 16;  // elements of V per lane = number of O tiles
  constexpr int kQTerms = BF16 ? 1 : NV ? 2 : 3;
  constexpr int kPTerms = BF16 ? 1 : 2;
  constexpr int kStep = kTileKeys * NW;
  __shared__ float s_o[NW][kRows][DP + 4];
  __shared__ float s_m[NW][kRows], s_l[NW][kRows];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int split = blockIdx.x % splits;
  const int th = blockIdx.x / splits;
  const int h = th % a.c.heads, tile = th / a.c.heads;
  RowTile r;
  if (!find_tile<kRows>(a, tile, r)) return;
  if (split >= tile_chunks(r, chunk)) return;
  const int c_lo = r.lo + (int)(split * chunk);
  const int c_hi = (int)min((int64_t)r.hi, c_lo + chunk);
  const int D = FULL ? DP : a.c.dim, G = a.group;

  // this lane's row: its query, and the keys [my_lo, my_hi) it sees
  const int row = r.row0 + c;
  const bool live = row < r.n * G;
  const int t = live ? row / G : r.n - 1;
  const int head = h * G + (live ? row - t * G : 0);
  const int my_hi = a.causal ? min(max(r.len - r.n + t + 1, 0), r.len) : r.len;
  const int my_lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)r.len - r.n + t + 1 - a.window) : 0;
  // keys that every row of the tile sees
  const int t_first = r.row0 / G, t_last = min((r.row0 + kRows - 1) / G, r.n - 1);
  const int all_hi = a.causal ? min(max(r.len - r.n + t_first + 1, 0), r.len) : r.len;
  const int all_lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)r.len - r.n + t_last + 1 - a.window) : 0;

  const int shift = a.c.page_shift, in_page = (1 << shift) - 1;
  const int32_t* table = a.table + r.b * a.table_stride;
  const int row_codes = D >> 1, row_scales = D / kBlk;
  const int last16 = (r.len - 1) & ~15;  // the last 16 keys that exist
  // lane offsets within a 16-key half; elements past the head size are read
  // from the row's beginning and meet queries of 0, or results not stored
  uint32_t k_at[Regs::kKWords], ks_at[Regs::kKScales];
#pragma unroll
  for (int w = 0; w < Regs::kKWords; w++) {
    const int d = g * (DP / 4) + 8 * w;
    k_at[w] = c * row_codes + (FULL || d < D ? d >> 1 : 0);
  }
#pragma unroll
  for (int i = 0; i < Regs::kKScales; i++) {
    const int b = g * (DP / 4) / kBlk + i;
    ks_at[i] = c * row_scales + (FULL || b < row_scales ? b : 0);
  }
  const int vd = FULL || kChunkV * c < D ? kChunkV * c : 0;
  const uint32_t v_at = 4 * g * row_codes + (vd >> 1), vs_at = 4 * g * row_scales + vd / kBlk;

  auto pages_of = [&](int kt) {
    TilePages p;
#pragma unroll
    for (int sub = 0; sub < 2; sub++) p.p[sub] = table[min(kt + 16 * sub, last16) >> shift];
    return p;
  };
  // 16 keys lie in one page. Keys past the end are read as they lie in the
  // last page (their scores are masked, their values zeroed below); a half
  // past the last page is read from there.
  auto load = [&](int kt, const TilePages& p, Regs& x) {
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      const int64_t page = min(max((int64_t)p.p[sub], (int64_t)0), a.c.pages - 1);
      const int row0 = (h << shift) + (min(kt + 16 * sub, last16) & in_page);
      const int64_t at_c = page * a.c.codes_ps + (int64_t)row0 * row_codes;
      const int64_t at_s = page * a.c.scales_ps + (int64_t)row0 * row_scales;
      const uint8_t *kc = a.c.kc + at_c, *ks = a.c.ks + at_s, *vc = a.c.vc + at_c, *vs = a.c.vs + at_s;
      if constexpr (FULL && Regs::kKWords == 2) {
        const u32x2 y = *reinterpret_cast<const u32x2*>(kc + k_at[0]);
        x.k[sub][0] = y.x;
        x.k[sub][1] = y.y;
      } else if constexpr (FULL) {
#pragma unroll
        for (int w = 0; w < Regs::kKWords; w += 4) {
          const u32x4 y = *reinterpret_cast<const u32x4*>(kc + k_at[w]);
#pragma unroll
          for (int i = 0; i < 4; i++) x.k[sub][w + i] = y[i];
        }
      } else {
#pragma unroll
        for (int w = 0; w < Regs::kKWords; w++) x.k[sub][w] = *reinterpret_cast<const uint32_t*>(kc + k_at[w]);
      }
#pragma unroll
      for (int i = 0; i < Regs::kKScales; i++) x.ks[sub][i] = ks[ks_at[i]];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint8_t* y = vc + (v_at + i * row_codes);
        if constexpr (DP == 64) {
          x.v[4 * sub + i][0] = *reinterpret_cast<const uint16_t*>(y);
        } else if constexpr (Regs::kVWords == 2) {
          const u32x2 z = *reinterpret_cast<const u32x2*>(y);
          x.v[4 * sub + i][0] = z.x;
          x.v[4 * sub + i][1] = z.y;
        } else {
          x.v[4 * sub + i][0] = *reinterpret_cast<const uint32_t*>(y);
        }
        x.vs[4 * sub + i] = vs[vs_at + i * row_scales];
      }
    }
  };

  // the first tile's codes are on their way while the queries are laid out
  Regs tiles[2];
  TilePages ahead{};
  int kt = c_lo + kTileKeys * wave;
  if (kt < c_hi) {
    load(kt, pages_of(kt), tiles[0]);
    if (kt + kStep < c_hi) ahead = pages_of(kt + kStep);
  }

  // queries, in the order of the K operand; a negative scale goes into them
  u32x4 q[kQTerms][DP / 32];
  float score_scale = __builtin_fabsf(a.scale);
  {
    float x[DP / 4];
#pragma unroll
    for (int w = 0; w < DP / 32; w++) {
      const int d = g * (DP / 4) + 8 * w;
#pragma unroll
      for (int i = 0; i < 8; i++) x[8 * w + i] = 0.0f;
      if (live && d < D) {
        const int64_t at = (int64_t)(r.q0 + t) * a.q_ts_ + (int64_t)head * a.q_hs + d;
        if constexpr (BF16) {
          const uint4 p = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at);
          x[8 * w + 0] = bf16_lo(p.x); x[8 * w + 1] = bf16_hi(p.x);
          x[8 * w + 2] = bf16_lo(p.y); x[8 * w + 3] = bf16_hi(p.y);
          x[8 * w + 4] = bf16_lo(p.z); x[8 * w + 5] = bf16_hi(p.z);
          x[8 * w + 6] = bf16_lo(p.w); x[8 * w + 7] = bf16_hi(p.w);
        } else {
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
          const float4 p0 = p[0], p1 = p[1];
          x[8 * w + 0] = p0.x; x[8 * w + 1] = p0.y; x[8 * w + 2] = p0.z; x[8 * w + 3] = p0.w;
          x[8 * w + 4] = p1.x; x[8 * w + 5] = p1.y; x[8 * w + 6] = p1.z; x[8 * w + 7] = p1.w;
        }
        if (a.scale < 0.0f) {
#pragma unroll
          for (int i = 0; i < 8; i++) x[8 * w + i] = -x[8 * w + i];
        }
      }
    }
    if constexpr (NV) {
      // the row's largest magnitude to [2^14, 2^15)
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < DP / 4; i++) amax = __builtin_fmaxf(amax, __builtin_fabsf(x[i]));
      amax = __builtin_fmaxf(amax, xor_shfl<16>(amax));
      amax = __builtin_fmaxf(amax, xor_shfl<32>(amax));
      const int up = 141 - (int)(__builtin_bit_cast(uint32_t, amax) >> 23);
#pragma unroll
      for (int i = 0; i < DP / 4; i++) x[i] = __builtin_ldexpf(x[i], up);
      score_scale = __builtin_ldexpf(score_scale * tensor_scale_of(a.c.k_ts, h), -up);
    }
#pragma unroll
    for (int k = 0; k < kQTerms; k++) {
#pragma unroll
      for (int w = 0; w < DP / 32; w++) {
#pragma unroll
        for (int i = 0; i < 4; i++) q[k][w][i] = split16bit<NV>(x[8 * w + 2 * i], x[8 * w + 2 * i + 1]);
      }
    }
  }
  const bool capped = a.softcap > 0.0f;
  const float cap2 = a.softcap * kLog2e;
  score_scale = capped ? score_scale / a.softcap : score_scale * kLog2e;

  f32x4 o[kChunkV];
#pragma unroll
  for (int j = 0; j < kChunkV; j++) o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kNoMax, l = 0.0f;

  auto compute = [&](int kt, Regs& x) {
    float s[8];
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < Regs::kKWords; w++) {
        const u32x4 kk = convert8<NV>(x.k[sub][w], x.ks[sub][w * 8 / kBlk < Regs::kKScales ? w * 8 / kBlk : 0]);
#pragma unroll
        for (int n = 0; n < kQTerms; n++) acc = mfma16<NV>(kk, q[n][w], acc);
      }
#pragma unroll
      for (int i = 0; i < 4; i++) s[4 * sub + i] = acc[i];
    }
    float factor = score_scale;  // of s, to scores in powers of two
    if (capped) {
#pragma unroll
      for (int i = 0; i < 8; i++) s[i] = cap2 * tanh_exp(s[i] * score_scale);
      factor = 1.0f;
    }
    if (kt + kTileKeys > all_hi || kt < all_lo) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int key = kt + 16 * (i >> 2) + 4 * g + (i & 3);
        s[i] = key < my_hi && key >= my_lo ? s[i] * factor : -__builtin_huge_valf();
        // a weight of 0 must meet a number
        if (key >= r.len) {
#pragma unroll
          for (int w = 0; w < Regs::kVWords; w++) x.v[i][w] = 0u;
          x.vs[i] = 0u;
        }
      }
      factor = 1.0f;
    }
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 8; i++) top = __builtin_fmaxf(top, s[i]);
    top *= factor;
    if (__any(top > m + kSlack)) {
      top = __builtin_fmaxf(top, xor_shfl<16>(top));
      top = __builtin_fmaxf(top, xor_shfl<32>(top));
      const float raised = __builtin_fmaxf(m, top);
      const float down = __builtin_amdgcn_exp2f(m - raised);
      l *= down;
#pragma unroll
      for (int j = 0; j < kChunkV; j++) o[j] *= down;
      m = raised;
    }
    const float base = NV ? m - kF16Lift : m;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; i++) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], factor, -base));
    l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    u32x4 pw[kPTerms];
#pragma unroll
    for (int n = 0; n < kPTerms; n++) {
#pragma unroll
      for (int i = 0; i < 4; i++) pw[n][i] = split16bit<NV>(p[2 * i], p[2 * i + 1]);
    }
#pragma unroll
    for (int w = 0; w < Regs::kVWords; w++) {
      constexpr int kPairs = kChunkV >= 8 ? 4 : 2;
      uint32_t vt[4][2 * kPairs];
#pragma unroll
      for (int i = 0; i < 4; i++)
        convert_key_pair<NV, kPairs>(x.v[2 * i][w], x.v[2 * i + 1][w], x.vs[2 * i], x.vs[2 * i + 1], vt[i]);
#pragma unroll
      for (int j = 0; j < 2 * kPairs; j++) {
        const u32x4 vv = {vt[0][j], vt[1][j], vt[2][j], vt[3][j]};
#pragma unroll
        for (int n = 0; n < kPTerms; n++) o[8 * w + j] = mfma16<NV>(vv, pw[n], o[8 * w + j]);
      }
    }
  };

  // two tiles' registers in turn: one is loaded while the other is used, and
  // the page numbers are fetched a tile earlier still
  for (; kt < c_hi; kt += 2 * kStep) {
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int now = kt + k * kStep;
      if (now + kStep < c_hi) {
        load(now + kStep, ahead, tiles[1 - k]);
        if (now + 2 * kStep < c_hi) ahead = pages_of(now + 2 * kStep);
      }
      if (now < c_hi) compute(now, tiles[k]);
    }
  }
  l += xor_shfl<16>(l);
  l += xor_shfl<32>(l);

  // join the waves: O tile j holds of row c the elements kChunkV * (4g + i) + j
  if (g == 0) {
    s_m[wave][c] = m;
    s_l[wave][c] = l;
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
#pragma unroll
    for (int j = 0; j < kChunkV; j++) s_o[wave][c][(4 * g + i) * kChunkV + j] = o[j][i];
  }
  __syncthreads();
  constexpr int kEach = kRows * DP / (64 * NW);  // elements a thread joins
  constexpr int kPerRow = DP / kEach;
  const int jr = threadIdx.x / kPerRow, d = threadIdx.x % kPerRow * kEach;
  const int jrow = r.row0 + jr;
  if (jrow >= r.n * G || d >= D) return;
  const int jt = jrow / G, jhead = h * G + jrow - jt * G;
  float top = s_m[0][jr];
#pragma unroll
  for (int w = 1; w < NW; w++) top = __builtin_fmaxf(top, s_m[w][jr]);
  float sum = 0.0f, acc[kEach];
#pragma unroll
  for (int j = 0; j < kEach; j++) acc[j] = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; w++) {
    const float f = __builtin_amdgcn_exp2f(s_m[w][jr] - top);
    sum += f * s_l[w][jr];
#pragma unroll
    for (int j = 0; j < kEach; j++) acc[j] += f * s_o[w][jr][d + j];
  }
  if (splits > 1) {
    float* part = a.ws + (int64_t)blockIdx.x * (kRows * (D + 2));
#pragma unroll
    for (int j = 0; j < kEach; j++) part[jr * D + d + j] = acc[j];
    if (d == 0) {
      part[kRows * D + jr] = top;
      part[kRows * (D + 1) + jr] = sum;
    }
  } else {
    const float f = row_factor<NV>(a, h, sum);
#pragma unroll
    for (int j = 0; j < kEach; j++) acc[j] *= f;
    store_row<BF16, kEach>(a, r.q0 + jt, jhead, d, acc);
    if (d == 0 && a.lse) a.lse[(int64_t)(r.q0 + jt) * a.q_heads + jhead] = row_lse<NV>(top, sum);
  }
}

// Joins the chunks of one row: DP / 4 lanes take four elements each, and the
// rest of the workgroup every kGroups-th chunk.
template <int DP, bool NV, bool BF16, int THREADS>
__global__ __launch_bounds__(THREADS) void kv_attn_join_kernel(KvAttnArgs a, int splits, int64_t chunk) {
  constexpr int kRows = 16;
  constexpr int kLanes = DP / 4, kGroups = THREADS / kLanes;
  __shared__ float s_acc[kGroups][DP + 4];
  __shared__ float s_m[kGroups], s_l[kGroups];
  const int jr = blockIdx.x % kRows, th = blockIdx.x / kRows;
  const int h = th % a.c.heads, tile = th / a.c.heads;
  RowTile r;
  if (!find_tile<kRows>(a, tile, r)) return;
  const int D = a.c.dim, G = a.group;
  const int row = r.row0 + jr;
  if (row >= r.n * G) return;
  const int n = tile_chunks(r, chunk);
  const int t = row / G, head = h * G + row - t * G;
  const int64_t step = kRows * (D + 2);
  const float* part = a.ws + (int64_t)th * splits * step;
  const int grp = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  float top = kNoMax, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (d < D) {
#pragma unroll 4
    for (int k = grp; k < n; k += kGroups) {
      const float* p = part + k * step;
      const float pm = p[kRows * D + jr], pl = p[kRows * (D + 1) + jr];
      const float4 v = *reinterpret_cast<const float4*>(p + jr * D + d);
      const float raised = __builtin_fmaxf(top, pm);
      const float fo = __builtin_amdgcn_exp2f(top - raised), fn = __builtin_amdgcn_exp2f(pm - raised);
      top = raised;
      sum = sum * fo + pl * fn;
      acc.x = acc.x * fo + v.x * fn;
      acc.y = acc.y * fo + v.y * fn;
      acc.z = acc.z * fo + v.z * fn;
      acc.w = acc.w * fo + v.w * fn;
    }
  }
  if (d == 0) {
    s_m[grp] = top;
    s_l[grp] = sum;
  }
  *reinterpret_cast<float4*>(&s_acc[grp][d]) = acc;
  __syncthreads();
  if (grp != 0 || d >= D) return;
  const int used = n < kGroups ? n : kGroups;
  float all = s_m[0];
  for (int k = 1; k < used; k++) all = __builtin_fmaxf(all, s_m[k]);
  sum = 0.0f;
  float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < used; k++) {
    const float f = __builtin_amdgcn_exp2f(s_m[k] - all);
    sum += f * s_l[k];
    const float4 v = *reinterpret_cast<const float4*>(&s_acc[k][d]);
    y[0] += f * v.x;
    y[1] += f * v.y;
    y[2] += f * v.z;
    y[3] += f * v.w;
  }
  const float f = row_factor<NV>(a, h, sum);
#pragma unroll
  for (int j = 0; j < 4; j++) y[j] *= f;
  store_row<BF16, 4>(a, r.q0 + t, head, d, y);
  if (d == 0 && a.lse) a.lse[(int64_t)(r.q0 + t) * a.q_heads + head] = row_lse<NV>(all, sum);
}

namespace {
constexpr int kWaves = 4;
// waves of the wide form: as many as its registers allow (heads past 128: no wide form)
constexpr int wide_waves(int dp) { return dp <= 128 ? 8 : kWaves; }
}  // namespace

KvAttnPlan plan_kv_attention(const KvAttnArgs& a) {
  KvAttnPlan p{};
  p.rows = 16;
  p.waves = kWaves;
  const int64_t rows = a.tokens * a.group;
  p.tiles = a.offs ? rows / p.rows + a.batch : a.batch * ((a.group + p.rows - 1) / p.rows);
  // keys a tile can see at most: all, or the windows of its queries
  int64_t keys = a.max_len;
  if (a.window > 0) {
    const int64_t w = a.window + p.rows + kTileKeys;
    keys = keys < w ? keys : w;
  }
  const int64_t work = p.tiles * a.c.heads;
  // Little work: one launch whose workgroups have many waves, rather than
  // chunks and a second launch to join them.
  const int wide = wide_waves(a.c.dim);
  if (work <= 256 && keys <= 4 * wide * kTileKeys) {
    p.waves = wide;
    p.chunk = keys > 0 ? keys : 1;
    p.splits = 1;
    return p;
  }
  const int64_t per_pass = kTileKeys * kWaves;
  const int64_t want = 4096;
  int64_t splits = work >= want ? 1 : (want + work - 1) / work;
  int64_t chunk = ((keys + splits - 1) / splits + per_pass - 1) / per_pass * per_pass;
  if (chunk < 4 * per_pass) chunk = 4 * per_pass;
  p.chunk = chunk;
  p.splits = keys <= chunk ? 1 : (keys + chunk - 1) / chunk;
  p.ws = p.splits > 1 ? (size_t)(work * p.splits) * (size_t)(p.rows * (a.c.dim + 2)) * sizeof(float) : 0;
  return p;
}

template <int DP, bool NV, bool BF16>
static hipError_t launch_rows(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  constexpr int kWide = wide_waves(DP);
  const int64_t work = p.tiles * a.c.heads;
  const dim3 grid((unsigned)(work * p.splits));
  const int n = (int)p.splits;
  if (p.waves == kWaves) {
    if (a.c.dim == DP)
      hipLaunchKernelGGL((kv_attn_kernel<DP, NV, BF16, true, kWaves>), grid, dim3(64 * kWaves), 0, s, a, n, p.chunk);
    else
      hipLaunchKernelGGL((kv_attn_kernel<DP, NV, BF16, false, kWaves>), grid, dim3(64 * kWaves), 0, s, a, n, p.chunk);
  } else {
    if (a.c.dim == DP)
      hipLaunchKernelGGL((kv_attn_kernel<DP, NV, BF16, true, kWide>), grid, dim3(64 * kWide), 0, s, a, n, p.chunk);
    else
      hipLaunchKernelGGL((kv_attn_kernel<DP, NV, BF16, false, kWide>), grid, dim3(64 * kWide), 0, s, a, n, p.chunk);
  }
  if (n > 1) {
    const dim3 rows((unsigned)(work * p.rows));
    // few chunks: more threads would have nothing to do
    if (n <= 16)
      hipLaunchKernelGGL((kv_attn_join_kernel<DP, NV, BF16, 128>), rows, dim3(128), 0, s, a, n, p.chunk);
    else
      hipLaunchKernelGGL((kv_attn_join_kernel<DP, NV, BF16, 1024>), rows, dim3(1024), 0, s, a, n, p.chunk);
  }
  return hipGetLastError();
}

template <int DP>
static hipError_t launch_dim(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  if (a.c.nvfp4) return a.bf16 ? launch_rows<DP, true, true>(a, p, s) : launch_rows<DP, true, false>(a, p, s);
  return a.bf16 ? launch_rows<DP, false, true>(a, p, s) : launch_rows<DP, false, false>(a, p, s);
}

hipError_t launch_kv_attention(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  if (a.c.dim <= 64) return launch_dim<64>(a, p, s);
  if (a.c.dim <= 128) return launch_dim<128>(a, p, s);
  return launch_dim<256>(a, p, s);
}

}  // namespace fp4impl
