// kv_attention.hip -- softmax attention over the paged 4-bit key-value cache.
//
//   s = scale (q . k), p = exp(s - max), out = sum(p v) / sum(p)
//
// in one pass over the keys with a running maximum and sum. A workgroup of
// four waves takes 16 rows (row = (query, head of the kv head's group)) of
// one sequence and kv head and a chunk of their visible keys; each wave takes
// every fourth 32-key tile of the chunk on its own, with no barrier until the
// four results are joined through LDS. Long key ranges are cut into chunks
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
#include "fp4_device.h"
#include "launch.h"

namespace fp4impl {
using namespace fp4dev;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;
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

template <bool BF16>
__device__ __forceinline__ void store_row(const KvAttnArgs& a, int token, int head, int d, const float* v, int n) {
  if constexpr (BF16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + token * a.o_ts_ + head * a.o_hs + d;
#pragma unroll
    for (int i = 0; i < n; i += 4)
      *reinterpret_cast<uint2*>(o + i) = make_uint2(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]));
  } else {
    float* o = static_cast<float*>(a.out) + token * a.o_ts_ + head * a.o_hs + d;
#pragma unroll
    for (int i = 0; i < n; i += 4)
      *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}

// A tile's codes and scale bytes in one lane's registers.
template <int DP, bool NV>
struct TileRegs {
  static constexpr int kBlk = NV ? 16 : 32;
  static constexpr int kKWords = DP / 32;                             // of one key row
  static constexpr int kKScales = DP / 4 > kBlk ? DP / 4 / kBlk : 1;  // blocks those cover
  static constexpr int kVWords = DP > 128 ? 2 : 1;
  uint32_t k[2][kKWords];
  uint32_t ks[2][kKScales];
  uint32_t v[8][kVWords];
  uint32_t vs[8];
};

template <int DP, bool NV, bool BF16>
__global__ __launch_bounds__(256) void kv_attn_kernel(KvAttnArgs a, int splits, int64_t chunk) {
  using Regs = TileRegs<DP, NV>;
  constexpr int kRows = 16;
  constexpr int kBlk = Regs::kBlk;
  constexpr int kChunkV = DP / 16;  // elements of V per lane = number of O tiles
  constexpr int kQTerms = BF16 ? 1 : NV ? 2 : 3;
  constexpr int kPTerms = BF16 ? 1 : 2;
  constexpr int kPart = kChunkV < 8 ? kChunkV : 8;  // elements a thread joins at once
  constexpr int kParts = kChunkV / kPart;
  __shared__ float s_o[kWaves][kRows][16 * kPart + 4];
  __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];

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
  const int D = a.c.dim, G = a.group;

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

  // queries, in the order of the K operand
  u32x4 q[kQTerms][DP / 32];
  float score_scale = a.scale;
  {
    float x[DP / 4];
#pragma unroll
    for (int w = 0; w < DP / 32; w++) {
      const int d = g * (DP / 4) + 8 * w;
#pragma unroll
      for (int i = 0; i < 8; i++) x[8 * w + i] = 0.0f;
      if (live && d < D) {
        const int64_t at = (r.q0 + t) * a.q_ts_ + head * a.q_hs + d;
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

  const int shift = a.c.page_shift, in_page = (1 << shift) - 1;
  const int32_t* table = a.table + r.b * a.table_stride;
  const int row_codes = D >> 1, row_scales = D / kBlk;

  auto load = [&](int kt, Regs& x) {
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      const int key0 = kt + 16 * sub;
      // 16 keys lie in one page; rows past the end hold nothing to be read as
      // a number, pages past it may not even exist
      if (key0 < r.len) {
        const int64_t page = min(max((int64_t)table[key0 >> shift], (int64_t)0), a.c.pages - 1);
        const int row0 = (h << shift) + (key0 & in_page);
        const uint8_t* kc = a.c.kc + page * a.c.codes_ps + (int64_t)row0 * row_codes;
        const uint8_t* ks = a.c.ks + page * a.c.scales_ps + (int64_t)row0 * row_scales;
        const uint8_t* vc = a.c.vc + page * a.c.codes_ps + (int64_t)row0 * row_codes;
        const uint8_t* vs = a.c.vs + page * a.c.scales_ps + (int64_t)row0 * row_scales;
#pragma unroll
        for (int w = 0; w < Regs::kKWords; w++) {
          const int d = g * (DP / 4) + 8 * w;
          x.k[sub][w] = d < D ? *reinterpret_cast<const uint32_t*>(kc + c * row_codes + (d >> 1)) : 0u;
        }
#pragma unroll
        for (int w = 0; w < Regs::kKScales; w++) {
          const int bi = g * (DP / 4) / kBlk + w;
          x.ks[sub][w] = bi < row_scales ? ks[c * row_scales + bi] : 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int k = 4 * g + i, d = kChunkV * c;
          const bool there = key0 + k < r.len && d < D;
          const uint8_t* p = vc + k * row_codes + (d >> 1);
          if constexpr (DP == 64) {
            x.v[4 * sub + i][0] = there ? *reinterpret_cast<const uint16_t*>(p) : 0u;
          } else {
#pragma unroll
            for (int w = 0; w < Regs::kVWords; w++)
              x.v[4 * sub + i][w] = there ? reinterpret_cast<const uint32_t*>(p)[w] : 0u;
          }
          x.vs[4 * sub + i] = there ? vs[k * row_scales + d / kBlk] : 0u;
        }
      } else {
#pragma unroll
        for (int w = 0; w < Regs::kKWords; w++) x.k[sub][w] = 0u;
#pragma unroll
        for (int w = 0; w < Regs::kKScales; w++) x.ks[sub][w] = 0u;
#pragma unroll
        for (int i = 0; i < 4; i++) {
#pragma unroll
          for (int w = 0; w < Regs::kVWords; w++) x.v[4 * sub + i][w] = 0u;
          x.vs[4 * sub + i] = 0u;
        }
      }
    }
  };

  Regs next;
  int kt = c_lo + kTileKeys * wave;
  if (kt < c_hi) load(kt, next);
  for (; kt < c_hi; kt += kTileKeys * kWaves) {
    const Regs x = next;
    if (kt + kTileKeys * kWaves < c_hi) load(kt + kTileKeys * kWaves, next);

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
      for (int i = 0; i < 4; i++) s[4 * sub + i] = acc[i] * score_scale;
    }
    if (capped) {
#pragma unroll
      for (int i = 0; i < 8; i++) s[i] = cap2 * tanh_exp(s[i]);
    }
    if (kt + kTileKeys > all_hi || kt < all_lo) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int key = kt + 16 * (i >> 2) + 4 * g + (i & 3);
        s[i] = key < my_hi && key >= my_lo ? s[i] : -__builtin_huge_valf();
      }
    }
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 8; i++) top = __builtin_fmaxf(top, s[i]);
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
    for (int i = 0; i < 8; i++) {
      p[i] = __builtin_amdgcn_exp2f(s[i] - base);
      l += p[i];
    }
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
  }
  l += xor_shfl<16>(l);
  l += xor_shfl<32>(l);

  // join the four waves
  if (g == 0) {
    s_m[wave][c] = m;
    s_l[wave][c] = l;
  }
  const int jr = threadIdx.x >> 4, jc = threadIdx.x & 15;  // row and V chunk this thread joins
  const int jrow = r.row0 + jr;
  const bool jlive = jrow < r.n * G;
  const int jt = jlive ? jrow / G : 0, jhead = jlive ? h * G + jrow - jt * G : 0;
  float* part = a.ws ? a.ws + (int64_t)blockIdx.x * (kRows * (D + 2)) : nullptr;
#pragma unroll
  for (int half = 0; half < kParts; half++) {
    if (half) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
      for (int j = 0; j < kPart; j++) s_o[wave][c][(4 * g + i) * kPart + j] = o[half * kPart + j][i];
    }
    __syncthreads();
    float top = s_m[0][jr];
#pragma unroll
    for (int w = 1; w < kWaves; w++) top = __builtin_fmaxf(top, s_m[w][jr]);
    float sum = 0.0f, acc[kPart];
#pragma unroll
    for (int j = 0; j < kPart; j++) acc[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      const float f = __builtin_amdgcn_exp2f(s_m[w][jr] - top);
      sum += f * s_l[w][jr];
#pragma unroll
      for (int j = 0; j < kPart; j++) acc[j] += f * s_o[w][jr][jc * kPart + j];
    }
    const int d = kChunkV * jc + half * kPart;
    if (jlive && d < D) {
      if (splits > 1) {
        float* po = part + jr * D + d;
#pragma unroll
        for (int j = 0; j < kPart; j += 4)
          *reinterpret_cast<float4*>(po + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        if (d == 0) {
          part[kRows * D + jr] = top;
          part[kRows * (D + 1) + jr] = sum;
        }
      } else {
        const float f = sum > 0.0f || sum != sum ? (NV ? tensor_scale_of(a.c.v_ts, h) : 1.0f) / sum : 0.0f;
#pragma unroll
        for (int j = 0; j < kPart; j++) acc[j] *= f;
        store_row<BF16>(a, r.q0 + jt, jhead, d, acc, kPart);
        if (d == 0 && a.lse)
          a.lse[(int64_t)(r.q0 + jt) * a.q_heads + jhead] =
              sum == 0.0f ? -__builtin_huge_valf() : kLn2 * ((NV ? top - kF16Lift : top) + __builtin_amdgcn_logf(sum));
      }
    }
  }
}

// Joins a row tile's chunks: thread (row, 1/16 of the head).
template <int DP, bool NV, bool BF16>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(KvAttnArgs a, int splits, int64_t chunk) {
  constexpr int kRows = 16;
  constexpr int kChunkV = DP / 16;
  const int h = blockIdx.x % a.c.heads, tile = blockIdx.x / a.c.heads;
  RowTile r;
  if (!find_tile<kRows>(a, tile, r)) return;
  const int n = tile_chunks(r, chunk);
  const int D = a.c.dim, G = a.group;
  const int jr = threadIdx.x >> 4, d = kChunkV * (threadIdx.x & 15);
  const int row = r.row0 + jr;
  if (row >= r.n * G || d >= D) return;
  const int t = row / G, head = h * G + row - t * G;
  const int64_t step = kRows * (D + 2);
  const float* part = a.ws + (int64_t)blockIdx.x * splits * step;
  float top = kNoMax;
  for (int k = 0; k < n; k++) top = __builtin_fmaxf(top, part[k * step + kRows * D + jr]);
  float sum = 0.0f, acc[kChunkV];
#pragma unroll
  for (int j = 0; j < kChunkV; j++) acc[j] = 0.0f;
#pragma unroll 4
  for (int k = 0; k < n; k++) {
    const float f = __builtin_amdgcn_exp2f(part[k * step + kRows * D + jr] - top);
    sum += f * part[k * step + kRows * (D + 1) + jr];
    const float* po = part + k * step + jr * D + d;
#pragma unroll
    for (int j = 0; j < kChunkV; j += 4) {
      const float4 v = *reinterpret_cast<const float4*>(po + j);
      acc[j] += f * v.x;
      acc[j + 1] += f * v.y;
      acc[j + 2] += f * v.z;
      acc[j + 3] += f * v.w;
    }
  }
  const float f = sum > 0.0f || sum != sum ? (NV ? tensor_scale_of(a.c.v_ts, h) : 1.0f) / sum : 0.0f;
#pragma unroll
  for (int j = 0; j < kChunkV; j++) acc[j] *= f;
  store_row<BF16>(a, r.q0 + t, head, d, acc, kChunkV);
  if (d == 0 && a.lse)
    a.lse[(int64_t)(r.q0 + t) * a.q_heads + head] =
        sum == 0.0f ? -__builtin_huge_valf() : kLn2 * ((NV ? top - kF16Lift : top) + __builtin_amdgcn_logf(sum));
}

KvAttnPlan plan_kv_attention(const KvAttnArgs& a) {
  KvAttnPlan p{};
  p.rows = 16;
  const int64_t rows = a.tokens * a.group;
  p.tiles = a.offs ? rows / p.rows + a.batch : a.batch * ((a.group + p.rows - 1) / p.rows);
  // keys a tile can see at most: all, or the windows of its queries
  int64_t keys = a.max_len;
  if (a.window > 0) {
    const int64_t w = a.window + p.rows + kTileKeys;
    keys = keys < w ? keys : w;
  }
  const int64_t per_pass = kTileKeys * kWaves;
  const int64_t want = 1024;
  const int64_t work = p.tiles * a.c.heads;
  int64_t splits = work >= want ? 1 : (want + work - 1) / work;
  int64_t chunk = ((keys + splits - 1) / splits + per_pass - 1) / per_pass * per_pass;
  if (chunk < per_pass) chunk = per_pass;
  p.chunk = chunk;
  p.splits = keys <= chunk ? 1 : (keys + chunk - 1) / chunk;
  p.ws = p.splits > 1 ? (size_t)(work * p.splits) * (size_t)(p.rows * (a.c.dim + 2)) * sizeof(float) : 0;
  return p;
}

template <int DP, bool NV, bool BF16>
static hipError_t launch_rows(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  const int64_t work = p.tiles * a.c.heads;
  hipLaunchKernelGGL((kv_attn_kernel<DP, NV, BF16>), dim3((unsigned)(work * p.splits)), dim3(256), 0, s, a,
                     (int)p.splits, p.chunk);
  if (p.splits > 1)
    hipLaunchKernelGGL((kv_attn_join_kernel<DP, NV, BF16>), dim3((unsigned)work), dim3(256), 0, s, a, (int)p.splits,
                       p.chunk);
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
