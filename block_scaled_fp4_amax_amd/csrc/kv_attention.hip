// kv_attention.hip -- softmax attention over the paged 4-bit key-value cache.
//
//   s = scale (q . k), p = exp(s - max), out = sum(p v) / sum(p)
//
// in one pass over the keys with a running maximum and sum, in tiles of 32
// keys. A row is (query, head of the kv head's group). Two forms:
//
// Few rows (a token or some per sequence; bound by reading the cache): a
// workgroup takes 16 or 32 rows of one sequence and kv head; each of its waves
// takes every n-th key tile on its own, with no barrier until the waves'
// results are joined through LDS. Where that alone would leave the GPU unevenly
// loaded, the key tiles of the whole batch are cut into equal runs, one for
// each workgroup that fits on the GPU at once; partial results (fp32 sum,
// maximum, denominator) of rows whose keys lie in several runs go to the
// workspace and are joined by a second kernel.
//
// Many rows (prompts; bound by arithmetic): a workgroup's four waves have rows
// of their own, 32 each, and go through the key tiles together. Each
// wave converts a quarter of the next tile and leaves it in LDS as the matrix
// instructions' operands, while all of them use the present one.
//
// One wave, one tile of 32 keys, on v_mfma_f32_16x16x32 (lane l: c = l % 16,
// g = l / 16):
//   S^T = K Q^T: the A operand's rows are 16 keys, lane (c, g) holding of key
//     c the head's elements g * D/4 .. g * D/4 + D/4 - 1, so one row's codes
//     are read by four lanes, D/8 bytes each, and converted in registers. The
//     result has a query per column: lane (c, g) holds row c's scores of four
//     keys of both 16-key halves.
//   O^T += V^T P^T: those eight scores are exactly the lane's part of the B
//     operand if the contraction runs over the keys in that order, so the
//     weights never leave their lane. The A operand needs, for one element d
//     per lane, the same eight keys: the lane reads D/32 bytes of each of
//     them (elements c * D/16 ..) and transposes pairs of keys in registers.
// MXFP4 elements times their power-of-two scale are exact in bf16 (and leave
// fp16's range), NVFP4 elements times their E4M3 scale in both, 6 bits; the
// NVFP4 tensor scales multiply the scores and the result. NVFP4 queries are
// brought to a common power of two per row first, so that none leaves the
// operand's range. bf16 calls round the weights once for the product with V,
// to the type V is exact in: bf16 for MXFP4, fp16 for NVFP4, whose three more
// bits and cheaper conversion it can take. fp32 calls split queries and
// weights into three bf16 terms (24 bits, fp32's range) and multiply every
// term, also for NVFP4: fp16 terms would lose weights below 2^-31 of the
// largest, which a long context may be made of.
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
// The running maximum starts at the lowest number, so that a masked score
// (-inf) weighs exp2(-inf) = 0 also before the first visible key, and every
// finite one counts.
constexpr float kNoMax = -3.40282347e38f;
// A row's maximum is only raised when a score passes it by more than 2^8
// (weights may grow to that without harm in fp32), so that most tiles need
// neither the exchange across lanes nor the rescaling.
constexpr float kSlack = 8.0f;
// fp16 weights (of bf16 calls) are held times 2^6, so that small ones stay
// clear of fp16's smallest number; the factor cancels in the division by their
// sum.
constexpr float kF16Lift = 6.0f;

// A weight is 2 to the exact product of score and factor, less the maximum,
// which is a rounded one: at 2^20 that rounding alone makes it 2^(1/16), and far
// past it would leave fp16 and fp32. From here on products are rounded alike.
constexpr float kLargeScore = 1048576.0f;

// What one row tile of one kv head has to do.
struct RowTile {
  int b;        // sequence
  int q0, n;    // its first query and their number
  int row0;     // first row of the tile (row = query in sequence * group + head in group)
  int len;      // cached rows
  int lo, hi;   // keys that any row of the tile may see; lo is a multiple of kTileKeys
};

// A sequence's queries (q0, n), cut into the tokens there are.
__device__ __forceinline__ void seq_queries(const KvAttnArgs& a, int b, int& q0, int& n) {
  q0 = b;
  n = 1;
  if (a.offs) {
    const int T = (int)a.tokens;
    q0 = min(max(a.offs[b], 0), T);
    n = max(min(max(a.offs[b + 1], 0), T) - q0, 0);
  }
}
__device__ __forceinline__ int seq_len(const KvAttnArgs& a, int b) { return min(max(a.lens[b], 0), (int)a.max_len); }

// First key that query t of a sequence may see, and the key after its last.
__device__ __forceinline__ int first_key(const KvAttnArgs& a, int len, int n, int t) {
  const int64_t k = (int64_t)len - n + t + 1 - a.window;
  return a.window > 0 && k > 0 ? (int)k : 0;
}
__device__ __forceinline__ int end_key(const KvAttnArgs& a, int len, int n, int t) {
  return a.causal ? min(max(len - n + t + 1, 0), len) : len;
}

// The keys of the tile of `rows` rows from r.row0 on.
__device__ __forceinline__ void tile_keys(const KvAttnArgs& a, int rows, RowTile& r) {
  // both ends grow with the query
  const int t0 = r.row0 / a.group, t1 = min((r.row0 + rows - 1) / a.group, r.n - 1);
  r.hi = end_key(a, r.len, r.n, t1);
  r.lo = min(first_key(a, r.len, r.n, t0), r.hi) & ~(kTileKeys - 1);
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_prefix(int x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}

// The tile-th row tile of the batch.
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
    const int lane = threadIdx.x & 63, B = (int)a.batch;
    int before = 0;
    bool found = false;
    for (int b0 = 0; b0 < B; b0 += 64) {
      const int b = b0 + lane;
      int s = 0, n = 0;
      if (b < B) seq_queries(a, b, s, n);
      const int mine = (int)(((int64_t)n * G + ROWS - 1) / ROWS);
      const int upto = wave_prefix(mine);
      const uint64_t hit = __ballot(before + upto > tile);
      if (hit) {
        const int src = __builtin_ctzll(hit);
        r.b = b0 + src;
        r.q0 = __builtin_amdgcn_readlane(s, src);
        r.n = __builtin_amdgcn_readlane(n, src);
        r.row0 = (tile - before - __builtin_amdgcn_readlane(upto - mine, src)) * ROWS;
        found = true;
        break;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (!found) return false;
  }
  r.len = seq_len(a, r.b);
  tile_keys(a, ROWS, r);
  return true;
}

// The balanced form. The items (sequence, row tile, kv head), in that order,
// each count the key tiles of their sequence (`span` of them from `lo` on),
// and all those key tiles, one after another, are cut into equal runs, one
// for each workgroup. An item within one run is finished there. Otherwise
// each run it touches leaves a partial result in one of its two slots: 2 w
// for an item that began before run w, 2 w + 1 for one that begins in it.
struct SeqWork {
  int b, q0, n, len;
  int lo, span;    // keys lo .. lo + span * kTileKeys hold all that any query sees
  int row_tiles;
};

template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const KvAttnArgs& a, int b) {
  SeqWork w;
  w.b = b;
  seq_queries(a, b, w.q0, w.n);
  w.len = seq_len(a, b);
  w.row_tiles = (w.n * a.group + ROWS - 1) / ROWS;
  w.lo = w.n > 0 ? min(first_key(a, w.len, w.n, 0), w.len) & ~(kTileKeys - 1) : 0;
  w.span = max((w.len - w.lo + kTileKeys - 1) / kTileKeys, 1);
  return w;
}

__device__ __forceinline__ int run_length(int total, int runs, int least) {
  return max((total + runs - 1) / runs, least);
}

// 64 sequences' work, one a lane, and its running sums.
template <int ROWS>
struct WorkScan {
  SeqWork mine;
  int tiles, items;            // of this lane's sequence
  int upto_tiles, upto_items;  // of the 64 up to it

  __device__ __forceinline__ WorkScan(const KvAttnArgs& a, int b0) {
    const int b = b0 + (threadIdx.x & 63);
    mine = seq_work<ROWS>(a, min(b, (int)a.batch - 1));
    items = b < a.batch ? mine.row_tiles * a.c.heads : 0;
    tiles = items * mine.span;
    upto_tiles = wave_prefix(tiles);
    upto_items = wave_prefix(items);
  }
  __device__ __forceinline__ int all_tiles() const { return __builtin_amdgcn_readlane(upto_tiles, 63); }
  __device__ __forceinline__ int all_items() const { return __builtin_amdgcn_readlane(upto_items, 63); }

  // The sequence that holds key tile `at` (ITEM: item `at`) of these 64;
  // `before` are the key tiles of those before it, and `at` becomes the place
  // within the sequence.
  template <bool ITEM>
  __device__ __forceinline__ bool find(int& at, SeqWork& w, int& before) const {
    const uint64_t hit = __ballot((ITEM ? upto_items : upto_tiles) > at);
    if (!hit) return false;
    const int src = __builtin_ctzll(hit);
    w.b = __builtin_amdgcn_readlane(mine.b, src);
    w.q0 = __builtin_amdgcn_readlane(mine.q0, src);
    w.n = __builtin_amdgcn_readlane(mine.n, src);
    w.len = __builtin_amdgcn_readlane(mine.len, src);
    w.lo = __builtin_amdgcn_readlane(mine.lo, src);
    w.span = __builtin_amdgcn_readlane(mine.span, src);
    w.row_tiles = __builtin_amdgcn_readlane(mine.row_tiles, src);
    before = __builtin_amdgcn_readlane(upto_tiles - tiles, src);
    at -= ITEM ? __builtin_amdgcn_readlane(upto_items - items, src) : before;
    return true;
  }
};

// Key tiles of the whole batch, of which `first` holds the first 64 sequences.
template <int ROWS>
__device__ __forceinline__ int total_work(const KvAttnArgs& a, const WorkScan<ROWS>& first) {
  int sum = first.all_tiles();
  for (int b0 = 64; b0 < a.batch; b0 += 64) sum += WorkScan<ROWS>(a, b0).all_tiles();
  return sum;
}

// The sequence that holds key tile (ITEM: item) `at` of the batch.
template <int ROWS, bool ITEM>
__device__ __forceinline__ bool find_work(const KvAttnArgs& a, const WorkScan<ROWS>& first, int& at, SeqWork& w,
                                          int& before) {
  if (first.template find<ITEM>(at, w, before)) return true;
  int tiles = first.all_tiles();
  at -= ITEM ? first.all_items() : tiles;
  for (int b0 = 64; b0 < a.batch; b0 += 64) {
    const WorkScan<ROWS> next(a, b0);
    if (next.template find<ITEM>(at, w, before)) {
      before += tiles;
      return true;
    }
    tiles += next.all_tiles();
    at -= ITEM ? next.all_items() : next.all_tiles();
  }
  return false;
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  const bf16x2 p = {(__bf16)x, (__bf16)y};
  return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  const f16x2 p = {(_Float16)x, (_Float16)y};
  return __builtin_bit_cast(uint32_t, p);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16bit(float x, float y) {
  return F16 ? pack_f16(x, y) : pack_bf16(x, y);
}
// x and y rounded to 16 bits, and what the rounding left.
template <bool F16>
__device__ __forceinline__ uint32_t split16bit(float& x, float& y) {
  const uint32_t w = pack16bit<F16>(x, y);
  if constexpr (F16) {
    const f16x2 p = __builtin_bit_cast(f16x2, w);
    x -= (float)p.x;
    y -= (float)p.y;
  } else {
    x -= bf16_lo(w);
    y -= bf16_hi(w);
  }
  return w;
}

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 y, f32x4 acc) {
  if constexpr (F16)
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
__device__ __forceinline__ f32x2 e2m1_pair_f32(uint32_t w, int sel) {
  return sel == 0 ? e2m1_unpack2<0>(w) : sel == 1 ? e2m1_unpack2<1>(w) : sel == 2 ? e2m1_unpack2<2>(w) : e2m1_unpack2<3>(w);
}
// The E4M3 values of the two low bytes of w in fp16 (exact).
__device__ __forceinline__ f16x2 e4m3_pair_f16(uint32_t w) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, f16x2 y) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x) * y);
}

// Eight consecutive codes under one scale byte as an MFMA operand (F16: fp16,
// else bf16).
template <bool NV, bool F16>
__device__ __forceinline__ u32x4 convert8(uint32_t w, uint32_t scale_byte) {
  if constexpr (NV && !F16) {
    const float s = e4m3_decode(scale_byte);
    const f32x2 a = e2m1_unpack2<0>(w), b = e2m1_unpack2<1>(w), c = e2m1_unpack2<2>(w), d = e2m1_unpack2<3>(w);
    return u32x4{pack_bf16(a.x * s, a.y * s), pack_bf16(b.x * s, b.y * s), pack_bf16(c.x * s, c.y * s),
                 pack_bf16(d.x * s, d.y * s)};
  } else if constexpr (NV) {
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
template <bool NV, bool F16, int PAIRS>
__device__ __forceinline__ void convert_key_pair(uint32_t x, uint32_t y, uint32_t sx, uint32_t sy, uint32_t* out) {
  if constexpr (NV) {
    // the two keys' nibbles of one element side by side in a byte
    const uint32_t even = (x & 0x0f0f0f0fu) | ((y & 0x0f0f0f0fu) << 4);
    const uint32_t odd = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
    if constexpr (F16) {
      const f16x2 s = e4m3_pair_f16(sx | (sy << 8));
#pragma unroll
      for (int i = 0; i < PAIRS; i++) {
        out[2 * i] = mul_f16x2(e2m1_pair_f16(even, i), s);
        out[2 * i + 1] = mul_f16x2(e2m1_pair_f16(odd, i), s);
      }
    } else {
      const float fx = e4m3_decode(sx), fy = e4m3_decode(sy);
#pragma unroll
      for (int i = 0; i < PAIRS; i++) {
        const f32x2 p = e2m1_pair_f32(even, i), q = e2m1_pair_f32(odd, i);
        out[2 * i] = pack_bf16(p.x * fx, p.y * fy);
        out[2 * i + 1] = pack_bf16(q.x * fx, q.y * fy);
      }
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

// cap tanh(s / cap), with 1 / cap given. Below |x| = 0.6 (SMALL: known to be
// below) the score times tanh(x) / x = 1 + x^2 P(x^2), P of least relative
// error there (2^-28, found by reweighted least squares): small scores under a
// large cap keep all their bits, where 1 - 2 / (1 + e^2x) would be off by 2^-24
// of the cap. Above, that form, 1 where the exponential overflows.
constexpr float kSmallTanh = 0.6f;
template <bool SMALL>
__device__ __forceinline__ float soft_cap(float s, float cap, float inv_cap) {
  const float x = s * inv_cap, u = x * x;
  float p = -0.00589515548f;
  p = __builtin_fmaf(p, u, 0.0207959693f);
  p = __builtin_fmaf(p, u, -0.0537838303f);
  p = __builtin_fmaf(p, u, 0.133319244f);
  p = __builtin_fmaf(p, u, -0.333332986f);
  const float small = __builtin_fmaf(s * u, p, s);
  if constexpr (SMALL) return small;
  const float ax = __builtin_fabsf(x);
  const float t = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(ax * (2.0f * kLog2e)));
  return ax < kSmallTanh ? small : __builtin_copysignf(cap * t, s);
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
template <bool F16>
__device__ __forceinline__ float row_lse(float top, float sum) {
  return sum == 0.0f ? -__builtin_huge_valf() : kLn2 * ((F16 ? top - kF16Lift : top) + __builtin_amdgcn_logf(sum));
}

// A 32-key tile's codes and scale bytes: in LDS as the copies lay them down,
// and where a lane finds its part. DP: the head size the kernel is made for
// (64, 128, 256), FULL: the head size is DP itself, else it is smaller.
template <int DP, bool NV>
struct Tile {
  static constexpr int kBlk = NV ? 16 : 32;
  // K: words of 8 codes of one key per lane, elements g * DP/4 on, and the
  // scale bytes over them
  static constexpr int kKWords = DP / 32;
  static constexpr int kKScales = DP / 4 > kBlk ? DP / 4 / kBlk : 1;
  // V: elements per lane and key, the number of O tiles, and their words
  static constexpr int kChunkV = DP / 16;
  static constexpr int kVWords = DP > 128 ? 2 : 1;
  static constexpr int kPairs = kChunkV >= 8 ? 4 : 2;  // of elements, in a word

  // LDS slot: the keys' codes of both 16-key halves, the values', then the
  // scales in the order K half 0, K half 1, V half 0, V half 1
  static constexpr int kHalf = 16 * DP / 2;
  static constexpr int kVAt = 2 * kHalf, kScalesAt = 4 * kHalf;
  static constexpr int kSlot = kScalesAt + 4 * 16 * DP / kBlk;
  // copies of 64 x 16 bytes: kCopies of K, as many of V, one of all the scales
  static constexpr int kCopies = 2 * kHalf / 1024;
  static constexpr int kLoads = 2 * kCopies + 1;
  static __device__ __forceinline__ constexpr int k_scale(int w) {
    return w * 8 / kBlk < kKScales ? w * 8 / kBlk : 0;
  }
};

// Direct-to-LDS copy of 16 bytes per active lane: lane i's bytes at its
// address (or base + offset) land at LDS address lds + 16 i (lds
// wave-uniform, passed in m0). Inline assembly, so that the compiler, which
// cannot match copies in flight to what is read from LDS, adds no waits of
// its own: every wait on these copies is explicit below. The instruction has
// no output register. It writes m0, which cannot be named as clobbered; the
// compiler sets m0 itself right before each instruction of its own that reads
// it.
__device__ __forceinline__ void copy16(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(p), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}
__device__ __forceinline__ void copy16(const uint8_t* base, uint32_t offset, uint32_t lds) {
  // base and lds are wave-uniform
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  const uint64_t u = (uint64_t)hi << 32 | lo;
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(offset), "s"(u), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}
// LDS byte address of a __shared__ object
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
// s_waitcnt vmcnt(N) and lgkmcnt(0) (gfx9 encoding), the other counters free
template <int N>
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
  asm volatile("" ::: "memory");
}

// The cached rows of one sequence and kv head, copied to LDS tile by tile.
// Score row c of a half is its key turned = 4 (c % 4) + c / 4, so that lane
// (c, g) gets the scores of keys 4 i + g, and its reads of V fall on other LDS
// banks than those of the other g.
template <int DP, bool NV, bool FULL>
struct CacheReader {
  using T = Tile<DP, NV>;
  const KvAttnArgs& a;
  // Read through the scalar cache (the kernel never writes it): a vector load
  // would be waited for in order with the copies in flight.
  const __attribute__((address_space(4))) int32_t* table;
  int h, len, last16, D, row_codes, row_scales;
  uint32_t k_from, v_from;      // this lane's part of a copy of K, of V
  const uint8_t* scales_from;   // and of the scales: part 0 and 1 of K's
  int part;                     // halves, 2 and 3 of V's, 4 on none

  __device__ __forceinline__ CacheReader(const KvAttnArgs& a_, const RowTile& r, int h_, int lane) : a(a_) {
    h = h_;
    len = r.len;
    last16 = (len - 1) & ~15;  // the last 16 keys that exist
    table = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)(a.table + r.b * a.table_stride);
    D = FULL ? DP : a.c.dim;
    row_codes = D >> 1;
    row_scales = D / T::kBlk;
    const int c = lane & 15, g = lane >> 4, turned = 4 * (c & 3) + (c >> 2);
    // K of a whole head size: a lane copies what lane (c, g) will read, so
    // that these reads are linear; else, and V, as the rows lie
    constexpr int kPerHalf = T::kHalf / 16;  // lanes
    v_from = 16 * (lane % kPerHalf);
    k_from = !FULL       ? v_from
             : DP == 64  ? turned * row_codes + 16 * (g & 1)
             : DP == 128 ? turned * row_codes + 16 * g
                         : turned * row_codes + 32 * g;
    part = lane / row_scales;  // a half's scales are row_scales copies of 16 bytes
    scales_from = (part & 2 ? a.c.vs : a.c.ks) + 16 * (lane - part * row_scales);
  }

  // Pages of the two halves of the tile at kt. Sequences end inside pages and
  // tiles: a half past the last page is read from there.
  __device__ __forceinline__ int2 pages(int kt) const {
    const int i = __builtin_amdgcn_readfirstlane(min(kt, last16) >> a.c.page_shift);
    const int j = __builtin_amdgcn_readfirstlane(min(kt + 16, last16) >> a.c.page_shift);
    return make_int2(table[i], table[j]);
  }

  // Byte offsets of a half's codes and scales. 16 keys lie in one page, their
  // rows back to back.
  __device__ __forceinline__ void half_at(int key, int page, uint64_t& codes, uint64_t& scales) const {
    const uint32_t pg = (uint32_t)min(max(page, 0), (int)a.c.pages - 1);
    const uint32_t row = ((uint32_t)h << a.c.page_shift) + (min(key, last16) & ((1 << a.c.page_shift) - 1));
    codes = (uint64_t)pg * (uint64_t)a.c.codes_ps + row * (uint32_t)row_codes;
    scales = (uint64_t)pg * (uint64_t)a.c.scales_ps + row * (uint32_t)row_scales;
  }

  // Starts copies of the tile at kt into an LDS slot: those whose bit in
  // `which` is set (bit i: copy i of K, kCopies + i: of V; the scales always).
  // Keys past the sequence's end are copied as they lie in the last page:
  // their scores are masked, their values zeroed before use.
  __device__ __forceinline__ void copy(int kt, int2 page, uint32_t slot, int lane, uint32_t which) const {
    uint64_t c0, s0, c1, s1;
    half_at(kt, page.x, c0, s0);
    if (a.c.page_shift >= 5 && kt + 16 <= last16) {
      c1 = c0 + 16 * row_codes;  // a tile lies in one page
      s1 = s0 + 16 * row_scales;
    } else {
      half_at(kt + 16, page.y, c1, s1);
    }
    if constexpr (DP == 64) {
      // one copy for both halves
      const uint64_t at = lane < 32 ? c0 : c1;
      if (FULL || (int)v_from < 16 * row_codes) {
        if (which & 1) copy16(a.c.kc + at + k_from, slot);
        if (which & 2) copy16(a.c.vc + at + v_from, slot + T::kVAt);
      }
    } else {
      constexpr int kEach = T::kCopies / 2;  // copies of a half
#pragma unroll
      for (int i = 0; i < T::kCopies; i++) {
        const int sub = i / kEach, n = i % kEach;
        const uint64_t at = sub ? c1 : c0;
        if (FULL || (int)v_from + n * 1024 < 16 * row_codes) {
          if (which >> i & 1) copy16(a.c.kc + at, k_from + n * (FULL ? 16 : 1024), slot + sub * T::kHalf + n * 1024);
          if (which >> (T::kCopies + i) & 1)
            copy16(a.c.vc + at, v_from + n * 1024, slot + T::kVAt + sub * T::kHalf + n * 1024);
        }
      }
    }
    if (part < 4) copy16(scales_from + (part & 1 ? s1 : s0), slot + T::kScalesAt);
  }

  // Where in a slot this lane's codes and scale bytes of one key lie: word w
  // (scale i) of K of half 0, V (its scale) of the half's key 4 i + g.
  __device__ __forceinline__ uint32_t k_word(int c, int g, int w) const {
    if (FULL && DP == 64) return (g >> 1) * 256 + c * 16 + (g & 1) * 8 + 4 * w;
    if (FULL) return (w / 4) * 1024 + (16 * g + c) * 16 + 4 * (w % 4);
    const int d = g * (DP / 4) + 8 * w;  // past the head size: meets queries of 0
    return (4 * (c & 3) + (c >> 2)) * row_codes + (d < D ? d >> 1 : 0);
  }
  __device__ __forceinline__ uint32_t k_scale(int c, int g, int i) const {
    const int b = g * (DP / 4) / T::kBlk + i;
    return T::kScalesAt + (4 * (c & 3) + (c >> 2)) * row_scales + (FULL || b < row_scales ? b : 0);
  }
  __device__ __forceinline__ uint32_t v_code(int c, int g) const {
    const int d = T::kChunkV * c;  // past the head size: results not stored
    return T::kVAt + g * row_codes + (FULL || d < D ? d >> 1 : 0);
  }
  __device__ __forceinline__ uint32_t v_scale(int c, int g) const {
    const int d = T::kChunkV * c;
    return T::kScalesAt + 2 * 16 * row_scales + g * row_scales + (FULL || d < D ? d / T::kBlk : 0);
  }
};

// A V word in LDS: the codes of up to 8 elements of one key.
template <int DP>
__device__ __forceinline__ uint32_t v_word(const uint8_t* p, int w) {
  if constexpr (DP == 64) return *reinterpret_cast<const uint16_t*>(p);
  else return reinterpret_cast<const uint32_t*>(p)[w];
}

// RT tiles of 16 rows in one wave: their queries, running statistics and
// weighted sums.
template <int DP, bool NV, bool BF16, bool FULL, int RT>
struct Rows {
  static constexpr int kChunkV = DP / 16;
  static constexpr bool kF16 = NV && BF16;  // fp16 operands, else bf16
  static constexpr int kTerms = BF16 ? 1 : 3;  // of the queries and of the weights
  bool live[RT];
  int token[RT], head[RT];
  int my_lo[RT], my_hi[RT];  // the keys this lane's rows see
  int all_lo, all_hi;        // keys that every row sees
  bool large = false;        // a maximum of these rows passed kLargeScore
  u32x4 q[RT][kTerms][DP / 32];
  float score_scale[RT];
  f32x4 o[RT][kChunkV];
  float m[RT], l[RT];

  // Rows r.row0 on of kv head h.
  __device__ __forceinline__ void start(const KvAttnArgs& a, const RowTile& r, int h, int c, int g) {
    const int D = FULL ? DP : a.c.dim, G = a.group;
    all_hi = end_key(a, r.len, r.n, r.row0 / G);
    all_lo = first_key(a, r.len, r.n, min((r.row0 + 16 * RT - 1) / G, r.n - 1));
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
      const int row = r.row0 + 16 * rt + c;
      live[rt] = row < r.n * G;
      const int t = live[rt] ? row / G : r.n - 1;
      token[rt] = r.q0 + t;
      head[rt] = h * G + (live[rt] ? row - t * G : 0);
      my_hi[rt] = end_key(a, r.len, r.n, t);
      my_lo[rt] = first_key(a, r.len, r.n, t);
      m[rt] = kNoMax;
      l[rt] = 0.0f;
#pragma unroll
      for (int j = 0; j < kChunkV; j++) o[rt][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // queries, in the order of the K operand; a negative scale goes into them
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
      float x[DP / 4];
#pragma unroll
      for (int w = 0; w < DP / 32; w++) {
        const int d = g * (DP / 4) + 8 * w;
#pragma unroll
        for (int i = 0; i < 8; i++) x[8 * w + i] = 0.0f;
        if (live[rt] && d < D) {
          const int64_t at = (int64_t)token[rt] * a.q_ts_ + (int64_t)head[rt] * a.q_hs + d;
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
      float f = __builtin_fabsf(a.scale);
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
        f = __builtin_ldexpf(f * tensor_scale_of(a.c.k_ts, h), -up);
      }
#pragma unroll
      for (int k = 0; k < kTerms; k++) {
#pragma unroll
        for (int w = 0; w < DP / 32; w++) {
#pragma unroll
          for (int i = 0; i < 4; i++) q[rt][k][w][i] = split16bit<kF16>(x[8 * w + 2 * i], x[8 * w + 2 * i + 1]);
        }
      }
      score_scale[rt] = f * kLog2e;
    }
  }

  // The products s[rt][i] (key kt + 4 i + g, or TURNED: its pairs of keys begun g
  // pairs earlier, round the four) to weights in 16 bits, in the order of V's
  // operand; the statistics and sums follow.
  template <bool TURNED, bool CAP>
  __device__ __forceinline__ void weigh(const KvAttnArgs& a, int kt, int g, float s[RT][8], u32x4 pw[RT][kTerms]) {
    float factor[RT];  // of s, to scores in powers of two
#pragma unroll
    for (int rt = 0; rt < RT; rt++) factor[rt] = score_scale[rt];
    if (CAP && a.cap > 0.0f) {
      float top = 0.0f;
#pragma unroll
      for (int rt = 0; rt < RT; rt++) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          s[rt][i] *= score_scale[rt];
          top = __builtin_fmaxf(top, __builtin_fabsf(s[rt][i]));
        }
        factor[rt] = 1.0f;
      }
      // mostly all small (prompt of 4096 under a cap of 30: 221 us; both forms
      // for every score: 250)
      if (__any(top * a.inv_cap >= kSmallTanh)) {
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
#pragma unroll
          for (int i = 0; i < 8; i++) s[rt][i] = soft_cap<false>(s[rt][i], a.cap, a.inv_cap);
        }
      } else {
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
#pragma unroll
          for (int i = 0; i < 8; i++) s[rt][i] = soft_cap<true>(s[rt][i], a.cap, a.inv_cap);
        }
      }
    }
    if (partly_seen(kt) || large) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int key = key_of<TURNED>(kt, g, i >> 1, i & 1);
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
          s[rt][i] = key < my_hi[rt] && key >= my_lo[rt] ? s[rt][i] * factor[rt] : -__builtin_huge_valf();
      }
#pragma unroll
      for (int rt = 0; rt < RT; rt++) factor[rt] = 1.0f;
    }
    float top[RT];
    bool raise = false;
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
      top[rt] = s[rt][0];
#pragma unroll
      for (int i = 1; i < 8; i++) top[rt] = __builtin_fmaxf(top[rt], s[rt][i]);
      top[rt] *= factor[rt];
      raise = raise || top[rt] > m[rt] + kSlack;
    }
    if (__any(raise)) {
#pragma unroll
      for (int rt = 0; rt < RT; rt++) {
        top[rt] = __builtin_fmaxf(top[rt], xor_shfl<16>(top[rt]));
        top[rt] = __builtin_fmaxf(top[rt], xor_shfl<32>(top[rt]));
        const float raised = __builtin_fmaxf(m[rt], top[rt]);
        const float down = __builtin_amdgcn_exp2f(m[rt] - raised);
        l[rt] *= down;
#pragma unroll
        for (int j = 0; j < kChunkV; j++) o[rt][j] *= down;
        m[rt] = raised;
      }
      bool passed = false;
#pragma unroll
      for (int rt = 0; rt < RT; rt++) passed |= __builtin_fabsf(m[rt]) > kLargeScore && m[rt] != kNoMax;
      large = __any(passed);
      if (large) {
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
#pragma unroll
          for (int i = 0; i < 8; i++) s[rt][i] *= factor[rt];
          factor[rt] = 1.0f;
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
      const float base = kF16 ? m[rt] - kF16Lift : m[rt];
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; i++) p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][i], factor[rt], -base));
      l[rt] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
      for (int n = 0; n < kTerms; n++) {
#pragma unroll
        for (int i = 0; i < 4; i++) pw[rt][n][i] = split16bit<kF16>(p[2 * i], p[2 * i + 1]);
      }
    }
  }

  // s += K operand . queries (word w); sums += V operand j . weights.
  __device__ __forceinline__ void times_k(u32x4 kk, int w, f32x4 acc[RT]) const {
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
#pragma unroll
      for (int n = 0; n < kTerms; n++) acc[rt] = mfma16<kF16>(kk, q[rt][n][w], acc[rt]);
    }
  }
  __device__ __forceinline__ void times_v(u32x4 vv, int j, const u32x4 pw[RT][kTerms]) {
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
#pragma unroll
      for (int n = 0; n < kTerms; n++) o[rt][j] = mfma16<kF16>(vv, pw[rt][n], o[rt][j]);
    }
  }

  // The key of the tile at kt that half `odd` of operand word i stands for.
  template <bool TURNED>
  static __device__ __forceinline__ int key_of(int kt, int g, int i, int odd) {
    return kt + 8 * (TURNED ? (i - g) & 3 : i) + 4 * odd + g;
  }
  // Whether some row does not see some key of the tile at kt.
  __device__ __forceinline__ bool partly_seen(int kt) const { return kt + kTileKeys > all_hi || kt < all_lo; }

  __device__ __forceinline__ void sum_denominators() {
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
      l[rt] += xor_shfl<16>(l[rt]);
      l[rt] += xor_shfl<32>(l[rt]);
    }
  }
};

// A weight of 0 hides a value only if that is a number: an infinity or NaN that
// some rows see would reach the sums of those that do not. So in a tile that
// not every row sees whole, a key with such a value (a block whose scale is
// NaN, or 2^126 and more, which passes bf16 and fp32) gets values of 0 and a key
// of NaN, which makes NaN of the rows that see it and is masked for the others;
// keys past the sequence's end, which may hold anything, get values of 0.
//
// The bytes of four such scales, by their highest bits.
template <bool NV>
__device__ __forceinline__ uint32_t no_numbers(uint32_t scales) {
  const uint32_t low = scales & 0x7f7f7f7fu;
  return (NV ? low + 0x01010101u : (low + 0x03030303u) & scales) & 0x80808080u;
}
// Whether the tile at kt, in a wave's LDS slot y, has keys past the end or with
// such values.
template <int DP, bool NV, bool FULL>
__device__ __forceinline__ bool unsettled(const CacheReader<DP, NV, FULL>& in, const uint8_t* y, int kt, int lane) {
  using T = Tile<DP, NV>;
  if (kt + kTileKeys > in.len) return true;
  asm volatile("" : "+v"(lane));  // its addresses are not kept through the loop over tiles
  const uint32_t* vs = reinterpret_cast<const uint32_t*>(y + T::kScalesAt + 2 * 16 * in.row_scales);
  uint32_t found = 0u;
#pragma unroll
  for (int i = 0; i < (8 * DP / T::kBlk + 63) / 64; i++) {
    const int at = 64 * i + lane;
    if (at < 8 * in.row_scales) found |= no_numbers<NV>(vs[at]);
  }
  return __any(found != 0u);
}
// Lanes 0 to 31 settle a key each.
template <int DP, bool NV, bool FULL>
__device__ __forceinline__ void settle(const CacheReader<DP, NV, FULL>& in, uint8_t* y, int kt, int lane) {
  using T = Tile<DP, NV>;
  asm volatile("" : "+v"(lane));
  if (lane < kTileKeys) {
    uint8_t* ks = y + T::kScalesAt + lane * in.row_scales;
    uint8_t* vs = ks + 2 * 16 * in.row_scales;
    const bool past = kt + lane >= in.len;
    uint32_t found = 0u;
#pragma unroll 1
    for (int i = 0; i < in.row_scales; i++) found |= no_numbers<NV>(vs[i]);
    if (past || found) {
#pragma unroll 1
      for (int i = 0; i < in.row_scales; i++) {
        vs[i] = 0;
        if (!past) ks[i] = 255;
      }
    }
  }
  asm volatile("" ::: "memory");  // a wave's LDS accesses keep their order
}

// Few rows: a workgroup's LDS, its waves' tiles and afterwards their results.
template <int DP, bool NV, int NW>
union FewSpace {
  // tiles on their way or in use per wave
  static constexpr int kDepth = 2;
  uint8_t tiles[NW][kDepth][Tile<DP, NV>::kSlot];
  struct {
    float o[NW][16][DP + 4];
    float m[NW][16], l[NW][16];
  } join;
};

// RT * 16 rows of kv head h over their keys from c_lo (a multiple of
// kTileKeys) to c_hi, each wave every NW-th tile; the result to `out`, or
// (part) the partial result to a slot.
template <int DP, bool NV, bool BF16, bool FULL, int NW, int RT>
__device__ __forceinline__ void attend_few(const KvAttnArgs& a, const RowTile& r, int h, int c_lo, int c_hi,
                                           float* part, FewSpace<DP, NV, NW>& lds) {
  using T = Tile<DP, NV>;
  constexpr int kRows = 16 * RT;
  constexpr int kStep = kTileKeys * NW;
  constexpr int kDepth = FewSpace<DP, NV, NW>::kDepth;
  constexpr uint32_t kAllCopies = (1u << 2 * T::kCopies) - 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int D = FULL ? DP : a.c.dim, G = a.group;
  const CacheReader<DP, NV, FULL> in(a, r, h, lane);
  const uint32_t ring = lds_address(&lds.tiles[wave][0][0]);

  // This wave's tiles, kDepth of them on their way or in use (the first while
  // the queries are laid out); the page numbers come one earlier still. Past
  // its last tile a wave copies that one again rather than nothing, so that
  // the number of copies in flight is always the same.
  int kt = c_lo + kTileKeys * wave;
  const int last = kt + (c_hi - 1 - kt) / kStep * kStep;
  int2 ahead = make_int2(0, 0);
  if (kt < c_hi) {
#pragma unroll
    for (int i = 0; i < kDepth; i++)
      in.copy(min(kt + i * kStep, last), in.pages(min(kt + i * kStep, last)), ring + i * T::kSlot, lane, kAllCopies);
    ahead = in.pages(min(kt + kDepth * kStep, last));
  }
  Rows<DP, NV, BF16, FULL, RT> rows;
  rows.start(a, r, h, c, g);

  uint32_t slot = 0;
  for (; kt < c_hi; kt += kStep) {
    wait_copies<(kDepth - 1) * T::kLoads>();
    uint8_t* y = &lds.tiles[wave][0][0] + slot;
    if (rows.partly_seen(kt) && unsettled(in, y, kt, lane)) settle(in, y, kt, lane);
    float s[RT][8];
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      f32x4 acc[RT];
#pragma unroll
      for (int rt = 0; rt < RT; rt++) acc[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < T::kKWords; w++) {
        const uint32_t code = *reinterpret_cast<const uint32_t*>(y + sub * T::kHalf + in.k_word(c, g, w));
        const uint32_t scale = y[in.k_scale(c, g, T::k_scale(w)) + sub * 16 * in.row_scales];
        rows.times_k(convert8<NV, NV && BF16>(code, scale), w, acc);
      }
#pragma unroll
      for (int rt = 0; rt < RT; rt++) {
#pragma unroll
        for (int i = 0; i < 4; i++) s[rt][4 * sub + i] = acc[rt][i];
      }
    }
    uint32_t v[8][T::kVWords], vs[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int key = 16 * (i >> 2) + 4 * (i & 3);
      vs[i] = y[in.v_scale(c, g) + key * in.row_scales];
#pragma unroll
      for (int w = 0; w < T::kVWords; w++)
        v[i][w] = v_word<DP>(y + in.v_code(c, g) + (i >> 2) * T::kHalf + 4 * (i & 3) * in.row_codes, w);
    }
    u32x4 pw[RT][Rows<DP, NV, BF16, FULL, RT>::kTerms];
    rows.template weigh<false, true>(a, kt, g, s, pw);
#pragma unroll
    for (int w = 0; w < T::kVWords; w++) {
      uint32_t vt[4][2 * T::kPairs];
#pragma unroll
      for (int i = 0; i < 4; i++)
        convert_key_pair<NV, NV && BF16, T::kPairs>(v[2 * i][w], v[2 * i + 1][w], vs[2 * i], vs[2 * i + 1], vt[i]);
#pragma unroll
      for (int j = 0; j < 2 * T::kPairs; j++) rows.times_v(u32x4{vt[0][j], vt[1][j], vt[2][j], vt[3][j]}, 8 * w + j, pw);
    }
    // the slot has been read: the next tile's copies may land in it
    wait_lds();
    in.copy(min(kt + kDepth * kStep, last), ahead, ring + slot, lane, kAllCopies);
    ahead = in.pages(min(kt + (kDepth + 1) * kStep, last));
    slot = slot == (kDepth - 1) * T::kSlot ? 0 : slot + T::kSlot;
  }
  wait_copies<0>();
  rows.sum_denominators();
  __syncthreads();

  // O tile j holds of row c the elements kChunkV * (4g + i) + j
#pragma unroll
  for (int rt = 0; rt < RT; rt++) {
    if (rt) __syncthreads();
    if (g == 0) {
      lds.join.m[wave][c] = rows.m[rt];
      lds.join.l[wave][c] = rows.l[rt];
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
      for (int j = 0; j < T::kChunkV; j++) lds.join.o[wave][c][(4 * g + i) * T::kChunkV + j] = rows.o[rt][j][i];
    }
    __syncthreads();
    constexpr int kEach = 16 * DP / (64 * NW);  // elements a thread joins
    constexpr int kPerRow = DP / kEach;
    const int jr = threadIdx.x / kPerRow, d = threadIdx.x % kPerRow * kEach;
    const int jrow = r.row0 + 16 * rt + jr;
    if (jrow >= r.n * G || d >= D) continue;
    const int jt = jrow / G, jhead = h * G + jrow - jt * G;
    float top = lds.join.m[0][jr];
#pragma unroll
    for (int w = 1; w < NW; w++) top = __builtin_fmaxf(top, lds.join.m[w][jr]);
    float sum = 0.0f, acc[kEach];
#pragma unroll
    for (int j = 0; j < kEach; j++) acc[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const float f = __builtin_amdgcn_exp2f(lds.join.m[w][jr] - top);
      sum += f * lds.join.l[w][jr];
#pragma unroll
      for (int j = 0; j < kEach; j++) acc[j] += f * lds.join.o[w][jr][d + j];
    }
    if (part) {
      const int pr = 16 * rt + jr;
#pragma unroll
      for (int j = 0; j < kEach; j++) part[pr * D + d + j] = acc[j];
      if (d == 0) {
        part[kRows * D + pr] = top;
        part[kRows * (D + 1) + pr] = sum;
      }
    } else {
      const float f = row_factor<NV>(a, h, sum);
#pragma unroll
      for (int j = 0; j < kEach; j++) acc[j] *= f;
      store_row<BF16, kEach>(a, r.q0 + jt, jhead, d, acc);
      if (d == 0 && a.lse) a.lse[(int64_t)(r.q0 + jt) * a.q_heads + jhead] = row_lse<NV && BF16>(top, sum);
    }
  }
}

// Waves a SIMD that the registers of the form for few rows allow: past heads of
// 128 two for bf16, so that two workgroups stay on a CU (8 sequences to 30000 of
// heads of 256: 49 us, 65 with one; of 192: 43 against 67). TWO: the launch has
// no more than two anyway (runs, or eight waves a workgroup past heads of 64),
// which fp32's terms need there (130001 keys: 24.8 us, 27.6 with registers for
// three; 300 sequences to 700 in four waves: 67 with two, 57 with three).
constexpr int few_waves(int dp, int rt, bool bf16, bool two) {
  return dp == 256 ? (bf16 ? 2 : 1) : dp == 128 && (rt > 1 || (!bf16 && two)) ? 2 : 3;
}

// One workgroup for each row tile and kv head.
//
// A tile of 32 keys of 128 elements in MXFP4 costs a wave about 190 vector
// instructions, 64 of them conversions (3.7 ns each, others 2 to 2.4), and 16
// matrix instructions: 0.57 us with two waves a SIMD. So little work is bound
// by the launch, the chain of first loads (lengths, page, tile: 6 us with one
// key) and the tiles one wave goes through: one sequence of 997 keys, 4 tiles
// a wave, 10 us. 32 sequences to 4096 keys (98 MB, 32 heads over 8 of 128):
// 27 us, 4.6 TB/s after the first 6 us, where a copy of that size reaches 4.8.
// Sixteen waves a workgroup: 31 us; a ring of three or four tiles a wave, or
// all of a tile's LDS reads ahead of its first use: no faster.
template <int DP, bool NV, bool BF16, bool FULL, int NW, int RT>
__global__ __launch_bounds__(64 * NW, few_waves(DP, RT, BF16, NW > 4)) void kv_attn_kernel(KvAttnArgs a) {
  __shared__ __attribute__((aligned(16))) FewSpace<DP, NV, NW> lds;
  const int h = blockIdx.x % a.c.heads, tile = blockIdx.x / a.c.heads;
  RowTile r;
  if (!find_tile<16 * RT>(a, tile, r)) return;
  attend_few<DP, NV, BF16, FULL, NW, RT>(a, r, h, r.lo, r.hi, nullptr, lds);
}

// The balanced form: one workgroup for each run of key tiles, two a CU. 64
// sequences to 16384 keys (699 MB, 64 heads over 8 of 128): 135 us, 5.2 TB/s,
// and 7 to join; reads of 4 to 8 KB from anywhere reach 5.7 to 5.9 here.
template <int DP, bool NV, bool BF16, bool FULL, int NW, int RT>
__global__ __launch_bounds__(64 * NW, few_waves(DP, RT, BF16, true)) void kv_attn_runs_kernel(KvAttnArgs a, int least) {
  constexpr int kRows = 16 * RT;
  __shared__ __attribute__((aligned(16))) FewSpace<DP, NV, NW> lds;
  const WorkScan<kRows> scan(a, 0);
  const int total = total_work<kRows>(a, scan);
  const int per = run_length(total, gridDim.x, least);
  int at = (int)min((int64_t)blockIdx.x * per, (int64_t)total);
  int left = min(per, total - at);
  if (left <= 0) return;
  SeqWork w;
  int before;
  if (!find_work<kRows, false>(a, scan, at, w, before)) return;
  int item = at / w.span, k = at - item * w.span;
  while (true) {
    const int take = min(w.span - k, left);
    RowTile r;
    r.b = w.b;
    r.q0 = w.q0;
    r.n = w.n;
    r.len = w.len;
    r.row0 = item / a.c.heads * kRows;
    tile_keys(a, kRows, r);
    const int c_lo = max(w.lo + k * kTileKeys, r.lo), c_hi = min(w.lo + (k + take) * kTileKeys, r.hi);
    float* part =
        take == w.span ? nullptr : a.ws + (int64_t)(2 * blockIdx.x + (k == 0 ? 1 : 0)) * (kRows * (a.c.dim + 2));
    attend_few<DP, NV, BF16, FULL, NW, RT>(a, r, item % a.c.heads, c_lo, c_hi, part, lds);
    left -= take;
    if (left == 0) return;
    k = 0;
    if (++item == w.row_tiles * a.c.heads) {
      item = 0;
      do {
        if (w.b + 1 >= a.batch) return;
        w = seq_work<kRows>(a, w.b + 1);
      } while (w.row_tiles == 0);
    }
    __syncthreads();  // the join's LDS is used again
  }
}

// 16-row tiles of a wave in the form for many rows. Three leave registers for
// two waves a SIMD instead of three: 590 against 559 us (the prompt of 8192
// below), and at heads of 64 327 against 314; past 128 three do not fit, and one
// is a third slower (1226 against 820 us, 4096 queries over 8192).
constexpr int kManyTiles = 2;

template <int DP, bool NV>
struct ManySpace {
  static constexpr int kRing = 4;  // raw tiles: one being converted, two on their way, one being started
  static constexpr int kKParts = 2 * (DP / 32), kVParts = DP / 16;  // operands of a tile, 64 lanes x 16 bytes each
  uint8_t raw[kRing][Tile<DP, NV>::kSlot];
  u32x4 k[2][kKParts][64];
  u32x4 v[2][kVParts][64];
};

// Many rows: NW waves with RT tiles of 16 rows each. CAP: under a softcap. (Its
// registers beside the loop's own, asked for in one kernel by a.cap: prompts of
// 4096 without one, heads of 96 197 against 184 us, of 256 340 against 306.)
//
// Bound by vector and matrix instructions together (issuing 56 and 40 % of the
// SIMDs' cycles by the counters, one or the other waiting for the rest): a
// weight costs an fma, an exponential (9.9 ns a wave's 64) and its parts of a
// maximum, a sum and a conversion, and each tile's conversion comes on top,
// which is why waves share it through LDS (each on its own: 737 us with two row
// tiles, then 620 in this form, for a prompt of 8192 of 32 heads over 8 of 128).
// LDS comes next (42 %): four waves read 64 KB of operands a tile. With every
// conversion's access on all of its banks 573 us, 960 TFLOP/s of the pairs seen;
// a large library product of bf16 runs at 1140. The next scores beside this
// tile's softmax within a wave were slower (620 to 695 us). Conversion and the
// product with V go before other waves' work: 4 x up to 1024 queries over up to
// 6000 keys (8 heads a kv head) took 312 us without and 286 with that, 272 now,
// 750 TFLOP/s: all 752 workgroups are on the GPU from the start, of 51 to 188
// key tiles each, and the fullest CU has 446 where the mean is 385.
template <int DP, bool NV, bool FULL, bool CAP>
__global__ __launch_bounds__(256, DP == 256 ? 1 : DP == 64 ? 4 : 3) void kv_attn_many_kernel(KvAttnArgs a) {
  using T = Tile<DP, NV>;
  using Space = ManySpace<DP, NV>;
  constexpr int NW = 4, RT = kManyTiles;
  constexpr int kRows = 16 * RT * NW;
  __shared__ __attribute__((aligned(16))) Space lds;
  // The last rows have the most keys under a causal order: they begin first.
  const int back = gridDim.x - 1 - blockIdx.x;
  const int h = back % a.c.heads;
  RowTile r;
  if (!find_tile<kRows>(a, back / a.c.heads, r)) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int D = FULL ? DP : a.c.dim;
  const CacheReader<DP, NV, FULL> in(a, r, h, lane);
  const int first = r.lo, end = r.hi;  // of the workgroup's keys
  const int last = first + (end - 1 - first) / kTileKeys * kTileKeys;
  // this wave's copies of a tile: every NW-th
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < 2 * T::kCopies; i++) mine |= i % NW == wave ? 1u << i : 0u;
  constexpr int kLoads = 2 * T::kCopies / NW + 1;  // per wave and tile, at least
  const uint32_t raw = lds_address(&lds.raw[0][0]);

  // This wave's quarter of a tile's conversion: a fourth of the K words of both
  // halves (heads of 64: one of the two words of half wave / 2), and the key
  // pair `wave` of V, a fourth of each of its operands. Which word, and which
  // fourth, moves on with g: lanes lie 16 bytes apart, and one and the same word
  // of each would meet 16 of the 64 banks only (prompt of 8192: 612 against 563
  // us). K's rows lie in the order that this gives the weights.
  uint32_t k_to[2];
#pragma unroll
  for (int sub = 0; sub < 2; sub++) {
    const int pair = (2 * sub + (c >> 1 & 1) + (c >> 2)) & 3;
    k_to[sub] = (pair >> 1) * T::kKWords * 64 + 16 * g + (c & 12) + 2 * (pair & 1) + (c & 1);
  }
  // Whether some row of the workgroup does not see some key of a tile.
  const int all_hi = end_key(a, r.len, r.n, r.row0 / a.group);
  const int all_lo = first_key(a, r.len, r.n, min((r.row0 + kRows - 1) / a.group, r.n - 1));
  auto partly_seen = [=](int kt) { return kt + kTileKeys > all_hi || kt < all_lo; };
  auto convert = [&](int kt, uint8_t* y, int to) {
    if (partly_seen(kt) && unsettled(in, y, kt, lane)) {  // all waves or none
      wait_lds();
      __syncthreads();
      if (wave == 0) settle(in, y, kt, lane);
      wait_lds();
      __syncthreads();
    }
    if constexpr (T::kKWords == 2) {
      const int sub = wave >> 1, w = (wave + (g >> 1)) & 1;
      const uint32_t code = *reinterpret_cast<const uint32_t*>(y + sub * T::kHalf + in.k_word(c, g, w));
      (&lds.k[to][w][0])[k_to[sub]] = convert8<NV, NV>(code, y[in.k_scale(c, g, 0) + sub * 16 * in.row_scales]);
    } else {
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
#pragma unroll
        for (int i = 0; i < T::kKWords / 4; i++) {
          const int w = ((wave + g) & 3) + 4 * i;
          const uint32_t code = *reinterpret_cast<const uint32_t*>(y + sub * T::kHalf + in.k_word(c, g, w));
          const uint32_t scale = y[in.k_scale(c, g, T::k_scale(w)) + sub * 16 * in.row_scales];
          (&lds.k[to][w][0])[k_to[sub]] = convert8<NV, NV>(code, scale);
        }
      }
    }
    // keys 16 sub + 4 i + g of the pair, i = 2 (wave % 2) and the next
    const int sub = wave >> 1, i = 2 * (wave & 1);
    const uint8_t* yv = y + in.v_code(c, g) + sub * T::kHalf + 4 * i * in.row_codes;
    const uint8_t* ys = y + in.v_scale(c, g) + (16 * sub + 4 * i) * in.row_scales;
    const uint32_t s0 = ys[0], s1 = ys[4 * in.row_scales];
#pragma unroll
    for (int w = 0; w < T::kVWords; w++) {
      const uint32_t x0 = v_word<DP>(yv, w), x1 = v_word<DP>(yv + 4 * in.row_codes, w);
      uint32_t vt[2 * T::kPairs];
      convert_key_pair<NV, NV, T::kPairs>(x0, x1, s0, s1, vt);
#pragma unroll
      for (int j = 0; j < 2 * T::kPairs; j++)
        reinterpret_cast<uint32_t*>(&lds.v[to][8 * w + j][lane])[(wave + g) & 3] = vt[j];
    }
  };
  auto slot_of = [](int n) { return n % Space::kRing * T::kSlot; };

  if (first < end) {
#pragma unroll
    for (int i = 0; i < 3; i++) {
      const int kt = min(first + i * kTileKeys, last);
      in.copy(kt, in.pages(kt), raw + slot_of(i), lane, mine);
    }
  }
  int2 ahead = make_int2(0, 0);
  if (first < end) ahead = in.pages(min(first + 3 * kTileKeys, last));

  r.row0 += 16 * RT * wave;
  const bool idle = r.row0 >= r.n * a.group;  // no rows for this wave: it only helps
  if (idle) r.row0 = 0;
  tile_keys(a, 16 * RT, r);
  Rows<DP, NV, true, FULL, RT> rows;
  rows.start(a, r, h, c, g);
  if (first < end) {
    wait_copies<2 * kLoads>();
    __syncthreads();
    convert(first, &lds.raw[0][0], 0);
    wait_copies<kLoads>();
    wait_lds();
    __syncthreads();
  }
  int n = 0;
  for (int kt = first; kt < end; kt += kTileKeys, n++) {
    // the tile after the next two begins its way, the next one is converted
    in.copy(min(kt + 3 * kTileKeys, last), ahead, raw + slot_of(n + 3), lane, mine);
    ahead = in.pages(min(kt + 4 * kTileKeys, last));
    __builtin_amdgcn_s_setprio(1);
    convert(min(kt + kTileKeys, last), &lds.raw[0][0] + slot_of(n + 1), (n + 1) & 1);
    __builtin_amdgcn_s_setprio(0);
    if (!idle && kt < r.hi && kt + kTileKeys > r.lo) {
      float s[RT][8];
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
        f32x4 acc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; rt++) acc[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < T::kKWords; w++) rows.times_k(lds.k[n & 1][sub * T::kKWords + w][lane], w, acc);
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
#pragma unroll
          for (int i = 0; i < 4; i++) s[rt][4 * sub + i] = acc[rt][i];
        }
      }
      u32x4 pw[RT][1];
      rows.template weigh<true, CAP>(a, kt, g, s, pw);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int j = 0; j < T::kChunkV; j++) rows.times_v(lds.v[n & 1][j][lane], j, pw);
      __builtin_amdgcn_s_setprio(0);
    }
    // the tile after next and what the waves wrote is there for all
    wait_copies<kLoads>();
    wait_lds();
    __syncthreads();
  }
  wait_copies<0>();
  if (idle) return;
  rows.sum_denominators();
#pragma unroll
  for (int rt = 0; rt < RT; rt++) {
    const float f = row_factor<NV>(a, h, rows.l[rt]);
    if (!rows.live[rt]) continue;
    // a lane has 4 kChunkV elements in a row
#pragma unroll
    for (int i = 0; i < 4; i++) {
      float y[T::kChunkV];
#pragma unroll
      for (int j = 0; j < T::kChunkV; j++) y[j] = rows.o[rt][j][i] * f;
      const int d = T::kChunkV * (4 * g + i);
      if (d < D) store_row<true, T::kChunkV>(a, rows.token[rt], rows.head[rt], d, y);
    }
    if (g == 0 && a.lse) a.lse[(int64_t)rows.token[rt] * a.q_heads + rows.head[rt]] = row_lse<NV>(rows.m[rt], rows.l[rt]);
  }
}

// Joins COLS columns of the partial results of one row of one item, if it has
// any: COLS / 4 lanes take four elements each, and the rest of the workgroup
// every kGroups-th partial result. Bound by latency: 6 to 7 us, 4 of them what
// any second launch takes.
template <int DP, bool NV, bool BF16, int RT, int THREADS, int COLS>
__global__ __launch_bounds__(THREADS) void kv_attn_join_kernel(KvAttnArgs a, int runs, int least, int rows_each) {
  constexpr int kRows = 16 * RT;
  constexpr int kLanes = COLS / 4, kGroups = THREADS / kLanes;
  __shared__ float s_acc[kGroups][COLS + 4];
  __shared__ float s_m[kGroups], s_l[kGroups];
  const int jr = blockIdx.x % rows_each;
  int item = blockIdx.x / rows_each, before;
  SeqWork w;
  const WorkScan<kRows> scan(a, 0);
  if (!find_work<kRows, true>(a, scan, item, w, before)) return;
  const int per = run_length(total_work<kRows>(a, scan), runs, least);
  const int begin = before + item * w.span;
  const int run0 = begin / per, n = (begin + w.span - 1) / per - run0 + 1;
  if (n == 1) return;
  const int h = item % a.c.heads;
  const int D = a.c.dim, G = a.group;
  const int row = item / a.c.heads * kRows + jr;
  if (row >= w.n * G) return;
  const int t = row / G, head = h * G + row - t * G;
  const int64_t step = kRows * (D + 2);
  const int grp = threadIdx.x / kLanes, dl = threadIdx.x % kLanes * 4, d = blockIdx.y * COLS + dl;
  float top = kNoMax, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (d < D) {
#pragma unroll 4
    for (int k = grp; k < n; k += kGroups) {
      const float* p = a.ws + (int64_t)(2 * (run0 + k) + (k == 0 ? 1 : 0)) * step;
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
  if (dl == 0) {
    s_m[grp] = top;
    s_l[grp] = sum;
  }
  *reinterpret_cast<float4*>(&s_acc[grp][dl]) = acc;
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
    const float4 v = *reinterpret_cast<const float4*>(&s_acc[k][dl]);
    y[0] += f * v.x;
    y[1] += f * v.y;
    y[2] += f * v.z;
    y[3] += f * v.w;
  }
  const float f = row_factor<NV>(a, h, sum);
#pragma unroll
  for (int j = 0; j < 4; j++) y[j] *= f;
  store_row<BF16, 4>(a, w.q0 + t, head, d, y);
  if (d == 0 && a.lse) a.lse[(int64_t)(w.q0 + t) * a.q_heads + head] = row_lse<NV && BF16>(all, sum);
}

namespace {
constexpr int kWaves = 4;
// waves of the wide form: as many as its registers allow (heads past 128: no wide form)
constexpr int wide_waves(int dp) { return dp <= 128 ? 8 : kWaves; }
// Most 16-row tiles of a wave in the form for few rows.
constexpr int few_tiles(int dp, bool bf16) { return bf16 && dp <= 128 ? 2 : 1; }
}  // namespace

// Lengths and offsets are on the device: max_len stands for every length, the
// mean rows for every sequence's. A bound of 131072 in place of the lengths: one
// sequence of 997 keys 11.0 us instead of 10.1, 32 to 4096 31.3 instead of 28.6.
// A prompt of 4096 beside forty tokens over 16384 keys: 634 us, 319 in two calls.
KvAttnPlan plan_kv_attention(const KvAttnArgs& a) {
  KvAttnPlan p{};
  const int64_t rows = a.tokens * a.group;
  const int64_t cus = device_cu_count();
  // Many rows a sequence, and enough of them for two workgroups a CU (heads of
  // up to 64 and more than a few tiles of keys: three): the form for many. Fewer
  // rows: each key tile's conversion and barrier serve too few (8 x 448 queries
  // of 20 heads of 64 over 1500 keys: 58 us in that form, 43 in the other); fewer
  // workgroups: the longest of them, whose keys nobody shares, set the time.
  // That form against the other, 32 heads over 8, at 512 workgroups and more:
  // heads of 128, prompts of 2 x 1024 58 against 63 us, 8 x 256 27 against 44, 2 x 2048
  // 118 against 159 (2048 alone: 92 against 86); heads of 64, 8 x 256 18 against 27, but 2048
  // 67 against 54; heads of 256, 2048 164 against 182. Below that: heads of 128, 1024
  // queries over 6000 225 against 145; heads of 256, 1536 over 8192 894 against 628.
  constexpr int kManyRows = 16 * kWaves * kManyTiles;
  const int64_t fill = (a.c.dim <= 64 && a.max_len > 512 ? 3 : 2) * cus;
  if (a.bf16 && a.offs && rows >= 128 * a.batch && (rows / kManyRows + a.batch / 2) * a.c.heads >= fill) {
    p.many = true;
    p.waves = kWaves;
    p.tiles = rows / kManyRows + a.batch;
    return p;
  }
  // Few. Keys a tile can see at most: all, or the windows of its queries.
  int64_t keys = a.max_len;
  if (a.window > 0) {
    const int64_t w = a.window + 32 + kTileKeys;
    keys = keys < w ? keys : w;
  }
  const int wide = wide_waves(a.c.dim);
  const int64_t each = keys / (wide * kTileKeys);  // key tiles of a wave of the wide form
  // Two row tiles share the conversion of their keys, but make half as many
  // workgroups and leave fewer waves a SIMD. They are taken where enough
  // workgroups are left (8 x 448 queries over 1500 keys, 20 heads of 64: 40
  // against 46 us), where one row tile each would need a second round of the
  // wide form (24 x 5 queries over 3000, heads of 128: 28 against 39; but 16 x 5
  // over 6000 of 4 kv heads, one round: 42 against 34), and for the runs of long
  // keys where there is work for them all (60 queries over 20000: 53 against 58;
  // but 16 over 8192: 23 against 21).
  auto tiles = [&](int64_t per) { return a.batch * ((rows / a.batch + per - 1) / per) * a.c.heads; };
  p.few_tiles = 1;
  if (rows > 16 * a.batch &&
      (tiles(32) >= 4 * cus ||
       (tiles(16) <= 2 * cus && (tiles(16) > cus || (each > 24 && tiles(16) >= cus / 4)))))
    p.few_tiles = few_tiles(a.c.dim, a.bf16);
  const int per = 16 * p.few_tiles;
  p.tiles = a.offs ? rows / per + a.batch : a.batch * ((a.group + per - 1) / per);
  const int64_t items = p.tiles * a.c.heads;
  p.waves = kWaves;
  // Little work, or at most a few tiles more for some workgroups than for
  // others: one launch whose workgroups have many waves, rather than runs and
  // a second launch to join them (24 sequences of 5 queries over 3000 keys:
  // 20 against 28 us; 32 to 4096 keys: 27 against 32). Where most CUs would
  // have no workgroup, only up to 8 tiles a wave.
  if (items <= 4 * cus && each <= (2 * items >= cus ? 24 : 8)) {
    p.waves = wide;
    return p;
  }
  // Enough items of few keys: the order in which workgroups end evens them out.
  // (Key tiles are counted in 32 bits, whatever the offsets are on the device.)
  const int64_t span = (a.max_len + kTileKeys - 1) / kTileKeys + 1;
  const int64_t most = (a.offs ? a.batch * (rows / per + 1) : p.tiles) * a.c.heads;
  if (items >= 4 * cus || keys <= 8 * kWaves * kTileKeys || most >= (int64_t(1) << 31) / span) return p;
  p.runs = 2 * cus;
  p.least = 2 * kWaves;
  p.ws = (size_t)(2 * p.runs) * (size_t)(per * (a.c.dim + 2)) * sizeof(float);
  return p;
}

template <int DP, bool NV, bool BF16, bool FULL, int RT>
static void launch_few(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  constexpr int kWide = wide_waves(DP);
  const int64_t items = p.tiles * a.c.heads;
  const dim3 grid((unsigned)items);
  if (p.runs > 0) {
    const int runs = (int)p.runs, least = (int)p.least;
    hipLaunchKernelGGL((kv_attn_runs_kernel<DP, NV, BF16, FULL, kWaves, RT>), dim3(runs), dim3(64 * kWaves), 0, s, a,
                       least);
    const int each = !a.offs && a.group < 16 * RT ? a.group : 16 * RT;
    const dim3 rows((unsigned)(items * each));
    // few partial results each: more threads would have nothing to do; many
    // (256 of a row of 128): 32 columns a workgroup (512 threads for all of
    // them: 22.3 against 21.8 us, 130001 keys)
    if (runs <= 8 * items)
      hipLaunchKernelGGL((kv_attn_join_kernel<DP, NV, BF16, RT, 128, DP>), rows, dim3(128), 0, s, a, runs, least, each);
    else
      hipLaunchKernelGGL((kv_attn_join_kernel<DP, NV, BF16, RT, 256, 32>), dim3(rows.x, (a.c.dim + 31) / 32),
                         dim3(256), 0, s, a, runs, least, each);
  } else if (p.waves == kWaves) {
    hipLaunchKernelGGL((kv_attn_kernel<DP, NV, BF16, FULL, kWaves, RT>), grid, dim3(64 * kWaves), 0, s, a);
  } else {
    hipLaunchKernelGGL((kv_attn_kernel<DP, NV, BF16, FULL, kWide, RT>), grid, dim3(64 * kWide), 0, s, a);
  }
}

template <int DP, bool NV, bool BF16, bool FULL>
static hipError_t launch_rows(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  if (p.many) {
    if constexpr (BF16) {
      const dim3 grid((unsigned)(p.tiles * a.c.heads)), block(64 * kWaves);
      if (a.cap > 0.0f) hipLaunchKernelGGL((kv_attn_many_kernel<DP, NV, FULL, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((kv_attn_many_kernel<DP, NV, FULL, false>), grid, block, 0, s, a);
    }
  } else if (p.few_tiles == 1) {
    launch_few<DP, NV, BF16, FULL, 1>(a, p, s);
  } else {
    launch_few<DP, NV, BF16, FULL, few_tiles(DP, BF16)>(a, p, s);
  }
  return hipGetLastError();
}

template <int DP, bool NV, bool BF16>
static hipError_t launch_full(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  return a.c.dim == DP ? launch_rows<DP, NV, BF16, true>(a, p, s) : launch_rows<DP, NV, BF16, false>(a, p, s);
}

template <int DP>
static hipError_t launch_dim(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  if (a.c.nvfp4) return a.bf16 ? launch_full<DP, true, true>(a, p, s) : launch_full<DP, true, false>(a, p, s);
  return a.bf16 ? launch_full<DP, false, true>(a, p, s) : launch_full<DP, false, false>(a, p, s);
}

hipError_t launch_kv_attention(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t s) {
  if (a.c.dim <= 64) return launch_dim<64>(a, p, s);
  if (a.c.dim <= 128) return launch_dim<128>(a, p, s);
  return launch_dim<256>(a, p, s);
}

}  // namespace fp4impl
