// moe_rows.hip -- (token, expert) pairs sorted by expert, the tokens' rows
// carried there, and the experts' rows brought back.
//
// Pair p = t * top_k + j is slot j of token t. group: a stable counting sort,
// place[p] = the pair's row, order[r] = row r's pair, offsets[e] = expert e's
// first row; pairs of no expert come last. dispatch: rows[place[p]] = x[t].
// combine: out[t] = sum_j w[p] rows[place[p]], in order of j.
//
// All are bound by memory, and the sort by latency. No sum and no place depends
// on the order in which workgroups or atomics run.
#include "fp4_device.h"
#include "launch.h"

namespace fp4impl {
using namespace fp4dev;

namespace {

constexpr int kGroupWaves = 16;                     // of a workgroup that sorts
constexpr int kGroupTurn = 64 * kGroupWaves;        // pairs of a round

// The wave's lanes whose id is this lane's: one ballot for each bit of an id.
__device__ __forceinline__ uint64_t same_id(int id, int bits) {
  uint64_t m = __builtin_amdgcn_ballot_w64(true);
  for (int i = 0; i < bits; i++) {
    const uint64_t b = __builtin_amdgcn_ballot_w64((id >> i) & 1);
    m &= (id >> i) & 1 ? b : ~b;
  }
  return m;
}

// A wave's lanes see what its other lanes wrote to LDS.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The workgroup's pairs, R times 64 consecutive ones for each wave; the lane's
// in registers, as buckets (a.experts: no expert; -1: no pair).
template <int R>
struct Pairs {
  int bucket[R];
  int first;  // the lane's pair of round 0
  __device__ __forceinline__ Pairs(const GroupArgs& a) {
    const int n = (int)a.pairs;
    first = blockIdx.x * (R * kGroupTurn) + (threadIdx.x >> 6) * (R * 64) + (threadIdx.x & 63);
#pragma unroll
    for (int r = 0; r < R; r++) bucket[r] = a.ids[first + r * 64 < n ? first + r * 64 : 0];
#pragma unroll
    for (int r = 0; r < R; r++) {
      const int e = (unsigned)bucket[r] < (unsigned)a.experts ? bucket[r] : a.experts;
      bucket[r] = first + r * 64 < n ? e : -1;
    }
  }
};

// counts[w * n + e] = pairs of bucket e in wave w's part, n the buckets
// rounded up to even: 16 bits each, added to by halves of words.
__device__ __forceinline__ int padded(int buckets) { return buckets + (buckets & 1); }
template <int R>
__device__ __forceinline__ void count_parts(const GroupArgs& a, const Pairs<R>& p, uint32_t* words) {
  const int n = padded(a.experts + 1);
  for (int i = threadIdx.x; i < n / 2 * kGroupWaves; i += 64 * kGroupWaves) words[i] = 0;
  __syncthreads();
  uint32_t* mine = words + (threadIdx.x >> 6) * (n / 2);
#pragma unroll
  for (int r = 0; r < R; r++) {
    if (p.bucket[r] >= 0) atomicAdd(&mine[p.bucket[r] >> 1], p.bucket[r] & 1 ? 1u << 16 : 1u);
  }
  __syncthreads();
}

}  // namespace

// Each workgroup's pairs of each bucket, for the scan that follows.
template <int R>
__global__ __launch_bounds__(64 * kGroupWaves) void group_count_kernel(GroupArgs a) {
  extern __shared__ uint32_t lds[];
  const Pairs<R> pairs(a);
  count_parts(a, pairs, lds);
  const uint16_t* counts = reinterpret_cast<uint16_t*>(lds);
  const int n = a.experts + 1;
  for (int e = threadIdx.x; e < n; e += 64 * kGroupWaves) {
    uint32_t sum = 0;
    for (int w = 0; w < kGroupWaves; w++) sum += counts[w * padded(n) + e];
    a.counts[(int64_t)blockIdx.x * n + e] = sum;
  }
}

// Scan and placement: a pair's row is its expert's first, and the pairs of that
// expert in earlier workgroups, in earlier waves and in earlier lanes (ballots).
// Bound by its chain of dependent steps and, at 16384 pairs, by scattered
// 4-byte stores: 128 pairs 2.7 us, 16384 pairs 3.0 + 4.6. With one workgroup the counts are its own; with more
// they come from group_count_kernel, and each workgroup adds up what lies
// before it.
template <int R>
__global__ __launch_bounds__(64 * kGroupWaves) void group_place_kernel(GroupArgs a) {
  extern __shared__ uint32_t lds[];
  const int n = a.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t* base = lds;         // [n]: first row of each bucket
  uint32_t* before = base + n;  // [n]: pairs of the bucket in earlier workgroups
  uint32_t* words = before + n;
  uint16_t* counts = reinterpret_cast<uint16_t*>(words);
  const Pairs<R> pairs(a);
  count_parts(a, pairs, words);
  for (int e = threadIdx.x; e < n; e += 64 * kGroupWaves) {
    uint32_t all = 0, early = 0;
    if (gridDim.x > 1) {
#pragma unroll 8
      for (unsigned g = 0; g < gridDim.x; g++) {
        const uint32_t c = a.counts[(int64_t)g * n + e];
        all += c;
        early += g < blockIdx.x ? c : 0;
      }
    }
    // each wave's next row of the bucket, counted from the workgroup's first
    uint32_t at = 0;
    for (int w = 0; w < kGroupWaves; w++) {
      const uint32_t c = counts[w * padded(n) + e];
      counts[w * padded(n) + e] = (uint16_t)at;
      at += c;
    }
    base[e] = gridDim.x > 1 ? all : at;
    before[e] = early;
  }
  __syncthreads();
  if (wave == 0) {  // exclusive scan of the buckets
    uint32_t carry = 0;
    for (int e0 = 0; e0 < n; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t own = e < n ? base[e] : 0;
      uint32_t s = own;
      for (int step = 1; step < 64; step <<= 1) {
        const uint32_t o = __shfl_up(s, step, 64);
        s += lane >= step ? o : 0;
      }
      if (e < n) {
        if (blockIdx.x == 0) a.offsets[e] = (int32_t)(carry + s - own);
        base[e] = carry + s - own + before[e];
      }
      carry += __shfl(s, 63, 64);
    }
  }
  __syncthreads();
  uint16_t* mine = counts + wave * padded(n);
#pragma unroll
  for (int r = 0; r < R; r++) {
    const int e = pairs.bucket[r];
    if (e >= 0) {
      const uint64_t m = same_id(e, a.id_bits), earlier = m & ((1ull << lane) - 1);
      const uint32_t row = base[e] + mine[e] + __builtin_popcountll(earlier);
      wave_sync();
      if (earlier == 0) mine[e] += __builtin_popcountll(m);  // (the lowest lane of each bucket)
      const int p = pairs.first + r * 64;
      a.order[row] = p;
      a.place[p] = (int32_t)row;
    }
    wave_sync();
  }
}

// Rounds of a workgroup: one workgroup up to 4096 pairs (one launch: 3.4 us for
// 1024 of 64 experts, 5.0 for 4096); beyond, workgroups of 1024 as long as there
// are 32 at most to add up, since one CU alone is slow at the scattered stores
// (16384 pairs: 13.8 us as one workgroup of 16 rounds, 7.6 so), then of 4096
// (131072 pairs: 3.0 + 7.5), then of 16384 (262144 pairs: 4.5 + 14.6).
static int group_rounds(int64_t pairs) {
  if (pairs <= kGroupTurn) return 1;
  if (pairs <= 4 * kGroupTurn) return 4;
  return pairs <= 32 * kGroupTurn ? 1 : pairs <= 128 * kGroupTurn ? 4 : 16;
}

int64_t moe_group_blocks(int64_t pairs) {
  const int64_t per = (int64_t)group_rounds(pairs) * kGroupTurn;
  return (pairs + per - 1) / per;
}

template <int R>
static hipError_t group_with(const GroupArgs& a, unsigned blocks, hipStream_t s) {
  const int n = a.experts + 1;
  const unsigned lds = (unsigned)(n * 8 + (n + (n & 1)) * kGroupWaves * 2);  // 41 KB at 1024 experts
  const dim3 grid(blocks > 0 ? blocks : 1), block(64 * kGroupWaves);
  if (blocks > 1) {
    hipLaunchKernelGGL(group_count_kernel<R>, grid, block, lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(group_place_kernel<R>, grid, block, lds, s, a);
  return hipGetLastError();
}

hipError_t launch_moe_group(GroupArgs a, hipStream_t s) {
  const unsigned blocks = (unsigned)moe_group_blocks(a.pairs);
  a.id_bits = 32 - __builtin_clz((unsigned)a.experts);
  if (a.pairs == 0) a.ids = a.offsets;  // (somewhere to read; no pair is one)
  switch (group_rounds(a.pairs)) {
    case 1: return group_with<1>(a, blocks, s);
    case 4: return group_with<4>(a, blocks, s);
    default: return group_with<16>(a, blocks, s);
  }
}

// ---------------------------------------------------------------------------
// dispatch: bytes only
// ---------------------------------------------------------------------------
namespace {

template <typename V>
__device__ __forceinline__ void carry(const uint8_t* src, uint8_t* rows, int64_t ld, int64_t bytes, const int32_t* place,
                                      int top_k, int64_t pairs, int64_t kept) {
  const int64_t n = bytes / (int64_t)sizeof(V);
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const V v = reinterpret_cast<const V*>(src)[i];
    for (int j = 0; j < top_k; j++) {
      const int64_t r = place[j];
      if ((uint64_t)r < (uint64_t)pairs) reinterpret_cast<V*>(rows + r * ld)[i] = r < kept ? v : V{};
    }
  }
}

}  // namespace

// A workgroup for each token: its row is read once and written to each of its
// places. V: the widest access that bases, pitches and row sizes allow (one byte
// at worst, for packed codes of odd pitch).
// 4096 tokens to 4 places each, rows of 5760 bytes: 19 us, 6.2 TB/s.
template <typename V, typename V2>
__global__ __launch_bounds__(256) void dispatch_kernel(DispatchArgs a) {
  const int64_t t = blockIdx.x;
  const int32_t* place = a.place + t * a.top_k;
  const int64_t pairs = a.tokens * a.top_k, kept = a.kept ? *a.kept : pairs;
  carry<V>(a.x + t * a.ld_x, a.rows, a.ld_rows, a.bytes, place, a.top_k, pairs, kept);
  if (a.bytes2 > 0)
    carry<V2>(a.x2 + t * a.ld_x2, a.rows2, a.ld_rows2, a.bytes2, place, a.top_k, pairs, kept);
}

namespace {

int widest(const void* p, const void* q, int64_t ld, int64_t ld2, int64_t bytes) {
  const uintptr_t m = (uintptr_t)p | (uintptr_t)q | (uintptr_t)ld | (uintptr_t)ld2 | (uintptr_t)bytes;
  return m % 16 == 0 ? 16 : m % 4 == 0 ? 4 : m % 2 == 0 ? 2 : 1;
}

template <typename V>
hipError_t dispatch_with(const DispatchArgs& a, int w2, hipStream_t s) {
  const dim3 grid((unsigned)a.tokens), block(256);
  if (w2 == 16) hipLaunchKernelGGL((dispatch_kernel<V, u32x4>), grid, block, 0, s, a);
  else if (w2 == 4) hipLaunchKernelGGL((dispatch_kernel<V, uint32_t>), grid, block, 0, s, a);
  else if (w2 == 2) hipLaunchKernelGGL((dispatch_kernel<V, uint16_t>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((dispatch_kernel<V, uint8_t>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_dispatch(const DispatchArgs& a, hipStream_t s) {
  const int w = widest(a.x, a.rows, a.ld_x, a.ld_rows, a.bytes);
  const int w2 = a.bytes2 > 0 ? widest(a.x2, a.rows2, a.ld_x2, a.ld_rows2, a.bytes2) : 16;
  if (w == 16) return dispatch_with<u32x4>(a, w2, s);
  if (w == 4) return dispatch_with<uint32_t>(a, w2, s);
  if (w == 2) return dispatch_with<uint16_t>(a, w2, s);
  return dispatch_with<uint8_t>(a, w2, s);
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------
namespace {

// Sixteen bytes of a row, wherever they start, or less at its end.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <bool BF16>
struct Elements {
  static constexpr int N = BF16 ? 8 : 4;
  float v[N];
  __device__ __forceinline__ void load(const void* p, int64_t i, int64_t width) {
    if (i + N <= width) {
      const u32x4 w = *reinterpret_cast<const u32x4_any*>(reinterpret_cast<const char*>(p) + i * (16 / N));
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const uint32_t x = w[k];
        if constexpr (BF16) {
          v[2 * k] = bf16_lo(x);
          v[2 * k + 1] = bf16_hi(x);
        } else {
          v[k] = __builtin_bit_cast(float, x);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; k++) {
        v[k] = 0.0f;
        if (i + k < width)
          v[k] = BF16 ? bf16_lo(reinterpret_cast<const uint16_t*>(p)[i + k]) : reinterpret_cast<const float*>(p)[i + k];
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i, int64_t width) const {
    if (i + N <= width) {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; k++) {
        if constexpr (BF16) w[k] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * k], (__bf16)v[2 * k + 1]});
        else w[k] = __builtin_bit_cast(uint32_t, v[k]);
      }
      *reinterpret_cast<u32x4_any*>(reinterpret_cast<char*>(p) + i * (16 / N)) = w;
    } else {
#pragma unroll
      for (int k = 0; k < N; k++) {
        if (i + k >= width) continue;
        if constexpr (BF16) reinterpret_cast<__bf16*>(p)[i + k] = (__bf16)v[k];
        else reinterpret_cast<float*>(p)[i + k] = v[k];
      }
    }
  }
};

__device__ __forceinline__ int64_t pair_row(const CombineArgs& a, int64_t p) { return a.place ? (int64_t)a.place[p] : p; }

// Rows that have a part: 0 to num_rows, whatever *kept says.
__device__ __forceinline__ int64_t rows_kept(const CombineArgs& a) {
  const int64_t n = a.kept ? *a.kept : a.num_rows;
  return n < 0 ? 0 : n < a.num_rows ? n : a.num_rows;
}

}  // namespace

// One lane, 16 bytes of one token's row: each slot's row in turn, four of them on
// their way at once. fp32 sums, rounded once where `out` is bf16; the order is
// that of the slots, so a result does not depend on the sort.
// 4096 tokens of 4 rows of 5760 bytes: 25.4 us, 4.6 TB/s; 32 tokens 3.9.
template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  constexpr int N = Elements<BF16>::N;
  const int64_t t = blockIdx.x;
  const int64_t i = ((int64_t)blockIdx.y * 256 + threadIdx.x) * N;
  if (i >= a.width) return;
  const int64_t kept = rows_kept(a);
  constexpr int64_t size = BF16 ? 2 : 4;
  Elements<BF16> sum, x;
#pragma unroll
  for (int k = 0; k < N; k++) sum.v[k] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < a.top_k; j++) {
    const int64_t p = t * a.top_k + j, r = pair_row(a, p);
    if ((uint64_t)r >= (uint64_t)kept) continue;
    const float w = a.weights ? a.weights[p] : 1.0f;
    x.load(reinterpret_cast<const char*>(a.rows) + r * a.ld_rows * size, i, a.width);
#pragma unroll
    for (int k = 0; k < N; k++) sum.v[k] = __builtin_fmaf(w, x.v[k], sum.v[k]);
  }
  sum.store(reinterpret_cast<char*>(a.out) + t * a.ld_out * size, i, a.width);
}

// A workgroup for four pairs of a token: the gradient's row is read once for
// them, four rows are on their way at once, and each gives its product with
// the gradient's, summed in fp32 (lanes, then waves, always in one order).
// 2048 tokens of 8 rows of 1001 fp32 numbers: 33 us, 4.2 TB/s. (A workgroup for
// each pair: 43, most of it the latency of one row after the other.)
constexpr int kBackPairs = 4;

template <bool BF16>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineBackwardArgs b) {
  constexpr int N = Elements<BF16>::N;
  const CombineArgs& a = b.a;
  const int64_t t = blockIdx.x;
  const int64_t kept = rows_kept(a);
  constexpr int64_t size = BF16 ? 2 : 4;
  const char* g = reinterpret_cast<const char*>(b.grad) + t * b.ld_grad * size;
  const int j0 = blockIdx.y * kBackPairs;
  const char* x[kBackPairs];
  char* out[kBackPairs];
  float w[kBackPairs], dot[kBackPairs];
  bool there[kBackPairs], write[kBackPairs];
#pragma unroll
  for (int q = 0; q < kBackPairs; q++) {
    const bool real = j0 + q < a.top_k;
    const int64_t p = t * a.top_k + (real ? j0 + q : j0), r = pair_row(a, p);
    there[q] = real && (uint64_t)r < (uint64_t)kept;
    write[q] = real && (uint64_t)r < (uint64_t)a.num_rows;
    w[q] = there[q] ? (a.weights ? a.weights[p] : 1.0f) : 0.0f;
    x[q] = reinterpret_cast<const char*>(a.rows) + r * a.ld_rows * size;
    out[q] = reinterpret_cast<char*>(b.grad_rows) + r * b.ld_grad_rows * size;
    dot[q] = 0.0f;
  }
  for (int64_t i = threadIdx.x * N; i < a.width; i += 256 * N) {
    Elements<BF16> gv, xv[kBackPairs];
    gv.load(g, i, a.width);
#pragma unroll
    for (int q = 0; q < kBackPairs; q++) {
      if (there[q] && b.grad_weights) xv[q].load(x[q], i, a.width);
    }
#pragma unroll
    for (int q = 0; q < kBackPairs; q++) {
      if (there[q] && b.grad_weights) {
#pragma unroll
        for (int k = 0; k < N; k++) dot[q] = __builtin_fmaf(gv.v[k], xv[q].v[k], dot[q]);
      }
      if (write[q]) {
        Elements<BF16> y;
        // (a pair without an expert: zeros, whatever the gradient holds)
#pragma unroll
        for (int k = 0; k < N; k++) y.v[k] = there[q] ? gv.v[k] * w[q] : 0.0f;
        y.store(out[q], i, a.width);
      }
    }
  }
  if (!b.grad_weights) return;
  __shared__ float part[kBackPairs][4];
#pragma unroll
  for (int q = 0; q < kBackPairs; q++) {
    float d = dot[q];
    d += xor_shfl<1>(d);
    d += xor_shfl<2>(d);
    d += xor_shfl<4>(d);
    d += xor_shfl<8>(d);
    d += xor_shfl<16>(d);
    d += xor_shfl<32>(d);
    if ((threadIdx.x & 63) == 0) part[q][threadIdx.x >> 6] = d;
  }
  __syncthreads();
  const int q = threadIdx.x;
  if (q < kBackPairs && j0 + q < a.top_k)
    b.grad_weights[t * a.top_k + j0 + q] = part[q][0] + part[q][1] + part[q][2] + part[q][3];
}

hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t s) {
  const int n = a.bf16 ? 8 : 4;
  const dim3 grid((unsigned)a.tokens, (unsigned)((a.width + 256 * n - 1) / (256 * n))), block(256);
  if (a.bf16) hipLaunchKernelGGL(combine_kernel<true>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(combine_kernel<false>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const CombineBackwardArgs& b, hipStream_t s) {
  const dim3 grid((unsigned)b.a.tokens, (unsigned)((b.a.top_k + kBackPairs - 1) / kBackPairs)), block(256);
  if (b.a.bf16) hipLaunchKernelGGL(combine_backward_kernel<true>, grid, block, 0, s, b);
  else hipLaunchKernelGGL(combine_backward_kernel<false>, grid, block, 0, s, b);
  return hipGetLastError();
}

}  // namespace fp4impl
