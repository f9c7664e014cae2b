// moe_rows.hip -- (token, expert) pairs sorted by expert, the tokens' rows
// carried there, and the experts' rows brought back.
//
// Pair p = t * top_k + j is slot j of token t. group: a stable counting sort,
// place[p] = the pair's row, order[r] = row r's pair, offsets[e] = expert e's
// first row; pairs of no expert come last. dispatch: rows[place[p]] = x[t].
// combine: out[t] = sum_j w[p] rows[place[p]], in order of j.
#include "fp4_device.h"
#include "launch.h"

namespace fp4impl {
using namespace fp4dev;

namespace {

constexpr int kGroupWaves = 16;      // of a workgroup that sorts
constexpr int kGroupPairs = 8192;    // pairs of one workgroup: 8 rounds of 64 a wave

// The wave's lanes whose id is this lane's: one ballot for each bit of an id.
__device__ __forceinline__ uint64_t same_id(int id, int bits) {
  uint64_t m = __builtin_amdgcn_ballot_w64(true);
  for (int i = 0; i < bits; i++) {
    const uint64_t b = __builtin_amdgcn_ballot_w64((id >> i) & 1);
    m &= (id >> i) & 1 ? b : ~b;
  }
  return m;
}

__device__ __forceinline__ int bucket(const GroupArgs& a, int64_t p) {
  const int id = a.ids[p];
  return (unsigned)id < (unsigned)a.experts ? id : a.experts;
}

// Pairs [first, last) of the workgroup, a consecutive part for each wave.
struct Part {
  int64_t first, last;
};
__device__ __forceinline__ Part wave_part(const GroupArgs& a) {
  const int64_t lo = (int64_t)blockIdx.x * kGroupPairs;
  const int64_t n = a.pairs - lo < kGroupPairs ? a.pairs - lo : kGroupPairs;
  const int64_t per = ((n + 64 * kGroupWaves - 1) / (64 * kGroupWaves)) * 64;
  const int w = threadIdx.x >> 6;
  const int64_t f = per * w < n ? per * w : n, l = per * (w + 1) < n ? per * (w + 1) : n;
  return {lo + f, lo + l};
}

// A wave's lanes see what its other lanes wrote to LDS.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// counts[w * (experts + 1) + e] = pairs of bucket e in wave w's part (at most
// kGroupPairs in all: 16 bits).
__device__ __forceinline__ void count_parts(const GroupArgs& a, uint16_t* counts) {
  const int n = a.experts + 1, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < n * kGroupWaves; i += blockDim.x) counts[i] = 0;
  __syncthreads();
  uint16_t* mine = counts + (threadIdx.x >> 6) * n;
  const Part part = wave_part(a);
  for (int64_t p = part.first + lane; p < part.last; p += 64) {
    const int e = bucket(a, p);
    const uint64_t m = same_id(e, a.id_bits);
    if ((m & ((1ull << lane) - 1)) == 0) mine[e] += __builtin_popcountll(m);  // (the lowest lane of each bucket)
    wave_sync();
  }
  __syncthreads();
}

}  // namespace

// Each workgroup's pairs of each bucket, for the scan that follows.
__global__ __launch_bounds__(64 * kGroupWaves) void group_count_kernel(GroupArgs a) {
  extern __shared__ uint32_t lds[];
  uint16_t* counts = reinterpret_cast<uint16_t*>(lds);
  count_parts(a, counts);
  const int n = a.experts + 1;
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    uint32_t sum = 0;
    for (int w = 0; w < kGroupWaves; w++) sum += counts[w * n + e];
    a.counts[(int64_t)blockIdx.x * n + e] = sum;
  }
}

// Scan and placement. With one workgroup the counts are its own; with more
// they come from group_count_kernel, and each workgroup adds up what lies
// before it.
__global__ __launch_bounds__(64 * kGroupWaves) void group_place_kernel(GroupArgs a) {
  extern __shared__ uint32_t lds[];
  const int n = a.experts + 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t* base = lds;        // [n]: first row of each bucket
  uint32_t* before = base + n; // [n]: pairs of the bucket in earlier workgroups
  uint16_t* counts = reinterpret_cast<uint16_t*>(before + n);
  count_parts(a, counts);
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    uint32_t all = 0, early = 0;
    if (gridDim.x == 1) {
      for (int w = 0; w < kGroupWaves; w++) all += counts[w * n + e];
    } else {
      for (unsigned g = 0; g < gridDim.x; g++) {
        const uint32_t c = a.counts[(int64_t)g * n + e];
        all += c;
        early += g < blockIdx.x ? c : 0;
      }
    }
    base[e] = all;
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
      if (e < n) base[e] = carry + s - own;
      carry += __shfl(s, 63, 64);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < n; e += blockDim.x) a.offsets[e] = (int32_t)base[e];
  // each wave's next row of each bucket, counted from the workgroup's first
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    base[e] += before[e];
    uint32_t at = 0;
    for (int w = 0; w < kGroupWaves; w++) {
      const uint32_t c = counts[w * n + e];
      counts[w * n + e] = at;
      at += c;
    }
  }
  __syncthreads();
  uint16_t* mine = counts + wave * n;
  const Part part = wave_part(a);
  for (int64_t p = part.first + lane; p < part.last; p += 64) {
    const int e = bucket(a, p);
    const uint64_t m = same_id(e, a.id_bits), earlier = m & ((1ull << lane) - 1);
    const uint32_t row = base[e] + mine[e] + __builtin_popcountll(earlier);
    wave_sync();
    if (earlier == 0) mine[e] += __builtin_popcountll(m);
    wave_sync();
    a.order[row] = (int32_t)p;
    a.place[p] = (int32_t)row;
  }
}

int64_t moe_group_blocks(int64_t pairs) { return (pairs + kGroupPairs - 1) / kGroupPairs; }

hipError_t launch_moe_group(GroupArgs a, hipStream_t s) {
  const unsigned blocks = (unsigned)moe_group_blocks(a.pairs);
  const int n = a.experts + 1;
  a.id_bits = 32 - __builtin_clz((unsigned)a.experts);
  const unsigned lds = (unsigned)(n * (kGroupWaves * 2 + 8));  // 41 KB at 1024 experts
  if (blocks > 1) {
    hipLaunchKernelGGL(group_count_kernel, dim3(blocks), dim3(64 * kGroupWaves), lds, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(group_place_kernel, dim3(blocks > 0 ? blocks : 1), dim3(64 * kGroupWaves), lds, s, a);
  return hipGetLastError();
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
// places. V: the widest access that bases, pitches and row sizes allow.
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

// N consecutive elements, 16 bytes of them (or one).
template <bool BF16, int N>
struct Elements {
  float v[N];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (N == 1) {
      v[0] = BF16 ? bf16_lo(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
    } else if constexpr (BF16) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p) + i);
#pragma unroll
      for (int k = 0; k < 4; k++) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
      }
    } else {
      const f32x4 w = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(p) + i);
#pragma unroll
      for (int k = 0; k < 4; k++) v[k] = w[k];
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    if constexpr (N == 1) {
      if (BF16) reinterpret_cast<__bf16*>(p)[i] = (__bf16)v[0];
      else reinterpret_cast<float*>(p)[i] = v[0];
    } else if constexpr (BF16) {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; k++) w[k] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * k], (__bf16)v[2 * k + 1]});
      *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p) + i) = w;
    } else {
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i) = f32x4{v[0], v[1], v[2], v[3]};
    }
  }
};

__device__ __forceinline__ int64_t pair_row(const CombineArgs& a, int64_t p) { return a.place ? (int64_t)a.place[p] : p; }

}  // namespace

// One lane, N elements of one token's row: each slot's row in turn.
template <bool BF16, int N>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const int64_t t = blockIdx.x;
  const int64_t i = ((int64_t)blockIdx.y * 256 + threadIdx.x) * N;
  if (i >= a.width) return;
  const int64_t kept = a.kept && *a.kept < a.num_rows ? *a.kept : a.num_rows;
  constexpr int64_t size = BF16 ? 2 : 4;
  Elements<BF16, N> sum, x;
#pragma unroll
  for (int k = 0; k < N; k++) sum.v[k] = 0.0f;
  for (int j = 0; j < a.top_k; j++) {
    const int64_t p = t * a.top_k + j, r = pair_row(a, p);
    if ((uint64_t)r >= (uint64_t)kept) continue;
    const float w = a.weights ? a.weights[p] : 1.0f;
    x.load(reinterpret_cast<const char*>(a.rows) + r * a.ld_rows * size, i);
#pragma unroll
    for (int k = 0; k < N; k++) sum.v[k] = __builtin_fmaf(w, x.v[k], sum.v[k]);
  }
  sum.store(reinterpret_cast<char*>(a.out) + t * a.ld_out * size, i);
}

// A workgroup for each pair: its gradient row, and the product of the two rows.
template <bool BF16, int N>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineBackwardArgs b) {
  const CombineArgs& a = b.a;
  const int64_t p = blockIdx.x, t = p / a.top_k, r = pair_row(a, p);
  const int64_t kept = a.kept && *a.kept < a.num_rows ? *a.kept : a.num_rows;
  constexpr int64_t size = BF16 ? 2 : 4;
  const bool there = (uint64_t)r < (uint64_t)kept, write = (uint64_t)r < (uint64_t)a.num_rows;
  const char* g = reinterpret_cast<const char*>(b.grad) + t * b.ld_grad * size;
  const char* x = reinterpret_cast<const char*>(a.rows) + r * a.ld_rows * size;
  char* out = reinterpret_cast<char*>(b.grad_rows) + r * b.ld_grad_rows * size;
  const float w = there ? (a.weights ? a.weights[p] : 1.0f) : 0.0f;
  float dot = 0.0f;
  for (int64_t i = threadIdx.x * N; i < a.width; i += 256 * N) {
    Elements<BF16, N> gv, xv;
    gv.load(g, i);
    if (there && b.grad_weights) {
      xv.load(x, i);
#pragma unroll
      for (int k = 0; k < N; k++) dot = __builtin_fmaf(gv.v[k], xv.v[k], dot);
    }
#pragma unroll
    for (int k = 0; k < N; k++) gv.v[k] = there ? gv.v[k] * w : 0.0f;
    if (write) gv.store(out, i);
  }
  if (!b.grad_weights) return;
  dot += xor_shfl<1>(dot);
  dot += xor_shfl<2>(dot);
  dot += xor_shfl<4>(dot);
  dot += xor_shfl<8>(dot);
  dot += xor_shfl<16>(dot);
  dot += xor_shfl<32>(dot);
  __shared__ float part[4];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
  __syncthreads();
  if (threadIdx.x == 0) b.grad_weights[p] = part[0] + part[1] + part[2] + part[3];
}

hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t s) {
  const int n = a.vec_ok ? (a.bf16 ? 8 : 4) : 1;
  const dim3 grid((unsigned)a.tokens, (unsigned)((a.width + 256 * n - 1) / (256 * n))), block(256);
  if (a.bf16 && n > 1) hipLaunchKernelGGL((combine_kernel<true, 8>), grid, block, 0, s, a);
  else if (a.bf16) hipLaunchKernelGGL((combine_kernel<true, 1>), grid, block, 0, s, a);
  else if (n > 1) hipLaunchKernelGGL((combine_kernel<false, 4>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((combine_kernel<false, 1>), grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const CombineBackwardArgs& b, hipStream_t s) {
  const dim3 grid((unsigned)(b.a.tokens * b.a.top_k)), block(256);
  if (b.a.bf16 && b.a.vec_ok) hipLaunchKernelGGL((combine_backward_kernel<true, 8>), grid, block, 0, s, b);
  else if (b.a.bf16) hipLaunchKernelGGL((combine_backward_kernel<true, 1>), grid, block, 0, s, b);
  else if (b.a.vec_ok) hipLaunchKernelGGL((combine_backward_kernel<false, 4>), grid, block, 0, s, b);
  else hipLaunchKernelGGL((combine_backward_kernel<false, 1>), grid, block, 0, s, b);
  return hipGetLastError();
}

}  // namespace fp4impl
