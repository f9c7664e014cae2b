// matvec.hip -- products of a few rows in 16 or 32 bits with 4-bit weights:
//   y[p, n] = sum_k deq(W_e)[n, k] x[p / repeat, k], e = ids[p] (or 0),
// accumulated in fp32. The weights' bytes are read once; activations are not
// rounded.
#include <type_traits>

#include "fp4_device.h"
#include "launch.h"

namespace fp4impl {
using namespace fp4dev;

namespace {

constexpr int kWaves = 8;
constexpr int kMaxPairs = 4096;    // of a call by experts
constexpr int kMaxExperts = 4096;

struct Bf16Terms {
  bf16x8 t[3];
};

// Eight numbers of an activation row as bf16 operands: themselves, or three
// terms that hold all 24 bits of fp32 (each the leading 8 bits of what is
// left, cut off, so that nothing overflows).
template <bool XBF>
__device__ __forceinline__ void load_x(const void* row, int64_t k, bool there, Bf16Terms& o) {
  if constexpr (XBF) {
    u32x4 w = {0, 0, 0, 0};
    if (there) w = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(row) + k);
    o.t[0] = __builtin_bit_cast(bf16x8, w);
  } else {
    f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
    if (there) {
      lo = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(row) + k)[0];
      hi = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(row) + k)[1];
    }
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint32_t part[3][2];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int e = 2 * i + h;
        float v = e < 4 ? lo[e] : hi[e - 4];
        const uint32_t b0 = __builtin_bit_cast(uint32_t, v);
        part[0][h] = b0 >> 16;
        const bool fin = (b0 & 0x7f800000u) != 0x7f800000u;
        const float r1 = fin ? v - __builtin_bit_cast(float, b0 & 0xffff0000u) : 0.0f;
        const uint32_t b1 = __builtin_bit_cast(uint32_t, r1);
        part[1][h] = b1 >> 16;
        const float r2 = r1 - __builtin_bit_cast(float, b1 & 0xffff0000u);
        part[2][h] = __builtin_bit_cast(uint32_t, r2) >> 16;
      }
#pragma unroll
      for (int q = 0; q < 3; q++) w[q][i] = part[q][0] | (part[q][1] << 16);
    }
#pragma unroll
    for (int q = 0; q < 3; q++) o.t[q] = __builtin_bit_cast(bf16x8, u32x4{w[q][0], w[q][1], w[q][2], w[q][3]});
  }
}

// The eight values of a word of codes, times their block's scale: exact in
// bf16 (E2M1 has 2 significant bits, E4M3 4).
template <bool NV>
__device__ __forceinline__ bf16x8 weights8(uint32_t w, float scale) {
  uint32_t o[4];
  if constexpr (!NV) {
    o[0] = e2m1_unpack2_bf16<0>(w, scale);
    o[1] = e2m1_unpack2_bf16<1>(w, scale);
    o[2] = e2m1_unpack2_bf16<2>(w, scale);
    o[3] = e2m1_unpack2_bf16<3>(w, scale);
  } else {
    const f32x2 v[4] = {e2m1_unpack2<0>(w), e2m1_unpack2<1>(w), e2m1_unpack2<2>(w), e2m1_unpack2<3>(w)};
#pragma unroll
    for (int i = 0; i < 4; i++)
      o[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(v[i].x * scale), (__bf16)(v[i].y * scale)});
  }
  return __builtin_bit_cast(bf16x8, u32x4{o[0], o[1], o[2], o[3]});
}

struct Experts {
  uint32_t seen[kMaxExperts / 32];
  int expert, count;
  uint16_t list[kMaxPairs];
};

// The blockIdx.y-th expert among those that the pairs name, and its pairs in
// order. expert = -1: there are not so many.
__device__ __forceinline__ void find_expert(const MatvecArgs& a, Experts& s) {
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kMaxExperts / 32; i += blockDim.x) s.seen[i] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < a.pairs; p += blockDim.x) {
    const int e = a.ids[p];
    if ((unsigned)e < (unsigned)a.experts) atomicOr(&s.seen[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    int left = blockIdx.y, expert = -1;
    for (int i = 0; i < (a.experts + 31) / 32; i++) {
      const uint32_t w = s.seen[i];
      const int n = __builtin_popcount(w);
      if (left < n) {
        uint32_t m = w;
        for (; left > 0; left--) m &= m - 1;
        expert = i * 32 + __builtin_ctz(m);
        break;
      }
      left -= n;
    }
    int count = 0;
    if (expert >= 0) {
      for (int p0 = 0; p0 < a.pairs; p0 += 64) {
        const bool mine = p0 + lane < a.pairs && a.ids[p0 + lane] == expert;
        const uint64_t m = __builtin_amdgcn_ballot_w64(mine);
        if (mine) s.list[count + __builtin_popcountll(m & ((1ull << lane) - 1))] = p0 + lane;
        count += __builtin_popcountll(m);
      }
    }
    if (lane == 0) {
      s.expert = expert;
      s.count = count;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void store_y(const MatvecArgs& a, int64_t p, int64_t n, float v) {
  if (a.y_bf16) reinterpret_cast<__bf16*>(a.y)[p * a.ld_y + n] = (__bf16)v;
  else reinterpret_cast<float*>(a.y)[p * a.ld_y + n] = v;
}

}  // namespace

// A workgroup for 16 rows of W (of one expert); its waves take every eighth
// piece of 128 along K, a lane 32 consecutive values of row lane % 16, which
// are four operands of v_mfma_f32_16x16x32_bf16 against 16 rows of x.
template <bool NV, bool XBF, bool BY_EXPERT>
__global__ __launch_bounds__(64 * kWaves) void matvec_kernel(MatvecArgs a) {
  __shared__ float red[kWaves][256];
  __shared__ typename std::conditional<BY_EXPERT, Experts, int>::type found;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  int64_t expert = 0, count = a.pairs;
  if constexpr (BY_EXPERT) {
    if (blockIdx.y == 0) {  // pairs without an expert
      for (int64_t i = threadIdx.x; i < a.pairs * 16; i += blockDim.x) {
        const int64_t n = n0 + (i & 15);
        if ((unsigned)a.ids[i >> 4] >= (unsigned)a.experts && n < a.N) store_y(a, i >> 4, n, 0.0f);
      }
    }
    find_expert(a, found);
    expert = found.expert;
    count = found.count;
    if (expert < 0) return;
  }
  const int64_t n = n0 + c16 < a.N ? n0 + c16 : a.N - 1;
  const uint8_t* codes = a.codes + expert * a.c_es + n * a.ld_c + g * 16;
  const uint8_t* scales = a.scales + expert * a.s_es + n * a.ld_s + (NV ? 2 * g : g);
  const float ts = NV ? a.ts[expert] : 1.0f;
  for (int64_t r0 = 0; r0 < count; r0 += 16) {
    const int64_t r = r0 + c16 < count ? r0 + c16 : count - 1;
    int64_t pair = r;
    if constexpr (BY_EXPERT) pair = found.list[r];
    const char* x = reinterpret_cast<const char*>(a.x) + (pair / a.repeat) * a.ld_x * (XBF ? 2 : 4);
    f32x4 acc = {0, 0, 0, 0};
#pragma unroll 4
    for (int64_t k0 = wave * 128; k0 < a.K; k0 += 128 * kWaves) {
      const int64_t k = k0 + g * 32;
      u32x4 w = {0, 0, 0, 0};
      uint32_t s = 0;
      const bool first = k < a.K, second = k + 16 < a.K;
      if (first) {
        w = *reinterpret_cast<const u32x4*>(codes + (k0 >> 1));
        if constexpr (NV) s = *reinterpret_cast<const uint16_t*>(scales + (k0 >> 4));
        else s = scales[k0 >> 5];
      }
      float s0, s1;
      if constexpr (NV) {
        s0 = e4m3_decode(s & 0xffu);
        s1 = second ? e4m3_decode(s >> 8) : 0.0f;
      } else {
        s0 = s1 = e8m0_scale_operand(s);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        Bf16Terms xv;
        load_x<XBF>(x, k + 8 * j, j < 2 ? first : second, xv);
        const bf16x8 b = weights8<NV>(w[j], j < 2 ? s0 : s1);
#pragma unroll
        for (int q = 0; q < (XBF ? 1 : 3); q++) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv.t[q], b, acc, 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) red[wave][(4 * g + i) * 16 + c16] = acc[i];
    __syncthreads();
    if (threadIdx.x < 256) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; w++) sum += red[w][threadIdx.x];
      const int64_t row = r0 + (threadIdx.x >> 4), col = n0 + (threadIdx.x & 15);
      if (row < count && col < a.N) {
        int64_t p = row;
        if constexpr (BY_EXPERT) p = found.list[row];
        store_y(a, p, col, sum * ts);
      }
    }
    __syncthreads();
  }
}

namespace {

template <bool NV, bool XBF>
hipError_t launch(const MatvecArgs& a, hipStream_t s) {
  const unsigned tiles = (unsigned)((a.N + 15) / 16);
  if (a.ids) {
    const int64_t slots = a.pairs < a.experts ? a.pairs : a.experts;
    hipLaunchKernelGGL((matvec_kernel<NV, XBF, true>), dim3(tiles, (unsigned)(slots > 0 ? slots : 1)), dim3(64 * kWaves), 0,
                       s, a);
  } else {
    hipLaunchKernelGGL((matvec_kernel<NV, XBF, false>), dim3(tiles), dim3(64 * kWaves), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t s) {
  if (a.nvfp4) return a.x_bf16 ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return a.x_bf16 ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace fp4impl
