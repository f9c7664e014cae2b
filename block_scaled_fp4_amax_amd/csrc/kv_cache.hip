// kv_cache.hip -- writing to and reading from the paged 4-bit key-value cache.
//
// Append: for each token, rotate the keys (and the step's queries) to the
// token's position, quantize keys and values in blocks along the head and
// store them at the token's slot. One lane takes 8 elements of a row, so that
// a wave's loads and stores are whole lines; the lanes of a block (2 for
// NVFP4, 4 for MXFP4) exchange its maximum and squared errors. Every step is
// that of quant_common.h's 16-element unit, so codes and scales are those of
// fp4_quantize under the same S_t, bit for bit (no rounding between the
// rotation and the quantizer).
//
// Bound by HBM: queries in and out, keys and values in, and a quarter of the
// latter out in 4 bits. 16384 tokens of 32 + 8 + 8 heads of 128 in bf16 to
// NVFP4 (364 MB): 83 us, 4.4 TB/s, where a large copy reaches 5.2. Few tokens
// are bound by the launch: 32 take 4 us. 16 elements a lane: 96 us.
#include "quant_common.h"

namespace fp4impl {

enum Rotation {
  kNoRotation = 0,
  kHalves = 1,       // pairs (i, i + R/2), R % 16 == 0: the partners of 8 elements are another lane's 8
  kInterleaved = 2,  // pairs (2i, 2i + 1): partners lie in the same lane
  kHalvesAny = 3,    // pairs (i, i + R/2), any even R: partners one by one
};

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  static constexpr int kWords = 8 * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
      const u32x4 x = reinterpret_cast<const u32x4*>(p)[i / 4];
#pragma unroll
      for (int j = 0; j < 4; j++) w[i + j] = x[j];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      reinterpret_cast<u32x4*>(p)[i / 4] = u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]};
  }
  __device__ __forceinline__ void get(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if constexpr (sizeof(T) == 4) v[i] = __builtin_bit_cast(float, w[i]);
      else v[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
  }
  __device__ __forceinline__ void set(const float v[8]) {
#pragma unroll
    for (int i = 0; i < kWords; i++) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __builtin_bit_cast(uint32_t, v[i]);
      } else {
        const bf16x2 pr = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
        w[i] = __builtin_bit_cast(uint32_t, pr);
      }
    }
  }
};
__device__ __forceinline__ float load1(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// Eight fp32 of 4-byte alignment.
__device__ __forceinline__ void load8_any(const float* p, float v[8]) {
  typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
  const f32x4_any a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// Cosines and signed sines of 8 elements from e0 on: element e becomes
// x[e] * c[e] + x[partner(e)] * s[e] (s negative for a pair's first
// element), the rounding of a c - b s and b c + a s step by step.
template <int ROT>
__device__ __forceinline__ void load_turn(const KvAppendArgs& a, int64_t pos, int e0, float c[8], float s[8]) {
  const int half = a.rotary >> 1;
  const float* ct = a.cos_t + pos * half;
  const float* st = a.sin_t + pos * half;
  if constexpr (ROT == kHalves) {
    if (e0 < a.rotary) {
      const int j = e0 < half ? e0 : e0 - half;
      load8_any(ct + j, c);
      load8_any(st + j, s);
#pragma unroll
      for (int i = 0; i < 8; i++) s[i] = e0 < half ? -s[i] : s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int e = e0 + i;
      if (e >= a.rotary) continue;
      const int j = ROT == kInterleaved ? e >> 1 : (e < half ? e : e - half);
      const bool first = ROT == kInterleaved ? (i & 1) == 0 : e < half;
      c[i] = ct[j];
      s[i] = first ? -st[j] : st[j];
    }
  }
}

// Codes of 8 scaled values, and a block's codes and scale byte from 8 of its
// values in each of its lanes (see quantize_unit).
__device__ __forceinline__ uint32_t pack8(const float q[8]) {
  uint32_t w = e2m1_pack2<0>(0u, q[0], q[1]);
  w = e2m1_pack2<1>(w, q[2], q[3]);
  w = e2m1_pack2<2>(w, q[4], q[5]);
  return e2m1_pack2<3>(w, q[6], q[7]);
}
template <bool NV, int SEL>
__device__ __forceinline__ uint32_t quantize8(const float v[8], const NvConsts& nc, uint32_t& sbyte) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[i]));
  amax = __builtin_fmaxf(amax, xor_shfl<1>(amax));
  float q[8];
  if constexpr (NV) {
    const NvCand c = nv_candidate<false>(amax, nc.k6, nc);
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = v[i] * c.r;
    uint32_t w = pack8(q);
    sbyte = c.code;
    if constexpr (SEL == 1) {
      const NvCand c4 = nv_candidate<false>(amax, nc.k4, nc);
      float q4[8];
#pragma unroll
      for (int i = 0; i < 8; i++) q4[i] = v[i] * c4.r;
      const uint32_t w4 = pack8(q4);
      float s6 = sq_chain8(q, w), s4 = sq_chain8(q4, w4);
      s6 += xor_shfl<1>(s6);
      s4 += xor_shfl<1>(s4);
      if (cand_error(c4, s4) < cand_error(c, s6)) {
        w = w4;
        sbyte = c4.code;
      }
    }
    return w;
  } else {
    amax = __builtin_fmaxf(amax, xor_shfl<2>(amax));
    sbyte = e8m0_from_amax(amax);
    if constexpr (SEL == 0) {
      const float sc = e8m0_scale_operand(sbyte);
      uint32_t w = e2m1_pack2_scaled<0>(0u, v[0], v[1], sc);
      w = e2m1_pack2_scaled<1>(w, v[2], v[3], sc);
      w = e2m1_pack2_scaled<2>(w, v[4], v[5], sc);
      return e2m1_pack2_scaled<3>(w, v[6], v[7], sc);
    }
    const int e = (int)sbyte - 127;
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = __builtin_ldexpf(v[i], -e);
    const uint32_t w = pack8(q);
    float q1[8];
#pragma unroll
    for (int i = 0; i < 8; i++) q1[i] = __builtin_ldexpf(v[i], -e - 1);
    const uint32_t w1 = pack8(q1);
    float s0 = sq_chain8(q, w), s1 = sq_chain8(q1, w1);
    s0 += xor_shfl<1>(s0);
    s1 += xor_shfl<1>(s1);
    s0 += xor_shfl<2>(s0);
    s1 += xor_shfl<2>(s1);
    if (e < 127 && 4.0f * s1 < s0) {
      sbyte += 1;
      return w1;
    }
    return w;
  }
}

__device__ __forceinline__ float sane_scale(const float* ts, int h) {
  const float s = ts[h];
  return s >= kFltMin && s <= 3.40282347e38f ? s : 1.0f;
}

// One wave per (token, group of passes): a pass takes 64 / (D / 8) rows, first
// the query rows', then the keys', then the values'. A lane keeps the same 8
// elements of every row it visits, so the token's cosines and sines stay in
// registers; the next pass's elements are on their way during a pass.
template <typename T, bool NV, int SEL, int ROT>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, int passes_per_wave) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.tokens) return;  // whole waves only: the lanes below exchange data
  const int lpr = a.c.dim >> 3;  // lanes of a row
  const int rpp = 64 / lpr;
  const int r_in = lane / lpr, u = lane - r_in * lpr;
  const int e0 = u << 3, half = a.rotary >> 1;
  const int64_t slot = a.slots[t];
  const bool stored = slot >= 0 && slot < (a.c.pages << a.c.page_shift);
  bool placed = true;
  float c[8], s[8];
  if constexpr (ROT != kNoRotation) {
    const int64_t pos = a.positions[t];
    placed = pos >= 0 && pos < a.max_position;
    if (placed) load_turn<ROT>(a, pos, e0, c, s);
  }
  // the lane with this lane's partners
  const int partner = e0 < half ? lane + (half >> 3) : e0 < a.rotary ? lane - (half >> 3) : lane;

  // 8 elements of a rotated row
  auto turn = [&](const Raw8<T>& now, const T* row, float v[8]) {
    now.get(v);
    if constexpr (ROT == kHalves) {
      Raw8<T> other;
#pragma unroll
      for (int i = 0; i < Raw8<T>::kWords; i++) other.w[i] = __builtin_amdgcn_ds_bpermute(4 * partner, now.w[i]);
      if (e0 < a.rotary) {  // all 8 or none
        float w[8];
        other.get(w);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = v[i] * c[i] + w[i] * s[i];
      }
    } else if constexpr (ROT != kNoRotation) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int e = e0 + i;
        if constexpr (ROT == kInterleaved) w[i] = v[i ^ 1];
        else w[i] = e < a.rotary ? load1(row + (e < half ? e + half : e - half)) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float y = v[i] * c[i] + w[i] * s[i];
        v[i] = e0 + i < a.rotary ? y : v[i];
      }
    }
  };

  const int q_passes = (a.q_heads + rpp - 1) / rpp, c_passes = (a.c.heads + rpp - 1) / rpp;
  const int first = blockIdx.y * passes_per_wave, end = first + passes_per_wave;
  const bool lane_on = r_in < rpp;

  // queries
  {
    const int p1 = min(end, q_passes);
    int r = first * rpp + r_in;
    const T* in = static_cast<const T*>(a.q) + t * a.q_ts_ + (int64_t)r * a.q_hs + e0;
    T* out = static_cast<T*>(a.q_out) + t * a.o_ts_ + (int64_t)r * a.o_hs + e0;
    const int64_t in_step = rpp * a.q_hs, out_step = rpp * a.o_hs;
    Raw8<T> raw{};
    if (first < p1 && lane_on && r < a.q_heads) raw.load(in);
    for (int p = first; p < p1; p++) {
      const Raw8<T> now = raw;
      const bool live = lane_on && r < a.q_heads;
      const T* row = live ? in - e0 : static_cast<const T*>(a.q);
      r += rpp;
      in += in_step;
      if (p + 1 < p1 && lane_on && r < a.q_heads) raw.load(in);
      float v[8];
      turn(now, row, v);
      if (!placed) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __builtin_nanf("");
      }
      if (live) {
        Raw8<T> y;
        y.set(v);
        y.store(out);
      }
      out += out_step;
    }
  }

  // keys, then values
  const int64_t page = slot >> a.c.page_shift;
  const int64_t in_page = slot & ((1 << a.c.page_shift) - 1);
  constexpr int kLanes = NV ? 2 : 4;  // of a block
#pragma unroll
  for (int kv = 0; kv < 2; kv++) {
    const int before = q_passes + kv * c_passes;
    const int p0 = max(first - before, 0), p1 = min(end - before, c_passes);
    if (p0 >= p1) continue;
    int h = p0 * rpp + r_in;
    const int64_t hs = kv ? a.v_hs : a.k_hs;
    const T* in = static_cast<const T*>(kv ? a.v : a.k) + t * (kv ? a.v_ts_ : a.k_ts_) + (int64_t)h * hs + e0;
    const int64_t row0 = ((int64_t)h << a.c.page_shift) + in_page;
    uint8_t* codes_to = (kv ? a.c.vc : a.c.kc) + page * a.c.codes_ps + row0 * (a.c.dim >> 1) + (e0 >> 1);
    uint8_t* scale_to = (kv ? a.c.vs : a.c.ks) + page * a.c.scales_ps + row0 * (lpr / kLanes) + u / kLanes;
    const int64_t rows_step = (int64_t)rpp << a.c.page_shift;
    Raw8<T> raw{};
    if (lane_on && h < a.c.heads) raw.load(in);
    for (int p = p0; p < p1; p++) {
      const Raw8<T> now = raw;
      const bool live = lane_on && h < a.c.heads;
      const int head = live ? h : 0;
      const T* row = live ? in - e0 : static_cast<const T*>(a.k);
      h += rpp;
      in += rpp * hs;
      if (p + 1 < p1 && lane_on && h < a.c.heads) raw.load(in);
      float v[8];
      if (kv) now.get(v);
      else turn(now, row, v);
      NvConsts nc{};
      if constexpr (NV) {
        nc.St = sane_scale(kv ? a.c.v_ts : a.c.k_ts, head);
        nc.k6 = 1.0f / (6.0f * nc.St);
        nc.k4 = 1.0f / (4.0f * nc.St);
      }
      uint32_t sbyte;
      const uint32_t codes = quantize8<NV, SEL>(v, nc, sbyte);
      if (live && stored && placed) {
        *reinterpret_cast<uint32_t*>(codes_to) = codes;
        if (u % kLanes == 0) *scale_to = (uint8_t)sbyte;
      }
      codes_to += rows_step * (a.c.dim >> 1);
      scale_to += rows_step * (lpr / kLanes);
    }
  }
}

template <typename T, bool NV, int SEL>
static hipError_t append_rot(const KvAppendArgs& a, hipStream_t s) {
  const int rpp = 64 / (a.c.dim >> 3);
  const int passes = (a.q_heads + rpp - 1) / rpp + 2 * ((a.c.heads + rpp - 1) / rpp);
  // few tokens: a wave takes one pass, so that the rows of a token spread
  // over the GPU; many: four, of which each but the first is loaded during
  // the one before (16384 tokens of 32 + 2 x 8 rows of 128: 83 us; six 87,
  // all twelve 85). A launch has up to 65535 workgroups along y; four passes
  // a wave need fewer for any number of heads.
  const int64_t waves = 4 * 2048;
  const int per_wave = a.tokens * passes <= waves && passes <= 65535 ? 1 : passes < 4 ? passes : 4;
  const dim3 grid((unsigned)((a.tokens + 3) / 4), (unsigned)((passes + per_wave - 1) / per_wave));
  if (a.rotary == 0) hipLaunchKernelGGL((kv_append_kernel<T, NV, SEL, kNoRotation>), grid, dim3(256), 0, s, a, per_wave);
  else if (a.interleaved)
    hipLaunchKernelGGL((kv_append_kernel<T, NV, SEL, kInterleaved>), grid, dim3(256), 0, s, a, per_wave);
  else if (a.rotary % 16 == 0)
    hipLaunchKernelGGL((kv_append_kernel<T, NV, SEL, kHalves>), grid, dim3(256), 0, s, a, per_wave);
  else hipLaunchKernelGGL((kv_append_kernel<T, NV, SEL, kHalvesAny>), grid, dim3(256), 0, s, a, per_wave);
  return hipGetLastError();
}

template <typename T>
static hipError_t append_fmt(const KvAppendArgs& a, hipStream_t s) {
  if (a.c.nvfp4) return a.four_over_six ? append_rot<T, true, 1>(a, s) : append_rot<T, true, 0>(a, s);
  return a.four_over_six ? append_rot<T, false, 1>(a, s) : append_rot<T, false, 0>(a, s);
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
  return a.bf16 ? append_fmt<uint16_t>(a, s) : append_fmt<float>(a, s);
}

// Read: one lane per 8 codes of a row, blockIdx.y 0 for keys and 1 for
// values. Bound by the stores (16 or 32 bytes for 4 bytes of codes): 16384
// tokens of 8 heads of 128 in bf16 (86 MB) take 22 us, 4 TB/s, also with 16
// codes a lane (32 tokens: 3.1 us; this way 2.8).
template <bool NV, typename T>
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  const uint32_t upr = a.c.dim >> 3, upt = a.c.heads * upr;  // units of a row, of a token
  const int64_t first = (int64_t)blockIdx.x * 256 / upt;     // of the workgroup's tokens
  const uint32_t from = (uint32_t)((int64_t)blockIdx.x * 256 - first * upt) + threadIdx.x;
  const uint32_t t_off = from / upt, unit = from - t_off * upt;
  const int64_t t = first + t_off;
  const int h = unit / upr, u = unit - h * upr;
  if (t >= a.tokens) return;
  const bool is_k = blockIdx.y == 0;
  const int64_t slot = a.slots[t];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = 0.0f;
  if (slot >= 0 && slot < (a.c.pages << a.c.page_shift)) {
    const int64_t page = slot >> a.c.page_shift;
    const int64_t row = ((int64_t)h << a.c.page_shift) + (slot & ((1 << a.c.page_shift) - 1));
    const uint32_t w =
        *reinterpret_cast<const uint32_t*>((is_k ? a.c.kc : a.c.vc) + page * a.c.codes_ps + row * (a.c.dim >> 1) + u * 4);
    const uint8_t* sc = (is_k ? a.c.ks : a.c.vs) + page * a.c.scales_ps + row * (NV ? upr >> 1 : upr >> 2);
    const uint32_t scale = sc[NV ? u >> 1 : u >> 2];
    const float step = NV ? 1.0f : e8m0_scale_operand(scale);
    const float eff = NV ? e4m3_decode(scale) * sane_scale(is_k ? a.c.k_ts : a.c.v_ts, h) : 1.0f;
    const f32x2 p[4] = {e2m1_unpack2<0>(w, step), e2m1_unpack2<1>(w, step), e2m1_unpack2<2>(w, step),
                        e2m1_unpack2<3>(w, step)};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[2 * j] = NV ? p[j].x * eff : p[j].x;
      v[2 * j + 1] = NV ? p[j].y * eff : p[j].y;
    }
  }
  Raw8<T> y;
  y.set(v);
  y.store(static_cast<T*>(is_k ? a.k : a.v) + ((t * a.c.heads + h) * upr + u) * 8);
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int64_t units = a.tokens * a.c.heads * (a.c.dim >> 3);
  const dim3 grid((unsigned)((units + 255) / 256), 2);
  if (a.c.nvfp4) {
    if (a.bf16) hipLaunchKernelGGL((kv_read_kernel<true, uint16_t>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv_read_kernel<true, float>), grid, dim3(256), 0, s, a);
  } else {
    if (a.bf16) hipLaunchKernelGGL((kv_read_kernel<false, uint16_t>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv_read_kernel<false, float>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace fp4impl
