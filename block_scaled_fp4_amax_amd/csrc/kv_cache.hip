// kv_cache.hip -- writing to and reading from the paged 4-bit key-value cache.
//
// Append: for each token, rotate the keys (and the step's queries) to the
// token's position, quantize keys and values in blocks along the head and
// store them at the token's slot. One lane takes a unit of 16 elements of a
// row, the unit of quantize_unit, so codes and scales are those of
// fp4_quantize under the same S_t, bit for bit (no rounding between the
// rotation and the quantizer).
//
// Bound by HBM: queries in and out, keys and values in, and a quarter of
// that again out in 4 bits; about 20 arithmetic instructions an element.
#include "quant_common.h"

namespace fp4impl {

enum Rotation {
  kNoRotation = 0,
  kHalves = 1,       // pairs (i, i + R/2), R % 16 == 0: the partners of 8 elements are 8 whole elements
  kInterleaved = 2,  // pairs (2i, 2i + 1): partners lie in the same unit
  kHalvesAny = 3,    // pairs (i, i + R/2), any even R: partners one by one
};

__device__ __forceinline__ float load1(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

template <typename T>
__device__ __forceinline__ void store8(T* p, const float v[8]);
template <>
__device__ __forceinline__ void store8<uint16_t>(uint16_t* p, const float v[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const bf16x2 pr = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
    o[i] = __builtin_bit_cast(uint32_t, pr);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float v[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

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

// Cosines and signed sines of a unit's 16 elements: element e becomes
// x[e] * c[e] + x[partner(e)] * s[e] (s negative for a pair's first
// element), the rounding of a c - b s and b c + a s step by step.
template <int ROT>
__device__ __forceinline__ void load_turn(const KvAppendArgs& a, int64_t pos, int e0, float c[16], float s[16]) {
  const int half = a.rotary >> 1;
  const float* ct = a.cos_t + pos * half;
  const float* st = a.sin_t + pos * half;
  if constexpr (ROT == kHalves) {
    // half % 8 == 0: 8 elements use 8 entries in a row
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int e = e0 + 8 * k;
      if (e >= a.rotary) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          c[8 * k + i] = 1.0f;
          s[8 * k + i] = 0.0f;
        }
        continue;
      }
      const int j = e < half ? e : e - half;
      load8_any(ct + j, c + 8 * k);
      load8_any(st + j, s + 8 * k);
#pragma unroll
      for (int i = 0; i < 8; i++) s[8 * k + i] = e < half ? -s[8 * k + i] : s[8 * k + i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int e = e0 + i;
    if (e < a.rotary) {
      const int j = ROT == kInterleaved ? e >> 1 : (e < half ? e : e - half);
      const bool first = ROT == kInterleaved ? (i & 1) == 0 : e < half;
      c[i] = ct[j];
      s[i] = first ? -st[j] : st[j];
    } else {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
  }
}

// 16 elements of a row from e0 on, rotated.
template <typename T, int ROT>
__device__ __forceinline__ void load_turned(const KvAppendArgs& a, const T* row, int e0, const float c[16],
                                            const float s[16], float v[16]) {
  load8<T>(row + e0, v);
  load8<T>(row + e0 + 8, v + 8);
  if constexpr (ROT == kNoRotation) return;
  const int half = a.rotary >> 1;
  float w[16];
  if constexpr (ROT == kInterleaved) {
#pragma unroll
    for (int i = 0; i < 16; i++) w[i] = v[i ^ 1];
  } else if constexpr (ROT == kHalves) {
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int e = e0 + 8 * k;
      const int from = e < half ? e + half : e < a.rotary ? e - half : e;
      load8<T>(row + from, w + 8 * k);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; i++) {
      const int e = e0 + i;
      w[i] = load1(row + (e < half ? e + half : e < a.rotary ? e - half : e));
    }
  }
#pragma unroll
  for (int i = 0; i < 16; i++) {
    // elements past the rotary part pass unchanged (also infinities, which a
    // product with 0 would turn into NaN)
    const float y = v[i] * c[i] + w[i] * s[i];
    v[i] = e0 + i < a.rotary ? y : v[i];
  }
}

__device__ __forceinline__ float sane_scale(const float* ts, int h) {
  const float s = ts[h];
  return s >= kFltMin && s <= 3.40282347e38f ? s : 1.0f;
}

// One wave per (token, group of row passes): 64 / (D / 16) rows at a time,
// the rows being q heads, then keys, then values. A lane keeps the same unit
// of every row it visits, so the token's cosines and sines stay in registers.
template <typename T, bool NV, int SEL, int ROT>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, int passes_per_wave) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.tokens) return;  // whole waves only: the lanes below exchange data
  const int upr = a.c.dim >> 4;
  const int rpp = 64 / upr;
  const int r_in = lane / upr, u = lane - r_in * upr;
  const int e0 = u << 4;
  const int rows = a.q_heads + 2 * a.c.heads;
  const int64_t slot = a.slots[t];
  const bool stored = slot >= 0 && slot < (a.c.pages << a.c.page_shift);
  bool placed = true;
  float c[16], s[16];
  if constexpr (ROT != kNoRotation) {
    const int64_t pos = a.positions[t];
    placed = pos >= 0 && pos < a.max_position;
    if (placed) load_turn<ROT>(a, pos, e0, c, s);
  }
  const int64_t page = slot >> a.c.page_shift;
  const int64_t in_page = slot & ((1 << a.c.page_shift) - 1);
  const int blk_units = NV ? 1 : 2;
  for (int pass = 0; pass < passes_per_wave; pass++) {
    const int base = (blockIdx.y * passes_per_wave + pass) * rpp;
    if (base >= rows) return;
    const int r = base + r_in;
    const bool live = r_in < rpp && r < rows;
    const bool is_q = r < a.q_heads, is_k = !is_q && r < a.q_heads + a.c.heads;
    const int h = is_q ? r : is_k ? r - a.q_heads : r - a.q_heads - a.c.heads;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = 0.0f;
    if (live && placed) {
      if (is_q) load_turned<T, ROT>(a, static_cast<const T*>(a.q) + t * a.q_ts_ + h * a.q_hs, e0, c, s, v);
      else if (is_k) load_turned<T, ROT>(a, static_cast<const T*>(a.k) + t * a.k_ts_ + h * a.k_hs, e0, c, s, v);
      else load_turned<T, kNoRotation>(a, static_cast<const T*>(a.v) + t * a.v_ts_ + h * a.v_hs, e0, c, s, v);
    }
    if (live && is_q) {
      if (!placed) {
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = __builtin_nanf("");
      }
      T* o = static_cast<T*>(a.q_out) + t * a.o_ts_ + h * a.o_hs + e0;
      store8<T>(o, v);
      store8<T>(o + 8, v + 8);
    }
    if (base + rpp <= a.q_heads) continue;  // queries only
    NvConsts nc{};
    if constexpr (NV) {
      nc.St = live && !is_q ? sane_scale(is_k ? a.c.k_ts : a.c.v_ts, h) : 1.0f;
      nc.k6 = 1.0f / (6.0f * nc.St);
      nc.k4 = 1.0f / (4.0f * nc.St);
    }
    uint32_t w0, w1, sbyte;
    quantize_unit<NV, SEL, false, false, false>(v, nc, 0, 0, 0, w0, w1, sbyte);
    if (live && !is_q && stored && placed) {
      const int64_t row = ((int64_t)h << a.c.page_shift) + in_page;
      uint8_t* codes = (is_k ? a.c.kc : a.c.vc) + page * a.c.codes_ps + row * (a.c.dim >> 1) + (e0 >> 1);
      *reinterpret_cast<uint2*>(codes) = make_uint2(w0, w1);
      uint8_t* scales = (is_k ? a.c.ks : a.c.vs) + page * a.c.scales_ps + row * (upr / blk_units);
      if (NV || (u & 1) == 0) scales[u / blk_units] = (uint8_t)sbyte;
    }
  }
}

template <typename T, bool NV, int SEL>
static hipError_t append_rot(const KvAppendArgs& a, hipStream_t s) {
  const int rows = a.q_heads + 2 * a.c.heads, rpp = 64 / (a.c.dim >> 4);
  const int passes = (rows + rpp - 1) / rpp;
  // few tokens: a wave takes one pass, so that the rows of a token spread
  // over the GPU; many: a wave takes them all and reads the tables once
  const int64_t waves = 4 * 2048;
  const int per_wave = a.tokens * passes <= waves ? 1 : passes;
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

// Read: one lane per 16 codes of a row, blockIdx.y 0 for keys and 1 for
// values. Bound by the stores (32 or 64 bytes for 8 bytes of codes).
template <bool NV, typename T>
__global__ __launch_bounds__(256) void kv_read_kernel(KvReadArgs a) {
  const int upr = a.c.dim >> 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t th = i / upr;
  const int u = (int)(i - th * upr);
  const int64_t t = th / a.c.heads;
  const int h = (int)(th - t * a.c.heads);
  if (t >= a.tokens) return;
  const bool is_k = blockIdx.y == 0;
  const int64_t slot = a.slots[t];
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; j++) v[j] = 0.0f;
  if (slot >= 0 && slot < (a.c.pages << a.c.page_shift)) {
    const int64_t page = slot >> a.c.page_shift;
    const int64_t row = ((int64_t)h << a.c.page_shift) + (slot & ((1 << a.c.page_shift) - 1));
    const uint2 w =
        *reinterpret_cast<const uint2*>((is_k ? a.c.kc : a.c.vc) + page * a.c.codes_ps + row * (a.c.dim >> 1) + u * 8);
    const uint8_t* sc = (is_k ? a.c.ks : a.c.vs) + page * a.c.scales_ps + row * (NV ? upr : upr >> 1);
    const float step = NV ? 1.0f : e8m0_scale_operand(sc[u >> 1]);
    const f32x2 p[8] = {e2m1_unpack2<0>(w.x, step), e2m1_unpack2<1>(w.x, step), e2m1_unpack2<2>(w.x, step),
                        e2m1_unpack2<3>(w.x, step), e2m1_unpack2<0>(w.y, step), e2m1_unpack2<1>(w.y, step),
                        e2m1_unpack2<2>(w.y, step), e2m1_unpack2<3>(w.y, step)};
    const float eff = NV ? e4m3_decode(sc[u]) * sane_scale(is_k ? a.c.k_ts : a.c.v_ts, h) : 1.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      v[2 * j] = NV ? p[j].x * eff : p[j].x;
      v[2 * j + 1] = NV ? p[j].y * eff : p[j].y;
    }
  }
  T* y = static_cast<T*>(is_k ? a.k : a.v) + th * a.c.dim + u * 16;
  store8<T>(y, v);
  store8<T>(y + 8, v + 8);
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int64_t units = a.tokens * a.c.heads * (a.c.dim >> 4);
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
