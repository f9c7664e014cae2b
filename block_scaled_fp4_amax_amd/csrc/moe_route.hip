// moe_route.hip -- a router's scores to each token's experts and weights, and
// the gradient of the scores.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)); choice c_e = s_e + b_e; the k
//   largest c (within the top groups of consecutive experts, if limited), ties
//   to the lowest index; w_j = scale * s_ij, over their sum if renormalized.
//
// L lanes (a DPP row of 16, or a wave) hold one token's E logits, VPL
// consecutive ones a lane, so that every reduction stays inside the row and a
// wave serves 64 / L tokens. A candidate is one double: the fp32 value with
// its expert's index in the mantissa's lowest bits (a float leaves 29 of them
// zero), turned so that the larger double is the better candidate and, of
// equal values, the lower index: one v_max_f64 compares both.
//
// Without a bias the order of the scores is that of the logits, which are
// compared as they are. With one (or where a group's rank is a sum of two
// scores) c is computed in fp32 with a known error; where two neighbours of the
// resulting order lie within it, those few candidates (or the best scores of
// each group) are done again in double, so that the choice is that of c in double.
//
// Bound by vector instructions, about 1700 a wave where four tokens have 256
// experts in groups: 16384 tokens of 256 fp32 logits (17.8 MB, which a copy
// moves in 3.5 us) take 16.5 us with a biased sigmoid and groups, 14.5 without
// groups; 1 token of 32 experts 2.8. (Every choice as a maximum over all keys
// took 53: instead each lane sorts its own keys once, and a choice is a maximum
// of the 16 heads and a shift of one lane's keys. A row done again as a whole
// held the kernel up for 9 us, where its candidates alone take 1.)
#include <float.h>

#include "fp4_device.h"
#include "launch.h"

namespace fp4impl {
using namespace fp4dev;

namespace {

// Keys of experts that may not be chosen: below kNone, where no float lies.
constexpr uint32_t kNoneHigh = 0xffe00000u;
constexpr double kNone = -0x1p1000;
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// exp(x) to about an ulp for x <= 88: 2^(x log2 e) by the hardware, and a
// first-order term for what the product's rounding lost.
__device__ __forceinline__ float exp_near(float x) {
  x = x < -200.0f ? -200.0f : x;  // (NaN passes)
  const float hi = x * kLog2e;
  const float lo = __builtin_fmaf(x, kLog2e, -hi) + x * kLog2eLow;
  const float r = __builtin_amdgcn_exp2f(hi);
  return __builtin_fmaf(r * lo, kLn2, r);
}

// value of lane ^ MASK within rows of 16 lanes (mirrors: the lanes they bring
// together differ in every lower bit too, which a reduction does not mind)
template <int STEP>
__device__ __forceinline__ int row_move(int x) {
  if constexpr (STEP == 1) return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true);        // quad_perm [1, 0, 3, 2]
  else if constexpr (STEP == 2) return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true);   // quad_perm [2, 3, 0, 1]
  else if constexpr (STEP == 4) return __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true);  // row_half_mirror
  else if constexpr (STEP == 8) return __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true);  // row_mirror
  else return __shfl_xor(x, STEP, 64);
}
template <int STEP>
__device__ __forceinline__ float move(float v) {
  return __builtin_bit_cast(float, row_move<STEP>(__builtin_bit_cast(int, v)));
}
template <int STEP>
__device__ __forceinline__ double move(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)row_move<STEP>((int)(uint32_t)u), hi = (uint32_t)row_move<STEP>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_fmaxf(a, b); }
  __device__ __forceinline__ double operator()(double a, double b) const { return __builtin_fmax(a, b); }
};
struct Min {
  __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_fminf(a, b); }
  __device__ __forceinline__ double operator()(double a, double b) const { return __builtin_fmin(a, b); }
};
struct Add {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};

// over the token's L lanes; every lane gets the result
template <int L, typename OP, typename T>
__device__ __forceinline__ T reduce(T v, OP op) {
  v = op(v, move<1>(v));
  v = op(v, move<2>(v));
  v = op(v, move<4>(v));
  v = op(v, move<8>(v));
  if constexpr (L == 64) {
    v = op(v, move<16>(v));
    v = op(v, move<32>(v));
  }
  return v;
}

template <int L>
__device__ __forceinline__ float from_lane(float v, int i) { return __shfl(v, i, L); }
template <int L>
__device__ __forceinline__ double from_lane(double v, int i) { return __shfl(v, i, L); }

// v of expert e; -inf and NaN make the key of one that may not be chosen.
__device__ __forceinline__ double make_key(float v, int e) {
  // (-0 and +0 are equal logits; +inf with an index would be a NaN)
  const uint64_t u = __builtin_bit_cast(uint64_t, (double)(__builtin_fminf(v, FLT_MAX) + 0.0f));
  const uint32_t hi = (uint32_t)(u >> 32), turn = ~(uint32_t)((int32_t)hi >> 31) & 1023u;
  const uint32_t lo = (uint32_t)u | ((uint32_t)e ^ turn);
  return __builtin_bit_cast(double, ((uint64_t)(v > -__builtin_inff() ? hi : kNoneHigh) << 32) | lo);
}
__device__ __forceinline__ int key_index(double k) {
  const uint64_t u = __builtin_bit_cast(uint64_t, k);
  return (int)(((uint32_t)u & 1023u) ^ ((int64_t)u < 0 ? 0u : 1023u));
}
__device__ __forceinline__ float key_value(double k) {
  return (float)__builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~(uint64_t)1023);
}

// The lane's VPL numbers of a row (logits, or the bias), `pad` past the last:
// 16 bytes (8 of bf16) at a time where rows are made of such pieces. No load
// waits for another: those past the end read the last piece again.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_part(const void* row, int n, bool vec, int lane, float pad, float (&l)[VPL]) {
  if constexpr (VPL >= 4) {
    if (vec) {
      uint32_t w[VPL];
#pragma unroll
      for (int i = 0; i < VPL; i += 4) {
        const int e = lane * VPL + i < n ? lane * VPL + i : n - 4;
        if constexpr (BF16) {
          const u32x2 h = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(row) + e);
          w[i] = h.x;
          w[i + 1] = h.y;
        } else {
          const u32x4 h = *reinterpret_cast<const u32x4*>(reinterpret_cast<const float*>(row) + e);
          w[i] = h.x;
          w[i + 1] = h.y;
          w[i + 2] = h.z;
          w[i + 3] = h.w;
        }
      }
#pragma unroll
      for (int v = 0; v < VPL; v++) {
        const uint32_t word = BF16 ? w[v / 4 * 4 + v % 4 / 2] : w[v];
        const float f = !BF16 ? __builtin_bit_cast(float, word) : v % 2 ? bf16_hi(word) : bf16_lo(word);
        l[v] = lane * VPL + v < n ? f : pad;
      }
      return;
    }
  }
  uint32_t w[VPL];
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    const int e = lane * VPL + v < n ? lane * VPL + v : n - 1;
    w[v] = BF16 ? (uint32_t)reinterpret_cast<const uint16_t*>(row)[e] << 16 : reinterpret_cast<const uint32_t*>(row)[e];
  }
#pragma unroll
  for (int v = 0; v < VPL; v++) l[v] = lane * VPL + v < n ? __builtin_bit_cast(float, w[v]) : pad;
}

template <int VPL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, const void* row, int lane, float pad, float (&l)[VPL]) {
  if (a.bf16) load_part<VPL, true>(row, a.experts, a.vec, lane, pad, l);
  else load_part<VPL, false>(row, a.experts, a.vec, lane, pad, l);
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, const void* row, int e) {
  return a.bf16 ? bf16_lo(reinterpret_cast<const uint16_t*>(row)[e]) : reinterpret_cast<const float*>(row)[e];
}

__device__ __forceinline__ const void* logit_row(const RouteArgs& a, int64_t t) {
  return reinterpret_cast<const char*>(a.logits) + t * a.ld * (a.bf16 ? 2 : 4);
}

// f(value of another lane of the row of 16, that lane) for each of the 15.
template <int N, typename T, typename F>
__device__ __forceinline__ void turns(T v, int lane, F f) {
  if constexpr (N < 16) {
    auto turn = [](int x) { return __builtin_amdgcn_mov_dpp(x, 0x120 + N, 0xF, 0xF, true); };  // row_ror:N
    T o;
    if constexpr (sizeof(T) == 8) {
      const uint64_t u = __builtin_bit_cast(uint64_t, v);
      o = __builtin_bit_cast(T, ((uint64_t)(uint32_t)turn((int)(u >> 32)) << 32) | (uint32_t)turn((int)(uint32_t)u));
    } else {
      o = __builtin_bit_cast(T, turn(__builtin_bit_cast(int, v)));
    }
    f(o, turn(lane));
    turns<N + 1>(v, lane, f);
  }
}

// The lane's keys in descending order (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_down(double (&key)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; i++)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const double x = key[i + j], y = key[i + j + k];
            key[i + j] = __builtin_fmax(x, y);
            key[i + j + k] = __builtin_fmin(x, y);
          }
}

// x joins a best and second best number.
template <typename T>
__device__ __forceinline__ void join_best(T& b1, T& b2, T x) {
  b2 = __builtin_elementwise_max(b2, __builtin_elementwise_min(b1, x));
  b1 = __builtin_elementwise_max(b1, x);
}

// What of two scores a group's rank is made of, and the larger magnitude in it.
template <typename T>
__device__ __forceinline__ T group_rank(const RouteArgs& a, T b1, T b2, T* mag) {
  const bool two = a.best == 2 && b2 > -(T)__builtin_inff();
  *mag = __builtin_elementwise_max(__builtin_elementwise_abs(b1), two ? __builtin_elementwise_abs(b2) : (T)0);
  if constexpr (sizeof(T) == 4) {
    // (a sum beyond fp32 is a group too, and one whose order is unsure: the gap to its like is 0)
    return two ? __builtin_amdgcn_fmed3f(b1 + b2, -FLT_MAX, FLT_MAX) : b1;
  }
  return two ? b1 + b2 : b1;
}

// Whether the lane's group is kept, where a.lanes_of_group (1, 2, 4 or 8) lanes
// of a row of 16 make a group, from the best two of each lane. `gap`: the
// difference between the last rank kept and the first left out, `size` the
// larger magnitude that entered either.
template <typename T>
__device__ __forceinline__ bool keep_lane(const RouteArgs& a, T b1, T b2, int lane, T* gap, T* size) {
  const T none = -(T)__builtin_inff(), big = (T)__builtin_inff();
  auto join = [&](T o1, T o2) {
    b2 = __builtin_elementwise_max(__builtin_elementwise_max(b2, o2), __builtin_elementwise_min(b1, o1));
    b1 = __builtin_elementwise_max(b1, o1);
  };
  const int q = a.lanes_of_group;
  if (q > 1) join(move<1>(b1), move<1>(b2));
  if (q > 2) join(move<2>(b1), move<2>(b2));
  if (q > 4) join(move<4>(b1), move<4>(b2));
  T mag;
  const T rank = group_rank(a, b1, b2, &mag);
  // lanes ahead of this one: those of better groups
  const int mine = lane & -q;
  int ahead = 0;
  turns<1>(rank, lane, [&](T r, int from) { ahead += (int)(r > rank) | ((int)(r == rank) & (int)(from < mine)); });
  const bool there = rank > none, kept = there && ahead < a.top_groups * q;
  *gap = reduce<16>(kept ? rank : big, Min()) - reduce<16>(there && !kept ? rank : none, Max());
  *size = reduce<16>(there ? mag : (T)0, Max());
  return kept;
}

// Which of the lane's experts belong to the groups kept (bit v), from the
// choice values c; c of experts that may not be chosen is -inf.
template <int L, int VPL, typename T>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& a, const T (&c)[VPL], int lane, T* gap, T* size) {
  const int gs = a.group_size, G = a.groups;
  const T none = -(T)__builtin_inff();
  T rank = none, mag = (T)0;  // of group `lane`
  if (L == 16 && a.lanes_of_group > 0) {
    T b1 = none, b2 = none;
#pragma unroll
    for (int v = 0; v < VPL; v++) join_best(b1, b2, c[v]);
    return keep_lane(a, b1, b2, lane, gap, size) ? ~0u : 0u;
  }
  for (int g = 0; g < G; g++) {
    T b1 = none, b2 = none;
    const int first = lane * VPL - g * gs;  // of the lane's experts, counted in the group
#pragma unroll
    for (int v = 0; v < VPL; v++) join_best(b1, b2, (unsigned)(first + v) < (unsigned)gs ? c[v] : none);
    auto join = [&](T o1, T o2) {
      b2 = __builtin_elementwise_max(__builtin_elementwise_max(b2, o2), __builtin_elementwise_min(b1, o1));
      b1 = __builtin_elementwise_max(b1, o1);
    };
    join(move<1>(b1), move<1>(b2));
    join(move<2>(b1), move<2>(b2));
    join(move<4>(b1), move<4>(b2));
    join(move<8>(b1), move<8>(b2));
    if constexpr (L == 64) {
      join(move<16>(b1), move<16>(b2));
      join(move<32>(b1), move<32>(b2));
    }
    if (lane == g) rank = group_rank(a, b1, b2, &mag);
  }
  int ahead = 0;
  for (int g = 0; g < G; g++) {
    const T r = from_lane<L>(rank, g);
    ahead += (r > rank || (r == rank && g < lane)) ? 1 : 0;
  }
  const bool there = lane < G && rank > none, kept = there && ahead < a.top_groups;
  const T big = (T)__builtin_inff();
  *gap = reduce<L>(kept ? rank : big, Min()) - reduce<L>(there && !kept ? rank : none, Max());
  *size = reduce<L>(there ? mag : (T)0, Max());
  uint64_t mask = __builtin_amdgcn_ballot_w64(kept);  // bit g for group g
  if constexpr (L == 16) mask = (mask >> (threadIdx.x & 48)) & 0xffffu;
  int g = lane * VPL / gs, left = gs - (lane * VPL - g * gs);
  uint32_t in = 0;
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    in |= (uint32_t)((mask >> (g & 63)) & 1) << v;
    if (--left == 0) {
      g++;
      left = gs;
    }
  }
  return in;
}

// The sum of exp(l - m) over the row in double, and m. spare: LDS for VPL
// numbers of each thread (four at a time, to keep these rare paths short).
template <int L, int VPL>
__device__ __forceinline__ double softmax_sum(const float (&l)[VPL], float m, double* spare) {
  double sum = 0;
#pragma unroll
  for (int v = 0; v < VPL; v++) spare[v * 256 + threadIdx.x] = l[v] > neg_inf() ? (double)l[v] - (double)m : -1e9;
#pragma unroll 4
  for (int v = 0; v < VPL; v++) sum += exp(spare[v * 256 + threadIdx.x]);
  return reduce<L>(sum, Add());
}

__device__ __forceinline__ double exact_score(const RouteArgs& a, double z, double m, double inv_sum) {
  const double p = exp(a.sigmoid ? -__builtin_fabs(z) : z - m);
  return a.sigmoid ? (z >= 0 ? 1.0 : p) / (1.0 + p) : p * inv_sum;
}

// keep_lane where errors make it unsure: the lane's best scores again in
// double, one after another, until the next is surely behind the second
// (`close`); two of them as a rule.
template <int VPL, typename CLOSE>
__device__ __forceinline__ bool keep_lane_exactly(const RouteArgs& a, const void* row, const float (&c)[VPL], int lane,
                                                  double m, double inv_sum, CLOSE close) {
  float left[VPL], second = neg_inf();
#pragma unroll
  for (int v = 0; v < VPL; v++) left[v] = c[v];
  double b1 = -(double)__builtin_inff(), b2 = b1, gap, size;
#pragma unroll 1
  for (int i = 0; i < VPL; i++) {
    float best = neg_inf();
    int at = 0;
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      at = left[v] > best ? v : at;
      best = __builtin_fmaxf(best, left[v]);
    }
    if (!(best > neg_inf()) || (i > 1 && !close(second, best))) break;
    second = i < 2 ? best : second;
#pragma unroll
    for (int v = 0; v < VPL; v++) left[v] = v == at ? neg_inf() : left[v];
    const int e = lane * VPL + at;
    join_best(b1, b2, exact_score(a, load_logit(a, row, e), m, inv_sum) + (a.bias ? a.bias[e] : 0.0f));
  }
  return keep_lane(a, b1, b2, lane, &gap, &size);
}

// The first n lanes hold one candidate each, in an order that their scores'
// errors make unsure; the row's other experts are surely behind them. The
// exact order: lane j gets the j-th. (Lanes of a row of 16.)
__device__ __forceinline__ int order_exactly(const RouteArgs& a, const void* row, int lane, int id, int n, double m,
                                             double inv_sum) {
  const bool there = lane < n;
  const double c = there ? exact_score(a, load_logit(a, row, id), m, inv_sum) + (a.bias ? a.bias[id] : 0.0f) : -DBL_MAX;
  int rank = 0;
  turns<1>(c, lane, [&](double o, int from) {
    const int oid = __shfl(id, from, 16);
    rank += (int)(from < n) & ((int)(o > c) | ((int)(o == c) & (int)(oid < id)));
  });
  const int to = (threadIdx.x & 48) | (there ? rank : lane);
  return __builtin_amdgcn_ds_permute(to * 4, id);
}

// The whole row's choice in double: slot j's expert goes to lane j (and j - L
// to its `more`).
template <int L, int VPL>
__device__ __forceinline__ void choose_exactly(const RouteArgs& a, int64_t t, int lane, float m, double* spare, int* mine,
                                               int* more) {
  const void* row = logit_row(a, t);
  const double none = -(double)__builtin_inff();
  double c[VPL], inv_sum = 1;
  {
    float l[VPL];
    load_logits<VPL>(a, row, lane, neg_inf(), l);
    if (!a.sigmoid) inv_sum = 1.0 / softmax_sum<L>(l, m, spare);
#pragma unroll
    for (int v = 0; v < VPL; v++) spare[v * 256 + threadIdx.x] = l[v] == l[v] ? (double)l[v] : none;
  }
#pragma unroll 4
  for (int v = 0; v < VPL; v++) {
    const int e = lane * VPL + v < a.experts ? lane * VPL + v : a.experts - 1;
    const double z = spare[v * 256 + threadIdx.x], b = a.bias ? (double)a.bias[e] : 0.0;
    const double s = exact_score(a, z, m, inv_sum) + b;
    spare[v * 256 + threadIdx.x] = z > none && b == b ? s : none;
  }
#pragma unroll
  for (int v = 0; v < VPL; v++) c[v] = spare[v * 256 + threadIdx.x];
  if (a.top_groups < a.groups) {
    double gap, size;
    const uint32_t in = keep_groups<L, VPL>(a, c, lane, &gap, &size);
#pragma unroll
    for (int v = 0; v < VPL; v++) c[v] = (in >> v) & 1 ? c[v] : none;
  }
  if (!a.bias) {  // the logits' order is that of the scores, also where those round to one number
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      if (c[v] > none) c[v] = (double)load_logit(a, row, lane * VPL + v);
    }
  }
  for (int j = 0; j < a.top_k; j++) {
    double best = none;
    int at = a.experts;  // (none)
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      if (c[v] > best) {
        best = c[v];
        at = lane * VPL + v;
      }
    }
    const double top = reduce<L>(best, Max());
    at = (int)reduce<L>(best == top ? (float)at : 4096.0f, Min());  // (indices are exact in fp32)
    best = top;
    if (lane == (j & (L - 1))) (j < L ? *mine : *more) = best > none ? at : -1;
#pragma unroll
    for (int v = 0; v < VPL; v++) c[v] = lane * VPL + v == at ? none : c[v];
  }
}

}  // namespace

// D: keys a lane may give: VPL, or no fewer than the choices, the one after
// them and what an unsure order may ask for.
template <int L, int VPL, int D>
__global__ __launch_bounds__(256, 4) void route_kernel(RouteArgs a) {
  __shared__ double spare[VPL * 256];
  const int lane = threadIdx.x & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (t >= a.tokens) return;  // (a token's lanes leave together)
  const void* row = logit_row(a, t);
  float l[VPL], m = neg_inf();
  load_logits<VPL>(a, row, lane, neg_inf(), l);
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    m = __builtin_fmaxf(m, l[v]);  // (NaN leaves it)
  }
  m = reduce<L>(m, Max());
  const bool by_score = a.bias != nullptr;
  const bool limited = a.top_groups < a.groups;
  const bool group_score = limited && (by_score || a.best == 2);
  double key[VPL];
  float sum = 1.0f, unsure = 0.0f;  // unsure: bound on a score's error
  bool sure = true;
  if (!a.sigmoid && (!a.renormalize || by_score || group_score)) {
    sum = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; v++) sum += exp_near(l[v] - m);
    sum = reduce<L>(sum, Add());
  }
  float c[VPL];  // choice value, -inf where there is none
#pragma unroll
  for (int v = 0; v < VPL; v++) c[v] = l[v] == l[v] ? l[v] : neg_inf();
  if (by_score || group_score) {
    // sigmoid, p = exp(-l): s (1 - s) times p's relative error, which is 2^-23
    // for exp2 and 1.5 |l| 2^-24 for its rounded argument, and s times 2^-24
    // for the sum and 2^-23 for the reciprocal; s (1 - s) is at most 1/4 and
    // |l| s (1 - s) below 0.23: in all below 2^-22.
    // softmax: (VPL + 6 + 3) 2^-24 relative for the sum, exponent as above:
    // below 2^-19 of the largest score, 1 / sum.
    float b[VPL];
    if (a.bias) {
      load_part<VPL, false>(a.bias, a.experts, a.vec_bias, lane, neg_inf(), b);
    } else {
#pragma unroll
      for (int v = 0; v < VPL; v++) b[v] = 0.0f;
    }
    const float inv = __builtin_amdgcn_rcpf(sum);
    unsure = a.sigmoid ? 0x1p-22f : 0x1p-19f * __builtin_fminf(inv, 1.0f) + 0x1p-24f;
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      const float x = a.sigmoid ? -l[v] : l[v] - m;
      const float p = __builtin_amdgcn_exp2f(x * kLog2e);
      const float s = (a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + p) : p * inv) + b[v];
      c[v] = c[v] > neg_inf() && s == s ? s : neg_inf();
    }
  }
  // Could two neighbours of the order be the other way round?
  auto close = [&](float x, float y) {
    return !(x - y > 2.0f * unsure + 0x1p-24f * (__builtin_fabsf(x) + __builtin_fabsf(y)));
  };
  uint32_t in = ~0u;
  if (limited) {
    float gap, size;
    in = keep_groups<L, VPL>(a, c, lane, &gap, &size);
    // two ranks of two scores: each score with its error and the rounding of
    // its bias (2^-24 size), each sum with one (2^-23 size); and what the
    // bound's own arithmetic rounds
    if (group_score) sure = !(gap <= 4.0f * unsure + 0x1.01p-21f * size);
    if (L == 16 && !sure && a.lanes_of_group > 0) {
      const double inv_sum = a.sigmoid ? 1.0 : 1.0 / softmax_sum<L>(l, m, spare);
      in = keep_lane_exactly<VPL>(a, row, c, lane, m, inv_sum, close) ? ~0u : 0u;
      sure = true;
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    key[v] = make_key((in >> v) & 1 ? (by_score ? c[v] : l[v]) : neg_inf(), lane * VPL + v);
  }
  int mine = -1, more = -1, found = 0;
  float last = 0.0f;
  // each lane's keys in order: the row's next is the best of their heads
  sort_down<VPL>(key);
  auto pop = [&]() {
    const double best = reduce<L>(key[0], Max());
    if (key[0] == best) {  // (one lane's, or nothing is left)
#pragma unroll
      for (int v = 0; v + 1 < D; v++) key[v] = key[v + 1];
      key[D - 1] = -DBL_MAX;
    }
    return best;
  };
  bool ordered = true, next = false;  // next: lane top_k of a row of 16 holds the one after the chosen
  for (int j = 0; j < a.top_k + (by_score ? 1 : 0); j++) {
    const double best = pop();
    if (lane == (j & (L - 1)) && j < 2 * L) (j < L ? mine : more) = best > kNone ? key_index(best) : -1;
    if (by_score) {
      const float now = key_value(best);
      if (j > 0 && best > kNone) {
        next = j == a.top_k && close(last, now);
        ordered = ordered && !close(last, now);
      }
      last = now;
      if (best > kNone) found = j + 1;
    }
  }
  if (!sure || (!ordered && a.top_k > 14)) {
    choose_exactly<L, VPL>(a, t, lane, m, spare, &mine, &more);
  } else if (!ordered) {
    // more candidates, until one is surely behind (found: those before it)
    if (!next && found > a.top_k) found = a.top_k;
    bool enough = !next;
    for (int j = a.top_k + 1; !enough && j < (D < VPL ? D : 16); j++) {
      const double best = pop();
      const float now = key_value(best);
      enough = !(best > kNone) || !close(last, now);
      if (!enough) {
        if (lane == j) mine = key_index(best);
        found = j + 1;
        last = now;
      }
    }
    if (enough) {
      const double inv_sum = a.sigmoid ? 1.0 : 1.0 / softmax_sum<L>(l, m, spare);
      mine = order_exactly(a, row, lane, mine, found, m, inv_sum);
      if (lane >= found) mine = -1;
    } else {
      choose_exactly<L, VPL>(a, t, lane, m, spare, &mine, &more);
    }
  }
  if (lane >= a.top_k) mine = -1;
  if (lane + L >= a.top_k) more = -1;
  // weights: lane j has slot j (and slot j + L)
  const bool have2 = L < 32 && a.top_k > L;
  const float z1 = mine >= 0 ? load_logit(a, row, mine) : neg_inf();
  const float z2 = have2 && more >= 0 ? load_logit(a, row, more) : neg_inf();
  float w1, w2;
  if (a.sigmoid) {
    // exp(min(z, 0)) / (1 + exp(-|z|)); over their sum the largest exponent
    // is taken out first, so that scores that underflow still have a ratio
    float top = 0.0f;
    if (a.renormalize) top = reduce<L>(__builtin_fminf(__builtin_fmaxf(z1, z2), 0.0f), Max());
    w1 = exp_near(__builtin_fminf(z1, 0.0f) - top) / (1.0f + exp_near(-__builtin_fabsf(z1)));
    w2 = exp_near(__builtin_fminf(z2, 0.0f) - top) / (1.0f + exp_near(-__builtin_fabsf(z2)));
  } else {
    const float top = a.renormalize ? reduce<L>(__builtin_fmaxf(z1, z2), Max()) : m;
    w1 = exp_near(z1 - top);
    w2 = exp_near(z2 - top);
  }
  w1 = mine >= 0 ? w1 : 0.0f;
  w2 = have2 && more >= 0 ? w2 : 0.0f;
  if (a.renormalize) sum = reduce<L>(w1 + w2, Add());
  const bool divide = a.renormalize || !a.sigmoid;
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = mine;
    a.weights[t * a.top_k + lane] = mine >= 0 ? (divide ? w1 / sum : w1) * a.scale : 0.0f;
  }
  if (have2 && lane + L < a.top_k) {
    a.ids[t * a.top_k + lane + L] = more;
    a.weights[t * a.top_k + lane + L] = more >= 0 ? (divide ? w2 / sum : w2) * a.scale : 0.0f;
  }
}

// dl from dw. Without renormalization softmax gives p_e (g_e - sum p g), g the
// scaled dw of the chosen and 0 elsewhere, sigmoid g_e s (1 - s); with it, and
// q_j the chosen scores over their sum, softmax q_j (g_j - sum q g), sigmoid
// that times (1 - s_j). One pass: the row is read once and written once.
// 16384 tokens of 160 fp32 logits, 6 chosen: 8.2 us, 2.6 TB/s (21 MB; a copy
// takes 4.3): bound by vector instructions, 592 a wave (57 % of the cycles), that
// stand behind one trip to memory. (As two passes over the row: 22.)
template <int L, int VPL>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteBackwardArgs b) {
  const RouteArgs& a = b.a;
  const int lane = threadIdx.x & (L - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (t >= a.tokens) return;
  const void* row = logit_row(a, t);
  const bool dense = !a.sigmoid && !a.renormalize;
  float p[VPL], m = neg_inf(), sum = 1.0f;
  if (dense) {
    load_logits<VPL>(a, row, lane, neg_inf(), p);
#pragma unroll
    for (int v = 0; v < VPL; v++) m = __builtin_fmaxf(m, p[v]);
    m = reduce<L>(m, Max());
    const float top = m > neg_inf() ? m : 0.0f;  // (a row of -inf has no part)
    sum = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; v++) {
      p[v] = exp_near(p[v] - top);
      sum += p[v];
    }
    sum = reduce<L>(sum, Add());
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; v++) p[v] = p[v] * inv;
    sum = inv;
  } else {
#pragma unroll
    for (int v = 0; v < VPL; v++) p[v] = 0.0f;
  }
  // slots j = lane and lane + L
  int e[2];
  float z[2], g[2], d[2];
  float top = neg_inf();
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int j = lane + i * L;
    e[i] = j < a.top_k ? a.ids[t * a.top_k + j] : -1;
    if ((unsigned)e[i] >= (unsigned)a.experts) e[i] = -1;
    z[i] = e[i] >= 0 ? load_logit(a, row, e[i]) : neg_inf();
    g[i] = e[i] >= 0 ? b.grad[t * a.top_k + j] * a.scale : 0.0f;
    top = __builtin_fmaxf(top, a.sigmoid ? __builtin_fminf(z[i], 0.0f) : z[i]);
  }
  if (dense) {
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      d[i] = e[i] >= 0 ? exp_near(z[i] - m) * sum * g[i] : 0.0f;
      dot += d[i];
    }
    dot = reduce<L>(dot, Add());
#pragma unroll
    for (int v = 0; v < VPL; v++) p[v] = -(p[v] * dot);
  } else {
    float q[2], r[2];  // score (times a power of e common to the row), 1 - s
    top = a.renormalize ? reduce<L>(top, Max()) : 0.0f;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      if (a.sigmoid) {
        const float small = exp_near(-__builtin_fabsf(z[i])), inv = 1.0f / (1.0f + small);
        q[i] = exp_near(__builtin_fminf(z[i], 0.0f) - top) * inv;
        r[i] = (z[i] >= 0.0f ? small : 1.0f) * inv;
      } else {
        q[i] = exp_near(z[i] - top);
        r[i] = 1.0f;
      }
      if (e[i] < 0) q[i] = 0.0f;
    }
    float dot = 0.0f;
    if (a.renormalize) {
      const float all = reduce<L>(q[0] + q[1], Add());
      const float inv = all > 0.0f ? 1.0f / all : 0.0f;
      q[0] *= inv;
      q[1] *= inv;
      dot = reduce<L>(q[0] * g[0] + q[1] * g[1], Add());
    }
#pragma unroll
    for (int i = 0; i < 2; i++) d[i] = e[i] >= 0 ? q[i] * r[i] * (g[i] - dot) : 0.0f;
  }
  for (int j = 0; j < a.top_k; j++) {
    const int at = __shfl(j < L ? e[0] : e[1], j & (L - 1), L) - lane * VPL;
    const float val = __shfl(j < L ? d[0] : d[1], j & (L - 1), L);
#pragma unroll
    for (int v = 0; v < VPL; v++) p[v] += at == v ? val : 0.0f;
  }
  char* out = reinterpret_cast<char*>(b.out) + t * b.ld_out * (a.bf16 ? 2 : 4);
  if constexpr (VPL >= 4) {
    if (b.vec_out) {
#pragma unroll
      for (int i = 0; i < VPL; i += 4) {
        const int at = lane * VPL + i;
        if (at >= a.experts) continue;
        if (a.bf16) {
          const bf16x2 lo = {(__bf16)p[i], (__bf16)p[i + 1]}, hi = {(__bf16)p[i + 2], (__bf16)p[i + 3]};
          *reinterpret_cast<u32x2*>(out + 2 * at) = u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
        } else {
          *reinterpret_cast<f32x4*>(out + 4 * at) = f32x4{p[i], p[i + 1], p[i + 2], p[i + 3]};
        }
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < VPL; v++) {
    const int at = lane * VPL + v;
    if (at < a.experts) {
      if (a.bf16) reinterpret_cast<__bf16*>(out)[at] = (__bf16)p[v];
      else reinterpret_cast<float*>(out)[at] = p[v];
    }
  }
}

namespace {

// Lanes for one token: a row of 16, but a wave for more than 256 experts or 16
// groups. (A wave for each of a few tokens is no sooner done: 1024 tokens of 32
// experts 4.3 us, rows 3.8; of 256 in groups 9.8 and 8.4; of 160 5.2 and 5.6.)
bool wide_route(const RouteArgs& a) { return a.experts > 256 || a.groups > 16; }

// The gradient, which has no steps from choice to choice, does gain from a
// wave's shorter turns up to some thousand tokens of many experts: 64 tokens of
// 256 4.3 us, rows 4.9; 4096 of them 5.6 and 6.3; 4096 of 160 4.9 and 5.2.
// (64 experts: 3.8 and 3.2.)
bool wide_backward(const RouteArgs& a) {
  return a.experts > 256 || (a.experts > 64 && a.tokens <= 16 * device_cu_count());
}

// Experts for each lane of a row of 16. 12 spare a quarter of the work of 16
// where they suffice and split no groups of whole lanes (the gradient of 16384
// tokens of 160 8.2 us for 10.0, the choice of 192 in 8 groups 15.4 for 24.2).
int row_share(const RouteArgs& a) {
  const int per = (a.experts + 15) / 16;
  if (per > 8 && per <= 12 && !(a.top_groups < a.groups && a.group_size % 16 == 0)) return 12;
  return per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : per <= 8 ? 8 : 16;
}

// What depends on the lanes' shares: 16-byte rows, and lanes that make a group.
void set_shares(RouteArgs& a) {
  const int64_t piece = a.bf16 ? 8 : 16;  // of four logits
  a.vec = (uintptr_t)a.logits % piece == 0 && (a.ld * (a.bf16 ? 2 : 4)) % piece == 0 && a.experts % 4 == 0;
  a.vec_bias = (uintptr_t)a.bias % 16 == 0 && a.experts % 4 == 0;
  const int vpl = row_share(a), q = a.group_size / vpl;
  a.lanes_of_group = a.group_size % vpl == 0 && (q & (q - 1)) == 0 && q <= 8 ? q : 0;
}

template <template <int, int> class LAUNCH, typename ARGS>
hipError_t route_by_size(bool wide, const RouteArgs& a, const ARGS& args, hipStream_t s) {
  if (wide) {
    const int per = (a.experts + 63) / 64;
    if (per <= 2) return LAUNCH<64, 2>::go(args, a.tokens, s);
    if (per <= 4) return LAUNCH<64, 4>::go(args, a.tokens, s);
    if (per <= 8) return LAUNCH<64, 8>::go(args, a.tokens, s);
    return LAUNCH<64, 16>::go(args, a.tokens, s);
  }
  switch (row_share(a)) {
    case 1: return LAUNCH<16, 1>::go(args, a.tokens, s);
    case 2: return LAUNCH<16, 2>::go(args, a.tokens, s);
    case 4: return LAUNCH<16, 4>::go(args, a.tokens, s);
    case 8: return LAUNCH<16, 8>::go(args, a.tokens, s);
    case 12: return LAUNCH<16, 12>::go(args, a.tokens, s);
    default: return LAUNCH<16, 16>::go(args, a.tokens, s);
  }
}

template <int L, int VPL>
struct Forward {
  static hipError_t go(const RouteArgs& a, int64_t tokens, hipStream_t s) {
    const dim3 grid((unsigned)((tokens + 256 / L - 1) / (256 / L))), block(256);
    constexpr int D = VPL < 12 ? VPL : 12;
    if (a.top_k < D) hipLaunchKernelGGL((route_kernel<L, VPL, D>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_kernel<L, VPL, VPL>), grid, block, 0, s, a);
    return hipGetLastError();
  }
};
template <int L, int VPL>
struct Backward {
  static hipError_t go(const RouteBackwardArgs& b, int64_t tokens, hipStream_t s) {
    hipLaunchKernelGGL((route_backward_kernel<L, VPL>), dim3((unsigned)((tokens + 256 / L - 1) / (256 / L))), dim3(256),
                       0, s, b);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_moe_route(RouteArgs a, hipStream_t s) {
  set_shares(a);
  return route_by_size<Forward>(wide_route(a), a, a, s);
}
hipError_t launch_moe_route_backward(RouteBackwardArgs b, hipStream_t s) {
  set_shares(b.a);
  const int64_t piece = b.a.bf16 ? 8 : 16;
  b.vec_out = (uintptr_t)b.out % piece == 0 && (b.ld_out * (b.a.bf16 ? 2 : 4)) % piece == 0 && b.a.experts % 4 == 0;
  return route_by_size<Backward>(wide_backward(b.a), b.a, b, s);
}

}  // namespace fp4impl
