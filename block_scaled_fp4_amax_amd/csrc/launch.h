// launch.h -- internal launch interface between the C ABI (fp4_api.cpp) and
// the HIP kernels. Arguments here are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4impl {

enum Flags : uint32_t {
  kFourOverSix = 1u,
  kBlock2D = 2u,
  kTranspose = 4u,
  kStochastic = 8u,
  kHadamard = 16u,
  kScaleSearch = 32u,
  kTensorScale = 64u,
};

struct QuantArgs {
  const void* x;
  bool x_bf16;
  int64_t batch, src_rows, src_cols;  // source matrix per batch item
  int64_t ld_x, bs_x;                 // elements
  int64_t R, C;                       // output matrix (C is the block direction)
  bool nvfp4;
  uint32_t flags;
  uint32_t signs;
  uint64_t seed, offset;
  const float* amax_in;   // [batch] or null
  uint8_t* codes;
  int64_t ld_c, bs_c;
  uint8_t* scales;
  int64_t ld_s, bs_s;
  float* tensor_scale;    // [batch] (NVFP4)
  float* partials;        // workspace [batch][nparts] (NVFP4 without amax_in)
  int nparts;
};

// Number of per-workgroup partial maxima the NVFP4 amax pre-pass writes for
// one batch item (also fixes its grid).
int amax_partials(int64_t src_rows, int64_t src_cols, uint32_t flags);

hipError_t launch_quantize(const QuantArgs& a, hipStream_t stream);

// Bytes of the library's own scratch array (one copy per GPU) that
// fp4_quantize_noalloc puts the NVFP4 amax partials in.
constexpr size_t kNoAllocScratchBytes = 262144;

// The current device's address of that array, looked up on the first call
// per device and cached; hipSuccess or the runtime's error.
hipError_t noalloc_scratch(float** ptr);

struct DequantArgs {
  bool nvfp4;
  int64_t batch, rows, cols;
  const uint8_t* codes;
  int64_t ld_c, bs_c;
  const uint8_t* scales;
  int64_t ld_s, bs_s;
  const float* tensor_scale;
  void* y;
  bool y_bf16;
  int64_t ld_y, bs_y;
};

hipError_t launch_dequantize(const DequantArgs& a, hipStream_t stream);

struct GemmArgs {
  bool nvfp4;
  int64_t groups, M, N, K;
  const uint8_t* a;
  int64_t lda, a_gs;
  const uint8_t* as;
  int64_t lda_s, as_gs;
  const float* a_ts;
  int64_t a_ts_gs;  // a_ts step per group: 1, or 0 when one scale covers all of A
  const uint8_t* b;
  int64_t ldb, b_gs;
  const uint8_t* bs;
  int64_t ldb_s, bs_gs;
  const float* b_ts;
  void* c;
  bool c_bf16;
  int64_t ldc, c_gs;
  bool c_vec_ok;  // C and its row / group pitches are 16-byte aligned
  // NULL: `groups` equal groups of M rows at the group strides. Else device
  // int32[groups + 1]: group g is rows [offs[g], offs[g + 1]) of one A and
  // one C of M rows (group strides of A and C zero).
  const int32_t* offs;
  // Quantized output instead of C (qc non-NULL; equal groups only): C_g
  // quantized along its rows into codes qc [M, N/2] and scales qs
  // [M, N/blk] per group; NVFP4 (q_nv) takes S_t from q_amax[g] and writes
  // it to q_ts[g].
  uint8_t* qc;
  int64_t ldqc, qc_gs;
  uint8_t* qs;
  int64_t ldqs, qs_gs;
  float* q_ts;
  const float* q_amax;
  bool q_nv, q_sr, q_rht;
  int q_sel;  // scale selection: 0 plain, 1 4/6, 2 search (NVFP4)
  uint32_t q_signs;
  uint64_t q_seed, q_offset;
};

hipError_t launch_gemm(const GemmArgs& g, hipStream_t stream);

// The paged key-value cache, as the kernels take it (strides in bytes).
struct KvCache {
  bool nvfp4;
  int64_t pages;
  int page_shift;  // page_size = 1 << page_shift
  int heads, dim;
  uint8_t *kc, *ks, *vc, *vs;
  int64_t codes_ps, scales_ps;
  const float *k_ts, *v_ts;
};

struct KvAppendArgs {
  KvCache c;
  bool bf16, four_over_six, interleaved;
  int64_t tokens;
  int q_heads, rotary;
  const void *k, *v, *q;
  void* q_out;
  int64_t k_ts_, k_hs, v_ts_, v_hs, q_ts_, q_hs, o_ts_, o_hs;  // token and head strides, elements
  const int64_t *slots, *positions;
  const float *cos_t, *sin_t;
  int64_t max_position;
};

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream);

struct KvReadArgs {
  KvCache c;
  int64_t tokens;
  const int64_t* slots;
  void *k, *v;
  bool bf16;
};

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t stream);

struct KvAttnArgs {
  KvCache c;
  bool bf16, causal;
  int q_heads, group;  // group = q_heads / kv heads
  int64_t batch, tokens;
  const int32_t *offs, *lens, *table;  // offs NULL: one query per sequence
  int64_t table_stride, max_len;
  const void* q;
  void* out;
  float* lse;
  int64_t q_ts_, q_hs, o_ts_, o_hs;
  float scale;
  float cap, inv_cap;  // the softcap in powers of two (0: off), and its inverse
  int64_t window;
  float* ws;
};

// How a call's work is cut.
struct KvAttnPlan {
  bool many;      // the form for many rows
  int few_tiles;  // few rows: 16-row tiles a wave
  int waves;      // of a workgroup
  int64_t tiles;  // row tiles of the batch per kv head, an upper bound
  int64_t runs;   // few rows, 0: a workgroup for each row tile and kv head; else equal runs of key tiles
  int64_t least;  // key tiles of a run, at least
  size_t ws;      // bytes of partial results
};

KvAttnPlan plan_kv_attention(const KvAttnArgs& a);
hipError_t launch_kv_attention(const KvAttnArgs& a, const KvAttnPlan& p, hipStream_t stream);

struct RouteArgs {
  bool bf16, sigmoid, renormalize;
  int64_t tokens, ld;  // ld: elements
  int experts, top_k, groups, group_size, top_groups, best;
  float scale;
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* ids;  // read by the backward pass
  // set at launch: rows readable four logits at a time; lanes that make a group, 0 if not whole lanes
  bool vec, vec_bias;
  int lanes_of_group;
};

struct RouteBackwardArgs {
  RouteArgs a;
  const float* grad;  // [tokens][top_k]
  void* out;
  int64_t ld_out;
  bool vec_out;
};

hipError_t launch_moe_route(RouteArgs a, hipStream_t stream);
hipError_t launch_moe_route_backward(RouteBackwardArgs b, hipStream_t stream);

struct GroupArgs {
  int64_t pairs;
  int experts, id_bits;  // id_bits: of `experts`, the bucket of pairs without an expert
  const int32_t* ids;
  int32_t *offsets, *order, *place;
  uint32_t* counts;  // workspace [workgroups][experts + 1] where there are several
};

// Workgroups of the sort, and whether it needs its workspace (more than one).
int64_t moe_group_blocks(int64_t pairs);
hipError_t launch_moe_group(GroupArgs a, hipStream_t stream);

struct DispatchArgs {
  int64_t tokens;
  int top_k;
  const int32_t *place, *kept;  // kept NULL: all rows
  const uint8_t* x;
  uint8_t* rows;
  int64_t bytes, ld_x, ld_rows;
  const uint8_t* x2;  // a second plane of bytes per row (bytes2 = 0: none)
  uint8_t* rows2;
  int64_t bytes2, ld_x2, ld_rows2;
};

hipError_t launch_moe_dispatch(const DispatchArgs& a, hipStream_t stream);

struct CombineArgs {
  bool bf16;
  int64_t tokens, width, num_rows;
  int top_k;
  const int32_t *place, *kept;  // NULL: row p, all rows
  const float* weights;         // NULL: 1
  const void* rows;
  void* out;
  int64_t ld_rows, ld_out;  // elements
};

struct CombineBackwardArgs {
  CombineArgs a;
  const void* grad;
  void* grad_rows;
  float* grad_weights;  // NULL: not asked for
  int64_t ld_grad, ld_grad_rows;
};

hipError_t launch_moe_combine(const CombineArgs& a, hipStream_t stream);
hipError_t launch_moe_combine_backward(const CombineBackwardArgs& b, hipStream_t stream);

struct MatvecArgs {
  bool nvfp4, x_bf16, y_bf16;
  int64_t pairs, repeat;  // row p of y belongs to row p / repeat of x
  int64_t N, K;
  const void* x;
  int64_t ld_x;  // elements
  const uint8_t* codes;
  int64_t ld_c, c_es;  // row pitch, and from one expert to the next, bytes
  const uint8_t* scales;
  int64_t ld_s, s_es;
  const float* ts;     // [experts]
  int experts;
  const int32_t* ids;  // [pairs], NULL: expert 0 for all
  void* y;
  int64_t ld_y;
};

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t stream);

// Compute units of the current device (cached per device).
int device_cu_count();

}  // namespace fp4impl
