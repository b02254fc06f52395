// Internal interface between the C-ABI layer (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/paged_kv.h"

namespace pkv {

// Number of pkv_kv_dtype values.
constexpr int kNumKvFormats = 4;

// KV formats of the pools (pkv_kv_dtype).
// One-byte element codes (E4M3, INT8)?
__host__ __device__ constexpr bool k8(int fmt) {
  return fmt == PKV_KV_FP8_E4M3 || fmt == PKV_KV_INT8;
}
// FP4: E2M1 code pairs plus E4M3 block scales?
__host__ __device__ constexpr bool fp4(int fmt) { return fmt == PKV_KV_NVFP4; }
// Quantised, with per-(page, kv head) scales (every format but bf16)?
__host__ __device__ constexpr bool quant(int fmt) { return fmt != PKV_KV_BF16; }

// Bytes of one token row of one kv head in a pool: element codes, and the
// FP4 block scales (stored after every row's codes).
__host__ __device__ constexpr int row_code_bytes(int fmt, int head_dim) {
  return fmt == PKV_KV_BF16 ? 2 * head_dim : fp4(fmt) ? head_dim / 2 : head_dim;
}
__host__ __device__ constexpr int row_scale_bytes(int fmt, int head_dim) {
  return fp4(fmt) ? head_dim / 16 : 0;
}

struct AppendParams {
  uint8_t* k_pool;
  uint8_t* v_pool;
  uint8_t* k_blocks;  // FP4: block scales of the K pool (after its codes); else null
  uint8_t* v_blocks;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* seq_lens_before;
  const int32_t* cu_new;
  const uint4* k_new;  // [T][Hkv][D] bf16, as 16-byte vectors
  const uint4* v_new;
  int32_t* flags;
  int32_t batch;
  int32_t total_new;
  int32_t max_pages;
  int32_t num_pages;
  int32_t page_size;
  int32_t num_kv_heads;
  int32_t head_dim;
};

struct DecodeParams {
  const __nv_bfloat16* q;  // [B][Hq][D]
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* k_scale;  // [pages][Hkv] (E4M3)
  const float* v_scale;
  __nv_bfloat16* out;  // [B][Hq][D]
  float* lse;          // [B][Hq] or null
  float* part_o;       // [U + C][G][D]
  float2* part_ml;     // [U + C][G]
  int2* unit_info;     // [U]: (first partial slot, number of segments)
  int32_t* flags;
  // Fused append (all null otherwise): one new token per sequence, at
  // position seq_lens[b] - 1, written into the pools before it is read.
  const __nv_bfloat16* k_new;  // [B][Hkv][D]
  const __nv_bfloat16* v_new;
  uint8_t* k_pool;
  uint8_t* v_pool;
  uint8_t* k_blocks_w;  // FP4 fused append: block-scale regions to write
  uint8_t* v_blocks_w;
  // FP4 pools: the block-scale regions (after the codes) that the loads read
  const uint8_t* k_blocks;
  const uint8_t* v_blocks;
  // Shared prefixes (null otherwise): the kernel then attends to each
  // sequence's own tokens alone and leaves every result as partials.
  const int32_t* cu_groups;    // [num_groups + 1]
  const int32_t* prefix_lens;  // [num_groups]
  int32_t num_groups;
  int32_t num_sms;      // of the device, and decode CTAs that share one
  int32_t ctas_per_sm;
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t max_pages;
  int32_t num_pages;
  int32_t page_size;
  float scale_log2;  // softmax_scale * log2(e)
};

// Shared prefixes: the members of a group from the first that holds the whole prefix to
// the last, how many hold it, and its tokens; all 0 where nothing is shared.
struct __align__(16) Span {
  int32_t b0, b1, holders, prefix;
};

// Shared-prefix attention: the partials of the prefix kernel.
struct SharedParams {
  DecodeParams d;    // the whole call; its partials hold the sequences' own tokens
  float* pre_o;      // prefix partials: float4 vectors, see shared.cu
  float2* pre_ml;    // (max, sum) of each partial row
  int4* pre_info;    // [batch * num_kv_heads]: where a unit's prefix partials are
  Span* spans;       // [num_groups], by the prefix kernel (every CTA writes the same)
  int32_t pre_rows;  // rows that pre_o and pre_ml hold
  int32_t own_slots; // partial slots of d (of group rows each)
};

// Head norms and position rotation of q and k rows, with (launch_append_rope)
// or without (launch_qk_norm_rope) the store of K and V into the pools.
struct RopeParams {
  const __nv_bfloat16* q;  // token t's heads at q + t * q_stride; null: none
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;  // append only
  int64_t q_stride;        // elements between tokens
  int64_t k_stride;
  int64_t v_stride;
  __nv_bfloat16* q_out;  // [T][Hq][D]
  __nv_bfloat16* k_out;  // [T][Hkv][D], without append
  const float* cos_sin;  // [max_positions][rot]: rot/2 cosines, then rot/2 sines
  const float* q_weight;  // [D] or null: no norm
  const float* k_weight;
  const int32_t* positions;  // [T]; append: null = the cache position
  int32_t tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t max_positions;
  int32_t rot;  // rotary_dim
  int32_t interleaved;
  int32_t rows_per_item;  // set by the launch
  float eps;
  // The error word, and for the append the page geometry and pools, as there
  // (k_new, v_new and total_new are not used).
  AppendParams a;
};

// fmt: the pool's pkv_kv_dtype
cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, int num_sms,
                                cudaStream_t stream);
cudaError_t launch_append_rope(const RopeParams& p, int fmt, int head_dim, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_append(const AppendParams& p, int fmt, int num_sms, cudaStream_t stream);
cudaError_t decode_occupancy(int head_dim, int fmt, int group, int* ctas_per_sm);
cudaError_t decode_run(int head_dim, int fmt, const CUtensorMap& tk, const CUtensorMap& tv,
                       const DecodeParams& p, int num_ctas, cudaStream_t stream);

// The prefix kernel with num_ctas CTAs (tq: 3-D map of the queries; tk, tv:
// maps of the pools with boxes of 64 rows), and the merge of its partials with
// those of the sequences' own tokens.
cudaError_t shared_prefix_run(int head_dim, int fmt, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const SharedParams& p, int num_ctas,
                              cudaStream_t stream);
cudaError_t shared_merge_run(int head_dim, const SharedParams& p, cudaStream_t stream);

cudaError_t launch_combine(const void* parts, const float* lse_parts, int num_parts, int rows,
                           int head_dim, void* out, float* lse, cudaStream_t stream);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();  // null: not to be had
int check_cache(const pkv_cache* c);
int check_group(const pkv_cache* c, int32_t num_q_heads, int32_t gqa_group);
int check_table_span(const pkv_cache* c, int32_t max_pages_per_seq);
int64_t block_region_offset(const pkv_cache* c);
int encode_pool_map(CUtensorMap* map, void* base, bool bytes, int64_t rows, int row_elems,
                    int box_cols, int box_rows);
int encode_q_map(CUtensorMap* map, const void* q, int total_q, int hq, int d, int group);
int prefill_entry(const pkv_cache* cache, const void* q, int32_t num_q_heads, int32_t gqa_group,
                  const int32_t* cu_q_lens, const int32_t* page_table, int32_t max_pages_per_seq,
                  const int32_t* seq_lens, int32_t num_chunks, int32_t total_q,
                  int32_t max_q_len, float softmax_scale, void* out, float* lse,
                  cudaStream_t stream);

}  // namespace pkv
