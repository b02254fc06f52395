// C ABI of libpagedkv.so (declared in include/paged_kv.h).
//
// Host side only: argument validation (every error is returned before any
// launch), decode planning, TMA tensor-map encoding and kernel launches.
// All device memory belongs to the caller.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "kernels.h"

namespace pkv {

// ------------------------------------------------------------- utilities
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int device_sms(int* sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices] = {};  // a device's count does not change
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices && (*sms = known[dev].load(std::memory_order_relaxed)) > 0)
    return PKV_OK;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PKV_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDevices) known[dev].store(*sms, std::memory_order_relaxed);
  return PKV_OK;
}

// Byte offset of an FP4 pool's block-scale region: all rows' codes come first.
int64_t block_region_offset(const pkv_cache* c) {
  return (int64_t)c->num_pages * c->num_kv_heads * c->page_size * (c->head_dim / 2);
}

// Validation shared by every entry point that reads the cache.
int check_cache(const pkv_cache* c) {
  if (!c) return PKV_ERR_NULL;
  if (!c->k_pool || !c->v_pool) return PKV_ERR_NULL;
  if (!aligned16(c->k_pool) || !aligned16(c->v_pool)) return PKV_ERR_ALIGN;
  if (c->num_pages < 1 || c->num_kv_heads < 1) return PKV_ERR_SHAPE;
  if (c->page_size != 64 && c->page_size != 128) return PKV_ERR_PAGE_SIZE;
  if (c->head_dim != 64 && c->head_dim != 128) return PKV_ERR_HEAD_DIM;
  if (c->kv_dtype != PKV_KV_BF16 && c->kv_dtype != PKV_KV_FP8_E4M3 &&
      c->kv_dtype != PKV_KV_INT8 && c->kv_dtype != PKV_KV_NVFP4)
    return PKV_ERR_DTYPE;
  if (c->kv_dtype != PKV_KV_BF16 && (!c->k_scale || !c->v_scale)) return PKV_ERR_DTYPE;
  // pool rows (pages * heads * page_size) index a TMA tensor: keep them in int32
  const long long rows = (long long)c->num_pages * c->num_kv_heads * c->page_size;
  if (rows >= INT_MAX) return PKV_ERR_SHAPE;
  return PKV_OK;
}

// Tokens a page-table row can address, max_pages_per_seq * page_size, must
// fit in int32: the kernels compare lengths against it in 32-bit arithmetic.
int check_table_span(const pkv_cache* c, int32_t max_pages_per_seq) {
  if ((int64_t)max_pages_per_seq * c->page_size > INT32_MAX) return PKV_ERR_SHAPE;
  return PKV_OK;
}

int check_group(const pkv_cache* c, int32_t num_q_heads, int32_t gqa_group) {
  if (gqa_group != 1 && gqa_group != 2 && gqa_group != 4 && gqa_group != 8) return PKV_ERR_GQA;
  if (num_q_heads != gqa_group * c->num_kv_heads) return PKV_ERR_GQA;
  return PKV_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D view [rows][row_elems] of a pool's codes (bytes, or bf16 elements)
// with a [box_rows][box_cols] box and the swizzle of the box's row width
// (128, 64 or 32 bytes).
int encode_pool_map(CUtensorMap* map, void* base, bool bytes, int64_t rows, int row_elems,
                    int box_cols, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return PKV_ERR_CUDA;
  const int eb = bytes ? 1 : 2;
  const int box_bytes = box_cols * eb;
  cuuint64_t dims[2] = {(cuuint64_t)row_elems, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_elems * eb};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUtensorMapSwizzle sw = box_bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                          : box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : CU_TENSOR_MAP_SWIZZLE_32B;
  CUresult r = fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_ERR_CUDA;
}

static int decode_ctas_per_sm(int head_dim, int fmt, int group, int* out) {
  // Cached per device and variant: a kernel's occupancy does not change at
  // run time, but the shared-memory attribute that decode_occupancy sets
  // belongs to the device that is current, so every device fills its own
  // entry (and sets its own attribute) on first use.
  constexpr int kMaxDevices = 64;
  static int cache[kMaxDevices][2][kNumKvFormats][4] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices || fmt < 0 || fmt >= kNumKvFormats) return PKV_ERR_UNSUPPORTED;
  const int gi = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3;
  std::lock_guard<std::mutex> lock(mu);
  int& slot = cache[dev][head_dim == 128][fmt][gi];
  if (slot == 0) {
    int n = 0;
    if (decode_occupancy(head_dim, fmt, group, &n) != cudaSuccess || n < 1) return PKV_ERR_CUDA;
    slot = n;
  }
  *out = slot;
  return PKV_OK;
}

// Where an append stores: the pools and the page geometry.
static void fill_append(const pkv_cache* cache, const int32_t* page_table,
                        int32_t max_pages_per_seq, const int32_t* seq_lens_before,
                        const int32_t* cu_new_tokens, int32_t batch, AppendParams* p) {
  p->k_pool = static_cast<uint8_t*>(cache->k_pool);
  p->v_pool = static_cast<uint8_t*>(cache->v_pool);
  p->k_blocks = fp4(cache->kv_dtype) ? p->k_pool + block_region_offset(cache) : nullptr;
  p->v_blocks = fp4(cache->kv_dtype) ? p->v_pool + block_region_offset(cache) : nullptr;
  p->k_scale = cache->k_scale;
  p->v_scale = cache->v_scale;
  p->page_table = page_table;
  p->seq_lens_before = seq_lens_before;
  p->cu_new = cu_new_tokens;
  p->flags = cache->error_flags;
  p->batch = batch;
  p->max_pages = max_pages_per_seq;
  p->num_pages = cache->num_pages;
  p->page_size = cache->page_size;
  p->num_kv_heads = cache->num_kv_heads;
  p->head_dim = cache->head_dim;
}

// The rotation and norms of a pkv_rope, checked.
static int check_rope(const pkv_rope* r, int32_t head_dim) {
  if (!r) return PKV_ERR_NULL;
  if (r->rotary_dim < 0 || r->rotary_dim > head_dim || r->rotary_dim % 16 != 0)
    return PKV_ERR_SHAPE;
  if (r->rotary_dim > 0) {
    if (!r->cos_sin) return PKV_ERR_NULL;
    if (!aligned16(r->cos_sin)) return PKV_ERR_ALIGN;
    if (r->max_positions < 1) return PKV_ERR_SHAPE;
  }
  if (!aligned16(r->q_norm_weight) || !aligned16(r->k_norm_weight)) return PKV_ERR_ALIGN;
  if (!std::isfinite(r->norm_eps) || r->norm_eps < 0.f) return PKV_ERR_SHAPE;
  return PKV_OK;
}

// Rows [tokens][heads][head_dim] whose tokens lie `stride` elements apart.
static int check_rows(const void* x, int64_t stride, int32_t heads, int32_t head_dim) {
  if (!x) return PKV_ERR_NULL;
  if (!aligned16(x) || stride % 8 != 0) return PKV_ERR_ALIGN;
  if (stride < (int64_t)heads * head_dim) return PKV_ERR_SHAPE;
  return PKV_OK;
}

static void fill_rope(const pkv_rope* r, RopeParams* p) {
  p->cos_sin = r->cos_sin;
  p->q_weight = r->q_norm_weight;
  p->k_weight = r->k_norm_weight;
  p->max_positions = r->max_positions;
  p->rot = r->rotary_dim;
  p->interleaved = r->interleaved != 0;
  p->eps = r->norm_eps;
}

// Upper bound of decode CTAs used for workspace sizing.
constexpr int kMaxDecodeCtasPerSm = 4;

// Groups of sequences that share a prefix (paged_decode_attention_shared).
struct Groups {
  const int32_t* cu;
  const int32_t* prefix_lens;
  int32_t num;
};

static size_t round16(size_t n) { return (n + 15) & ~size_t(15); }

// CTAs of the prefix kernel (one per SM, no more than it can have steps) and
// the rows of its partials; false if those do not fit int32.
static bool prefix_plan(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                        int32_t max_seq_len, int32_t num_groups, int sms, int32_t* ctas,
                        int32_t* rows) {
  const double group = (double)num_q_heads / num_kv_heads;
  const double steps = (batch * group / 128 + num_groups) * num_kv_heads *
                       (((int64_t)max_seq_len + 127) / 128);
  *ctas = steps < 1 ? 1 : steps < sms ? (int32_t)steps : sms;
  const int64_t n = 2 * (int64_t)batch * num_q_heads + 256 * (int64_t)*ctas;
  *rows = (int32_t)n;
  return n <= INT32_MAX;
}

// Bytes of the prefix partials, behind the decode workspace.
static size_t prefix_bytes(int32_t rows, int32_t units, int32_t groups, int32_t head_dim) {
  return (size_t)rows * head_dim * sizeof(float) + round16((size_t)rows * sizeof(float2)) +
         (size_t)units * sizeof(int4) + (size_t)groups * sizeof(Span);
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_abi_version(void) { return (1 << 16) | 2; }

const char* pkv_status_string(int status) {
  switch (status) {
    case PKV_OK: return "ok";
    case PKV_ERR_NULL: return "a required pointer is NULL";
    case PKV_ERR_SHAPE: return "a count or size is negative or inconsistent";
    case PKV_ERR_PAGE_SIZE: return "page_size must be 64 or 128";
    case PKV_ERR_HEAD_DIM: return "head_dim must be 64 or 128";
    case PKV_ERR_GQA: return "num_q_heads must equal gqa_group * num_kv_heads, group in {1,2,4,8}";
    case PKV_ERR_DTYPE: return "unknown kv dtype, or E4M3 pools without scales";
    case PKV_ERR_WORKSPACE: return "decode workspace is NULL, misaligned or too small";
    case PKV_ERR_CUDA: return "a CUDA call or kernel launch failed";
    case PKV_ERR_ALIGN: return "a pointer that must be 16-byte aligned is not";
    case PKV_ERR_UNSUPPORTED: return "this combination is not implemented";
    case PKV_ERR_SCRATCH_LIMIT:
      return "the request needs more decode scratch than the library's static 16 MiB array";
    case PKV_ERR_NO_PAGES: return "the free pages cannot cover the growth request";
    default: return "unknown status";
  }
}

int paged_kv_append(const pkv_cache* cache, const int32_t* page_table, int32_t max_pages_per_seq,
                    const int32_t* seq_lens_before, const int32_t* cu_new_tokens, int32_t batch,
                    int32_t total_new_tokens, const void* k_new, const void* v_new,
                    void* stream) {
  int st = check_cache(cache);
  if (st) return st;
  if (batch < 0 || total_new_tokens < 0 || max_pages_per_seq < 1) return PKV_ERR_SHAPE;
  if ((st = check_table_span(cache, max_pages_per_seq))) return st;
  if (total_new_tokens == 0 || batch == 0) return PKV_OK;
  if (!page_table || !seq_lens_before || !cu_new_tokens || !k_new || !v_new) return PKV_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new)) return PKV_ERR_ALIGN;
  int sms = 0;
  if ((st = device_sms(&sms))) return st;
  AppendParams p{};
  fill_append(cache, page_table, max_pages_per_seq, seq_lens_before, cu_new_tokens, batch, &p);
  p.k_new = static_cast<const uint4*>(k_new);
  p.v_new = static_cast<const uint4*>(v_new);
  p.total_new = total_new_tokens;
  cudaError_t e = launch_append(p, cache->kv_dtype, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int pkv_qk_norm_rope(const pkv_rope* rope, const void* q, int64_t q_stride, int32_t num_q_heads,
                     const void* k, int64_t k_stride, int32_t num_kv_heads, int32_t head_dim,
                     const int32_t* positions, int32_t tokens, void* q_out, void* k_out,
                     int32_t* error_flags, void* stream) {
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_HEAD_DIM;
  int st = check_rope(rope, head_dim);
  if (st) return st;
  if (tokens < 0 || num_q_heads < 0 || num_kv_heads < 0) return PKV_ERR_SHAPE;
  if (tokens == 0 || num_q_heads + (int64_t)num_kv_heads == 0) return PKV_OK;
  if (num_q_heads && ((st = check_rows(q, q_stride, num_q_heads, head_dim)) ||
                      (st = check_rows(q_out, (int64_t)num_q_heads * head_dim, num_q_heads, head_dim))))
    return st;
  if (num_kv_heads && ((st = check_rows(k, k_stride, num_kv_heads, head_dim)) ||
                       (st = check_rows(k_out, (int64_t)num_kv_heads * head_dim, num_kv_heads, head_dim))))
    return st;
  if (rope->rotary_dim && !positions) return PKV_ERR_NULL;
  int sms = 0;
  if ((st = device_sms(&sms))) return st;
  RopeParams p{};
  fill_rope(rope, &p);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.positions = positions;
  p.tokens = tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.a.flags = error_flags;
  cudaError_t e = launch_qk_norm_rope(p, head_dim, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int paged_kv_append_rope(const pkv_cache* cache, const pkv_rope* rope, const int32_t* page_table,
                         int32_t max_pages_per_seq, const int32_t* seq_lens_before,
                         const int32_t* cu_new_tokens, int32_t batch, int32_t total_new_tokens,
                         const void* k_new, int64_t k_stride, const void* v_new,
                         int64_t v_stride, const void* q, int64_t q_stride, int32_t num_q_heads,
                         void* q_out, const int32_t* positions, void* stream) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_rope(rope, cache->head_dim))) return st;
  if (batch < 0 || total_new_tokens < 0 || max_pages_per_seq < 1 || num_q_heads < 0)
    return PKV_ERR_SHAPE;
  if ((st = check_table_span(cache, max_pages_per_seq))) return st;
  if (total_new_tokens == 0 || batch == 0) return PKV_OK;
  if (!page_table || !seq_lens_before || !cu_new_tokens) return PKV_ERR_NULL;
  const int D = cache->head_dim, Hkv = cache->num_kv_heads;
  if ((st = check_rows(k_new, k_stride, Hkv, D))) return st;
  if ((st = check_rows(v_new, v_stride, Hkv, D))) return st;
  if (num_q_heads && ((st = check_rows(q, q_stride, num_q_heads, D)) ||
                      (st = check_rows(q_out, (int64_t)num_q_heads * D, num_q_heads, D))))
    return st;
  int sms = 0;
  if ((st = device_sms(&sms))) return st;
  RopeParams p{};
  fill_rope(rope, &p);
  fill_append(cache, page_table, max_pages_per_seq, seq_lens_before, cu_new_tokens, batch, &p.a);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k_new);
  p.v = static_cast<const __nv_bfloat16*>(v_new);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.positions = positions;
  p.tokens = total_new_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = Hkv;
  cudaError_t e =
      launch_append_rope(p, cache->kv_dtype, D, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int paged_decode_plan(int32_t batch, int32_t num_kv_heads, int32_t max_seq_len,
                      int32_t num_sms, int32_t num_ctas, int32_t ctas_per_sm,
                      int32_t* out_ctas) {
  if (!out_ctas) return PKV_ERR_NULL;
  if (batch < 0 || num_kv_heads < 1 || max_seq_len < 0 || num_sms < 1 || num_ctas < 0 ||
      ctas_per_sm < 1)
    return PKV_ERR_SHAPE;
  // 64-token work-list tiles of the largest possible batch (an upper bound on
  // the tiles of every format; the kernel lets only min(C, T) CTAs work).
  const long long max_tiles = (long long)batch * num_kv_heads * ((max_seq_len + 63) / 64);
  long long c = num_ctas > 0 ? num_ctas : (long long)num_sms * ctas_per_sm;
  if (c > max_tiles) c = max_tiles;
  if (c < 1) c = 1;
  *out_ctas = (int32_t)c;
  return PKV_OK;
}

size_t paged_decode_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t head_dim, int32_t max_seq_len, int32_t num_ctas) {
  if (batch < 0 || num_kv_heads < 1 || num_q_heads < num_kv_heads || head_dim < 1 ||
      max_seq_len < 0 || num_ctas < 0)
    return 0;
  int sms = 0;
  if (device_sms(&sms)) return 0;
  int32_t c = 0;
  if (paged_decode_plan(batch, num_kv_heads, max_seq_len, sms, num_ctas, kMaxDecodeCtasPerSm,
                        &c))
    return 0;
  const size_t G = (size_t)num_q_heads / num_kv_heads;
  const size_t units = (size_t)batch * num_kv_heads;
  const size_t slots = units + (size_t)c;
  size_t bytes = slots * G * head_dim * sizeof(float);  // partial o
  bytes = (bytes + 15) & ~size_t(15);
  bytes += slots * G * 2 * sizeof(float);  // partial (m, l)
  bytes = (bytes + 15) & ~size_t(15);
  bytes += units * sizeof(int2);  // per-unit (first slot, segments)
  return (bytes + 255) & ~size_t(255);
}

size_t paged_decode_shared_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                           int32_t num_kv_heads, int32_t head_dim,
                                           int32_t max_seq_len, int32_t num_groups) {
  const size_t own = paged_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim,
                                                  max_seq_len, 0);
  int sms = 0;
  int32_t ctas = 0, rows = 0;
  if (own == 0 || num_groups < 0 || (int64_t)batch * num_kv_heads > INT32_MAX || device_sms(&sms) ||
      !prefix_plan(batch, num_q_heads, num_kv_heads, max_seq_len, num_groups, sms, &ctas, &rows))
    return 0;
  if (num_groups == 0) return own;
  const size_t n = own + prefix_bytes(rows, batch * num_kv_heads, num_groups, head_dim);
  return (n + 255) & ~size_t(255);
}

// Decode, with the fused append of one new token per sequence when k_new
// and v_new are given (both null otherwise), or with the shared prefixes of
// `groups` read once (null otherwise).
static int decode_entry(const pkv_cache* cache, const void* q, int32_t num_q_heads,
                        int32_t gqa_group, const int32_t* page_table, int32_t max_pages_per_seq,
                        const int32_t* seq_lens, int32_t batch, int32_t max_seq_len,
                        float softmax_scale, const void* k_new, const void* v_new,
                        const Groups* groups, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int32_t num_ctas, void* stream) {
  int st = check_cache(cache);
  if (st) return st;
  if ((st = check_group(cache, num_q_heads, gqa_group))) return st;
  if (batch < 0 || max_pages_per_seq < 1 || max_seq_len < 0 || num_ctas < 0) return PKV_ERR_SHAPE;
  if (!std::isfinite(softmax_scale)) return PKV_ERR_SHAPE;
  if (batch == 0) return PKV_OK;
  if (!q || !page_table || !seq_lens || !out) return PKV_ERR_NULL;
  if (!aligned16(q) || !aligned16(out)) return PKV_ERR_ALIGN;
  if ((st = check_table_span(cache, max_pages_per_seq))) return st;
  if ((int64_t)max_seq_len > (int64_t)max_pages_per_seq * cache->page_size) return PKV_ERR_SHAPE;
  const size_t own_bytes = paged_decode_workspace_bytes(
      batch, num_q_heads, cache->num_kv_heads, cache->head_dim, max_seq_len, num_ctas);
  const size_t need =
      groups ? paged_decode_shared_workspace_bytes(batch, num_q_heads, cache->num_kv_heads,
                                                   cache->head_dim, max_seq_len, groups->num)
             : own_bytes;
  if (own_bytes == 0 || need == 0) return PKV_ERR_CUDA;
  if (!workspace || !aligned16(workspace) || workspace_bytes < need) return PKV_ERR_WORKSPACE;

  const int fmt = cache->kv_dtype;
  int sms = 0, per_sm = 0;
  if ((st = device_sms(&sms))) return st;
  if ((st = decode_ctas_per_sm(cache->head_dim, fmt, gqa_group, &per_sm))) return st;
  if (per_sm > kMaxDecodeCtasPerSm) per_sm = kMaxDecodeCtasPerSm;
  int32_t ctas = 0;
  if ((st = paged_decode_plan(batch, cache->num_kv_heads, max_seq_len, sms, num_ctas, per_sm,
                              &ctas)))
    return st;

  const int D = cache->head_dim;
  const int64_t rows = (int64_t)cache->num_pages * cache->num_kv_heads * cache->page_size;
  // quantised pools are viewed as bytes: a row holds D codes (one-byte
  // formats) or D/2 (FP4); bf16 rows are loaded in 64-element boxes
  const bool bytes = quant(fmt);
  const int row_elems = fp4(fmt) ? D / 2 : D;
  const int box_cols = bytes ? (row_elems >= 128 ? 128 : row_elems) : 64;
  CUtensorMap tk, tv;
  if ((st = encode_pool_map(&tk, cache->k_pool, bytes, rows, row_elems, box_cols, 64))) return st;
  if ((st = encode_pool_map(&tv, cache->v_pool, bytes, rows, row_elems, box_cols, 64))) return st;

  const size_t G = (size_t)gqa_group;
  const size_t units = (size_t)batch * cache->num_kv_heads;
  int32_t c_ws = 0;
  paged_decode_plan(batch, cache->num_kv_heads, max_seq_len, sms, num_ctas, kMaxDecodeCtasPerSm,
                    &c_ws);
  const size_t slots = units + (size_t)c_ws;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  size_t off = slots * G * D * sizeof(float);
  off = (off + 15) & ~size_t(15);
  float* part_o = reinterpret_cast<float*>(ws);
  float2* part_ml = reinterpret_cast<float2*>(ws + off);
  off += slots * G * 2 * sizeof(float);
  off = (off + 15) & ~size_t(15);
  int2* unit_info = reinterpret_cast<int2*>(ws + off);

  DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part_o = part_o;
  p.part_ml = part_ml;
  p.unit_info = unit_info;
  p.flags = cache->error_flags;
  if (fp4(fmt)) {
    p.k_blocks = static_cast<const uint8_t*>(cache->k_pool) + block_region_offset(cache);
    p.v_blocks = static_cast<const uint8_t*>(cache->v_pool) + block_region_offset(cache);
  }
  if (k_new) {
    p.k_new = static_cast<const __nv_bfloat16*>(k_new);
    p.v_new = static_cast<const __nv_bfloat16*>(v_new);
    p.k_pool = static_cast<uint8_t*>(cache->k_pool);
    p.v_pool = static_cast<uint8_t*>(cache->v_pool);
    if (fp4(fmt)) {
      p.k_blocks_w = p.k_pool + block_region_offset(cache);
      p.v_blocks_w = p.v_pool + block_region_offset(cache);
    }
  }
  p.batch = batch;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.group = gqa_group;
  p.max_pages = max_pages_per_seq;
  p.num_pages = cache->num_pages;
  p.page_size = cache->page_size;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!groups) {
    e = decode_run(D, fmt, tk, tv, p, ctas, s);
  } else {
    p.cu_groups = groups->cu;
    p.prefix_lens = groups->prefix_lens;
    p.num_groups = groups->num;
    p.num_sms = sms;
    p.ctas_per_sm = per_sm;
    SharedParams sp{};
    sp.d = p;
    sp.own_slots = (int32_t)slots;
    int32_t pre_ctas = 0;
    if (!prefix_plan(batch, num_q_heads, cache->num_kv_heads, max_seq_len, groups->num, sms,
                     &pre_ctas, &sp.pre_rows))
      return PKV_ERR_SHAPE;
    uint8_t* pre = ws + own_bytes;
    sp.pre_o = reinterpret_cast<float*>(pre);
    pre += (size_t)sp.pre_rows * D * sizeof(float);
    sp.pre_ml = reinterpret_cast<float2*>(pre);
    pre += round16((size_t)sp.pre_rows * sizeof(float2));
    sp.pre_info = reinterpret_cast<int4*>(pre);
    sp.spans = reinterpret_cast<Span*>(pre + units * sizeof(int4));
    CUtensorMap tq;
    if ((st = encode_q_map(&tq, q, batch, num_q_heads, D, gqa_group))) return st;
    e = shared_prefix_run(D, fmt, tq, tk, tv, sp, pre_ctas, s);
    if (e == cudaSuccess) e = decode_run(D, fmt, tk, tv, p, ctas, s);
    if (e == cudaSuccess) e = shared_merge_run(D, sp, s);
  }
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int paged_decode_attention(const pkv_cache* cache, const void* q, int32_t num_q_heads,
                           int32_t gqa_group, const int32_t* page_table,
                           int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t batch,
                           int32_t max_seq_len, float softmax_scale, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, int32_t num_ctas,
                           void* stream) {
  return decode_entry(cache, q, num_q_heads, gqa_group, page_table, max_pages_per_seq, seq_lens,
                      batch, max_seq_len, softmax_scale, nullptr, nullptr, nullptr, out, lse,
                      workspace, workspace_bytes, num_ctas, stream);
}

int paged_decode_attention_shared(const pkv_cache* cache, const void* q, int32_t num_q_heads,
                                  int32_t gqa_group, const int32_t* page_table,
                                  int32_t max_pages_per_seq, const int32_t* seq_lens,
                                  int32_t batch, int32_t max_seq_len, const int32_t* cu_groups,
                                  const int32_t* prefix_lens, int32_t num_groups,
                                  float softmax_scale, void* out, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (num_groups < 0) return PKV_ERR_SHAPE;
  if (batch > 0 && num_groups > 0 && (!cu_groups || !prefix_lens)) return PKV_ERR_NULL;
  const Groups groups = {cu_groups, prefix_lens, num_groups};
  return decode_entry(cache, q, num_q_heads, gqa_group, page_table, max_pages_per_seq, seq_lens,
                      batch, max_seq_len, softmax_scale, nullptr, nullptr,
                      num_groups > 0 ? &groups : nullptr, out, lse, workspace, workspace_bytes, 0,
                      stream);
}

int paged_decode_attention_append(const pkv_cache* cache, const void* q, int32_t num_q_heads,
                                  int32_t gqa_group, const int32_t* page_table,
                                  int32_t max_pages_per_seq, const int32_t* seq_lens,
                                  int32_t batch, int32_t max_seq_len, float softmax_scale,
                                  const void* k_new, const void* v_new, void* out, float* lse,
                                  void* workspace, size_t workspace_bytes, int32_t num_ctas,
                                  void* stream) {
  if (batch > 0 && (!k_new || !v_new)) return PKV_ERR_NULL;
  if (batch > 0 && (!aligned16(k_new) || !aligned16(v_new))) return PKV_ERR_ALIGN;
  return decode_entry(cache, q, num_q_heads, gqa_group, page_table, max_pages_per_seq, seq_lens,
                      batch, max_seq_len, softmax_scale, k_new, v_new, nullptr, out, lse,
                      workspace, workspace_bytes, num_ctas, stream);
}

int paged_attention_combine(const void* parts, const float* lse_parts, int32_t num_parts,
                            int32_t rows, int32_t head_dim, void* out, float* lse,
                            void* stream) {
  if (num_parts < 1 || rows < 0) return PKV_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_HEAD_DIM;
  if (rows == 0) return PKV_OK;
  if (!parts || !lse_parts || !out) return PKV_ERR_NULL;
  if (!aligned16(parts) || !aligned16(out)) return PKV_ERR_ALIGN;
  if ((int64_t)num_parts * rows * head_dim >= INT64_C(1) << 40) return PKV_ERR_SHAPE;
  cudaError_t e = launch_combine(parts, lse_parts, num_parts, rows, head_dim, out, lse,
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int paged_prefill_chunk_attention(const pkv_cache* cache, const void* q, int32_t num_q_heads,
                                  int32_t gqa_group, const int32_t* cu_q_lens,
                                  const int32_t* page_table, int32_t max_pages_per_seq,
                                  const int32_t* seq_lens, int32_t num_chunks, int32_t total_q,
                                  int32_t max_q_len, float softmax_scale, void* out, float* lse,
                                  void* stream) {
  return prefill_entry(cache, q, num_q_heads, gqa_group, cu_q_lens, page_table,
                       max_pages_per_seq, seq_lens, num_chunks, total_q, max_q_len,
                       softmax_scale, out, lse, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
