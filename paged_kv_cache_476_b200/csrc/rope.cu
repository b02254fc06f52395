// Head norms and position rotation of queries and keys, alone or on the way
// into the paged cache.
//
// The attention entry points take q and K as the scores need them: normalised
// per head where the model does so, and rotated by their position.  The pages
// leave that step to the model; here it is one pass over the projections'
// output.  For a row x of D values at position pos,
//   y = x * w / sqrt(mean(x^2) + eps)             (with weights; else y = x)
//   z_i = y_i c_i - y_j s_i,  z_j = y_j c_i + y_i s_i
// for the rot/2 pairs (i, j) = (i, i + rot/2), or (2i, 2i + 1) interleaved,
// with c_i, s_i the table's cosine and sine of pos * angle_i; values past
// rot keep y.  All in fp32 from the bf16 inputs and rounded once: to bf16, or
// for the cached K of a quantised pool straight to its codes (no bf16 step
// between, which would round twice).  V is stored as paged_kv_append stores
// it.
//
// Bound: HBM bytes (about ten operations a value) for long batches, latency
// for decode steps.  D/16 lanes hold a row, 16 values (two 16-byte vectors)
// a lane, chosen so that both members of every pair sit in one lane: vectors
// u and u + rot/16 of the rotated part (and likewise two of the rest).  The
// rotation then needs no exchange, the norm log2(D/16) shuffles.  A lane
// takes kRows rows of one token, so the table values (64 bytes a lane) and
// the page lookup are fetched once for them and all their loads are in
// flight together.
#include "common.cuh"
#include "kernels.h"

namespace pkv {

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& r, float* x) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(p[k]);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ void load8(const float* src, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(src));
  const float4 b = __ldg(reinterpret_cast<const float4*>(src) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// Which 8-value vectors of a row of 2L vectors lane u holds: the first 2h
// vectors in pairs (u, u + h), the rest in pairs (L - h) apart.
template <int L>
struct Halves {
  int h;
  __device__ __forceinline__ int first(int u) const { return u < h ? u : h + u; }
  __device__ __forceinline__ int second(int u) const { return u < h ? u + h : L + u; }
  // lane and slot (0 first, 1 second) that hold vector v
  __device__ __forceinline__ int lane(int v) const {
    return v < h ? v : v < 2 * h ? v - h : v < L + h ? v - h : v - L;
  }
  __device__ __forceinline__ int slot(int v) const {
    return v < 2 * h ? (v >= h ? 1 : 0) : (v >= L + h ? 1 : 0);
  }
};

// Sequence of new token `tok` by a search of the L lanes of a row together
// (L probes a step): the last b with cu[b] <= tok; -1 for tokens before the
// first sequence or behind the last.  Every lane of the warp calls it.
template <int L>
__device__ __forceinline__ int owner_of_lanes(const int32_t* cu, int batch, int tok, int u,
                                              int lane) {
  // a decode step's common case, one token each, costs one round of loads
  const bool in = tok >= 0 && tok < batch;
  const int lo_c = in ? __ldg(cu + tok) : 1, hi_c = in ? __ldg(cu + tok + 1) : 0;
  const int last = __ldg(cu + batch), first = __ldg(cu);
  const bool direct = in && lo_c <= tok && tok < hi_c;
  if (__all_sync(0xffffffffu, direct || tok >= last || tok < first)) {
    return direct ? tok : -1;
  }
  int lo = 0, n = batch;  // the answer lies in [lo, lo + n)
  while (n > 1) {         // n is the same in every lane
    const int step = (n + L) / (L + 1);
    const int at = lo + (u + 1) * step;
    const bool below = at < batch && (u + 1) * step < n && __ldg(cu + at) <= tok;
    const uint32_t votes = __ballot_sync(0xffffffffu, below) >> (lane & ~(L - 1)) & ((1u << L) - 1);
    lo += __popc(votes) * step;  // cu ascends, so the votes are a prefix
    n = step;
  }
  return tok >= first && tok < last ? lo : -1;
}

// One 8-value vector of K or V to its place in a one-byte pool, or its codes
// of an FP4 pool (unit d of its block).
template <int kFmt>
__device__ __forceinline__ void store_codes(uint8_t* pool, int64_t row, int D, int vec,
                                            const float* x, float s, float d) {
  if constexpr (fp4(kFmt)) {
    *reinterpret_cast<uint32_t*>(pool + row * (D / 2) + vec * 4) = nvfp4_codes8(x, d);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = (uint32_t)encode8x2<kFmt>(make_float2(x[4 * k], x[4 * k + 1]), s) |
             (uint32_t)encode8x2<kFmt>(make_float2(x[4 * k + 2], x[4 * k + 3]), s) << 16;
    *reinterpret_cast<uint2*>(pool + row * D + vec * 8) = make_uint2(w[0], w[1]);
  }
}

__device__ __forceinline__ float amax8(const float* x) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));  // fmaxf drops NaN
  return m;
}

// kFmt < 0: no cache, rotated k to k_out.
template <int D, int kFmt, int kRows>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  constexpr bool kAppend = kFmt >= 0;
  constexpr int L = D / 16;
  const int lane = threadIdx.x & 31;
  const int u = lane & (L - 1);
  // items: kRows rows of q, of k or (append) of v, of one token
  const int nq = (p.num_q_heads + kRows - 1) / kRows;
  const int nk = (p.num_kv_heads + kRows - 1) / kRows;
  const int per_token = nq + (kAppend ? 2 : 1) * nk;
  const int64_t item = (blockIdx.x * (int64_t)kRopeThreads + threadIdx.x) / L;
  bool live = item < (int64_t)p.tokens * per_token;
  const int tok = live ? (int)(item / per_token) : 0;
  const int part = live ? (int)(item - (int64_t)tok * per_token) : 0;
  const int kind = part < nq ? 0 : part < nq + nk ? 1 : 2;  // q, k, v
  const int row0 = (part - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * kRows;
  const int heads = kind == 0 ? p.num_q_heads : p.num_kv_heads;

  // All of the item's loads, before anything waits on them.
  const Halves<L> hv{kind == 2 ? L : p.rot / 16};
  const int va = hv.first(u), vb = hv.second(u);
  uint4 ra[kRows], rb[kRows];
  {
    const __nv_bfloat16* src = kind == 0   ? p.q + tok * p.q_stride
                               : kind == 1 ? p.k + tok * p.k_stride
                                           : p.v + tok * p.v_stride;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      ra[r] = rb[r] = make_uint4(0, 0, 0, 0);
      if (live && row0 + r < heads) {
        const uint4* x = reinterpret_cast<const uint4*>(src + (int64_t)(row0 + r) * D);
        ra[r] = x[va];  // plain loads: the output may be the input's buffer
        rb[r] = x[vb];
      }
    }
  }

  // Position of the token, and (append) its place in the cache.
  int64_t pos = 0;
  int32_t page = -1;
  int slot = 0;
  if constexpr (kAppend) {
    const int b = owner_of_lanes<L>(p.a.cu_new, p.a.batch, live ? tok : -1, u, lane);
    if (b < 0) live = false;
    if (live) {
      const int64_t at = (int64_t)__ldg(p.a.seq_lens_before + b) + (tok - __ldg(p.a.cu_new + b));
      pos = p.positions ? __ldg(p.positions + tok) : at;
      if (kind != 0) {
        const int64_t j = at / p.a.page_size;
        const bool report = kind == 1 && row0 == 0 && u == 0;
        if (at < 0 || j >= p.a.max_pages) {
          if (report) flag_error(p.a.flags, PKV_FLAG_BAD_LENGTH);
        } else {
          slot = (int)(at - j * p.a.page_size);
          page = __ldg(p.a.page_table + (int64_t)b * p.a.max_pages + j);
          if (page < 0 || page >= p.a.num_pages) {
            if (report) flag_error(p.a.flags, PKV_FLAG_BAD_PAGE);
            page = -1;
          }
        }
        if (page < 0) live = false;
      }
    }
  } else {
    if (live && p.rot) pos = __ldg(p.positions + tok);
  }
  if (p.rot && (pos < 0 || pos >= p.max_positions)) {
    // a token without a rotation is skipped whole, its V included
    if (live && part == 0 && u == 0) flag_error(p.a.flags, PKV_FLAG_BAD_LENGTH);
    live = false;
  }

  // cos and sin of this lane's eight pairs
  const bool turns = kind != 2 && u < p.rot / 16;
  float cs[8], sn[8];
  if (turns && live) {
    const float* row = p.cos_sin + pos * p.rot;
    if (p.interleaved) {
      const float4 c0 = __ldg(reinterpret_cast<const float4*>(row + 4 * va));
      const float4 c1 = __ldg(reinterpret_cast<const float4*>(row + 4 * vb));
      const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2 + 4 * va));
      const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2 + 4 * vb));
      cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
      cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
      sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
      sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    } else {
      load8(row + 8 * u, cs);
      load8(row + p.rot / 2 + 8 * u, sn);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = sn[i] = 0.f;
  }
  const float* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  float wa[8], wb[8];
  if (weight) {
    load8(weight + 8 * va, wa);
    load8(weight + 8 * vb, wb);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) wa[i] = wb[i] = 1.f;
  }

#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const bool row_live = live && row0 + r < heads;
    float xa[8], xb[8];
    unpack8(ra[r], xa);
    unpack8(rb[r], xb);
    if (kind != 2) {
      // every lane takes the shuffles: rows of a warp may differ in kind
      if (weight) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += xa[i] * xa[i] + xb[i] * xb[i];
        const uint32_t mask = (L == 32 ? 0xffffffffu : ((1u << L) - 1)) << (lane & ~(L - 1));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(mask, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xa[i] *= inv * wa[i];
          xb[i] *= inv * wb[i];
        }
      }
      if (turns) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = xa[2 * i], a1 = xa[2 * i + 1], b0 = xb[2 * i], b1 = xb[2 * i + 1];
            xa[2 * i] = a0 * cs[i] - a1 * sn[i];
            xa[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
            xb[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
            xb[2 * i + 1] = b1 * cs[4 + i] + b0 * sn[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = xa[i], b = xb[i];
            xa[i] = a * cs[i] - b * sn[i];
            xb[i] = b * cs[i] + a * sn[i];
          }
        }
      }
    }
    if (kind == 0 || !kAppend) {
      if (row_live) {
        __nv_bfloat16* out = kind == 0 ? p.q_out + (int64_t)tok * p.num_q_heads * D
                                       : p.k_out + (int64_t)tok * p.num_kv_heads * D;
        uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)(row0 + r) * D);
        dst[va] = pack8(xa);
        dst[vb] = pack8(xb);
      }
    } else if constexpr (kAppend) {
      const int g = row0 + r;
      uint8_t* pool = kind == 1 ? p.a.k_pool : p.a.v_pool;
      const int64_t prow = ((int64_t)page * p.num_kv_heads + g) * p.a.page_size + slot;
      if constexpr (kFmt == PKV_KV_BF16) {
        if (row_live) {
          uint4* dst = reinterpret_cast<uint4*>(pool + prow * D * 2);
          dst[va] = kind == 1 ? pack8(xa) : ra[r];  // V: the input bits
          dst[vb] = kind == 1 ? pack8(xb) : rb[r];
        }
      } else {
        float s = 1.f;
        if (row_live) {
          s = __ldg((kind == 1 ? p.a.k_scale : p.a.v_scale) +
                    (int64_t)page * p.num_kv_heads + g);
          if (!(s > 0.f && s <= 32768.f) && u == 0) flag_error(p.a.flags, PKV_FLAG_BAD_SCALE);
        }
        float da = 0.f, db = 0.f;
        if constexpr (fp4(kFmt)) {
          // a block is vectors 2m and 2m + 1; the other one's largest value
          // comes from the lane (of this row) that holds it
          const uint32_t mask = ((1u << L) - 1) << (lane & ~(L - 1));
          const float ma = amax8(xa), mb = amax8(xb);
          const int ja = hv.lane(va ^ 1), jb = hv.lane(vb ^ 1);
          const float fa0 = __shfl_sync(mask, ma, ja, L), fa1 = __shfl_sync(mask, mb, ja, L);
          const float fb0 = __shfl_sync(mask, ma, jb, L), fb1 = __shfl_sync(mask, mb, jb, L);
          uint32_t sba, sbb;
          da = nvfp4_block_unit(fmaxf(ma, hv.slot(va ^ 1) ? fa1 : fa0), s, &sba);
          db = nvfp4_block_unit(fmaxf(mb, hv.slot(vb ^ 1) ? fb1 : fb0), s, &sbb);
          if (row_live) {
            uint8_t* blocks = (kind == 1 ? p.a.k_blocks : p.a.v_blocks) + prow * (D / 16);
            if (!(va & 1)) blocks[va >> 1] = (uint8_t)sba;
            if (!(vb & 1)) blocks[vb >> 1] = (uint8_t)sbb;
          }
        }
        if (row_live) {
          store_codes<kFmt>(pool, prow, D, va, xa, s, da);
          store_codes<kFmt>(pool, prow, D, vb, xb, s, db);
        }
      }
    }
  }
}

template <int D, int kFmt, int kRows>
cudaError_t rope_launch(const RopeParams& p, cudaStream_t stream) {
  const int nq = (p.num_q_heads + kRows - 1) / kRows;
  const int nk = (p.num_kv_heads + kRows - 1) / kRows;
  const int64_t items = (int64_t)p.tokens * (nq + (kFmt >= 0 ? 2 : 1) * nk);
  const int64_t blocks = (items * (D / 16) + kRopeThreads - 1) / kRopeThreads;
  if (blocks == 0) return cudaSuccess;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  rope_kernel<D, kFmt, kRows><<<(unsigned)blocks, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// kFmt -1: no cache
template <int kFmt>
cudaError_t rope_run(const RopeParams& p, int head_dim, int num_sms, cudaStream_t stream) {
  const int64_t rows =
      (int64_t)p.tokens * (p.num_q_heads + (kFmt >= 0 ? 2 : 1) * p.num_kv_heads);
  // One row a lane while that still leaves SMs idle; then four.
  const bool few = rows * (head_dim / 16) <= (int64_t)num_sms * 1024;
  if (head_dim == 128)
    return few ? rope_launch<128, kFmt, 1>(p, stream) : rope_launch<128, kFmt, 4>(p, stream);
  return few ? rope_launch<64, kFmt, 1>(p, stream) : rope_launch<64, kFmt, 4>(p, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeParams& p, int head_dim, int num_sms,
                                cudaStream_t stream) {
  return rope_run<-1>(p, head_dim, num_sms, stream);
}

cudaError_t launch_append_rope(const RopeParams& p, int fmt, int head_dim, int num_sms,
                               cudaStream_t stream) {
  switch (fmt) {
    case PKV_KV_NVFP4: return rope_run<PKV_KV_NVFP4>(p, head_dim, num_sms, stream);
    case PKV_KV_INT8: return rope_run<PKV_KV_INT8>(p, head_dim, num_sms, stream);
    case PKV_KV_FP8_E4M3: return rope_run<PKV_KV_FP8_E4M3>(p, head_dim, num_sms, stream);
    default: return rope_run<PKV_KV_BF16>(p, head_dim, num_sms, stream);
  }
}

}  // namespace pkv
