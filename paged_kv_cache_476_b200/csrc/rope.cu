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
// takes several rows of one token, so the table values (64 bytes a lane) and
// the page lookup are fetched once for them.
#include "common.cuh"
#include "kernels.h"
#include "tensor.cuh"

namespace pkv {

namespace {

using pf::fma2;
using pf::mul2;

constexpr int kRopeThreads = 64;
// Blocks of an SM (128 registers a thread) and rows a lane works on together, the
// next ones loading meanwhile, in items of more than one row.  Measured (us a call:
// 16,384 tokens of 32 / 8 heads; bf16 append of 8,900 tokens), in 512 threads an SM:
// 66 and 53 in blocks of 64 threads, 67.6 and 53 of 128, 70 and 55 of 256 (whose last
// warps hold the others' places); of 256, without the load ahead 80 and 68, with 4
// rows 77 and 65; in 768 threads 1 row 70 and 60, 2 rows 90 and 72 (spills).
constexpr int kRopeBlocks = 8;
constexpr int kRopeRows = 2;

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
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
template <int D, int kFmt, int kRows, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_kernel(const RopeParams p) {
  constexpr bool kAppend = kFmt >= 0;
  constexpr int L = D / 16;
  const int lane = threadIdx.x & 31;
  const int u = lane & (L - 1);
  // items: `per` rows of q, of k or (append) of v, of one token
  const int per = p.rows_per_item;
  const int nq = (p.num_q_heads + per - 1) / per;
  const int nk = (p.num_kv_heads + per - 1) / per;
  const uint32_t per_token = nq + (kAppend ? 2 : 1) * nk;
  const uint32_t item = (blockIdx.x * (uint32_t)kRopeThreads + threadIdx.x) / L;
  bool live = item < (uint32_t)p.tokens * per_token;
  const int tok = live ? (int)(item / per_token) : 0;
  const int part = live ? (int)(item - tok * per_token) : 0;
  const int kind = part < nq ? 0 : part < nq + nk ? 1 : 2;  // q, k, v
  const int row0 = (part - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * per;
  const int heads = kind == 0 ? p.num_q_heads : p.num_kv_heads;
  const int rows = live ? min(per, heads - row0) : 0;

  // The first rows' loads go out before anything waits.
  const Halves<L> hv{kind == 2 ? L : p.rot / 16};
  const int va = hv.first(u), vb = hv.second(u);
  const uint4* const src = reinterpret_cast<const uint4*>(
      (kind == 0   ? p.q + tok * p.q_stride
       : kind == 1 ? p.k + tok * p.k_stride
                   : p.v + tok * p.v_stride) + (int64_t)row0 * D);
  uint4 ra[kRows], rb[kRows];
  auto load = [&](int r0, uint4* a, uint4* b) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      a[r] = b[r] = make_uint4(0, 0, 0, 0);
      if (r0 + r < rows) {
        a[r] = src[(r0 + r) * (D / 8) + va];  // plain loads: the output may be the input's buffer
        b[r] = src[(r0 + r) * (D / 8) + vb];
      }
    }
  };
  load(0, ra, rb);

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
        const bool report = kind == 1 && row0 == 0 && u == 0;
        if (at < 0 || at >= (int64_t)p.a.max_pages * p.a.page_size) {
          if (report) flag_error(p.a.flags, PKV_FLAG_BAD_LENGTH);
        } else {
          const int shift = p.a.page_size == 128 ? 7 : 6;  // (64 otherwise)
          const int j = (int)at >> shift;
          slot = (int)at - (j << shift);
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

  // What a lane's 16 values are multiplied with: z_a = x_a P + y_a Q and z_b =
  // x_b R + y_b S, where y is the pair's other value.  P, Q, R and S hold cosine
  // and sine times the weight of the value they meet, so that with the row's
  // 1 / rms a value costs three operations; two values go in one instruction.
  const bool turns = kind != 2 && u < p.rot / 16;
  const float* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
  float2 P[4], Q[4], R[4], S[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    P[i] = R[i] = make_float2(1.f, 1.f);
    Q[i] = S[i] = make_float2(0.f, 0.f);
  }
  if (weight) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(weight + 8 * va) + h);
      const float4 y = __ldg(reinterpret_cast<const float4*>(weight + 8 * vb) + h);
      P[2 * h] = make_float2(x.x, x.y), P[2 * h + 1] = make_float2(x.z, x.w);
      R[2 * h] = make_float2(y.x, y.y), R[2 * h + 1] = make_float2(y.z, y.w);
    }
  }
  if (turns && live) {
    const float* row = p.cos_sin + pos * p.rot;
    if constexpr (kInterleaved) {
      // pairs (2i, 2i + 1) of one vector: z = x (c, c) + swapped x (-s, s)
      auto turn = [&](int v, float2* x, float2* y) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * v));
        const float4 n = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2 + 4 * v));
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = make_float2(-x[i].y * sn[i], x[i].x * sn[i]);
          x[i] = make_float2(x[i].x * cs[i], x[i].y * cs[i]);
        }
      };
      turn(va, P, Q);
      turn(vb, R, S);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(row + 8 * u) + h);
        const float4 n = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2 + 8 * u) + h);
        const float2 cs[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
        const float2 sn[2] = {make_float2(n.x, n.y), make_float2(n.z, n.w)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 x = P[2 * h + i], y = R[2 * h + i];
          P[2 * h + i] = make_float2(x.x * cs[i].x, x.y * cs[i].y);
          Q[2 * h + i] = make_float2(-y.x * sn[i].x, -y.y * sn[i].y);
          R[2 * h + i] = make_float2(y.x * cs[i].x, y.y * cs[i].y);
          S[2 * h + i] = make_float2(x.x * sn[i].x, x.y * sn[i].y);
        }
      }
    }
  }

  // (every lane of a warp takes as many turns: the shuffles are its groups' own,
  // but rows of a warp may differ in kind)
  const int turns_all = __reduce_max_sync(0xffffffffu, rows);
  for (int r0 = 0; r0 < turns_all; r0 += kRows) {
    uint4 na[kRows], nb[kRows];
    load(r0 + kRows, na, nb);  // the next rows (if any), while these are worked on
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const bool row_live = live && r0 + r < rows;
      const uint32_t* wa = reinterpret_cast<const uint32_t*>(&ra[r]);
      const uint32_t* wb = reinterpret_cast<const uint32_t*>(&rb[r]);
      // every lane takes the shuffles: rows of a warp may differ in kind
      float inv = 1.f;
      if (kind != 2 && weight) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 xa = bf16_pair(wa[i]), xb = bf16_pair(wb[i]);
          ss = fma2(xa, xa, ss);
          ss = fma2(xb, xb, ss);
        }
        float sum = ss.x + ss.y;
        const uint32_t mask = (L == 32 ? 0xffffffffu : ((1u << L) - 1)) << (lane & ~(L - 1));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(mask, sum, o);
        inv = rsqrtf(sum * (1.f / D) + p.eps);
      }
      float xa[8], xb[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = bf16_pair(wa[i]), b = bf16_pair(wb[i]);
        float2 za = a, zb = b;
        if (kind != 2) {
          const float2 inv2 = make_float2(inv, inv);
          za = mul2(a, P[i]);
          zb = mul2(b, R[i]);
          if (turns) {  // (a branch, not zeros: 0 times an infinity is NaN)
            const float2 ya = kInterleaved ? make_float2(a.y, a.x) : b;
            const float2 yb = kInterleaved ? make_float2(b.y, b.x) : a;
            za = fma2(ya, Q[i], za);
            zb = fma2(yb, S[i], zb);
          }
          za = mul2(za, inv2);
          zb = mul2(zb, inv2);
        }
        xa[2 * i] = za.x, xa[2 * i + 1] = za.y;
        xb[2 * i] = zb.x, xb[2 * i + 1] = zb.y;
      }
      if (kind == 0 || !kAppend) {
        if (row_live) {
          __nv_bfloat16* out = kind == 0 ? p.q_out + (int64_t)tok * p.num_q_heads * D
                                         : p.k_out + (int64_t)tok * p.num_kv_heads * D;
          uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)(row0 + r0 + r) * D);
          dst[va] = pack8(xa);
          dst[vb] = pack8(xb);
        }
      } else if constexpr (kAppend) {
        const int g = row0 + r0 + r;
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
#pragma unroll
    for (int r = 0; r < kRows; ++r) ra[r] = na[r], rb[r] = nb[r];
  }
}

template <int D, int kFmt, int kRows>
cudaError_t rope_launch(const RopeParams& p, int64_t items, cudaStream_t stream) {
  const int64_t blocks = (items * (D / 16) + kRopeThreads - 1) / kRopeThreads;
  if (blocks == 0) return cudaSuccess;
  if (blocks * kRopeThreads > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (p.interleaved)
    rope_kernel<D, kFmt, kRows, true>
        <<<(unsigned)blocks, kRopeThreads, 0, stream>>>(p);
  else
    rope_kernel<D, kFmt, kRows, false>
        <<<(unsigned)blocks, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// kFmt -1: no cache
template <int kFmt>
cudaError_t rope_run(RopeParams p, int head_dim, int num_sms, cudaStream_t stream) {
  auto items = [&](int per) -> int64_t {
    const int nq = (p.num_q_heads + per - 1) / per, nk = (p.num_kv_heads + per - 1) / per;
    return (int64_t)p.tokens * (nq + (kFmt >= 0 ? 2 : 1) * nk);
  };
  // As many rows an item as leave every SM 384 threads: the way to the first product
  // costs a lane as much as two rows.
  const int64_t enough = (int64_t)num_sms * 384 / (head_dim / 16);
  int per = 8;
  while (per > 1 && items(per) < enough) per /= 2;
  p.rows_per_item = per;
  const int64_t n = items(per);
  if (head_dim == 128)
    return per > 1 ? rope_launch<128, kFmt, kRopeRows>(p, n, stream)
                   : rope_launch<128, kFmt, 1>(p, n, stream);
  return per > 1 ? rope_launch<64, kFmt, kRopeRows>(p, n, stream)
                 : rope_launch<64, kFmt, 1>(p, n, stream);
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
