// Groups of sequences that share a prefix: what each sequence shares, and how
// the SMs are divided between the prefix kernel and the decode kernel.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace pkv {

// Tokens that the sequences of group g share: sequences [cu_groups[g],
// cu_groups[g + 1]) share their first prefix_lens[g] tokens, rounded down to
// whole pages.  0 for a group of one sequence, whose prefix is read no more
// often than any other token of it, and for bounds outside the batch.
__device__ __forceinline__ int32_t group_tokens(const DecodeParams& p, int g) {
  const int32_t b0 = __ldg(p.cu_groups + g), b1 = __ldg(p.cu_groups + g + 1);
  const int32_t pages = __ldg(p.prefix_lens + g) / p.page_size;  // < 1 for negative lengths
  if (b0 < 0 || b1 > p.batch || b1 - b0 < 2) return 0;
  return max(0, min(pages, p.max_pages)) * p.page_size;
}

// Tokens of sequence b (of `len` tokens) that it shares with its group: 0
// outside the groups.  A sequence that does not hold the whole prefix shares
// nothing: all its tokens are its own, so it needs no mask in the prefix part,
// and no value behind its end can reach it.
__device__ __forceinline__ int32_t shared_tokens(const DecodeParams& p, int b, int32_t len) {
  int lo = 0, hi = p.num_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu_groups + mid) <= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  if (b < __ldg(p.cu_groups + lo) || b >= __ldg(p.cu_groups + lo + 1)) return 0;
  const int32_t n = group_tokens(p, lo);
  return len >= n ? n : 0;
}

// A group's prefix work for one kv head: key tiles of 128, Q tiles of 128
// rows; a step is one of the one against one of the other.
struct GroupWork {
  int32_t b0, b1, prefix, tiles, q_tiles;
  int64_t steps;
};

__device__ __forceinline__ GroupWork group_work(const DecodeParams& p, int g) {
  GroupWork w;
  w.b0 = __ldg(p.cu_groups + g);
  w.b1 = __ldg(p.cu_groups + g + 1);
  w.prefix = group_tokens(p, g);
  w.tiles = (w.prefix + 127) / 128;
  w.q_tiles = w.prefix > 0 ? ((w.b1 - w.b0) * p.group + 127) / 128 : 0;
  w.steps = (int64_t)w.tiles * w.q_tiles;
  return w;
}

// The two kernels run side by side: the prefix kernel's CTAs (one per SM) that
// find no work leave at once, and decode CTAs take their SMs.  Both work out
// the same division, in time of one SM; results do not depend on it.
struct Division {
  int64_t steps;   // of the prefix kernel
  bool pairs;      // some group has two Q tiles
  int prefix_sms;  // SMs for the prefix kernel
};

// Measured SM-microseconds (B200, D = 128): a 128-key tile costs the prefix
// kernel its bytes at the SM's share of HBM (44 GB/s a thousandth: 1.48 for bf16,
// 0.74 for one-byte codes), 0.95 for a quantised tile's conversion, and 0.57 a Q
// tile for the products and the softmax, whichever is most; it costs the decode
// kernel its bytes, or about 1.5 for quantised codes, and each unit's end 0.5.
template <int kFmt>
__device__ __forceinline__ float prefix_tile_cost(const DecodeParams& p, int q_tiles, int d) {
  const float bytes = 2.f * 128.f * (row_code_bytes(kFmt, d) + row_scale_bytes(kFmt, d));
  const float once = fmaxf(bytes * (1.f / 44300.f), quant(kFmt) ? 0.95f * d / 128.f : 0.f);
  return fmaxf(once, 0.57f * q_tiles);
}

template <int kFmt>
__device__ __forceinline__ float own_tile_cost(int d) {
  const float bytes = 2.f * 128.f * (row_code_bytes(kFmt, d) + row_scale_bytes(kFmt, d));
  return fmaxf(bytes * (1.f / 44300.f), quant(kFmt) ? 1.5f * d / 128.f : 0.f);
}
constexpr float kOwnUnitCost = 0.5f;

// Warp-wide.
template <int D, int kFmt>
__device__ Division divide_sms(const DecodeParams& p, int lane) {
  float own = 0.f, pre = 0.f;
  int64_t steps = 0;
  bool two = false;
  const int32_t cap = p.max_pages * p.page_size;
  for (int b = lane; b < p.batch; b += 32) {
    const int32_t len = max(0, min(__ldg(p.seq_lens + b), cap));
    if (len > 0) own += (float)((len + 127) / 128) * own_tile_cost<kFmt>(D) + kOwnUnitCost;
  }
  for (int g = lane; g < p.num_groups; g += 32) {
    const GroupWork w = group_work(p, g);
    if (w.steps == 0) continue;
    steps += w.steps;
    two |= w.q_tiles > 1;
    own -= (float)(w.b1 - w.b0) * w.tiles * own_tile_cost<kFmt>(D);
    for (int q = 0; q < w.q_tiles; q += 2)
      pre += w.tiles * prefix_tile_cost<kFmt>(p, min(2, w.q_tiles - q), D);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    own += __shfl_xor_sync(0xffffffffu, own, o);
    pre += __shfl_xor_sync(0xffffffffu, pre, o);
    steps += __shfl_xor_sync(0xffffffffu, steps, o);
  }
  Division d;
  d.steps = steps * p.num_kv_heads;
  d.pairs = __any_sync(0xffffffffu, two);
  own = fmaxf(own, 0.f);
  const int sms = p.num_sms;
  d.prefix_sms = (int)rintf(sms * pre / fmaxf(pre + own, 1e-6f));
  d.prefix_sms = max(d.steps > 0 ? 1 : 0, min(d.prefix_sms, own > 0.f ? sms - 1 : sms));
  return d;
}

}  // namespace pkv
