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

// Where a group's prefix is held.  Only members that hold the whole prefix share it,
// so its rows go from the first such member (whose table row names the pages) to the
// last: shorter members and padded rows at a group's ends cost nothing.  All 0 where
// nobody holds it.  Warp-wide.
__device__ __forceinline__ Span group_span(const DecodeParams& p, int g, int lane) {
  Span s = {0, 0, 0, 0};
  const int32_t n = group_tokens(p, g);
  if (n == 0) return s;
  const int32_t b0 = __ldg(p.cu_groups + g), b1 = __ldg(p.cu_groups + g + 1);
#pragma unroll 1
  for (int base = b0; base < b1; base += 32) {
    const int b = base + lane;
    const uint32_t hit =
        __ballot_sync(0xffffffffu, b < b1 && __ldg(p.seq_lens + min(b, b1 - 1)) >= n);
    if (hit == 0) continue;
    if (s.holders == 0) s.b0 = base + __ffs(hit) - 1;
    s.b1 = base + 32 - __clz(hit);
    s.holders += __popc(hit);
    s.prefix = n;
  }
  return s;
}

// The span of group base + lane (of none past the last): small groups a lane each,
// larger ones by the warp.  Warp-wide.
__device__ __forceinline__ Span make_span(const DecodeParams& p, int base, int lane) {
  Span mine = {0, 0, 0, 0};
  const int g = base + lane;
  const int32_t n = g < p.num_groups ? group_tokens(p, g) : 0;
  bool large = false;
  if (n > 0) {
    const int32_t b0 = __ldg(p.cu_groups + g), b1 = __ldg(p.cu_groups + g + 1);
    large = b1 - b0 > 32;
    if (!large) {
#pragma unroll 4
      for (int b = b0; b < b1; ++b) {
        if (__ldg(p.seq_lens + b) < n) continue;
        if (mine.holders == 0) mine.b0 = b;
        mine.b1 = b + 1;
        ++mine.holders;
        mine.prefix = n;
      }
    }
  }
#pragma unroll 1
  for (uint32_t todo = __ballot_sync(0xffffffffu, large); todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1;
    const Span s = group_span(p, base + l, lane);
    if (l == lane) mine = s;
  }
  return mine;
}

// All groups' spans to `a` and `b` (either may be null), by `warps` warps together.
__device__ __forceinline__ void plan_spans(const DecodeParams& p, Span* a, Span* b, int warp,
                                           int warps, int lane) {
  if (p.num_groups <= 4 * warps) {  // a warp each
#pragma unroll 1
    for (int g = warp; g < p.num_groups; g += warps) {
      const Span s = group_span(p, g, lane);
      if (lane == 0 && a) a[g] = s;
      if (lane == 0 && b) b[g] = s;
    }
    return;
  }
#pragma unroll 1
  for (int base = 32 * warp; base < p.num_groups; base += 32 * warps) {
    const Span s = make_span(p, base, lane);
    if (base + lane < p.num_groups) {
      if (a) a[base + lane] = s;
      if (b) b[base + lane] = s;
    }
  }
}

// The span of group base + lane: as planned, or (kMake, null) made here.  Warp-wide.
template <bool kMake>
__device__ __forceinline__ Span span_of(const DecodeParams& p, const Span* spans, int base,
                                        int lane) {
  if (kMake && !spans) return make_span(p, base, lane);
  Span mine = {0, 0, 0, 0};
  if (base + lane < p.num_groups)
    *reinterpret_cast<int4*>(&mine) = *reinterpret_cast<const int4*>(spans + base + lane);
  return mine;
}

// A group's prefix work for one kv head: key tiles of 128, Q tiles of 128
// rows; a step is one of the one against one of the other.
struct GroupWork {
  int32_t b0, b1, prefix, tiles, q_tiles;
  int64_t steps;
};

__device__ __forceinline__ GroupWork group_work(const DecodeParams& p, const Span& s) {
  GroupWork w;
  w.b0 = s.b0;
  w.b1 = s.b1;
  w.prefix = s.prefix;
  w.tiles = (w.prefix + 127) / 128;
  w.q_tiles = ((w.b1 - w.b0) * p.group + 127) / 128;
  w.steps = (int64_t)w.tiles * w.q_tiles;
  return w;
}

// The two kernels run side by side: prefix CTAs (one per SM) that find no work
// leave at once, and decode CTAs take their SMs.  Both kernels work out the same
// division, in SM-microseconds as measured on B200 at D = 128 with both kernels
// running (of quantised pools more than the prefix kernel alone takes; used at D = 64
// too, where a bf16 tile takes 0.65 of it); results do not depend on it.
struct Division {
  int64_t steps;   // of the prefix kernel
  bool pairs;      // some group has two Q tiles
  int prefix_sms;  // SMs for the prefix kernel
};

// A 128-key tile against one or two Q tiles in the prefix kernel: bf16 its bytes
// at the SM's share of HBM (1.48) and the hand-offs between products and softmax
// (2.35); quantised the converters.
template <int kFmt>
__host__ __device__ constexpr float prefix_tile_cost(bool two) {
  return !quant(kFmt) ? (two ? 2.35f : 1.48f) : two ? 3.1f : fp4(kFmt) ? 1.75f : 1.45f;
}
// A group's heads beyond the first of a CTA: queries to fetch, partials to write.
template <int kFmt>
__host__ __device__ constexpr float prefix_unit_cost() { return quant(kFmt) ? 3.f : 2.f; }
// The same tile in the decode kernel: bf16 its bytes, quantised its arithmetic;
// and the end of a sequence's tiles.
template <int kFmt>
__host__ __device__ constexpr float own_tile_cost() {
  return quant(kFmt) ? 1.05f : 1.25f;
}
template <int kFmt>
__host__ __device__ constexpr float own_unit_cost() { return quant(kFmt) ? 0.85f : 0.35f; }
// How much longer the prefix kernel's way to its first product and from its last is.
template <int kFmt>
__host__ __device__ constexpr float prefix_lead() { return quant(kFmt) ? 2.5f : 1.5f; }

// Sum over the warp of counts (exact): one instruction where they are small.
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
  if (__all_sync(0xffffffffu, x < (1 << 26)))
    return __reduce_add_sync(0xffffffffu, (uint32_t)x);
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What the decode kernel would have to read if nothing were shared, a lane's part of
// the batch.
template <int kFmt>
__device__ __forceinline__ float unshared_cost(const DecodeParams& p, int lane) {
  float own = 0.f;
  const int32_t cap = p.max_pages * p.page_size;
#pragma unroll 1
  for (int b = lane; b < p.batch; b += 32) {
    const int32_t len = max(0, min(__ldg(p.seq_lens + b), cap));
    if (len > 0) own += (float)((len + 127) / 128) * own_tile_cost<kFmt>() + own_unit_cost<kFmt>();
  }
  return own;
}

// Warp-wide, from the lanes' unshared_cost; a prefix saves its holders' tiles.
template <int kFmt, bool kMake>
__device__ Division divide_sms(const DecodeParams& p, const Span* spans, float own, int lane) {
  float pre = 0.f;
  int64_t steps = 0, tiles = 0;
  bool two = false;
#pragma unroll 1
  for (int base = 0; base < p.num_groups; base += 32) {
    const Span s = span_of<kMake>(p, spans, base, lane);
    const GroupWork w = group_work(p, s);
    steps += w.steps;
    tiles += (int64_t)w.tiles * ((w.q_tiles + 1) >> 1);
    two |= w.q_tiles > 1;
    own -= (float)s.holders * w.tiles * own_tile_cost<kFmt>();
    pre += w.tiles * ((w.q_tiles >> 1) * prefix_tile_cost<kFmt>(true) +
                      (w.q_tiles & 1) * prefix_tile_cost<kFmt>(false)) +
           ((w.q_tiles + 1) >> 1) * prefix_unit_cost<kFmt>();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    own += __shfl_xor_sync(0xffffffffu, own, o);
    pre += __shfl_xor_sync(0xffffffffu, pre, o);
  }
  Division d;
  d.steps = warp_sum(steps) * p.num_kv_heads;
  d.pairs = __any_sync(0xffffffffu, two);
  const float n_tiles = (float)warp_sum(tiles) * p.num_kv_heads;
  own = fmaxf(own, 0.f) * p.num_kv_heads;
  pre *= p.num_kv_heads;
  // n SMs for the prefix so that both end together: pre / n + lead = own / (sms - n),
  // a quadratic in n; then no more of them than make the same number of tiles each.
  const float sms = (float)p.num_sms, lead = prefix_lead<kFmt>();
  const float h = lead * sms - pre - own;
  float n = own > 0.f ? (h + sqrtf(h * h + 4.f * lead * pre * sms)) / (2.f * lead) : sms;
  n = fmaxf(1.f, fminf(fminf(rintf(n), own > 0.f ? sms - 1.f : sms), n_tiles));
  n = ceilf(__fdividef(n_tiles, ceilf(__fdividef(n_tiles, n))));
  d.prefix_sms = d.steps > 0 ? max(1, min((int)n, p.num_sms)) : 0;
  return d;
}

}  // namespace pkv
