// Decode attention for a batch whose sequences share long prefixes (sm_100a,
// tcgen05): the prefix part and the merge.
//
// What it computes: paged_decode_attention's function, for groups of
// sequences whose first tokens are the same pages.  Softmax over a union of
// key sets is the sum of the sets' parts,
//   M = max_i m_i,  out = sum_i e^(m_i - M) o_i / sum_i e^(m_i - M) l_i,
// with m_i, l_i = sum e^(s - m_i), o_i = sum e^(s - m_i) v over part i.  So
// the queries of a whole group (n sequences x G heads of a kv head) attend to
// the prefix together, one read of its K and V for all, the decode kernel
// attends to each sequence's own tokens, and a merge adds the parts up.
//
// The prefix kernel.
//  * Bound: HBM bytes of the prefix for one Q tile of bf16 (1.4 us a 128-key tile
//    and SM at head_dim 128: the SM's share); the cycle of a slot, its softmax, the
//    products and the hand-offs between them, for two (2.35 us a tile; E4M3 2.2, INT8
//    and FP4 2.5); the converters for one Q tile of quantised pools (E4M3 1.25 us,
//    INT8 and FP4 1.45).  These are the kernel's alone; beside the decode kernel the
//    quantised ones take longer (3.0 for two E4M3 tiles).  At head_dim 64: 0.95 and
//    2.0 (bf16), 1.15 to 1.2 and 2.15.  16 sequences behind 65,536 bf16 tokens of 8 kv
//    heads: 54 us, 4.9 TB/s, of which 6 us pass before the first tile has landed.
//  * Items.  A group's rows of one kv head are cut into pairs of 128-row Q
//    tiles, A and B.  An item is (group, kv head, pair) over the prefix's
//    128-key tiles.  The items' steps (a tile times one Q tile) in order are
//    split into equal ranges, one per CTA (one CTA per SM), as decode splits
//    its work list; a range's part of an item is a segment, whose (m, l, o)
//    goes to the workspace.
//  * An item with one Q tile alternates the key tiles between the two
//    accumulators (slot 0 the even ones, slot 1 the odd), so that one slot's
//    softmax runs under the other's products there too; both slots leave
//    partials.
//  * Roles: warps 0-3 and 4-7 softmax of slot 0 and 1, one TMEM lane a row;
//    warp 8 loads (Q by a 3-D map, K and V tiles page by page into rings);
//    warp 9 issues the MMAs, S = Q K^T and O += P V with P from TMEM; warp 10
//    walks the work list and hands out segments.  Step i of a segment belongs
//    to slot i & 1 whatever the mode: step i's PV, then step i + 2's S.
//  * Each role walks the segments on its own; only barriers on the data tie
//    them, so loads (and conversions) run ahead across segments.
//  * Quantised K and V: four warps convert K's codes exactly to f16 and four V's
//    and, at a segment's start, Q's rows (times powers of two); the K scales
//    multiply the scores of their 64-key block, the V scales ride on P.  The
//    softmax warps take the registers that the other warps give up.  (K and V
//    apart: a conversion is 0.6 us and the hand-offs around it 0.4, and V's wait
//    for the softmax must not hold K up.)
//  * Every wait is bounded; a timeout ends the CTA with the error flag set.
#include <mutex>

#include "common.cuh"
#include "groups.cuh"
#include "kernels.h"
#include "tensor.cuh"

namespace pkv {

namespace sh {

using namespace pf;

// Warps: 0-3 and 4-7 softmax of slot 0 and 1, then the roles below; quantised
// pools add two warpgroups of converters.
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kSchedWarp = 10;  // warp 11 only checks the groups
constexpr int kConvWarp0 = 12;
constexpr int kConvWarps = 4;  // for K, and as many for V
constexpr int kConvThreads = kConvWarps * 32;
constexpr int kSegRing = 2;  // segment descriptors ahead
// Barriers that say Q is converted.  A one-tile segment's queries give way to the
// next one's once its S is issued, with no word from the softmax, and a slot
// without steps holds nobody up: a softmax warp that is about to wait for segment
// k's Q may find k + 1's and k + 2's converted (not k + 3's: its descriptor
// waits for every warp to take k + 1's).  With fewer than four barriers the
// parity it waits for could have gone by.
constexpr int kQRing = 4;
// A facts slot is refilled when the K ring has let go of a tile (at most
// kMaxStages tiles back); the softmax may be three tiles behind that.
constexpr int kMaxStages = 5;
constexpr int kFactsRing = 16;
constexpr int kPairRows = 2 * kRows;
constexpr int kMaxSegments = 1 << 16;     // more than any GPU has SMs
constexpr float kTiny = 1.17549435e-38f;       // smallest normal fp32
constexpr float kSumUnit = 1.f / (1ull << 60);  // unit of l for quantised pools
// A V scale more than 2^64 below the segment's largest so far (a page of zeros may
// have the smallest float) would take P, and with it the row sum's share, out of
// fp32's range.  Such a block's weights are held as if its scale were 2^64 below,
// for the sum; its values, 2^-64 of the others', are left out.
constexpr float kScaleReach = 64.f;

// Registers of the softmax, the load / product / scheduler and the converter
// warps for quantised pools: 256 x 144 + 128 x 64 + 256 x 64 = 640 x 96, what
// the block is launched with.  (152 / 80 / 48: 29 in place of 26 us for the FP4
// prefixes of 48 rows, 168 / 64 / 40: 31; one-byte pools within 3 %.)
constexpr int kSoftmaxRegs = 144, kIssueRegs = 64, kConvRegs = 64, kLaunchRegs = 96;
static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs + 256 * kConvRegs <= 640 * kLaunchRegs, "");

constexpr int kNoValue = 4;
struct TileFacts {
  int32_t bad;  // bit per 64-key block: rejected page; times kNoValue: for the sum alone
  float ks[2];  // K scales of the blocks' pages
  float lv[2];  // log2 of the V scales
  float iv[2];  // kSumUnit over the V scales
};

// One CTA's part of an item.
struct Segment {
  int32_t b0, b1;    // sequences of the item
  int32_t b_table;   // sequence whose table row holds the prefix's pages
  int32_t head;
  int32_t rows;      // (b1 - b0) * G
  int32_t prefix;    // tokens
  int32_t tile0, n;  // key tiles of the segment; n = 0: no more segments
  int32_t row_base;  // first partial row of the segment
};

// Barriers and small state in front of the tiles.
struct Control {
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  uint64_t q_full, q_empty;       // Q landed, free again
  uint64_t qc_full[kQRing];       // Q converted, by segment in turn
  uint64_t k_full[kMaxStages + 1], k_empty[kMaxStages + 1];
  uint64_t v_full[kMaxStages + 1], v_empty[kMaxStages + 1];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t kc_full[2], kc_free[2], vc_full[2], vc_free[2];  // converted tiles
  uint64_t facts_full[kFactsRing];
  uint64_t done;
  TileFacts facts[kFactsRing];
  Segment seg[kSegRing];
  uint32_t tmem;
  int32_t idle;  // this CTA's range is empty
  // quantised pools: Q rows are 2^q_exp times f16, by segment parity and tile
  int8_t q_exp[2][2][kRows];
};

constexpr int kSmemLimit = 227 * 1024;
constexpr int kControlB = 2048;
static_assert(sizeof(Control) <= kControlB, "");

template <int D, int kFmt>
struct Smem {
  static constexpr int kHalves = D / 64;        // 128-byte column boxes per bf16 row
  static constexpr int kQB = kRows * D * 2;     // one Q tile
  static constexpr int kTileB = kKeys * D * 2;  // 16-bit K (or V) tile
  static constexpr int kHalfB = kKeys * 128;    // one 64-column half of a 16-bit tile
  static constexpr int kCodeRowB = row_code_bytes(kFmt, D);
  static constexpr int kScaleRowB = row_scale_bytes(kFmt, D);
  static constexpr int kCodesB = kKeys * kCodeRowB;
  static constexpr int kTileQB = kCodesB + kKeys * kScaleRowB;
  static constexpr int kOperandB = quant(kFmt) ? kTileQB : kTileB;  // K (or V) of a stage
  static constexpr int kStageB = 2 * kOperandB;
  static constexpr int kConvB = quant(kFmt) ? 3 * kTileB : 0;  // converted K, K, V
  static constexpr int kRoom = kSmemLimit - 1024 - kControlB - 2 * kQB - kConvB;
  static constexpr int kStages = kRoom / kStageB < kMaxStages ? kRoom / kStageB : kMaxStages;
  // An item with one Q tile leaves the other's place free.  Quantised pools use
  // it for a second converted V; bf16 at D = 128 for the K of a third stage, whose
  // V takes the rest of the room.
  static constexpr bool kExtra = !quant(kFmt) && kStages == 2 && kOperandB <= kQB &&
                                 kRoom - kStages * kStageB >= kOperandB;
  // (1024: the tiles' alignment)
  static constexpr int kBytes = 1024 + kControlB + 2 * kQB + kStages * kStageB + kConvB +
                                (kExtra ? kOperandB : 0);
  static_assert(kBytes <= kSmemLimit, "");
  static constexpr int kThreads = (kConvWarp0 + (quant(kFmt) ? 2 * kConvWarps : 0)) * 32;
  static_assert(kStages >= 2, "");
};

// A role's place in the K/V ring: the slot of its next tile and the parity of
// each slot's next fill.  Every role walks the same slots.
struct Ring {
  int slot = 0;
  uint32_t parities = 0;
  __device__ __forceinline__ void enter(int depth) {
    if (slot >= depth) slot = 0;
  }
  __device__ __forceinline__ uint32_t parity() const { return (parities >> slot) & 1; }
  __device__ __forceinline__ void advance(int depth) {
    parities ^= 1u << slot;
    if (++slot >= depth) slot = 0;
  }
};

// ---------------------------------------------------------------- work list
// a / b for a >= 0, b > 0: in 32 bits where they suffice (a 64-bit division
// costs the start of every CTA half a microsecond).
__device__ __noinline__ int64_t long_quotient(int64_t a, int64_t b) { return a / b; }

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return long_quotient(a, b);
}

// T steps over C CTAs: the first `rest` take `each` + 1, the others `each`.
struct Split {
  int64_t each, rest;
  __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + min(c, rest); }
  // CTA whose range holds step x
  __device__ __forceinline__ int64_t cta_of(int64_t x) const {
    const int64_t big = rest * (each + 1);
    return x < big ? quotient(x, each + 1) : rest + quotient(x - big, each);
  }
};

// Position in the work list: group's work, head, pair of Q tiles, key tile.
struct Cursor {
  GroupWork w;
  int32_t head, pair, tile;
  int64_t item_x;  // step index of the item's first step
};

// Q tiles of a group's pair.
__device__ __forceinline__ int pair_tiles(const GroupWork& w, int pair) {
  return min(2, w.q_tiles - 2 * pair);
}

// Warp-wide: the tile that step x belongs to (x < T); tiles go to the range
// that holds their last step.
__device__ Cursor locate(const DecodeParams& p, const Span* spans, int64_t x, int lane) {
  Cursor c;
  int64_t run = 0;
  for (int base = 0; base < p.num_groups; base += 32) {
    Span mine = span_of<false>(p, spans, base, lane);
    const int64_t s = group_work(p, mine).steps * p.num_kv_heads;
    int64_t incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int64_t all = __shfl_sync(0xffffffffu, incl, 31);
    if (run + all > x) {
      const int l0 = __ffs(__ballot_sync(0xffffffffu, run + incl > x)) - 1;
      const int64_t before = run + __shfl_sync(0xffffffffu, incl - s, l0);
      mine.b0 = __shfl_sync(0xffffffffu, mine.b0, l0);
      mine.b1 = __shfl_sync(0xffffffffu, mine.b1, l0);
      mine.prefix = __shfl_sync(0xffffffffu, mine.prefix, l0);
      c.w = group_work(p, mine);
      int64_t off = x - before;
      c.head = (int)quotient(off, c.w.steps);
      off -= c.head * c.w.steps;
      c.pair = (int)quotient(off, 2 * (int64_t)c.w.tiles);
      off -= c.pair * 2 * (int64_t)c.w.tiles;
      c.tile = (int)(pair_tiles(c.w, c.pair) == 2 ? off >> 1 : off);
      c.item_x = x - off;
      return c;
    }
    run += all;
  }
  c.w = GroupWork{};  // not reached for x < T
  c.head = c.pair = c.tile = 0;
  c.item_x = run;
  return c;
}

// Groups that run backwards or leave the batch, and negative prefixes.  Warp-wide.
__device__ void check_groups(const DecodeParams& p, int lane) {
  for (int g = lane; g < p.num_groups; g += 32) {
    const int32_t b0 = __ldg(p.cu_groups + g), b1 = __ldg(p.cu_groups + g + 1);
    if (b0 < 0 || b1 < b0 || b1 > p.batch || __ldg(p.prefix_lens + g) < 0)
      flag_error(p.flags, PKV_FLAG_BAD_LENGTH);
  }
}

// A landed tile of codes to f16 (exact: every E4M3 and INT8 value is one, and an
// FP4 value times its block scale has at most 6 significant bits in [2^-10,
// 2688]), laid out as TMA lays out 16-bit tiles.  Half h (64 rows, one page) is
// written as zeros unless bit h of `live` is set.  A thread makes 16-byte
// chunks of one column, eight threads a 128-byte line, so that neither its loads
// nor its stores meet in a bank; four units' loads come before their stores.
template <int D, int kFmt>
__device__ __forceinline__ void convert_codes(uint32_t src, uint32_t dst, int t, int live) {
  constexpr int kCols = D / 8;                  // 8-value columns of a row
  constexpr int kStep = kConvThreads / kCols;   // rows that the threads take at once
  constexpr int kUnits = 4;                     // a thread's units in flight
  constexpr int kRowB = row_code_bytes(kFmt, D);
  const int col = t % kCols, r0 = t / kCols;
  // rows kStep (8 or 16) apart have the same swizzle phase in both tiles
  const uint32_t to = bf16_chunk<D>(dst, r0, col);
  uint32_t from;
  if constexpr (fp4(kFmt))
    from = code_chunk<kRowB>(src, r0, col >> 2) + (col & 3) * 4;
  else
    from = code_chunk<kRowB>(src, r0, col >> 1) + (col & 1) * 8;
  const uint32_t scales = src + kKeys * kRowB + r0 * (D / 16) + (col >> 1);  // FP4
#pragma unroll 1
  for (int row0 = 0; row0 < kKeys; row0 += kUnits * kStep) {
    const bool on = (live >> (row0 >> 6)) & 1;
    uint32_t w[kUnits][2];
    if (on) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const int row = row0 + i * kStep;
        if constexpr (fp4(kFmt)) {
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i][0]) : "r"(from + row * kRowB));
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(w[i][1]) : "r"(scales + row * (D / 16)));
        } else {
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                       : "=r"(w[i][0]), "=r"(w[i][1])
                       : "r"(from + row * kRowB));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      uint32_t o[4] = {0u, 0u, 0u, 0u};
      if (on) {
        if constexpr (fp4(kFmt)) {
          const uint32_t s = e4m3_splat_f16x2(w[i][1], 0);
          e2m1x8_to_f16x2(w[i][0], o);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = hmul2_u32(o[e], s);
        } else {
          kv8x4_to_f16x2<kFmt>(w[i][0], o[0], o[1]);
          kv8x4_to_f16x2<kFmt>(w[i][1], o[2], o[3]);
        }
      }
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + (row0 + i * kStep) * 128),
                   "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                   : "memory");
    }
  }
}

// `rows` rows of a bf16 Q tile (128-byte swizzled column boxes) to f16 in place,
// row r times 2^q_exp[r], the power of two that puts its largest value in [2^14,
// 2^15): bf16's 8 bits fit f16's 11, and what is small enough to lose bits is
// 2^-28 of the largest.  Four threads share a row.
template <int D>
__device__ __forceinline__ void q_rows_to_f16(uint32_t base, int t, int rows, int8_t* q_exp,
                                              bool store) {
  constexpr int kChunks = D / 32;  // 16-byte chunks of a thread
#pragma unroll 1
  for (int r = t >> 2; r < ((rows + 7) & ~7); r += kConvThreads / 4) {  // whole warps
    uint32_t w[kChunks][4];
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c][2]), "=r"(w[c][3])
                   : "r"(bf16_chunk<D>(base, r, 4 * c + (t & 3))));
    __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // (drops NaN)
        top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[c][i])));
    uint32_t amax = __float_as_uint(fmaxf(__low2float(top), __high2float(top)));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // amax < 2^(field - 126); zeros and subnormals: 2^100
    const int e = min(100, 141 - (int)(amax >> 23));
    const float pre = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[c][i]));
        w[c][i] = pack_f16(f.x * pre, f.y * pre);
      }
      if (store)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                         bf16_chunk<D>(base, r, 4 * c + (t & 3))),
                     "r"(w[c][0]), "r"(w[c][1]), "r"(w[c][2]), "r"(w[c][3])
                     : "memory");
    }
    if (store && (t & 3) == 0) q_exp[r] = (int8_t)e;
  }
}

template <int kRegs, bool kMore>
__device__ __forceinline__ void set_registers() {
  if constexpr (kMore)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int D, int kFmt>
__global__ void __launch_bounds__(Smem<D, kFmt>::kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, const SharedParams sp) {
  using Sm = Smem<D, kFmt>;
  const DecodeParams& p = sp.d;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  Control& ct = *reinterpret_cast<Control*>(smem);
  uint8_t* sq = smem + kControlB;                // Q tile A, then Q tile B
  uint8_t* sconv = sq + 2 * Sm::kQB;             // quantised: 16-bit K, K, V
  uint8_t* skv = sconv + Sm::kConvB;             // stage s: K at s * kStageB, V after it
  auto k_slot = [&](int st) -> uint8_t* {
    if (Sm::kExtra && st == Sm::kStages) return sq + Sm::kQB;
    return skv + st * Sm::kStageB;
  };
  auto v_slot = [&](int st) -> uint8_t* {
    if (Sm::kExtra && st == Sm::kStages)
      return skv + Sm::kStages * Sm::kStageB;
    return skv + st * Sm::kStageB + Sm::kOperandB;
  };
  auto ring_depth = [](bool pairs) { return Sm::kStages + (Sm::kExtra && !pairs ? 1 : 0); };
  // converted V tiles: the second lies in Q tile B's place
  auto v_made = [&](int buf) -> uint8_t* { return buf ? sq + Sm::kQB : sconv + 2 * Sm::kTileB; };
  auto v_buffers = [](bool pairs) { return pairs ? 1 : 2; };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = p.group;
  const int TQ = kRows / G;  // sequences per Q tile

  // The decode kernel behind this one reads none of its results: its CTAs take
  // the SMs as they come free.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 1 && lane == 0) {
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(&ct.seg_full[s], 1);
      // producer, MMA, softmax warps, converters
      mbar_init(&ct.seg_empty[s], 2 + 8 + (quant(kFmt) ? 2 * kConvWarps : 0));
    }
    mbar_init(&ct.q_full, 1);
    mbar_init(&ct.q_empty, 1);
    for (int s = 0; s < kQRing; ++s) mbar_init(&ct.qc_full[s], kConvWarps);
    for (int s = 0; s < kMaxStages + 1; ++s) {
      mbar_init(&ct.k_full[s], 1);
      mbar_init(&ct.v_full[s], 1);
      // quantised: released by the converter warps
      mbar_init(&ct.k_empty[s], quant(kFmt) ? kConvWarps : 1);
      mbar_init(&ct.v_empty[s], quant(kFmt) ? kConvWarps : 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ct.s_full[x], 1);
      mbar_init(&ct.p_full[x], 4);
      mbar_init(&ct.o_full[x], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ct.kc_full[s], kConvWarps);
      mbar_init(&ct.kc_free[s], 1);
      mbar_init(&ct.vc_full[s], kConvWarps);
      mbar_init(&ct.vc_free[s], 1);
    }
    for (int s = 0; s < kFactsRing; ++s) mbar_init(&ct.facts_full[s], 1);
    mbar_init(&ct.done, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&ct.tmem, kTmemCols);
  if (warp == kSchedWarp + 1 && blockIdx.x == 0) check_groups(p, lane);
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
  }
  // This CTA's range of the work list and its first item, under the set-up.
  Split split{1, 0};
  int64_t x = 0, x_end = 0;
  Cursor cur{};
  // The groups' spans: for the start in place of the first tiles where they fit, for
  // later segments in the workspace.  By the warps that set nothing else up, with a
  // barrier of their own and the scheduler's (which would wait 1 us for the others).
  Span* const near = p.num_groups <= (int)(2 * Sm::kStageB / sizeof(Span))
                         ? reinterpret_cast<Span*>(skv) : nullptr;
  constexpr int kPlanWarp0 = 2, kPlanWarps = 6;
  constexpr int kPlanners = (kPlanWarps + 1) * 32;  // with the scheduler
  if (warp >= kPlanWarp0 && warp < kPlanWarp0 + kPlanWarps) {
    plan_spans(p, near, sp.spans, warp - kPlanWarp0, kPlanWarps, lane);
    asm volatile("bar.arrive 1, %0;" ::"n"(kPlanners) : "memory");
  }
  if (warp == kSchedWarp) {
    const float unshared = unshared_cost<kFmt>(p, lane);
    asm volatile("bar.sync 1, %0;" ::"n"(kPlanners) : "memory");
    const Span* spans = near ? near : sp.spans;
    const Division dv = divide_sms<kFmt, false>(p, spans, unshared, lane);
    const int64_t T = dv.steps;
    // Every range holds a whole tile (two steps of an item with two Q tiles).
    const int64_t most = min((int)gridDim.x, dv.prefix_sms);
    const int64_t ctas = max((int64_t)1, min(most, dv.pairs ? T >> 1 : T));
    split.each = quotient(T, ctas);
    split.rest = T - split.each * ctas;
    if (blockIdx.x < ctas) {
      x = split.begin(blockIdx.x);
      x_end = split.begin(blockIdx.x + 1);
    }
    if (x < x_end) {
      cur = locate(p, spans, x, lane);
      // the producer's first page ids
      const int64_t key0 = (int64_t)cur.tile * kKeys + lane * 64;
      if (key0 < cur.w.prefix)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(
            p.page_table + (int64_t)cur.w.b0 * p.max_pages + key0 / p.page_size));
    }
    if (lane == 0) ct.idle = x < x_end ? 0 : 1;
  }
  fence_async_smem();  // (the spans' place is the loads' from here on)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ct.tmem;
  if (ct.idle) {  // its SM goes to the decode kernel
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  // Segment number `k` (each warp that works on segments takes every one).
  auto take_segment = [&](uint32_t k, Segment* sg) -> bool {
    if (!mbar_wait(&ct.seg_full[k % kSegRing], (k / kSegRing) & 1, p.flags)) return false;
    *sg = ct.seg[k % kSegRing];
    return sg->n > 0;
  };

  if (warp < 8) {
    if constexpr (quant(kFmt)) set_registers<kSoftmaxRegs, true>();
    // ------------------------------------------------------------- softmax
    const int x = warp >> 2;   // slot
    const int wq = warp & 3;   // TMEM lane quadrant of this warp
    const int r = wq * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t colS = col_s(x), colO = col_o(x);
    uint32_t j0 = 0, steps = 0, outs = 0;  // key tiles, steps and O tiles so far
    bool ok = true;
    Segment sg{};
    // The first pass runs on whatever TMEM holds and leaves nothing behind: while
    // the first tiles load it brings the instructions of the loop to this SM,
    // which would cost the first real step 1.8 us.
    bool dry = take_segment(0, &sg);
    ok = dry;
    sg.rows = 0, sg.n = 1, sg.tile0 = 0, sg.prefix = kKeys;
    for (uint32_t k = 0; ok; k += dry ? 0 : 1, dry = false) {
      if (!dry) {
        if (!take_segment(k, &sg)) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.seg_empty[k % kSegRing]);
      }
      const bool pairs = sg.rows > kRows;
      const int mine = pairs ? sg.n : dry ? 1 : (sg.n + 1 - x) >> 1;  // steps of this slot
      float m_ref = -INFINITY, l = 0.f;
      float row_mul = p.scale_log2;
      if (quant(kFmt) && !dry) {  // (every segment: a phase left out would be mistaken later)
        if (!mbar_wait(&ct.qc_full[k % kQRing], (k / kQRing) & 1, p.flags)) { ok = false; break; }
        row_mul = ldexpf(p.scale_log2, -ct.q_exp[k & 1][pairs ? x : 0][r]);
      }
      for (int q = 0; q < mine; ++q) {
        const int i = pairs ? q : 2 * q + x;  // local key tile
        const uint32_t j = j0 + i;
        if (!dry && (!mbar_wait(&ct.s_full[x], (steps + q) & 1, p.flags) ||
                     !mbar_wait(&ct.facts_full[j % kFactsRing], (j / kFactsRing) & 1, p.flags))) {
          ok = false;
          break;
        }
        TileFacts tf = ct.facts[j % kFactsRing];
        if (dry) tf.bad = 0;
        tc_fence_after();
        const int32_t key0 = (sg.tile0 + i) * kKeys;
        const float mul0 = quant(kFmt) ? row_mul * tf.ks[0] : row_mul;
        const float mul1 = quant(kFmt) ? row_mul * tf.ks[1] : row_mul;
        // Quantised pools: the V scale of a 64-key block rides on P as an
        // exponent, P = 2^(s - m + log2 vs), and m bounds s + log2 vs, so that
        // the f16 P keeps its 11 bits whatever the scales are; the row sum takes
        // P / vs.  (m is a reference only: l and o carry the same 2^-m.)  l is
        // held 2^-60 smaller, so that it stays in range for every scale.
        const float lv0 = quant(kFmt) ? tf.lv[0] : 0.f, lv1 = quant(kFmt) ? tf.lv[1] : 0.f;
        const float iv0 = quant(kFmt) ? tf.iv[0] : 1.f, iv1 = quant(kFmt) ? tf.iv[1] : 1.f;
        // A block is live whole or not at all: pages, and with them the prefix,
        // end on 64 keys.
        const bool on0 = !(tf.bad & 1);
        const bool on1 = !(tf.bad & 2) && key0 + 64 < sg.prefix;
        // Max of a block: of the raw scores for positive multipliers (max(s) * mul
        // = max(s * mul)), else of the products.
        auto block_max = [&](const float* sv, float mul) -> float {
          float m0 = -INFINITY, m1 = -INFINITY;
          if (mul > 0.f) {
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              m0 = fmax3(m0, sv[e], sv[e + 1]);
              m1 = fmax3(m1, sv[e + 2], sv[e + 3]);
            }
            return fmaxf(m0, m1) * mul;
          }
#pragma unroll
          for (int e = 0; e < 64; ++e) m0 = fmaxf(m0, sv[e] * mul);
          return m0;
        };
        // The reference rises lazily, when a row's max has grown by 2^8 (P <= 2^8
        // in bf16 and in f16).  S of this step done implies the slot's earlier
        // products are, so O may be rescaled; this step's PV waits for its P.
        float alpha = 1.f;
        auto set_max = [&](float mt) -> float {
          const bool need = mt > m_ref + 8.f;
          const float m_new = need ? mt : m_ref;
          if (q >= 1 && need) {
            if constexpr (quant(kFmt)) {
              // (the sum reaches from 2^-75 to 2^94 and takes a factor below fp32's range)
              const float half = fast_exp2(0.5f * (m_ref - m_new));
              alpha = half * half;
              l = (l * half) * half;
            } else {
              alpha = fast_exp2(m_ref - m_new);
              l *= alpha;
            }
          }
          m_ref = m_new;
          return m_ref == -INFINITY ? 0.f : m_ref;
        };
        float mt = -INFINITY;
#pragma unroll
        for (int cb = 0; cb < kKeys; cb += 64) {
          float sv[64];
          tmem_ld32(tmem + lane_base + colS + cb, sv);
          tmem_ld32(tmem + lane_base + colS + cb + 32, sv + 32);
          tmem_wait_ld();
          if (cb < 64 ? on0 : on1)
            mt = fmaxf(mt, block_max(sv, cb < 64 ? mul0 : mul1) + (cb < 64 ? lv0 : lv1));
        }
        const float m_use = set_max(mt);
        float rs = 0.f;
#pragma unroll
        for (int cb = 0; cb < kKeys; cb += 64) {
          float sv[64];
          tmem_ld32(tmem + lane_base + colS + cb, sv);
          tmem_ld32(tmem + lane_base + colS + cb + 32, sv + 32);
          tmem_wait_ld();
          uint32_t pk[32];
          if (cb < 64 ? on0 : on1) {
            const float mul = cb < 64 ? mul0 : mul1, off = (cb < 64 ? lv0 : lv1) - m_use;
            float2 racc = make_float2(0.f, 0.f);
            const float2 mul_2 = make_float2(mul, mul), off_2 = make_float2(off, off);
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              const float2 t = fma2(make_float2(sv[e], sv[e + 1]), mul_2, off_2);
              const float2 pp = make_float2(fast_exp2(t.x), fast_exp2(t.y));
              racc = add2(racc, pp);
              pk[e / 2] = quant(kFmt) ? pack_f16(pp.x, pp.y) : pack_bf16(pp.x, pp.y);
            }
            rs += (racc.x + racc.y) * (cb < 64 ? iv0 : iv1);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) pk[e] = 0u;
          }
          // P column c/2 lies in an S column already read
          if (!dry) {
            tmem_st16(tmem + lane_base + colS + cb / 2, pk);
            tmem_st16(tmem + lane_base + colS + cb / 2 + 16, pk + 16);
          }
        }
        if (__any_sync(0xffffffffu, alpha != 1.f)) rescale_o<D>(tmem + lane_base + colO, alpha);
        l += rs;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !dry) mbar_arrive(&ct.p_full[x]);
      }
      // --------------------------------------------------------- partials
      // Rows of slot x: float4 vectors [D/4][rows of the slot], so that a warp's
      // lanes write consecutive 16 bytes; (m, l) beside them.  For quantised
      // pools o takes l's unit, and m makes up for it.
      if (!ok) break;
      constexpr float kUnit = quant(kFmt) ? kSumUnit : 1.f;
      const int nr = pairs ? (x ? sg.rows - kRows : kRows) : sg.rows;  // rows of the slot
      const bool out_ok = r < nr;
      const int64_t row0 = (int64_t)sg.row_base + (x ? min(sg.rows, kRows) : 0);
      // (no step or no live key: l = 0; NaN passes)
      if (out_ok) sp.pre_ml[row0 + r] = make_float2(m_ref + (quant(kFmt) ? 60.f : 0.f), l);
      if (mine > 0) {
        if (!dry) {
          if (!mbar_wait(&ct.o_full[x], outs & 1, p.flags)) { ok = false; break; }
          ++outs;
        }
        tc_fence_after();
        float4* dst = reinterpret_cast<float4*>(sp.pre_o) + row0 * (D / 4) + r;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tmem + lane_base + colO + c, o);
          tmem_wait_ld();
          if (out_ok) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              dst[(int64_t)((c + e) / 4) * nr] = make_float4(o[e] * kUnit, o[e + 1] * kUnit,
                                                             o[e + 2] * kUnit, o[e + 3] * kUnit);
          }
        }
      }
      if (!dry) {
        steps += mine;
        j0 += sg.n;
      }
    }
  } else if (warp < kConvWarp0) {
    if constexpr (quant(kFmt)) set_registers<kIssueRegs, false>();
    if (warp == kSchedWarp) {
      // ------------------------------------------------------------ scheduler
      // One descriptor per item that this CTA's range reaches.
      const int64_t c = blockIdx.x;
      uint32_t k = 0;
      bool first = true;  // `cur` is the item at x
      while (true) {
        Segment s{};
        if (x < x_end) {
          if (!first) cur = locate(p, sp.spans, x, lane);
          first = false;
          const int w = pair_tiles(cur.w, cur.pair);
          s.b0 = cur.w.b0 + cur.pair * 2 * TQ;
          s.b1 = min(cur.w.b1, s.b0 + 2 * TQ);
          s.b_table = cur.w.b0;
          s.head = cur.head;
          s.rows = (s.b1 - s.b0) * G;
          s.prefix = cur.w.prefix;
          s.tile0 = cur.tile;
          // tiles whose last step lies before the range's end
          const int64_t left = x_end - cur.item_x;
          s.n = (int)min((int64_t)cur.w.tiles, w == 2 ? left >> 1 : left) - s.tile0;
          // Items of one CTA lie 2 * rows apart, parts of an item kPairRows: no two
          // segments overlap, and the last ends by 2 * batch * heads + kPairRows * CTAs.
          const int64_t base = 2 * ((int64_t)p.num_kv_heads * cur.w.b0 * G +
                                    (int64_t)cur.head * (cur.w.b1 - cur.w.b0) * G +
                                    (int64_t)cur.pair * kPairRows);
          s.row_base = (int32_t)(base + (int64_t)kPairRows * c);
          if (s.tile0 == 0 && s.n > 0) {
            const int64_t c0 = split.cta_of(cur.item_x + w - 1);
            const int64_t c1 = split.cta_of(cur.item_x + (int64_t)cur.w.tiles * w - 1);
            const int4 info =
                make_int4((int)(base + kPairRows * c0), (int)(c1 - c0 + 1), s.b0, s.rows);
            for (int b = s.b0 + lane; b < s.b1; b += 32)
              sp.pre_info[(int64_t)b * p.num_kv_heads + s.head] = info;
          }
          x = cur.item_x + (int64_t)cur.w.tiles * w;
          if (s.n <= 0) continue;
        }
        if (!mbar_wait(&ct.seg_empty[k % kSegRing], ((k / kSegRing) & 1) ^ 1, p.flags)) break;
        if (lane == 0) {
          ct.seg[k % kSegRing] = s;
          mbar_arrive(&ct.seg_full[k % kSegRing]);
        }
        __syncwarp();
        ++k;
        if (s.n == 0) break;
      }
    } else if (warp == kProducerWarp) {
      // ------------------------------------------------------------- producer
      // The whole warp walks the tiles, lane 0 issues.  A lane looks up one of 32
      // consecutive 64-key blocks (16 tiles): page id, scales.
      const uint64_t pol = policy_evict_first();
      // bytes of one operand (K or V) per live 64-key block
      constexpr uint32_t kBlockBytes =
          quant(kFmt) ? 64u * (Sm::kCodeRowB + Sm::kScaleRowB) : Sm::kHalves * 64u * 128u;
      Ring ring;
      Ring v_ring;               // (quantised) as the converters walk V's buffers
      uint32_t j = 0, used = 0;  // key tiles so far; slots with a fill
      bool ok = true;
      Segment sg;
      for (uint32_t k = 0; ok && take_segment(k, &sg); ++k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.seg_empty[k % kSegRing]);
        const bool pairs = sg.rows > kRows;
        const int depth = ring_depth(pairs);
        ring.enter(depth);
        v_ring.enter(v_buffers(pairs));
        int my_bad = 0, my_live = 0;  // this lane's block: rejected page; to load
        int32_t my_y = 0;             // its first pool row
        float my_ks = 1.f, my_lv = 0.f, my_iv = 1.f;
        auto lookup = [&](int i) {
          const int32_t key0 = (sg.tile0 + i) * kKeys + lane * 64;
          my_bad = my_live = 0;
          if (key0 >= sg.prefix || key0 >= (sg.tile0 + sg.n) * kKeys) return;
          const int32_t pid =
              __ldg(p.page_table + (int64_t)sg.b_table * p.max_pages + key0 / p.page_size);
          if (pid < 0 || pid >= p.num_pages) {
            flag_error(p.flags, PKV_FLAG_BAD_PAGE);
            my_bad = 1;
            return;
          }
          if constexpr (quant(kFmt)) {
            my_ks = __ldg(p.k_scale + (int64_t)pid * p.num_kv_heads + sg.head);
            const float vs = __ldg(p.v_scale + (int64_t)pid * p.num_kv_heads + sg.head);
            if (!(my_ks > 0.f && my_ks <= 32768.f && vs > 0.f && vs <= 32768.f)) {
              flag_error(p.flags, PKV_FLAG_BAD_SCALE);
              my_bad = 1;
              return;
            }
            my_lv = log2f(fmaxf(vs, kTiny));
            my_iv = kSumUnit / fmaxf(vs, kTiny);
          }
          my_y = (int32_t)(((int64_t)pid * p.num_kv_heads + sg.head) * p.page_size +
                           key0 % p.page_size);
          my_live = 1;
        };
        float top = -INFINITY;  // log2 of the segment's largest V scale so far
        for (int i = 0; i < sg.n; ++i, ++j) {
          if ((i & 15) == 0) lookup(i);
          TileFacts tf;
          int32_t ys[2];
          int live = 0;
          tf.bad = 0;
#pragma unroll
          for (int sb = 0; sb < 2; ++sb) {
            const int from = 2 * (i & 15) + sb;
            tf.bad |= __shfl_sync(0xffffffffu, my_bad, from) << sb;
            live |= __shfl_sync(0xffffffffu, my_live, from) << sb;
            ys[sb] = __shfl_sync(0xffffffffu, my_y, from);
            if constexpr (quant(kFmt)) {  // (of no meaning in blocks that are not live)
              tf.ks[sb] = __shfl_sync(0xffffffffu, my_ks, from);
              tf.lv[sb] = __shfl_sync(0xffffffffu, my_lv, from);
              tf.iv[sb] = __shfl_sync(0xffffffffu, my_iv, from);
              if ((live >> sb) & 1) top = fmaxf(top, tf.lv[sb]);
            }
          }
          if constexpr (quant(kFmt)) {
            const float least = top - kScaleReach;
#pragma unroll
            for (int sb = 0; sb < 2; ++sb)
              if (((live >> sb) & 1) && tf.lv[sb] < least) {
                tf.bad |= kNoValue << sb;
                tf.lv[sb] = least;
                tf.iv[sb] = kSumUnit * fast_exp2(-least);
              }
          }
          auto load = [&](const CUtensorMap* map, const uint8_t* blocks, uint8_t* dst,
                          uint64_t* bar) {
            mbar_arrive_expect_tx(bar, (uint32_t)__popc(live) * kBlockBytes);
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
              if (!((live >> sb) & 1)) continue;
              if constexpr (quant(kFmt)) {
                tma_load_2d(dst + sb * 64 * Sm::kCodeRowB, map, 0, ys[sb], bar, pol);
                if constexpr (fp4(kFmt))
                  bulk_load(dst + Sm::kCodesB + sb * 64 * Sm::kScaleRowB,
                            blocks + (int64_t)ys[sb] * Sm::kScaleRowB, 64u * Sm::kScaleRowB, bar);
              } else {
#pragma unroll
                for (int h = 0; h < Sm::kHalves; ++h)
                  tma_load_2d(dst + h * Sm::kHalfB + sb * 64 * 128, map, h * 64, ys[sb], bar,
                              pol);
              }
            }
          };
          const int st = ring.slot;
          const uint32_t free_parity = ring.parity() ^ 1;
          if (!mbar_wait(&ct.k_empty[st], free_parity, p.flags)) { ok = false; break; }
          if (lane == 0) {
            ct.facts[j % kFactsRing] = tf;
            mbar_arrive(&ct.facts_full[j % kFactsRing]);
            load(&tmap_k, p.k_blocks, k_slot(st), &ct.k_full[st]);
          }
          __syncwarp();
          if (i == 0) {  // the queries: behind the last S of the segment before
            if (!mbar_wait(&ct.q_empty, (k & 1) ^ 1, p.flags)) { ok = false; break; }
            // (which has read the K in tile B's place, if one was there), and behind
            // the PV that reads the V there
            if (quant(kFmt) && pairs &&
                !mbar_wait(&ct.vc_free[1], ((v_ring.parities >> 1) & 1) ^ 1, p.flags)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(&ct.q_full, (uint32_t)(pairs ? 2 : 1) * Sm::kQB);
              for (int x = 0; x < (pairs ? 2 : 1); ++x)
#pragma unroll
                for (int h = 0; h < Sm::kHalves; ++h)
                  tma_load_3d(sq + x * Sm::kQB + h * (kRows * 128), &tmap_q, h * 64, sg.head * G,
                              sg.b0 + x * TQ, &ct.q_full);
            }
            __syncwarp();
          }
          if (!mbar_wait(&ct.v_empty[st], free_parity, p.flags)) { ok = false; break; }
          if (lane == 0) load(&tmap_v, p.v_blocks, v_slot(st), &ct.v_full[st]);
          __syncwarp();
          used |= 1u << st;
          ring.advance(depth);
          v_ring.advance(v_buffers(pairs));
        }
      }
      // No copy may be on its way to this CTA's shared memory when it ends.  (One
      // issued before a wait that gave up had that wait's whole limit to land.)
      for (int st = 0; st <= Sm::kStages; ++st)
        if ((used >> st) & 1) {
          mbar_wait(&ct.k_full[st], ((ring.parities >> st) & 1) ^ 1, p.flags);
          mbar_wait(&ct.v_full[st], ((ring.parities >> st) & 1) ^ 1, p.flags);
        }
    } else if (warp == kMmaWarp) {
      // ----------------------------------------------------------------- MMA
      const uint32_t id_s = idesc_f16kind(kRows, kKeys, 0, !quant(kFmt));
      const uint32_t id_o = idesc_f16kind(kRows, D, 1, !quant(kFmt));
      const uint32_t q_addr = smem_u32(sq);
      Ring kring, vring;        // slots of the next K and V tile (quantised: V's buffers)
      uint32_t jk = 0, jv = 0;  // key tiles so far, as S and as PV sees them
      uint32_t steps0 = 0, steps1 = 0;  // of each slot, before this segment
      uint32_t k_addr = 0, v_addr = 0;
      bool ok = true;
      Segment sg;
      for (uint32_t k = 0; ok && take_segment(k, &sg); ++k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.seg_empty[k % kSegRing]);
        const bool pairs = sg.rows > kRows;
        const int depth = ring_depth(pairs);
        kring.enter(depth);
        const int v_depth = quant(kFmt) ? v_buffers(pairs) : depth;
        vring.enter(v_depth);
        const int nsteps = pairs ? 2 * sg.n : sg.n;
        // whether a step is its tile's first / last
        auto first_of = [&](int s) { return !pairs || !(s & 1); };
        auto last_of = [&](int s) { return !pairs || (s & 1); };
        // S of step s: wait for its K tile, issue, release the tile after its last step
        auto issue_s = [&](int s) -> bool {
          if (first_of(s)) {
            if constexpr (quant(kFmt)) {
              k_addr = smem_u32(sconv) + (jk & 1) * Sm::kTileB;
              if (!mbar_wait(&ct.kc_full[jk & 1], (jk >> 1) & 1, p.flags)) return false;
            } else {
              k_addr = smem_u32(k_slot(kring.slot));
              if (!mbar_wait(&ct.k_full[kring.slot], kring.parity(), p.flags)) return false;
            }
          }
          const int x = s & 1;
          tc_fence_after();
          if (elect_one()) {
            // (the descriptors' low bits are the address in 16-byte units)
            const uint64_t ad = sdesc(q_addr + (pairs ? x * Sm::kQB : 0), 16, 1024);
            const uint64_t bd = sdesc(k_addr, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const int h = kk >> 2, w = kk & 3;
              mma_ss(tmem + col_s(x), ad + ((h * (kRows * 128) + w * 32) >> 4),
                     bd + ((h * Sm::kHalfB + w * 32) >> 4), id_s, kk > 0 ? 1u : 0u);
            }
            tc_commit(&ct.s_full[x]);
            if (last_of(s)) tc_commit(quant(kFmt) ? &ct.kc_free[jk & 1] : &ct.k_empty[kring.slot]);
            if (s == nsteps - 1) tc_commit(&ct.q_empty);
          }
          __syncwarp();
          if (last_of(s)) {
            kring.advance(depth);
            ++jk;
          }
          return true;
        };
        // O += P V of step s; V rows past the end or of a rejected page are zeroed
        auto issue_pv = [&](int s) -> bool {
          if (first_of(s)) {
            if constexpr (quant(kFmt)) {
              v_addr = smem_u32(v_made(vring.slot));
              if (!mbar_wait(&ct.vc_full[vring.slot], vring.parity(), p.flags)) return false;
            } else {
              if (!mbar_wait(&ct.v_full[vring.slot], vring.parity(), p.flags)) return false;
              const int32_t key0 = (sg.tile0 + (pairs ? s >> 1 : s)) * kKeys;
              const int bad = ct.facts[jv % kFactsRing].bad;
              const int zlo = min(kKeys, sg.prefix - key0);
              uint8_t* vd = v_slot(vring.slot);
              if (zlo < kKeys || bad) {
                for (int idx = lane; idx < kKeys * Sm::kHalves * 8; idx += 32) {
                  const int row = idx / (Sm::kHalves * 8);
                  const int rem = idx - row * (Sm::kHalves * 8);
                  const int h = rem >> 3, c = rem & 7;
                  if (row >= zlo || ((bad >> (row >> 6)) & 1))
                    *reinterpret_cast<uint4*>(vd + h * Sm::kHalfB + row * 128 + c * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
              }
              v_addr = smem_u32(vd);
            }
          }
          const int x = s & 1;
          if (!mbar_wait(&ct.p_full[x], ((x ? steps1 : steps0) + (s >> 1)) & 1, p.flags)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t bd = sdesc(v_addr, Sm::kHalfB, 1024);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              mma_ts(tmem + col_o(x), tmem + col_s(x) + kk * 8, bd + (kk * 2048 >> 4), id_o,
                     (s >= 2 || kk > 0) ? 1u : 0u);
            if (last_of(s)) tc_commit(quant(kFmt) ? &ct.vc_free[vring.slot] : &ct.v_empty[vring.slot]);
            if (s + 2 >= nsteps) tc_commit(&ct.o_full[x]);  // the slot's last step
          }
          __syncwarp();
          if (last_of(s)) {
            vring.advance(v_depth);
            ++jv;
          }
          return true;
        };
        if (quant(kFmt))
          ok = mbar_wait(&ct.qc_full[k % kQRing], (k / kQRing) & 1, p.flags);
        else
          ok = mbar_wait(&ct.q_full, k & 1, p.flags);
        if (ok) ok = issue_s(0);
        if (ok && nsteps > 1) ok = issue_s(1);
        for (int s = 0; s < nsteps && ok; ++s) {
          if (!(ok = issue_pv(s))) break;
          if (s + 2 < nsteps) ok = issue_s(s + 2);
        }
        steps0 += (nsteps + 1) >> 1;
        steps1 += nsteps >> 1;
      }
      // every product must finish before TMEM is released, also after a wait that gave
      // up: the commit is the elected thread's, which issued them
      __syncwarp();
      if (elect_one()) tc_commit(&ct.done);
      __syncwarp();
    }
  } else if constexpr (quant(kFmt)) {
    set_registers<kConvRegs, false>();
    // ------------------------------------------- codes -> f16 converters
    // One warpgroup converts K, the other V and, at a segment's start, Q.
    const bool v = warp >= kConvWarp0 + kConvWarps;
    const int t = threadIdx.x & (kConvThreads - 1);
    uint64_t* const full = v ? ct.v_full : ct.k_full;
    uint64_t* const empty = v ? ct.v_empty : ct.k_empty;
    uint64_t* const made = v ? ct.vc_full : ct.kc_full;
    uint64_t* const free = v ? ct.vc_free : ct.kc_free;
    Ring ring, out;  // slots of the codes, buffers of what they become
    uint32_t j = 0;  // key tiles so far
    bool ok = true;
    Segment sg{};
    bool dry = true;  // as in the softmax: the first pass only fetches, here at once
    sg.rows = kRows, sg.n = 1;
    for (uint32_t k = 0; ok; k += dry ? 0 : 1, dry = false) {
      if (!dry) {
        if (!take_segment(k, &sg)) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ct.seg_empty[k % kSegRing]);
      }
      const int tiles_q = sg.rows > kRows ? 2 : 1;
      const int depth = ring_depth(tiles_q == 2);
      const int buffers = v ? v_buffers(tiles_q == 2) : 2;
      ring.enter(depth);
      out.enter(buffers);
      if (v) {
        if (!dry && !mbar_wait(&ct.q_full, k & 1, p.flags)) break;
        for (int x = 0; x < tiles_q; ++x)
          q_rows_to_f16<D>(smem_u32(sq) + x * Sm::kQB, t, min(kRows, sg.rows - x * kRows),
                           ct.q_exp[k & 1][x], !dry);
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && !dry) mbar_arrive(&ct.qc_full[k % kQRing]);
      }
#pragma unroll 1
      for (int i = 0; i < sg.n; ++i) {
        const int st = ring.slot;
        int live = 3;
        if (!dry) {
          if (!mbar_wait(&full[st], ring.parity(), p.flags) ||
              !mbar_wait(&free[out.slot], out.parity() ^ 1, p.flags)) {
            ok = false;
            break;
          }
          // (pages, and with them the prefix, end on 64 keys)
          const int bad = ct.facts[j % kFactsRing].bad;
          live = ~(v ? bad | bad / kNoValue : bad) &
                 ((sg.tile0 + i) * kKeys + 64 < sg.prefix ? 3 : 1);
        }
        const uint8_t* to = v ? v_made(out.slot) : sconv + out.slot * Sm::kTileB;
        convert_codes<D, kFmt>(smem_u32(v ? v_slot(st) : k_slot(st)), smem_u32(to), t, live);
        fence_async_smem();
        __syncwarp();
        if (dry) break;
        if (lane == 0) {
          mbar_arrive(&made[out.slot]);
          mbar_arrive(&empty[st]);
        }
        ring.advance(depth);
        ++j;
        out.advance(buffers);
      }
    }
  }

  // ------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    mbar_wait(&ct.done, 0, p.flags);
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------- merge
// One to four warps (kW, by the unit's G * D outputs) per (sequence, kv head)
// add up the prefix partials of its G rows and the partials of the sequence's own
// tokens.  The (m, l) of all parts come first, spread over the threads, and give
// every part its weight 2^(m_i - M); the sum over the o_i then has no chain
// through it: a warp takes its share of the outputs, eight vectors in flight a
// lane.  Bound by its four trips to memory (7 us alone for 512
// units of three parts; 62 us with a chain through the parts).  Launched as a
// programmatic dependent of the decode kernel, whose completion (and memory) it
// awaits.
constexpr int kMergeThreads = 128;

__host__ __device__ constexpr int merge_warps(int gd) { return gd >= 512 ? 4 : gd >= 256 ? 2 : 1; }

template <int D, int G>
__global__ void __launch_bounds__(kMergeThreads) shared_merge_kernel(const SharedParams sp) {
  constexpr int kW = merge_warps(G * D);
  constexpr int kThreads = 32 * kW;             // of a unit
  constexpr int kUnits = kMergeThreads / kThreads;
  constexpr int kChunk = 2048 / G / kUnits;     // parts whose weights fit the shared array
  constexpr int kVecs = G * D / 4;              // float4 vectors of the unit's output
  constexpr int kN = (kVecs / kW + 31) / 32;    // of a lane
  constexpr int kInFlight = 8 / kN;             // parts a lane loads together
  __shared__ float s_w_all[kUnits][kChunk * G];
  __shared__ float s_red_all[kUnits][2][kW][G];
  const DecodeParams& p = sp.d;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % kW;
  const int tid = threadIdx.x % kThreads, slot = threadIdx.x / kThreads;
  auto& s_w = s_w_all[slot];
  auto& s_red = s_red_all[slot];
  auto unit_sync = [&]() {
    if constexpr (kW == 4)
      __syncthreads();
    else if constexpr (kW == 2)
      asm volatile("bar.sync %0, 64;" ::"r"(1 + slot) : "memory");
    else
      __syncwarp();
  };
  const int u = blockIdx.x * kUnits + slot;
  if (u >= p.batch * p.num_kv_heads) return;  // (the whole unit's threads)
  const int b = u / p.num_kv_heads;
  const int g = u - b * p.num_kv_heads;
  // (the arguments do not change under the kernels: read before the wait)
  const int32_t cap = p.max_pages * p.page_size;
  const int32_t len = max(0, min(__ldg(p.seq_lens + b), cap));
  const int32_t shared = shared_tokens(p, b, len);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // Where the parts lie (a CTA that gave up may have left its word unwritten).
  int n_pre = 0, n_own = 0, per = 1, rows = 0;  // parts; parts and rows of a segment
  int64_t pre_row = 0, own_row = 0;
  const int4 info = __ldcg(sp.pre_info + u);  // first row, segments, first sequence, rows
  const int2 own = __ldcg(p.unit_info + u);   // (both read whether of use or not: one trip)
  if (shared > 0) {
    rows = info.w;
    per = rows > kRows ? 1 : 2;
    if (info.x >= 0 && info.y > 0 && info.y <= kMaxSegments && b >= info.z &&
        (b - info.z) * G < rows && rows <= kPairRows &&
        info.x + (info.y - 1) * (int64_t)kPairRows + per * rows <= sp.pre_rows) {
      n_pre = info.y * per;
      pre_row = info.x;
      rows |= (b - info.z) * G << 16;  // low half: rows, high half: this unit's first row
    }
  }
  if (len > shared && own.x >= 0 && own.y > 0 && (int64_t)own.x + own.y <= sp.own_slots) {
    n_own = own.y;
    own_row = (int64_t)own.x * G;
  }
  const int r0 = rows >> 16;
  rows &= 0xffff;
  // Prefix part i: slot 0 or 1 of segment i / per.  The rows of a slot start
  // at `first`, `nr` of them; this unit's row 0 is row `r` there.
  struct Place {
    int64_t first;
    int nr, r;
  };
  auto place = [&](int i) -> Place {
    if (per == 1) {  // two Q tiles: the unit's rows lie in one of them
      const int64_t base = pre_row + (int64_t)i * kPairRows;
      return r0 < kRows ? Place{base, kRows, r0} : Place{base + kRows, rows - kRows, r0 - kRows};
    }
    return {pre_row + (int64_t)(i >> 1) * kPairRows + (i & 1) * rows, rows, r0};
  };
  auto ml_of = [&](int i, int row) -> float2 {
    if (i < n_pre) {
      const Place pl = place(i);
      return __ldcg(sp.pre_ml + pl.first + pl.r + row);
    }
    return __ldcg(p.part_ml + own_row + (int64_t)(i - n_pre) * G + row);
  };

  // The largest reference of each row: thread t of a unit looks at row t % G.
  const int n = n_pre + n_own;
  const int my_row = tid % G, my_part = tid / G;
  constexpr int kStep = kThreads / G;
  float M = -INFINITY;
  // (the first of them stays here: few units have more)
  const float2 my_ml = my_part < n ? ml_of(my_part, my_row) : make_float2(0.f, 0.f);
  for (int i = my_part; i < n; i += kStep) {
    const float2 ml = i == my_part ? my_ml : ml_of(i, my_row);
    if (ml.y != 0.f) M = fmaxf(M, ml.x);  // l = 0: a part without keys, its o is not written
  }
#pragma unroll
  for (int o = G; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane < G) s_red[0][warp][lane] = M;
  unit_sync();
#pragma unroll
  for (int w = 0; w < kW; ++w) M = fmaxf(M, s_red[0][w][my_row]);

  float4 acc[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int v0 = warp * (32 * kN) + lane;  // this lane's vectors: v0 + 32 j
  float L = 0.f;
  for (int c0 = 0; c0 < n; c0 += kChunk) {
    const int cn = min(n - c0, kChunk);
    if (c0 > 0) unit_sync();  // the last chunk's weights have been used
    for (int i = my_part; i < cn; i += kStep) {
      const float2 ml = c0 + i == my_part ? my_ml : ml_of(c0 + i, my_row);
      // in two factors: the sums of quantised pools' parts reach from 2^-75 to 2^94, and
      // where the weight is below fp32's range the weighted sum is not
      const float half = ml.y != 0.f ? fast_exp2(0.5f * (ml.x - M)) : 0.f;
      s_w[i * G + my_row] = half * half;
      L += (half * ml.y) * half;
    }
    unit_sync();
    for (int i0 = 0; i0 < cn; i0 += kInFlight) {
      float4 o[kInFlight][kN];
      float w[kInFlight][kN];
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int i = c0 + i0 + k;
        const bool pre = i < n_pre;
        const Place pl = pre ? place(i) : Place{own_row + (int64_t)(i - n_pre) * G, 0, 0};
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const int v = v0 + 32 * j;  // row v % G, dims 4 * (v / G)
          w[k][j] = i0 + k < cn && v < kVecs ? s_w[(i0 + k) * G + v % G] : 0.f;
          o[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (w[k][j] != 0.f)
            o[k][j] = pre ? __ldcg(reinterpret_cast<const float4*>(sp.pre_o) + pl.first * (D / 4) +
                                   (int64_t)(v / G) * pl.nr + pl.r + v % G)
                          : __ldcg(reinterpret_cast<const float4*>(p.part_o) +
                                   (pl.first + v % G) * (D / 4) + v / G);
        }
      }
#pragma unroll
      for (int k = 0; k < kInFlight; ++k)
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          acc[j].x += w[k][j] * o[k][j].x;
          acc[j].y += w[k][j] * o[k][j].y;
          acc[j].z += w[k][j] * o[k][j].z;
          acc[j].w += w[k][j] * o[k][j].w;
        }
    }
  }
#pragma unroll
  for (int o = G; o < 32; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane < G) s_red[1][warp][lane] = L;
  unit_sync();
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int v = v0 + 32 * j;
    if (v >= kVecs) break;
    const int row = v % G;  // (which is tid % G: M belongs to it)
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) l += s_red[1][w][row];
    const int64_t orow = (int64_t)b * p.num_q_heads + g * G + row;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(p.out + orow * D + 4 * (v / G)) = make_uint2(
        pack_bf16(acc[j].x * inv, acc[j].y * inv), pack_bf16(acc[j].z * inv, acc[j].w * inv));
    if (p.lse && v < G)
      p.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
  }
}

template <int D>
cudaError_t merge_for(const SharedParams& sp, cudaStream_t stream) {
  const int64_t units = (int64_t)sp.d.batch * sp.d.num_kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int a_block = 4 / merge_warps(sp.d.group * D);
  cfg.gridDim = dim3((unsigned)((units + a_block - 1) / a_block));
  switch (sp.d.group) {
    case 1: return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D, 1>, sp);
    case 2: return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D, 2>, sp);
    case 4: return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D, 4>, sp);
    default: return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D, 8>, sp);
  }
}

template <int D, int kFmt>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const SharedParams& p, int num_ctas, cudaStream_t stream) {
  const size_t smem = Smem<D, kFmt>::kBytes;
  // The shared-memory attribute belongs to the current device: set it once
  // per device and instantiation.
  constexpr int kMaxDevices = 64;
  static bool attr[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr[dev]) {
      // The register exchange counts on what the block is launched with (the build
      // checks it too); with fewer it would wait for ever.
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, prefix_kernel<D, kFmt>)) != cudaSuccess) return e;
      if (quant(kFmt) && fa.numRegs < kLaunchRegs) return cudaErrorLaunchOutOfResources;
      e = cudaFuncSetAttribute(prefix_kernel<D, kFmt>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
      attr[dev] = true;
    }
  }
  prefix_kernel<D, kFmt><<<num_ctas, Smem<D, kFmt>::kThreads, smem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

}  // namespace sh

cudaError_t shared_prefix_run(int head_dim, int fmt, const CUtensorMap& tq, const CUtensorMap& tk,
                              const CUtensorMap& tv, const SharedParams& p, int num_ctas,
                              cudaStream_t stream) {
  const bool d128 = head_dim == 128;
  switch (fmt) {
    case PKV_KV_NVFP4:
      return d128 ? sh::launch<128, PKV_KV_NVFP4>(tq, tk, tv, p, num_ctas, stream)
                  : sh::launch<64, PKV_KV_NVFP4>(tq, tk, tv, p, num_ctas, stream);
    case PKV_KV_INT8:
      return d128 ? sh::launch<128, PKV_KV_INT8>(tq, tk, tv, p, num_ctas, stream)
                  : sh::launch<64, PKV_KV_INT8>(tq, tk, tv, p, num_ctas, stream);
    case PKV_KV_FP8_E4M3:
      return d128 ? sh::launch<128, PKV_KV_FP8_E4M3>(tq, tk, tv, p, num_ctas, stream)
                  : sh::launch<64, PKV_KV_FP8_E4M3>(tq, tk, tv, p, num_ctas, stream);
    default:
      return d128 ? sh::launch<128, PKV_KV_BF16>(tq, tk, tv, p, num_ctas, stream)
                  : sh::launch<64, PKV_KV_BF16>(tq, tk, tv, p, num_ctas, stream);
  }
}

cudaError_t shared_merge_run(int head_dim, const SharedParams& p, cudaStream_t stream) {
  return head_dim == 128 ? sh::merge_for<128>(p, stream) : sh::merge_for<64>(p, stream);
}

}  // namespace pkv
