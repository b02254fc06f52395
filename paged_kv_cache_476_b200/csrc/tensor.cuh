// tcgen05 helpers shared by the kernels that run attention on the fifth-
// generation tensor cores: TMEM and MMA wrappers, descriptors, packed fp32
// arithmetic, and the conversion of one-byte and FP4 tiles to 16-bit ones.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace pkv {

namespace pf {

constexpr int kRows = 128;  // M of a Q tile
constexpr int kKeys = 128;  // N of the S tile (keys per KV tile)
constexpr uint32_t kTmemCols = 512;
// TMEM columns: S of tile A and B (P is written over S as 16-bit pairs), O
// of tile A and B.
__device__ __forceinline__ uint32_t col_s(int x) { return x ? 128u : 0u; }
__device__ __forceinline__ uint32_t col_o(int x) { return x ? 384u : 256u; }

// --------------------------------------------------------- tcgen05 helpers
// True in one lane of the (converged) warp.  Products issued under this, and
// not under lane == 0, let the compiler see that one thread alone gives their
// operands, which a warp takes from uniform registers (prefix kernel: 10 %).
__device__ __forceinline__ bool elect_one() {
  uint32_t one = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t@p mov.s32 %0, 1;\n\t}"
      : "+r"(one));
  return one != 0;
}

__device__ __forceinline__ void tmem_alloc(uint32_t* dst_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Arrive on `bar` once every tcgen05 operation this thread issued is done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 consecutive fp32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Store 16 consecutive 32-bit columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// max(a, b, c) in one instruction (three-input form of sm_100).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two fp32 lanes at once (sm_100 packed FMA / add / mul): each lane rounds
// exactly as its scalar instruction would.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)),
        "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}

// O row (this thread's TMEM lane, D fp32 columns from taddr) *= alpha.
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t taddr, float alpha) {
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_ld32(taddr + c, o);
    tmem_wait_ld();
    uint32_t u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * alpha);
    tmem_st16(taddr + c, u);
    tmem_st16(taddr + c + 16, u + 16);
  }
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Shared-memory matrix descriptor (tcgen05 format): start address, leading
// and stride byte offsets (16-byte units), version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo_bytes >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for sm_100
  d |= (uint64_t)2 << 61;  // SWIZZLE_128B
  return d;
}

// Instruction descriptor of kind::f16 with f32 accumulation: A and B both
// bf16 (or both f16), M x N, B K- or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16kind(int M, int N, int b_mn_major, bool bf16) {
  return (1u << 4)                           // D format f32
         | ((bf16 ? 1u : 0u) << 7)           // A: 1 bf16, 0 f16
         | ((bf16 ? 1u : 0u) << 10)          // B: same type as A
         | ((uint32_t)b_mn_major << 16)      // B major: 0 K, 1 MN
         | ((uint32_t)(N >> 3) << 17)        // N / 8
         | ((uint32_t)(M >> 4) << 24);       // M / 16
}

// Shared-memory byte address of 16-byte chunk c (0..D/8-1) of row r of a bf16
// tile laid out as TMA writes it: 64-column halves kHalfB apart, 128-byte
// rows, 128-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t bf16_chunk(uint32_t base, int r, int c) {
  return base + (c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Same for a tile of codes as TMA writes it: rows of kRowB bytes with the
// swizzle of that width (128, 64 or 32 bytes).
template <int kRowB>
__device__ __forceinline__ uint32_t code_chunk(uint32_t base, int r, int c) {
  if constexpr (kRowB == 128)
    return base + r * 128 + ((c ^ (r & 7)) << 4);
  else if constexpr (kRowB == 64)
    return base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return base + r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

// E4M3 tile -> bf16 or f16 tile (both exact: every E4M3 value is an f16 and a
// bf16), rows in `zero_mask` (bit per 64-row block) or at/after `zero_from`
// written as zeros.  64 threads share the work.
template <int D, int kFmt, bool kToF16>
__device__ __forceinline__ void convert_tile(uint32_t src, uint32_t dst, int t, int zero_from,
                                             int zero_mask) {
  constexpr int kChunks = kKeys * D / 16;  // 16-byte E4M3 chunks
#pragma unroll 4
  for (int ci = t; ci < kChunks; ci += 64) {
    const int r = ci / (D / 16);
    const int c = ci - r * (D / 16);
    uint32_t o[8];
    if (r >= zero_from || ((zero_mask >> (r >> 6)) & 1)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = 0u;
    } else {
      uint32_t w[4];
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(code_chunk<D>(src, r, c)));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t h01 = kv8x2_to_f16x2<kFmt>(w[k] & 0xffff);
        const uint32_t h23 = kv8x2_to_f16x2<kFmt>(w[k] >> 16);
        if constexpr (kToF16) {
          o[2 * k] = h01;
          o[2 * k + 1] = h23;
        } else {
          const float2 f01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
          const float2 f23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
          o[2 * k] = pack_bf16(f01.x, f01.y);
          o[2 * k + 1] = pack_bf16(f23.x, f23.y);
        }
      }
    }
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(bf16_chunk<D>(dst, r, 2 * c)),
                 "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                 : "memory");
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                     bf16_chunk<D>(dst, r, 2 * c + 1)),
                 "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
  }
}

// FP4 tile (codes, then one E4M3 block scale per 16 values of a row) ->
// bf16 or f16 tile, values e2m1(code) * decode(sb): exact in both, since the
// product has at most 6 significant bits and lies in [2^-10, 2688].  Rows
// in `zero_mask` or at/after `zero_from` are written as zeros.  64 threads.
template <int D, bool kToF16>
__device__ __forceinline__ void convert_fp4_tile(uint32_t src, uint32_t dst, int t, int zero_from,
                                                 int zero_mask) {
  constexpr int kRowB = D / 2;            // code bytes of a row
  constexpr int kChunks = kKeys * D / 32;  // 16-byte chunks of codes (32 values, 2 blocks)
  const uint32_t scales = src + kKeys * kRowB;
#pragma unroll 2
  for (int ci = t; ci < kChunks; ci += 64) {
    const int r = ci / (D / 32);
    const int c = ci - r * (D / 32);
    uint32_t o[16];
    if (r >= zero_from || ((zero_mask >> (r >> 6)) & 1)) {
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = 0u;
    } else {
      uint32_t w[4];
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(code_chunk<kRowB>(src, r, c)));
      uint32_t sb2;
      asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sb2) : "r"(scales + r * (D / 16) + 2 * c));
      const uint32_t s0 = e4m3_splat_f16x2(sb2, 0), s1 = e4m3_splat_f16x2(sb2, 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e2m1x8_to_f16x2(w[k], o + 4 * k);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[4 * k + i] = hmul2_u32(o[4 * k + i], k < 2 ? s0 : s1);
      }
      if constexpr (!kToF16) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
          o[k] = pack_bf16(f.x, f.y);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(bf16_chunk<D>(dst, r, 4 * c + q)),
                   "r"(o[4 * q]), "r"(o[4 * q + 1]), "r"(o[4 * q + 2]), "r"(o[4 * q + 3])
                   : "memory");
  }
}

}  // namespace pf

}  // namespace pkv
