// w4.cuh — weights in 4 bits with group scales: how they lie in memory and how a
// thread turns its codes into bf16 values.
//
// A matrix [K, N] stands as W[k, n] = value(code[k, n]) * scale[k / group, n].
// Kinds: int4, -8 .. 7; fp4, +-{0, 1/2, 1, 3/2, 2, 3, 4, 6} (a sign, two bits of
// exponent, one of mantissa). Scales are bf16.
//
// Codes lie in tiles of 16 columns n by 64 rows k, 512 bytes each. 8 x 4 of them, 128
// columns by 256 rows, are one contiguous piece (16 KB, one copy into shared memory), column
// block after column block and in one row after row; then come the next 256 rows of the
// same columns (w4_tile_at). At the right and lower edge pieces are as small as what there is.
// In a tile lane (g, t) = (lane / 4, lane % 4) owns 16 bytes, columns g and g + 8 at the
// rows 16j + 4t .. + 3, word j = 0 .. 3. So word j is
//   - the A operand of an m16n8k16 product whose B operand is four neighbouring
//     elements of a row of x (the order of k inside a product is free as long as
//     both sides agree): pair i of the word is register i; and
//   - a lane's part of 16 rows by 16 k of a tensor-memory operand (the 16x256b
//     shape), columns of 32 bits in the natural order of k.
// Register i of word j takes, low and high half: i & 1 = 0: column g, 1: column g + 8;
// rows 16j + 4t + 2 (i / 2) + {0, 1}.
// Where a pair's bits lie in the low 16 bits of its word (the high 16 bits hold
// the odd row alike):
//   int4: bits 4i .. 4i + 3, the code plus 8
//   fp4:  sign and three magnitude bits where a shift leaves them in a bf16's
//         place: i = 0: 15, 8..6; 1: 12, 5..3; 2: 9, 2..0; 3: 14, 11..10 and 13
//
// Scales lie in the same pieces, by steps of 128 rows: a step of 16 columns holds
// [g][groups of the step][columns g, g + 8] (w4_scales_at).
#pragma once
#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kW4Tile = 512;                       // bytes of a tile of codes
__host__ __device__ constexpr int w4_kblocks(int K) { return (K + 63) / 64; }
__host__ __device__ constexpr int w4_nblocks(int N) { return (N + 15) / 16; }
__host__ __device__ constexpr int w4_steps(int K) { return (K + 127) / 128; }
// groups of a step of 128 rows
__host__ __device__ constexpr int w4_gps(int group) { return 128 / group; }
__host__ __device__ constexpr int64_t w4_codes_per_expert(int K, int N) {
  return (int64_t)w4_nblocks(N) * w4_kblocks(K) * kW4Tile;
}
// elements
__host__ __device__ constexpr int64_t w4_scales_per_expert(int K, int N, int group) {
  return (int64_t)w4_nblocks(N) * w4_steps(K) * 16 * w4_gps(group);
}

// bytes in front of the tile of column block nb and row block kb, in an expert
__host__ __device__ __forceinline__ int64_t w4_tile_at(int nb, int kb, int nbs, int kbs) {
  const int b = nb & ~7, cb = nbs - b < 8 ? nbs - b : 8;
  const int c = kb & ~3, m = kbs - c < 4 ? kbs - c : 4;
  return ((int64_t)b * kbs + (int64_t)c * cb + (nb - b) * m + (kb - c)) * kW4Tile;
}
// elements in front of the scales of column block nb and step `st`
__host__ __device__ __forceinline__ int64_t w4_scales_at(int nb, int st, int nbs, int steps,
                                                         int gps) {
  const int b = nb & ~7, cb = nbs - b < 8 ? nbs - b : 8;
  const int c = st & ~1, m = steps - c < 2 ? 1 : 2;
  return ((int64_t)b * steps + (int64_t)c * cb + (nb - b) * m + (st - c)) * 16 * gps;
}

// what a code (two's complement, or sign and magnitude) stands for
__device__ __forceinline__ float w4_value(uint32_t code, bool fp4) {
  if (!fp4) return (float)((int)(code ^ 8u) - 8);
  const uint32_t e = (code >> 1) & 3u, m = code & 1u;
  const float a = e ? (float)((2 + m) << (e - 1)) * 0.5f : 0.5f * (float)m;
  return code & 8u ? -a : a;
}

// The experts' gated activation (moe_swiglu); NaN stays NaN.
__device__ __forceinline__ float gated(float g, float u, const ActParams& a) {
  const float gc = g > a.limit ? a.limit : g;
  const float uc = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
  return __fdividef(gc, 1.0f + __expf(-a.alpha * gc)) * (uc + a.c);
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// A word's four pairs as bf16. In place, or moved by a shift for two or three of them, a
// masked code is a bf16 already, a very small one:
//   int4: bits 0-3 or 4-7 hold u = value + 8; bf16's first two binades are one even scale,
//         so that is u 2^-133 or u 2^-129, and value * f = fma(that, f 2^133 or 2^129, -8 f)
//   fp4:  the code's exponent and mantissa are the low end of bf16's, which has subnormals
//         where fp4 has them: 2^-126 value
// values: the code's value (fp4), or 2^-13 of it (int4: 2^133 is no bf16), exact; kUnit gives
//   the factor back.
// scaled: 2^-16 code * scale, rounded to bf16 once, one operation a pair; for scales in the
//   wide range of plain_scale. general: code * scale for any other scale.
// The constants are held in registers that the compiler does not know the contents of: it
// would load them again for every pair.
template <bool FP4>
struct W4Decoder {
  static constexpr float kUnit = FP4 ? 1.f : 8192.f;        // of values
  static constexpr float kScaled = 65536.f;                 // of scaled
  uint32_t m0, m1, m2, f0, f1, c;
  __device__ __forceinline__ W4Decoder() {
    if (FP4) {
      asm volatile("mov.u32 %0, 0x81C081C0;" : "=r"(m0));
      asm volatile("mov.u32 %0, 0x01800180;" : "=r"(m1));
      asm volatile("mov.u32 %0, 0x00400040;" : "=r"(m2));
      asm volatile("mov.u32 %0, 0x7E807E80;" : "=r"(f0));       // 2^126
      f1 = c = 0;
    } else {
      asm volatile("mov.u32 %0, 0x000F000F;" : "=r"(m0));
      asm volatile("mov.u32 %0, 0x00F000F0;" : "=r"(m1));
      asm volatile("mov.u32 %0, 0x7B807B80;" : "=r"(f0));       // 2^120
      asm volatile("mov.u32 %0, 0x79807980;" : "=r"(f1));       // 2^116
      asm volatile("mov.u32 %0, 0xBA80BA80;" : "=r"(c));        // -2^-10
      m2 = 0;
    }
  }
  static __device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));   // (a & b) | c
    return r;
  }
  __device__ __forceinline__ void raw(uint32_t w, uint32_t* r) const {
    if (FP4) {
      r[0] = w & m0;
      r[1] = (w << 3) & m0;
      r[2] = (w << 6) & m0;
      r[3] = and_or(w >> 3, m1, (w << 1) & 0x80008000u);
      r[3] = and_or(w >> 7, m2, r[3]);
    } else {
      r[0] = w & m0;
      r[1] = w & m1;
      r[2] = (w >> 8) & m0;
      r[3] = (w >> 8) & m1;
    }
  }
  __device__ __forceinline__ void values(uint32_t w, uint32_t* r) const {
    raw(w, r);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = FP4 ? mul_bf16x2(r[i], f0) : fma_bf16x2(r[i], (i & 1) ? f1 : f0, c);
  }
  // a column's scale (both halves the same) for `scaled`: of column g (HI = 0) or g + 8
  struct Factor {
    uint32_t f, c;
  };
  template <int HI>
  static __device__ __forceinline__ Factor factor(uint32_t s2) {
    if (FP4) return Factor{mul_bf16x2(s2, 0x76807680u), 0u};                  // 2^110
    return Factor{mul_bf16x2(s2, HI ? 0x78007800u : 0x7A007A00u),             // 2^113, 2^117
                  mul_bf16x2(s2, 0xB900B900u)};                               // -2^-13
  }
  __device__ __forceinline__ void scaled(uint32_t w, const Factor& lo, const Factor& hi,
                                         uint32_t* r) const {
    raw(w, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Factor& k = (i & 1) ? hi : lo;
      r[i] = FP4 ? mul_bf16x2(r[i], k.f) : fma_bf16x2(r[i], k.f, k.c);
    }
  }
  __device__ __forceinline__ void general(uint32_t w, uint32_t lo2, uint32_t hi2,
                                          uint32_t* r) const {
    values(w, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!FP4) r[i] = mul_bf16x2(r[i], 0x46004600u);                          // 2^13
      r[i] = mul_bf16x2(r[i], (i & 1) ? hi2 : lo2);
    }
  }
};

// Whether `scaled` takes a scale (bf16 bits): 2^-100 <= |scale| < 2^9, 0 or NaN.
__device__ __forceinline__ bool plain_scale(uint32_t bits) {
  const uint32_t a = bits & 0x7FFFu;
  return a == 0u || a > 0x7F80u || (a >= 0x0D80u && a < 0x4400u);
}
// The arrays of scales end with a word an expert: not 0 where some scale is not plain.
__host__ __device__ __forceinline__ int64_t w4_flags_at(int64_t E, int K, int N, int group) {
  return E * w4_scales_per_expert(K, N, group);          // elements; a multiple of 16
}

}  // namespace moe
