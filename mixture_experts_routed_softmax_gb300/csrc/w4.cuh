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

// the bit of a pair's low half that holds bit b (0: lowest) of the fp4 code
__host__ __device__ constexpr int fp4_bit(int i, int b) {
  return i == 0   ? (b == 3 ? 15 : 6 + b)
         : i == 1 ? (b == 3 ? 12 : 3 + b)
         : i == 2 ? (b == 3 ? 9 : b)
                  : (b == 3 ? 14 : b == 0 ? 13 : 9 + b);
}

// a code (two's complement, or sign and magnitude) at its place in a word
__device__ __forceinline__ uint32_t w4_place(uint32_t code, int i, int odd, bool fp4) {
  uint32_t v;
  if (fp4) {
    v = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) v |= ((code >> b) & 1u) << fp4_bit(i, b);
  } else {
    v = (code ^ 8u) << (4 * i);
  }
  return v << (16 * odd);
}
__device__ __forceinline__ uint32_t w4_code_at(uint32_t word, int i, int odd, bool fp4) {
  const uint32_t v = word >> (16 * odd);
  if (!fp4) return ((v >> (4 * i)) & 15u) ^ 8u;
  uint32_t c = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) c |= ((v >> fp4_bit(i, b)) & 1u) << b;
  return c;
}
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

// A word's four pairs as bf16 values (exact), from an offset or factor of the kind:
//   int4: 128 + 8 + value (0x4300 holds 128 with steps of 1)
//   fp4:  2^-126 value: the code's exponent and mantissa as the low end of bf16's,
//         which has subnormals where fp4 has them
// scaled: value * scale, rounded to bf16 once. `plain` scales (plain_scale) take one
// operation a pair instead of two:
//   int4: 160 + 4 value in place of 136 + value, fma(that, scale / 4, -40 scale): with five
//         significant bits in a scale 40 scale has eight, so the sum rounds as the product does
//   fp4:  scale * 2^126 in one factor
// The constants are held in registers that the compiler does not know the contents of: it
// would load them again for every pair.
template <bool FP4>
struct W4Decoder {
  uint32_t mask, base, last, mask2;
  __device__ __forceinline__ W4Decoder() {
    if (FP4) {
      asm volatile("mov.u32 %0, 0x81C081C0;" : "=r"(mask));
      asm volatile("mov.u32 %0, 0x01800180;" : "=r"(base));
      asm volatile("mov.u32 %0, 0x00400040;" : "=r"(mask2));
      asm volatile("mov.u32 %0, 0x7E807E80;" : "=r"(last));       // 2^126
    } else {
      asm volatile("mov.u32 %0, 0x000F000F;" : "=r"(mask));
      asm volatile("mov.u32 %0, 0x43004300;" : "=r"(base));
      asm volatile("mov.u32 %0, 0x43084308;" : "=r"(last));       // 136
      asm volatile("mov.u32 %0, 0x003C003C;" : "=r"(mask2));
    }
  }
  static __device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));   // (a & b) | c
    return r;
  }
  __device__ __forceinline__ void raw_fp4(uint32_t w, uint32_t* r) const {
    r[0] = w & mask;
    r[1] = (w << 3) & mask;
    r[2] = (w << 6) & mask;
    r[3] = and_or(w >> 3, base, (w << 1) & 0x80008000u);
    r[3] = and_or(w >> 7, mask2, r[3]);
  }
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t* r) const {
    if (FP4) {
      raw_fp4(w, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2(r[i], last);
    } else {
      r[0] = and_or(w, mask, base);
      r[1] = and_or(w >> 4, mask, base);
      r[2] = and_or(w >> 8, mask, base);
      r[3] = and_or(w >> 12, mask, base);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = sub_bf16x2(r[i], last);
    }
  }
  // factors of a scale pair (both halves the same) for `scaled`
  struct Factor {
    uint32_t f, c;
  };
  template <bool PLAIN>
  __device__ __forceinline__ Factor factor(uint32_t s2) const {
    if (!PLAIN) return Factor{s2, 0u};
    if (FP4) return Factor{mul_bf16x2(s2, last), 0u};
    return Factor{mul_bf16x2(s2, 0x3E803E80u), mul_bf16x2(s2, 0xC220C220u)};   // 1/4, -40
  }
  template <bool PLAIN>
  __device__ __forceinline__ void scaled(uint32_t w, const Factor& lo, const Factor& hi,
                                         uint32_t* r) const {
    if (!PLAIN) {
      (*this)(w, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2(r[i], (i & 1) ? hi.f : lo.f);
    } else if (FP4) {
      raw_fp4(w, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = mul_bf16x2(r[i], (i & 1) ? hi.f : lo.f);
    } else {
      r[0] = and_or(w << 2, mask2, base);
      r[1] = and_or(w >> 2, mask2, base);
      r[2] = and_or(w >> 6, mask2, base);
      r[3] = and_or(w >> 10, mask2, base);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = fma_bf16x2(r[i], (i & 1) ? hi.f : lo.f, (i & 1) ? hi.c : lo.c);
    }
  }
};

// Whether a scale (bf16 bits) takes the short form of `scaled`: int4, at most five
// significant bits and far from either end of the range; fp4, below 2. NaN and 0 do.
__device__ __forceinline__ bool plain_scale(uint32_t bits, bool fp4) {
  const uint32_t a = bits & 0x7FFFu;
  if (a == 0u || a > 0x7F80u) return true;
  if (fp4) return a < 0x4000u;
  return (a & 7u) == 0u && a >= 0x0800u && a < 0x7700u;
}
// The arrays of scales end with a word an expert: not 0 where some scale is not plain.
__host__ __device__ __forceinline__ int64_t w4_flags_at(int64_t E, int K, int N, int group) {
  return E * w4_scales_per_expert(K, N, group);          // elements; a multiple of 16
}

}  // namespace moe
