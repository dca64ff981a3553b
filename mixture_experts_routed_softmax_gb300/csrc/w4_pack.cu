// w4_pack.cu — weights into 4 bits and back (layout: w4.cuh).
//
// Quantisation, group by group of `group` rows of a column:
//   a = max |w|
//   int4: scale = a / 7, its significand rounded up to five bits; codes are the
//         nearest of -7 .. 7 steps
//   fp4:  scale = the least power of two that keeps a within 6; codes are the nearest value
// halves to the even code; one step less where bf16 does not hold that value. A code has at most three significant bits, so with
// such scales code * scale is a bf16 value: nothing is rounded on the way to
// the tensor cores (five bits cost an int4 group at most 1/32 of its range).
// A group whose a is below 2^-120 becomes zeros (scale 0); one with an infinity
// or NaN gets scale NaN and stays visible as such.
//
// Bound by memory in floor (2 bytes read and 1/2 + 2/group written a weight). Quantisation: a
// warp takes 16 columns by 128 rows in registers, a lane two neighbouring columns, so
// that a word is a load, maxima and conversions work on pairs, and the codes of four rows of both are
// one word, which goes to the lanes that store it by two shuffles. (32 x 2880 x 2880: 129 us;
// through shared memory, a weight at a time, 181.) Given codes and the way back: a block takes
// 64 columns by 128 rows through shared memory, rows on one side, whole tiles of 512 bytes on
// the other.
#include "w4.cuh"

namespace moe {

constexpr int kPackN = 64;            // columns of a block: four tiles, a warp each
constexpr int kPackThreads = 128;
constexpr int kPackPitch = kPackN + 2;   // bf16 a row: 33 words, so that rows shift banks

struct W4View {
  uint8_t* codes;
  moe_bf16* scales;
  int E, K, N, group;
};

static W4View w4_view(const moe_w4& w) {
  return W4View{w.codes, w.scales, w.E, w.K, w.N, w.group};
}

__device__ __forceinline__ float group_scale(float a, bool fp4) {
  if (!(a < INFINITY)) return __uint_as_float(0x7FC00000u);
  if (a < 7.5231638e-37f) return 0.f;                        // 2^-120
  if (!fp4) {
    const uint32_t b = __float_as_uint(__fdiv_rn(a, 7.0f));
    return __uint_as_float((b + 0x7FFFFu) & ~0x7FFFFu);
  }
  // a = m 2^E, m in [1, 2): a <= 6 2^(E - 2) where m <= 3/2
  const uint32_t b = __float_as_uint(a);
  const uint32_t up = (b & 0x7FFFFFu) > 0x400000u ? 1u : 2u;
  return __uint_as_float(((b >> 23) - up) << 23);
}

// The code of one weight in any case: at the top of the range the nearest value may be one that
// bf16 does not hold.
__device__ __noinline__ uint32_t nearest_code(float w, float s, bool fp4) {
  if (!(s > 0.f)) return 0u;
  const float q = __fdiv_rn(w, s);
  const float a = fabsf(q);
  // the codes count steps of 1; or of 1/2 up to 2, of 1 up to 4, of 2 beyond
  int n = !fp4      ? __float2int_rn(a)
          : a < 2.f ? __float2int_rn(2.f * a)
          : a < 4.f ? __float2int_rn(a) + 2
                    : __float2int_rn(0.5f * a) + 4;
  if (s > 1e37f && n > 0 && w4_value((uint32_t)n, fp4) * s > 3.3895314e38f) --n;
  if (!fp4) return (uint32_t)(q < 0.f ? -n : n) & 15u;
  return (uint32_t)n | (n && q < 0.f ? 8u : 0u);
}

// A weight to an int4 code (the low four bits), by r = 1 / scale rounded. w / scale is half a step or at least
// 2^-9 away from one (w has eight significant bits, scale five, the quotient is below
// 7.5), w r is off by 2^-20: rounded to 2^-10 (the first two additions) it is on the right side, or
// on the half itself, which the third rounds to the even code. The sum's last bits
// are the code in two's complement.
__device__ __forceinline__ uint32_t int4_code(float w, float r) {
  const float q = __fadd_rn(__fadd_rn(__fmul_rn(w, r), 12288.0f), -12288.0f);
  return __float_as_uint(__fadd_rn(q, 12582912.0f));
}
// Two neighbouring weights of four rows to codes, a byte a row, rows 0, 2, 1, 3, the first weight's
// in the low four bits. (fp4: w r is exact, r is a power of two.)
template <bool FP4>
__device__ __forceinline__ uint32_t eight_codes(const uint32_t* w, float r0, float r1) {
  float a[4], b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    a[q] = __uint_as_float(w[q] << 16);
    b[q] = __uint_as_float(w[q] & 0xFFFF0000u);
  }
  uint32_t d;
  if (FP4) {
    asm("{\n\t.reg .b8 p, q, r, s;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 r, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
        "mov.b32 %0, {p, q, r, s};\n\t}\n"
        : "=r"(d)
        : "f"(a[0] * r0), "f"(b[0] * r1), "f"(a[1] * r0), "f"(b[1] * r1), "f"(a[2] * r0),
          "f"(b[2] * r1), "f"(a[3] * r0), "f"(b[3] * r1));
  } else {
    // the low bytes together, then their low halves
    const uint32_t even =
        __byte_perm(__byte_perm(int4_code(a[0], r0), int4_code(a[2], r0), 0x0040),
                    __byte_perm(int4_code(a[1], r0), int4_code(a[3], r0), 0x0040), 0x5410);
    const uint32_t odd =
        __byte_perm(__byte_perm(int4_code(b[0], r1), int4_code(b[2], r1), 0x0040),
                    __byte_perm(int4_code(b[1], r1), int4_code(b[3], r1), 0x0040), 0x5410);
    d = (even & 0x0F0F0F0Fu) | ((odd << 4) & 0xF0F0F0F0u);
  }
  return d;
}
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b) {      // NaN stays NaN
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b & 0x7FFF7FFFu));
  return a;
}
// A word of codes side by side (pair i in bits 4i of either half) to the kind's places
template <bool FP4>
__device__ __forceinline__ uint32_t w4_arrange(uint32_t x) {
  if (!FP4) return x ^ 0x88888888u;
  return ((x << 6) & 0x01C001C0u) | ((x << 12) & 0x80008000u) | ((x >> 1) & 0x40384038u) |
         ((x << 5) & 0x10001000u) | ((x >> 8) & 0x00070007u) | ((x >> 2) & 0x02000200u) |
         ((x << 1) & 0x20002000u) | ((x >> 3) & 0x0C000C00u);
}

// bf16 weights [E, K, N]
template <bool FP4>
__global__ void __launch_bounds__(kPackThreads) w4_quantise_kernel(
    W4View w, const moe_bf16* __restrict__ src) {
  pdl_enter();
  const int lane = threadIdx.x & 31, e = blockIdx.z, step = blockIdx.y;
  const int nb = blockIdx.x * (kPackN / 16) + threadIdx.x / 32;
  const int nbs = w4_nblocks(w.N), kbs = w4_kblocks(w.K);
  if (nb >= nbs) return;
  // columns n and n + 1 at rows 16j + 4t + q
  const int p = lane >> 2, t = lane & 3, n = 16 * nb + 2 * p, k0 = 128 * step + 4 * t;
  const int gps = w4_gps(w.group);
  const uint32_t* from =
      reinterpret_cast<const uint32_t*>(src + ((int64_t)e * w.K + k0) * w.N + n);
  const int left = n < w.N ? w.K - k0 : 0, pitch = w.N / 2;
  uint32_t v[32];
  if (128 * (step + 1) <= w.K && 16 * (nb + 1) <= w.N) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      v[i] = __ldcs(from + (int64_t)(16 * (i >> 2) + (i & 3)) * pitch);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int k = 16 * (i >> 2) + (i & 3);
      v[i] = k < left ? __ldcs(from + (int64_t)k * pitch) : 0u;
    }
  }
  // magnitudes by 32 rows, then by groups
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max_magnitude(a, v[8 * i + j]);
    a = max_magnitude(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    m[i] = max_magnitude(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
  }
  if (gps < 4) {
    m[0] = m[1] = max_magnitude(m[0], m[1]);
    m[2] = m[3] = max_magnitude(m[2], m[3]);
    if (gps < 2) m[0] = m[1] = m[2] = m[3] = max_magnitude(m[0], m[2]);
  }
  // lane t works out the scales of the group that rows 32t lie in
  const uint32_t a = t == 0 ? m[0] : t == 1 ? m[1] : t == 2 ? m[2] : m[3];
  const float s0 = group_scale(bf16_lo(a), FP4), s1 = group_scale(bf16_hi(a), FP4);
  const float r0 = s0 > 0.f ? 1.0f / s0 : 0.f, r1 = s1 > 0.f ? 1.0f / s1 : 0.f;
  // (scales near the top of bf16's range, which the fast forms do not take)
  const bool slow = __any_sync(0xFFFFFFFFu, s0 > 1e37f || s1 > 1e37f);
  if ((t * gps & 3) == 0) {
    moe_bf16* out = w.scales + (int64_t)e * w4_scales_per_expert(w.K, w.N, w.group) +
                    w4_scales_at(nb, step, nbs, w4_steps(w.K), gps) +
                    2 * (((2 * p) & 7) * gps + (t * gps >> 2)) + (p >> 2);
    const moe_bf16 b0 = __bfloat16_as_ushort(__float2bfloat16_rn(s0));
    const moe_bf16 b1 = __bfloat16_as_ushort(__float2bfloat16_rn(s1));
    out[0] = b0;
    out[2 * gps] = b1;
    // (or-ed: the order does not matter)
    if (!plain_scale(b0) || !plain_scale(b1))
      atomicOr(reinterpret_cast<uint32_t*>(w.scales + w4_flags_at(w.E, w.K, w.N, w.group)) + e, 1u);
  }
  uint4* dst = reinterpret_cast<uint4*>(w.codes + (int64_t)e * w4_codes_per_expert(w.K, w.N));
  float q0 = 0.f, q1 = 0.f;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    uint32_t word[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int by = (lane & ~3) | (2 * kb + (j >> 1));        // the lane with these rows' scales
      // columns n and n + 1; columns g and g + 8 after an exchange
      const uint32_t* x = v + 16 * kb + 4 * j;
      uint32_t mine;
      if (!slow) {
        if ((j & 1) == 0) {
          q0 = __shfl_sync(0xFFFFFFFFu, r0, by);
          q1 = __shfl_sync(0xFFFFFFFFu, r1, by);
        }
        mine = eight_codes<FP4>(x, q0, q1);
      } else {
        q0 = __shfl_sync(0xFFFFFFFFu, s0, by);
        q1 = __shfl_sync(0xFFFFFFFFu, s1, by);
        mine = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mine |= (nearest_code(bf16_lo(x[q]), q0, FP4) | (nearest_code(bf16_hi(x[q]), q1, FP4) << 4))
                  << (16 * (q & 1) + 8 * (q >> 1));
      }
      const int g = lane >> 2, at = (g & 1) * 4;
      const uint32_t lo = __shfl_sync(0xFFFFFFFFu, mine, (g >> 1) * 4 + t) >> at;
      const uint32_t hi = __shfl_sync(0xFFFFFFFFu, mine, 16 + (g >> 1) * 4 + t) >> at;
      word[j] = w4_arrange<FP4>((lo & 0x0F0F0F0Fu) | ((hi & 0x0F0F0F0Fu) << 4));
    }
    if (2 * step + kb < kbs)
      dst[w4_tile_at(nb, 2 * step + kb, nbs, kbs) / 16 + lane] =
          make_uint4(word[0], word[1], word[2], word[3]);
  }
}

// The caller's codes [E, K, N] (a byte each) and scales [E, groups, N]
template <bool FP4>
__global__ void __launch_bounds__(kPackThreads) w4_pack_kernel(
    W4View w, const uint8_t* __restrict__ codes, const moe_bf16* __restrict__ scales) {
  pdl_enter();
  __shared__ __align__(16) uint16_t tile[128 * kPackPitch];
  const int e = blockIdx.z, step = blockIdx.y, n0 = blockIdx.x * kPackN;
  const int tid = threadIdx.x;
  const int gps = w4_gps(w.group), groups = (w.K + w.group - 1) / w.group;
#pragma unroll 4
  for (int i = tid; i < 128 * (kPackN / 8); i += kPackThreads) {
    const int r = i / (kPackN / 8), c = (i % (kPackN / 8)) * 8;
    const int k = step * 128 + r;
    uint2 b = make_uint2(0u, 0u);
    if (k < w.K && n0 + c < w.N)
      b = *reinterpret_cast<const uint2*>(codes + ((int64_t)e * w.K + k) * w.N + n0 + c);
    uint32_t* d = reinterpret_cast<uint32_t*>(tile + r * kPackPitch + c);      // a byte to 16 bits
    d[0] = __byte_perm(b.x, 0, 0x4140);
    d[1] = __byte_perm(b.x, 0, 0x4342);
    d[2] = __byte_perm(b.y, 0, 0x4140);
    d[3] = __byte_perm(b.y, 0, 0x4342);
  }
  __syncthreads();
  // a warp a tile of 16 columns, its two tiles of 64 rows one after the other
  const int lane = tid & 31, nb = n0 / 16 + tid / 32, g = lane >> 2, t = lane & 3;
  if (nb >= w4_nblocks(w.N)) return;
  const int c0 = 16 * (tid / 32);
  const int kbs = w4_kblocks(w.K), nbs = w4_nblocks(w.N);
  for (int kb = 2 * step; kb < 2 * step + 2 && kb < kbs; ++kb) {
    uint32_t word[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r0 = 64 * (kb & 1) + 16 * j + 4 * t;
      uint32_t x = 0;
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {                 // column g, column g + 8
        const uint16_t* p = tile + r0 * kPackPitch + c0 + g + 8 * hi;
        // rows 0, 1 are pair hi, rows 2, 3 pair 2 + hi; odd rows in the high half
#pragma unroll
        for (int q = 0; q < 4; ++q)
          x |= (p[q * kPackPitch] & 15u) << (4 * hi + 8 * (q >> 1) + 16 * (q & 1));
      }
      word[j] = w4_arrange<FP4>(x);
    }
    uint4* dst = reinterpret_cast<uint4*>(w.codes +
                                          (int64_t)e * w4_codes_per_expert(w.K, w.N) +
                                          w4_tile_at(nb, kb, nbs, kbs));
    dst[lane] = make_uint4(word[0], word[1], word[2], word[3]);
  }
  moe_bf16* out = w.scales + (int64_t)e * w4_scales_per_expert(w.K, w.N, w.group) +
                  w4_scales_at(nb, step, nbs, w4_steps(w.K), gps);
  bool plain = true;
  for (int i = lane; i < 16 * gps; i += 32) {
    const int gg = i / (2 * gps), gr = (i / 2) % gps, hi = i & 1;
    const int gk = step * gps + gr, n = n0 + c0 + gg + 8 * hi;
    const moe_bf16 b =
        gk < groups && n < w.N ? scales[((int64_t)e * groups + gk) * w.N + n] : (moe_bf16)0;
    out[i] = b;
    plain = plain && plain_scale(b);
  }
  // (or-ed: the order does not matter)
  if (!plain)
    atomicOr(reinterpret_cast<uint32_t*>(w.scales + w4_flags_at(w.E, w.K, w.N, w.group)) + e, 1u);
}

// Back to bf16 [E, K, N]: code * scale, rounded (exact for the scales above).
// The same blocks the other way.
template <bool FP4>
__global__ void __launch_bounds__(kPackThreads) w4_unpack_kernel(W4View w,
                                                                 moe_bf16* __restrict__ dst) {
  pdl_enter();
  __shared__ moe_bf16 tile[128][kPackN + 8];
  const int e = blockIdx.z, step = blockIdx.y, n0 = blockIdx.x * kPackN;
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int nb = n0 / 16 + tid / 32, c0 = 16 * (tid / 32);
  const int gps = w4_gps(w.group), kbs = w4_kblocks(w.K);
  const W4Decoder<FP4> decode;
  if (nb < w4_nblocks(w.N)) {
    const moe_bf16* sp = w.scales + (int64_t)e * w4_scales_per_expert(w.K, w.N, w.group) +
                         w4_scales_at(nb, step, w4_nblocks(w.N), w4_steps(w.K), gps) +
                         2 * gps * g;
    for (int kb = 2 * step; kb < 2 * step + 2 && kb < kbs; ++kb) {
      const uint4 v = *reinterpret_cast<const uint4*>(
          w.codes + (int64_t)e * w4_codes_per_expert(w.K, w.N) +
          w4_tile_at(nb, kb, w4_nblocks(w.N), kbs) + 16 * lane);
      const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r0 = 64 * (kb & 1) + 16 * j + 4 * t;
        const int gr = (r0 * gps) >> 7;
        uint32_t p[4];
        decode.values(word[j], p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float s = __bfloat162float(__ushort_as_bfloat16(sp[2 * gr + (i & 1)]));
          const int n = c0 + g + 8 * (i & 1), r = r0 + 2 * (i >> 1);
          const uint32_t o =
              pack_bf16(bf16_lo(p[i]) * decode.kUnit * s, bf16_hi(p[i]) * decode.kUnit * s);
          tile[r][n] = (moe_bf16)(o & 0xFFFFu);
          tile[r + 1][n] = (moe_bf16)(o >> 16);
        }
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < 128 * (kPackN / 8); i += kPackThreads) {
    const int r = i / (kPackN / 8), c = (i % (kPackN / 8)) * 8;
    const int k = step * 128 + r;
    if (k < w.K && n0 + c < w.N)
      *reinterpret_cast<uint4*>(dst + ((int64_t)e * w.K + k) * w.N + n0 + c) =
          *reinterpret_cast<const uint4*>(&tile[r][c]);
  }
}

static dim3 pack_grid(const moe_w4& w) {
  return dim3((w.N + kPackN - 1) / kPackN, w4_steps(w.K), w.E);
}

cudaError_t launch_w4_pack(const moe_w4& w, const moe_bf16* src, const uint8_t* codes,
                           const moe_bf16* scales, cudaStream_t s) {
  timer_before(MOE_KERNEL_W4_PACK, s);
  const bool fp4 = w.kind == MOE_W4_FP4;
  cudaError_t e = cudaMemsetAsync(w.scales + w4_flags_at(w.E, w.K, w.N, w.group), 0,
                                  (size_t)w.E * 4, s);
  if (e == cudaSuccess)
    e = src ? launch_pdl(false, fp4 ? w4_quantise_kernel<true> : w4_quantise_kernel<false>,
                         pack_grid(w), dim3(kPackThreads), 0, s, w4_view(w), src)
            : launch_pdl(false, fp4 ? w4_pack_kernel<true> : w4_pack_kernel<false>, pack_grid(w),
                         dim3(kPackThreads), 0, s, w4_view(w), codes, scales);
  note_launches(1);
  timer_after(MOE_KERNEL_W4_PACK, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_w4_unpack(const moe_w4& w, moe_bf16* dst, cudaStream_t s) {
  timer_before(MOE_KERNEL_W4_PACK, s);
  const auto kernel = w.kind == MOE_W4_FP4 ? w4_unpack_kernel<true> : w4_unpack_kernel<false>;
  const cudaError_t e =
      launch_pdl(false, kernel, pack_grid(w), dim3(kPackThreads), 0, s, w4_view(w), dst);
  note_launches(1);
  timer_after(MOE_KERNEL_W4_PACK, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
