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
// Memory-bound: 2 bytes read and 1/2 + 2/group written a weight. A block takes 64
// columns by 128 rows through shared memory: rows of 128 bytes come in, whole
// tiles of 512 bytes go out.
#include "w4.cuh"

namespace moe {

constexpr int kPackN = 64;            // columns of a block: four tiles
constexpr int kPackThreads = 128;

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

__device__ __forceinline__ uint32_t nearest_code(float w, float s, bool fp4) {
  if (!(s > 0.f)) return 0u;
  const float q = __fdiv_rn(w, s);
  const float a = fabsf(q);
  // the codes count steps of 1; or of 1/2 up to 2, of 1 up to 4, of 2 beyond
  int n = !fp4      ? __float2int_rn(a)
          : a < 2.f ? __float2int_rn(2.f * a)
          : a < 4.f ? __float2int_rn(a) + 2
                    : __float2int_rn(0.5f * a) + 4;
  // at the top of the range the nearest value may be one that bf16 does not hold
  if (s > 1e37f && n > 0 && w4_value((uint32_t)n, fp4) * s > 3.3895314e38f) --n;
  if (!fp4) return (uint32_t)(q < 0.f ? -n : n) & 15u;
  return (uint32_t)n | (n && q < 0.f ? 8u : 0u);
}

// SRC 0: bf16 weights [E, K, N], quantised here; 1: codes [E, K, N] (a byte each) and
// scales [E, groups, N] of the caller's
template <int SRC, bool FP4>
__global__ void __launch_bounds__(kPackThreads) w4_pack_kernel(
    W4View w, const moe_bf16* __restrict__ src, const uint8_t* __restrict__ codes,
    const moe_bf16* __restrict__ scales) {
  pdl_enter();
  __shared__ float tile[128][kPackN + 1];             // weights, then codes
  __shared__ float amax[8][kPackN];                   // of 16 rows each
  __shared__ float sc[4][kPackN];                     // the step's groups
  const int e = blockIdx.z, step = blockIdx.y, n0 = blockIdx.x * kPackN;
  const int tid = threadIdx.x;
  const int gps = w4_gps(w.group), groups = (w.K + w.group - 1) / w.group;
  // rows of 64 columns, 16 bytes (8 with one byte a code) a thread
  for (int i = tid; i < 128 * (kPackN / 8); i += kPackThreads) {
    const int r = i / (kPackN / 8), c = (i % (kPackN / 8)) * 8;
    const int k = step * 128 + r;
    float v[8] = {};
    if (k < w.K && n0 + c < w.N) {
      const int64_t at = ((int64_t)e * w.K + k) * w.N + n0 + c;
      if (SRC == 0) {
        unpack8(*reinterpret_cast<const uint4*>(src + at), v);
      } else {
        const uint2 b = *reinterpret_cast<const uint2*>(codes + at);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = __uint_as_float(((j < 4 ? b.x : b.y) >> (8 * (j & 3))) & 15u);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[r][c + j] = v[j];
  }
  __syncthreads();
  if (SRC == 0) {
    for (int i = tid; i < 8 * kPackN; i += kPackThreads) {
      const int n = i % kPackN, part = i / kPackN;
      float a = 0.f;
      bool odd = false;                // an infinity or NaN
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float v = fabsf(tile[16 * part + r][n]);
        odd |= !(v < INFINITY);
        a = fmaxf(a, v);
      }
      amax[part][n] = odd ? INFINITY : a;
    }
    __syncthreads();
    for (int i = tid; i < gps * kPackN; i += kPackThreads) {
      const int n = i % kPackN, gr = i / kPackN, parts = 8 / gps;
      float a = 0.f;
      for (int p = 0; p < parts; ++p) a = fmaxf(a, amax[gr * parts + p][n]);
      sc[gr][n] = group_scale(a, FP4);
    }
  } else {
    for (int i = tid; i < gps * kPackN; i += kPackThreads) {
      const int n = i % kPackN, gr = i / kPackN, g = step * gps + gr;
      sc[gr][n] = g < groups && n0 + n < w.N
                      ? __bfloat162float(__ushort_as_bfloat16(
                            scales[((int64_t)e * groups + g) * w.N + n0 + n]))
                      : 0.f;
    }
  }
  __syncthreads();
  // a warp a tile of 16 columns, its two tiles of 64 rows one after the other
  const int lane = tid & 31, nb = n0 / 16 + tid / 32, g = lane >> 2, t = lane & 3;
  if (nb >= w4_nblocks(w.N)) return;
  const int c0 = 16 * (tid / 32);
  const int kbs = w4_kblocks(w.K);
  for (int kb = 2 * step; kb < 2 * step + 2 && kb < kbs; ++kb) {
    uint32_t word[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          const int n = c0 + g + 8 * (i & 1);
          const int r = 64 * (kb & 1) + 16 * j + 4 * t + 2 * (i >> 1) + odd;
          const float v = tile[r][n];
          // a group is 32, 64 or 128 rows: r / group without a division
          const uint32_t code =
              SRC == 0 ? nearest_code(v, sc[(r * gps) >> 7][n], FP4) : __float_as_uint(v);
          word[j] |= w4_place(code, i, odd, FP4);
        }
    uint4* dst = reinterpret_cast<uint4*>(w.codes +
                                          (int64_t)e * w4_codes_per_expert(w.K, w.N) +
                                          w4_tile_at(nb, kb, w4_nblocks(w.N), kbs));
    dst[lane] = make_uint4(word[0], word[1], word[2], word[3]);
  }
  moe_bf16* out = w.scales + (int64_t)e * w4_scales_per_expert(w.K, w.N, w.group) +
                  w4_scales_at(nb, step, w4_nblocks(w.N), w4_steps(w.K), gps);
  bool plain = true;
  for (int i = lane; i < 16 * gps; i += 32) {
    const int gg = i / (2 * gps), gr = (i / 2) % gps, hi = i & 1;
    out[i] = __bfloat16_as_ushort(__float2bfloat16_rn(sc[gr][c0 + gg + 8 * hi]));
    plain = plain && plain_scale(out[i]);
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
  const auto kernel = src ? (fp4 ? w4_pack_kernel<0, true> : w4_pack_kernel<0, false>)
                          : (fp4 ? w4_pack_kernel<1, true> : w4_pack_kernel<1, false>);
  cudaError_t e = cudaMemsetAsync(w.scales + w4_flags_at(w.E, w.K, w.N, w.group), 0,
                                  (size_t)w.E * 4, s);
  if (e == cudaSuccess)
    e = launch_pdl(false, kernel, pack_grid(w), dim3(kPackThreads), 0, s, w4_view(w), src, codes,
                   scales);
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
