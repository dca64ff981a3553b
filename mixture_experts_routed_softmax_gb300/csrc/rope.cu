// rope.cu — rotary positions with one to several axes, alone (moe_rope) or on
// the way into a paged cache (moe_kv_append).
//
// A pair (x1, x2) of a head turns by the angle pos * w: y1 = c x1 - s x2,
// y2 = c x2 + s x1 (the transpose: s -> -s). The frequency comes as a 64-bit
// binary fraction of a turn, so position * fraction mod 2^64 is the angle's
// fraction of a turn with an error of |pos| 2^-65 turns: an integer product
// does the range reduction that floating-point angles of far positions lose.
// Its top 32 bits (2^-32 turns) go to sincospif.
//
// Bound: memory. Every element is read once and written once in 16-byte
// pieces; a token's sines and cosines are computed once per block and shared
// by all its heads through shared memory. 16384 tokens of 64 + 8 heads, D = 64:
// moe_rope 56 us = 5.3 TB/s (52 us, 5.8 TB/s, back to back; a plain copy 6.8),
// the append 67 us = 5.0 TB/s (63 us). More loads in flight per thread cost
// registers and so resident blocks, and were slower. Halves of rd / 2 elements
// that no 16-byte piece divides go two bytes at a time, at half that rate: 32 + 4
// heads of 72, 16384 tokens, 73 us = 2.3 TB/s where heads of 80 take 42 us = 4.5
// TB/s; 64 + 8 heads of 40 83 us, by neighbours 42; the append of 16384 tokens, 32 +
// 4 heads of 72, 85 us, of 80 48 us.
#include "attn.cuh"
#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTok = 4;       // tokens of one block
constexpr int kRopeMaxPairs = kAttnMaxD / 2;

struct RopeArgs {
  const uint64_t* turns;
  const int32_t* axis;
  const int32_t* pos;
  int rd, n_axes;
  float scale, sign;
  int64_t T;
  int D, Hq, Hk;
  const moe_bf16* q;
  moe_bf16* q_out;
  int64_t q_stride, qo_stride;
  const moe_bf16* k;
  moe_bf16* k_out;       // moe_rope: [T, Hk, D]; the append: the cache's keys
  int64_t k_stride, ko_stride;
  const moe_bf16* v;     // the append only
  moe_bf16* v_out;
  int64_t v_stride;
  int64_t head_stride;   // of k_out and v_out
  AttnBatch bt;          // the append only
  int* status;
};

// How a pair's elements are reached: eight pairs at a time in 16-byte pieces,
// halves (pairs i, i + rd/2) or neighbours (2i, 2i + 1); or one pair per step
// with 2-byte accesses, for rd/2 (halves) or rd (neighbours) that no 16-byte
// piece divides.
enum class PairLoad { kHalves8, kNeighbours8, kHalves1, kNeighbours1 };

template <PairLoad L, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a, int ntok) {
  pdl_enter();
  __shared__ float2 cs[kRopeMaxTok][kRopeMaxPairs];
  __shared__ int64_t kv_at[kRopeMaxTok];    // element offset of the token's slot, -1: none
  __shared__ int s_pos[kRopeMaxTok];        // its cache position (0: none)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = (int64_t)blockIdx.x * ntok;
  const int nt = (int)(a.T - t0 < ntok ? a.T - t0 : ntok);
  const int np = a.rd / 2;

  if constexpr (APPEND) {
    if (warp < nt) {
      // one warp a token: its sequence, its cache position and its slot
      const int64_t t = t0 + warp;
      int64_t at = -1;
      int c = 0;
      const int b = find_sequence(a.bt.cu_q, a.bt.B, (int)t, lane);
      if (b >= 0 && lane == 0) {
        const int end = a.bt.cu_q[b + 1], n = a.bt.kv_len[b];
        bool ok = n >= 0 && n <= a.bt.max_pages * a.bt.page_size && end <= a.bt.T;
        if (ok) c = n - end + (int)t;      // kv_len - n_q + (t - cu_q[b])
        ok = ok && c >= 0 && c < n && a.bt.cu_q[b] <= t;
        if (ok) {
          const int pg = c / a.bt.page_size;
          const int page = a.bt.table[(int64_t)b * a.bt.table_stride + pg];
          ok = page >= 0 && page < a.bt.n_pages;
          if (ok)
            at = (int64_t)page * a.bt.page_stride +
                 (int64_t)(c - pg * a.bt.page_size) * a.bt.token_stride;
        }
        if (!ok) {
          raise_status(a.status, MOE_ERR_DEVICE_INDEX);
          c = 0;
        }
      }
      if (lane == 0) {
        kv_at[warp] = at;
        s_pos[warp] = c;
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < nt * np; i += kRopeThreads) {
    const int tk = i / np, p = i - tk * np;
    int ax = a.axis ? a.axis[p] : 0;
    if (ax < 0 || ax >= a.n_axes) {
      raise_status(a.status, MOE_ERR_DEVICE_INDEX);
      ax = 0;
    }
    int pos;
    if (APPEND && !a.pos) pos = s_pos[tk];
    else pos = a.pos[(int64_t)ax * a.T + t0 + tk];
    const uint64_t turn = (uint64_t)(int64_t)pos * a.turns[p];
    // the signed top half: the angle in units of 2^-32 turns = 2^-31 half turns
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077392578125e-10f, &s, &c);
    cs[tk][p] = make_float2(c * a.scale, s * a.scale * a.sign);
  }
  __syncthreads();

  // rotated pieces: thread -> a fixed group of pairs, heads in strides
  const int H = a.Hq + a.Hk;
  const int per = L == PairLoad::kHalves8 ? np / 8 : L == PairLoad::kNeighbours8 ? np / 4 : np;
  if (per > 0) {
    const int piece = tid % per;
    const int rstep = kRopeThreads / per;
    // the threads left over when `per` does not divide the block have no group
    const int first = tid / per < rstep ? tid / per : nt * H;
    for (int j = first; j < nt * H; j += rstep) {
      const int tk = j / H, h = j - tk * H;
      const int64_t t = t0 + tk;
      const moe_bf16* src;
      moe_bf16* dst;
      if (h < a.Hq) {
        src = a.q + t * a.q_stride + (int64_t)h * a.D;
        dst = a.q_out + t * a.qo_stride + (int64_t)h * a.D;
      } else {
        src = a.k + t * a.k_stride + (int64_t)(h - a.Hq) * a.D;
        if constexpr (APPEND) {
          if (kv_at[tk] < 0) continue;
          dst = a.k_out + kv_at[tk] + (int64_t)(h - a.Hq) * a.head_stride;
        } else {
          dst = a.k_out + t * a.ko_stride + (int64_t)(h - a.Hq) * a.D;
        }
      }
      if constexpr (L == PairLoad::kHalves8) {
        const uint4 lo = *reinterpret_cast<const uint4*>(src + piece * 8);
        const moe_bf16* s2 = src + np + piece * 8;
        const uint4 hi = *reinterpret_cast<const uint4*>(s2);
        float x[8], y[8], u[8], w[8];
        unpack8(lo, x);
        unpack8(hi, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = cs[tk][piece * 8 + e];
          u[e] = v.x * x[e] - v.y * y[e];
          w[e] = v.x * y[e] + v.y * x[e];
        }
        *reinterpret_cast<uint4*>(dst + piece * 8) = pack8(u);
        *reinterpret_cast<uint4*>(dst + np + piece * 8) = pack8(w);
      } else if constexpr (L == PairLoad::kNeighbours8) {
        const uint4 v4 = *reinterpret_cast<const uint4*>(src + piece * 8);
        float x[8], u[8];
        unpack8(v4, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = cs[tk][piece * 4 + e];
          u[2 * e] = v.x * x[2 * e] - v.y * x[2 * e + 1];
          u[2 * e + 1] = v.x * x[2 * e + 1] + v.y * x[2 * e];
        }
        *reinterpret_cast<uint4*>(dst + piece * 8) = pack8(u);
      } else {
        const int i1 = L == PairLoad::kHalves1 ? piece : 2 * piece;
        const int i2 = L == PairLoad::kHalves1 ? piece + np : 2 * piece + 1;
        const float x = bf16_lo(src[i1]), y = bf16_lo(src[i2]);
        const float2 v = cs[tk][piece];
        const uint32_t o = pack_bf16(v.x * x - v.y * y, v.x * y + v.y * x);
        dst[i1] = (moe_bf16)(o & 0xFFFFu);
        dst[i2] = (moe_bf16)(o >> 16);
      }
    }
  }
  // the elements past rd, copied; in 16-byte pieces where they start on one
  const int rest = a.D - a.rd;
  if (rest > 0) {
    const bool wide = (a.rd % 8) == 0;
    const int n = wide ? rest / 8 : rest;
    for (int j = tid; j < nt * H * n; j += kRopeThreads) {
      const int th = j / n, e = j - th * n;
      const int tk = th / H, h = th - tk * H;
      const int64_t t = t0 + tk;
      const moe_bf16* src;
      moe_bf16* dst;
      if (h < a.Hq) {
        src = a.q + t * a.q_stride + (int64_t)h * a.D + a.rd;
        dst = a.q_out + t * a.qo_stride + (int64_t)h * a.D + a.rd;
      } else {
        src = a.k + t * a.k_stride + (int64_t)(h - a.Hq) * a.D + a.rd;
        if constexpr (APPEND) {
          if (kv_at[tk] < 0) continue;
          dst = a.k_out + kv_at[tk] + (int64_t)(h - a.Hq) * a.head_stride + a.rd;
        } else {
          dst = a.k_out + t * a.ko_stride + (int64_t)(h - a.Hq) * a.D + a.rd;
        }
      }
      if (wide) reinterpret_cast<uint4*>(dst)[e] = reinterpret_cast<const uint4*>(src)[e];
      else dst[e] = src[e];
    }
  }
  if constexpr (APPEND) {
    const int n = a.D / 8;
    for (int j = tid; j < nt * a.Hk * n; j += kRopeThreads) {
      const int th = j / n, e = j - th * n;
      const int tk = th / a.Hk, h = th - tk * a.Hk;
      if (kv_at[tk] < 0) continue;
      const uint4* src = reinterpret_cast<const uint4*>(a.v + (t0 + tk) * a.v_stride +
                                                        (int64_t)h * a.D);
      uint4* dst = reinterpret_cast<uint4*>(a.v_out + kv_at[tk] + (int64_t)h * a.head_stride);
      dst[e] = src[e];
    }
  }
}

template <bool APPEND>
static cudaError_t launch_rope_kernel(const RopeArgs& a, int interleaved, cudaStream_t s) {
  // One token a block while blocks are few, then four (1 / 4 tokens a block, back
  // to back, 32 + 4 heads of 128: 500 tokens 6.5 / 6.7 us, 2432 tokens 15.9 / 14.2,
  // 16384 tokens 63.8 / 53.9).
  const int ntok = a.T >= 4 * kRopeMaxTok * (int64_t)num_sms() ? kRopeMaxTok : 1;
  const dim3 grid((unsigned)((a.T + ntok - 1) / ntok));
  const bool pdl = pdl_for_tokens(a.T);
  timer_before(MOE_KERNEL_ROPE, s);
  cudaError_t e;
  if (interleaved && a.rd % 8 == 0)
    e = launch_pdl(pdl, rope_kernel<PairLoad::kNeighbours8, APPEND>, grid, dim3(kRopeThreads), 0, s,
                   a, ntok);
  else if (interleaved)
    e = launch_pdl(pdl, rope_kernel<PairLoad::kNeighbours1, APPEND>, grid, dim3(kRopeThreads), 0, s,
                   a, ntok);
  else if (a.rd % 16 == 0)
    e = launch_pdl(pdl, rope_kernel<PairLoad::kHalves8, APPEND>, grid, dim3(kRopeThreads), 0, s, a,
                   ntok);
  else
    e = launch_pdl(pdl, rope_kernel<PairLoad::kHalves1, APPEND>, grid, dim3(kRopeThreads), 0, s, a,
                   ntok);
  note_launches(1);
  timer_after(MOE_KERNEL_ROPE, s);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

static RopeArgs rotary_args(const moe_rotary* rot, const int32_t* pos, int transpose, int64_t T,
                            int D, int* status) {
  RopeArgs a = {};
  if (rot) {
    a.turns = rot->turns;
    a.axis = rot->axis;
    a.rd = rot->rd;
    a.n_axes = rot->n_axes;
    a.scale = rot->scale;
  }
  a.sign = transpose ? -1.f : 1.f;
  a.pos = pos;
  a.T = T;
  a.D = D;
  a.status = status;
  return a;
}

cudaError_t launch_rope(const moe_rotary* rot, const int32_t* pos, int64_t T, int D,
                        int transpose, const moe_bf16* q, int64_t q_stride, int Hq,
                        moe_bf16* q_out, int64_t qo_stride, const moe_bf16* k, int64_t k_stride,
                        int Hk, moe_bf16* k_out, int64_t ko_stride, int* status,
                        cudaStream_t s) {
  RopeArgs a = rotary_args(rot, pos, transpose, T, D, status);
  a.q = q; a.q_out = q_out; a.q_stride = q_stride; a.qo_stride = qo_stride; a.Hq = Hq;
  a.k = k; a.k_out = k_out; a.k_stride = k_stride; a.ko_stride = ko_stride;
  a.Hk = k ? Hk : 0;
  return launch_rope_kernel<false>(a, rot->interleaved, s);
}

cudaError_t launch_kv_append(const moe_kv_cache& c, const moe_kv_batch& b, const moe_rotary* rot,
                             const int32_t* pos, const moe_bf16* k, int64_t k_stride,
                             const moe_bf16* v, int64_t v_stride, const moe_bf16* q,
                             int64_t q_stride, int Hq, moe_bf16* q_out, int64_t qo_stride,
                             int* status, cudaStream_t s) {
  RopeArgs a = rotary_args(rot, pos, 0, b.T, c.D, status);
  a.q = q; a.q_out = q_out; a.q_stride = q_stride; a.qo_stride = qo_stride;
  a.Hq = q ? Hq : 0;
  a.k = k; a.k_stride = k_stride; a.k_out = c.k;
  a.v = v; a.v_stride = v_stride; a.v_out = c.v;
  a.Hk = c.Hkv;
  a.head_stride = c.head_stride;
  a.bt = attn_batch(c, b);
  return launch_rope_kernel<true>(a, rot ? rot->interleaved : 0, s);
}

}  // namespace moe
