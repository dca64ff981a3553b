// attn_join.cuh — the launch after an attention kernel: units that the schedule
// cut are joined from their parts.
#pragma once

#include "attn.cuh"

namespace moe {

// Block c has the cut in front of CTA c: where it is the first of its unit, the
// block joins the unit's parts, CTA c - 1's slot 1, then slot 0 of c, c + 1, ...
// up to the unit's end, in this order.
constexpr int kJoinThreads = 256;

// Where columns 4 c4 .. 4 c4 + 3 of a part's row are: rows next to each other, as
// the chunk kernel's threads (one a row) write them.
template <int TM, int DP>
__device__ __forceinline__ int64_t part_at(int64_t slot, int r, int c4) {
  return ((slot * (DP / 4) + c4) * TM + r) * 4;
}

struct Part {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void join_part(Part& t, float m, float l, const float4& o) {
  const float nm = fmaxf(t.m, m);
  const float ref = nm == neg_inf() ? 0.f : nm;
  const float f = ex2(t.m - ref), g = ex2(m - ref);
  t.m = nm;
  t.l = t.l * f + l * g;
  t.o.x = t.o.x * f + o.x * g;
  t.o.y = t.o.y * f + o.y * g;
  t.o.z = t.o.z * f + o.z * g;
  t.o.w = t.o.w * f + o.w * g;
}

template <int TM, int DP, int LN>
__device__ __forceinline__ void join_rows(const AttnArgs& a, const Cut& c) {
  constexpr int kItems = 32 / LN;       // a warp's at a time
  const int lane = threadIdx.x & 31, it = lane % kItems, ln = lane / kItems;
  const int warps = kJoinThreads / 32 * gridDim.y;
  const int total = c.nrows * (DP / 4);
  for (int i0 = (blockIdx.y * (kJoinThreads / 32) + threadIdx.x / 32) * kItems; i0 < total;
       i0 += warps * kItems) {
    // lanes past the last item do it over, and write nothing
    const int i = min(i0 + it, total - 1), c4 = i / c.nrows, r = i - c4 * c.nrows;
    Part t{neg_inf(), 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    // four parts' loads in flight
    for (int p0 = c.first + ln; p0 < c.last; p0 += 4 * LN) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int p = p0 + k * LN;
        const int64_t slot = (int64_t)p * 2 + (p == c.first ? 1 : 0);
        ml[k] = make_float2(neg_inf(), 0.f);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < c.last) {
          ml[k] = a.part_ml[slot * TM + r];
          v[k] = *reinterpret_cast<const float4*>(a.part_o + part_at<TM, DP>(slot, r, c4));
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) join_part(t, ml[k].x, ml[k].y, v[k]);
    }
#pragma unroll
    for (int o = kItems; o < 32; o <<= 1) {
      const float m = __shfl_xor_sync(0xFFFFFFFFu, t.m, o);
      const float l = __shfl_xor_sync(0xFFFFFFFFu, t.l, o);
      const float4 v = make_float4(__shfl_xor_sync(0xFFFFFFFFu, t.o.x, o),
                                   __shfl_xor_sync(0xFFFFFFFFu, t.o.y, o),
                                   __shfl_xor_sync(0xFFFFFFFFu, t.o.z, o),
                                   __shfl_xor_sync(0xFFFFFFFFu, t.o.w, o));
      join_part(t, m, l, v);
    }
    if (ln > 0 || i0 + it >= total) continue;
    const int tok = div_group(a, c.r0 + r), head = c.h * a.G + (c.r0 + r) - tok * a.G;
    const RowEnd e = row_end(t.m, t.l, a.sinks, head);
    if (c4 * 4 < a.D)
      *reinterpret_cast<uint2*>(a.out + (int64_t)(c.q0 + tok) * a.out_stride +
                                (int64_t)head * a.D + c4 * 4) =
          make_uint2(pack_bf16(t.o.x * e.factor, t.o.y * e.factor),
                     pack_bf16(t.o.z * e.factor, t.o.w * e.factor));
    if (a.lse && c4 == 0) a.lse[(int64_t)(c.q0 + tok) * a.Hq + head] = e.lse;
  }
}

template <int TM, int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(
    const __grid_constant__ AttnArgs a) {
  pdl_enter();
  const Cut c = a.cuts[blockIdx.x + 1];
  if (c.first < 0) return;
  // LN lanes an item (four columns of a row), each every LN-th part, by which is
  // fewer rounds of loads, four parts a round: eight for few rows cut many times.
  // Bound: the latency of a round. One lane always: 8 tokens over 400 to 9000 keys
  // 44 instead of 32 us in all, 5 tokens over 100k keys 62 instead of 48; eight
  // always: 128 tokens over 2500 keys 67 instead of 42.
  const int parts = c.last - c.first, items = c.nrows * (DP / 4);
  const int threads = kJoinThreads * gridDim.y;
  const int one = ((items - 1) / threads + 1) * ((parts + 3) / 4);
  const int eight = ((items * 8 - 1) / threads + 1) * ((parts + 31) / 32);
  if (one < eight) join_rows<TM, DP, 1>(a, c);
  else join_rows<TM, DP, 8>(a, c);
}

}  // namespace moe
