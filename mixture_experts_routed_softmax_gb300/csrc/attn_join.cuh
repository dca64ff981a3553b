// attn_join.cuh — the launch after an attention kernel: units that the schedule
// cut are joined from their parts.
#pragma once

#include "attn.cuh"

namespace moe {

// Block c has the cut in front of CTA c: where it is the first of its unit, the
// block joins the unit's parts, CTA c - 1's slot 1, then slot 0 of c, c + 1, ...
// up to the unit's end, in this order.
constexpr int kJoinThreads = 256;

template <int TM, int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(
    const __grid_constant__ AttnArgs a) {
  pdl_enter();
  const Cut c = a.cuts[blockIdx.x + 1];
  if (c.first < 0) return;
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < c.nrows * (DP / 4);
       i += kJoinThreads * gridDim.y) {
    const int r = i / (DP / 4), c4 = i - r * (DP / 4);
    float m = neg_inf(), l = 0.f;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    // four parts' loads in flight
    for (int p0 = c.first; p0 < c.last; p0 += 4) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int p = p0 + k;
        const int64_t row = ((int64_t)p * 2 + (p == c.first ? 1 : 0)) * TM + r;
        if (p < c.last) {
          ml[k] = a.part_ml[row];
          v[k] = *reinterpret_cast<const float4*>(a.part_o + row * DP + c4 * 4);
        } else {
          ml[k] = make_float2(neg_inf(), 0.f);
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float nm = fmaxf(m, ml[k].x);
        const float ref = nm == neg_inf() ? 0.f : nm;
        const float f = ex2(m - ref), g = ex2(ml[k].x - ref);
        m = nm;
        l = l * f + ml[k].y * g;
        t.x = t.x * f + v[k].x * g; t.y = t.y * f + v[k].y * g;
        t.z = t.z * f + v[k].z * g; t.w = t.w * f + v[k].w * g;
      }
    }
    const int tok = div_group(a, c.r0 + r), head = c.h * a.G + (c.r0 + r) - tok * a.G;
    const RowEnd e = row_end(m, l, a.sinks, head);
    if (c4 * 4 < a.D)
      *reinterpret_cast<uint2*>(a.out + (int64_t)(c.q0 + tok) * a.out_stride +
                                (int64_t)head * a.D + c4 * 4) =
          make_uint2(pack_bf16(t.x * e.factor, t.y * e.factor),
                     pack_bf16(t.z * e.factor, t.w * e.factor));
    if (a.lse && c4 == 0) a.lse[(int64_t)(c.q0 + tok) * a.Hq + head] = e.lse;
  }
}

}  // namespace moe
