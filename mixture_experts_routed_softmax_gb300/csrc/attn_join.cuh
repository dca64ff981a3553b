// attn_join.cuh — the launch after an attention kernel: units that the schedule
// cut are joined from their parts.
#pragma once

#include "attn.cuh"

namespace moe {

// Block c looks at the boundary in front of CTA c. When it lies inside a unit
// and no earlier boundary does, the block joins the unit's parts: CTA c - 1's
// slot 1, then slot 0 of c, c + 1, ... up to the unit's end, in this order.
constexpr int kJoinThreads = 256;

template <int TM, int TN, int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnArgs a, int n) {
  __shared__ Place pl;
  pdl_enter();
  const int cta = blockIdx.x + 1;
  if (!locate<TM, TN, kJoinThreads>(a, cta, n, pl)) return;
  const Line line = pl.line;
  const long long unit0 = line.start(cta) - pl.off;
  if (pl.off == 0 || line.start(cta - 1) > unit0) return;
  const Seq s = load_seq(a, pl.b);
  const long long unit1 = unit0 + Tiling<TM, TN>::weight(a, s, pl.m);
  int last = cta;             // the parts are those of CTAs cta - 1 .. last - 1
  while (last < n && line.start(last) < unit1) ++last;
  const int r0 = pl.m * TM;
  const int nrows = min(TM, s.nq * a.G - r0);
  const int stripes = gridDim.y;
  for (int i = blockIdx.y * kJoinThreads + threadIdx.x; i < nrows * (DP / 4);
       i += kJoinThreads * stripes) {
    const int r = i / (DP / 4), c4 = i - r * (DP / 4);
    float m = neg_inf(), l = 0.f;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = cta - 1; p < last; ++p) {
      // a CTA without steps left no part
      if (line.start(p + 1) == line.start(p)) continue;
      const int64_t slot = (int64_t)p * 2 + (p == cta - 1 ? 1 : 0);
      const float2 ml = a.part_ml[slot * TM + r];
      const float4 v = *reinterpret_cast<const float4*>(a.part_o + (slot * TM + r) * DP + c4 * 4);
      const float nm = fmaxf(m, ml.x);
      const float ref = nm == neg_inf() ? 0.f : nm;
      const float f = ex2(m - ref), g = ex2(ml.x - ref);
      m = nm;
      l = l * f + ml.y * g;
      t.x = t.x * f + v.x * g; t.y = t.y * f + v.y * g;
      t.z = t.z * f + v.z * g; t.w = t.w * f + v.w * g;
    }
    const int tok = div_group(a, r0 + r), head = pl.h * a.G + (r0 + r) - tok * a.G;
    const RowEnd e = row_end(m, l, a.sinks, head);
    if (c4 * 4 < a.D)
      *reinterpret_cast<uint2*>(a.out + (int64_t)(s.q0 + tok) * a.out_stride +
                                (int64_t)head * a.D + c4 * 4) =
          make_uint2(pack_bf16(t.x * e.factor, t.y * e.factor),
                     pack_bf16(t.z * e.factor, t.w * e.factor));
    if (a.lse && c4 == 0) a.lse[(int64_t)(s.q0 + tok) * a.Hq + head] = e.lse;
  }
}

}  // namespace moe
