// attn_rows.cu — attention over the paged cache for few rows per key/value
// head (decode, draft verification), and for page sizes the chunk kernel does
// not take; the launch that joins cut units.
//
// out = sum_j p_j v_j / sum_j p_j with p_j = exp(s_j - max): one pass over the
// keys with a running maximum and sum. With R rows over the keys the work is
// 4 R D operations for 4 D bytes of a key and value, so up to a few dozen rows
// the bound is reading the cache once. Hence: warps that never wait for each
// other, each with its own keys (16 of a 64-key tile), its own ring of 16-byte
// asynchronous copies, its own maxima, sums and accumulator, joined through
// shared memory once per unit. The products run on mma.sync (m16n8k16): its
// rate is far above what the copies feed, and it takes 16 rows where tcgen05
// takes 128.
#include "attn.cuh"
#include "attn_join.cuh"
#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kRowsWarps = 4;
constexpr int kRowsThreads = 32 * kRowsWarps;
constexpr int kChunk = 16;                        // keys of a warp's step
constexpr int kRowsTN = kChunk * kRowsWarps;

template <int DP, int MB>
struct RowsGeo {
  static constexpr int TM = 16 * MB;
  static constexpr int row_bytes = DP * 2;
  static constexpr int stage = 2 * kChunk * row_bytes;           // K and V
  static constexpr int stages = DP == 128 ? 3 : 4;
  static constexpr int ring = kRowsWarps * stages * stage;
  static constexpr int merge = kRowsWarps * TM * DP * 4;         // reuses the ring
  static constexpr int q_bytes = TM * row_bytes;
  static constexpr int smem = (ring > merge ? ring : merge) + q_bytes;
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// byte offset of 16-byte piece c of row r; the pieces of 8 rows are permuted so
// that ldmatrix reads 8 rows of one piece from 8 different banks groups
template <int DP>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t ld_shared32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// No infinity or NaN among the chunk's values (by the whole warp).
template <int DP>
__device__ __forceinline__ bool chunk_finite(uint32_t sv) {
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kChunk * DP / 64; ++i) {
    const uint32_t v = ld_shared32(sv + (i * 32 + (threadIdx.x & 31)) * 4);
    bad = bad || (v & 0x7F800000u) == 0x7F800000u || (v & 0x7F80u) == 0x7F80u;
  }
  return !__any_sync(0xFFFFFFFFu, bad);
}

// The offset of key `key`'s slot in the cache (elements, before the head), or
// -1: outside [lo, hi), or a page outside the cache.
__device__ __forceinline__ int64_t key_at(const AttnArgs& a, int b, int key, int lo, int hi) {
  if (key < lo || key >= hi) return -1;
  const int pg = page_of(a.bt, key);
  const int page = a.bt.table[(int64_t)b * a.bt.table_stride + pg];
  if (page < 0 || page >= a.bt.n_pages) {
    raise_status(a.status, MOE_ERR_DEVICE_INDEX);
    return -1;
  }
  return (int64_t)page * a.bt.page_stride +
         (int64_t)(key - pg * a.bt.page_size) * a.bt.token_stride;
}

template <int DP, int MB>
__global__ void __launch_bounds__(kRowsThreads) attn_rows_kernel(const __grid_constant__ AttnArgs a) {
  using G = RowsGeo<DP, MB>;
  constexpr int TM = G::TM, TN = kRowsTN, S = G::stages;
  constexpr int ND = DP / 8;               // 8-wide column tiles of the accumulator
  constexpr int NC = DP / 8;               // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Place pl;
  __shared__ Unit un;
  __shared__ float2 s_ml[kRowsWarps][TM];
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!locate<TM, TN, kRowsThreads>(a, blockIdx.x, gridDim.x, pl)) return;
  if (tid == 0) unit_first<TM, TN>(a, pl, blockIdx.x, true, un);
  __syncthreads();

  const uint32_t s_ring = smem_u32(smem) + warp * S * G::stage;
  const uint32_t s_q = smem_u32(smem) + (uint32_t)(G::smem - G::q_bytes);
  float* const merge = reinterpret_cast<float*>(smem);
  const int lr = lane >> 2, lc = lane & 3;      // accumulator row and column pair

  while (un.more()) {
    const Unit wk = un;
    const Seq s = wk.s;
    const int rows = s.nq * a.G;
    const int r0 = wk.m * TM;
    const int nrows = min(TM, rows - r0);
    const int h = wk.h;
    // ---- the rows' queries into shared memory (rows past the unit: zeros) --
    for (int i = tid; i < TM * NC; i += kRowsThreads) {
      const int r = i / NC, c = i - r * NC;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < nrows && c * 8 < a.D) {
        const int tok = div_group(a, r0 + r), g = (r0 + r) - tok * a.G;
        v = *reinterpret_cast<const uint4*>(a.q + (int64_t)(s.q0 + tok) * a.q_stride +
                                            (int64_t)(h * a.G + g) * a.D + c * 8);
      }
      *reinterpret_cast<uint4*>(smem + (G::smem - G::q_bytes) + tile_at<DP>(r, c)) = v;
    }
    // ---- each row's keys; the range every row sees needs no mask -----------
    int lo[MB][2], hi[MB][2];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mb * 16 + lr + 8 * e;
        const int tok = div_group(a, r0 + min(r, nrows - 1));
        lo[mb][e] = key_lo(a, s, tok);
        hi[mb][e] = r < nrows ? key_hi(a, s, tok) : 0;
      }
    const int all_lo = wk.all_lo;
    const int all_hi = wk.all_hi;
    const bool rows_differ = all_lo > wk.lo || all_hi < wk.hi;

    float o[MB][ND][4];
    float mx[MB][2], sum[MB][2];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
      for (int n = 0; n < ND; ++n) o[mb][n][0] = o[mb][n][1] = o[mb][n][2] = o[mb][n][3] = 0.f;
      mx[mb][0] = mx[mb][1] = neg_inf();
      sum[mb][0] = sum[mb][1] = 0.f;
    }
    const int ntile = wk.nt;
    const int tile0 = wk.t0;
    const moe_bf16* kh = a.k + (int64_t)h * a.head_stride;
    const moe_bf16* vh = a.v + (int64_t)h * a.head_stride;

    // chunk j of this warp: keys [first_key(j), + 16)
    auto first_key = [&](int j) { return (tile0 + j) * TN + warp * kChunk; };
    auto lookup = [&](int j) -> int64_t {
      if (j >= ntile) return -1;
      return key_at(a, wk.b, first_key(j) + (lane & 15), wk.lo, wk.hi);
    };
    auto issue = [&](int j, int64_t at) {
      if (j < ntile) {
        const uint32_t dst = s_ring + (j % S) * G::stage;
        constexpr int kRowsPer = 32 / NC;           // rows covered by one warp-wide copy
        const int c = lane % NC;
#pragma unroll
        for (int i = 0; i < kChunk / kRowsPer; ++i) {
          const int r = i * kRowsPer + lane / NC;
          const int64_t off = __shfl_sync(0xFFFFFFFFu, at, r);
          const bool ok = off >= 0 && c * 8 < a.D;
          const int64_t e = ok ? off + c * 8 : 0;
          cp_async16(dst + tile_at<DP>(r, c), kh + e, ok);
          cp_async16(dst + kChunk * G::row_bytes + tile_at<DP>(r, c), vh + e, ok);
        }
      }
      cp_async_commit();
    };
    int64_t ahead = -1;      // the next chunk's slots, looked up a step early
    for (int j = 0; j < S - 1; ++j) issue(j, lookup(j));
    ahead = lookup(S - 1);
    __syncthreads();         // the queries are in shared memory

    uint32_t qf[MB == 1 ? DP / 16 : 1][4];
    if constexpr (MB == 1) {
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
        ldmatrix4(s_q + tile_at<DP>(lane & 15, kk * 2 + (lane >> 4)), qf[kk]);
    }

    for (int j = 0; j < ntile; ++j) {
      issue(j + S - 1, ahead);
      ahead = lookup(j + S);
      cp_async_wait<S - 1>();
      __syncwarp();
      const uint32_t sk = s_ring + (j % S) * G::stage;
      const uint32_t sv = sk + kChunk * G::row_bytes;
      float c[MB][2][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int n = 0; n < 2; ++n) c[mb][n][0] = c[mb][n][1] = c[mb][n][2] = c[mb][n][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        // B of two 8-key tiles: (keys 0-7, d lo), (0-7, d hi), (8-15, d lo), (8-15, d hi)
        uint32_t kf[4];
        ldmatrix4(sk + tile_at<DP>((lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)),
                  kf);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          if constexpr (MB == 1) {
            mma16816(c[mb][0], qf[kk], kf[0], kf[1]);
            mma16816(c[mb][1], qf[kk], kf[2], kf[3]);
          } else {
            uint32_t q4[4];
            ldmatrix4(s_q + tile_at<DP>(mb * 16 + (lane & 15), kk * 2 + (lane >> 4)), q4);
            mma16816(c[mb][0], q4, kf[0], kf[1]);
            mma16816(c[mb][1], q4, kf[2], kf[3]);
          }
        }
      }
      const int k0 = first_key(j);
      const bool masked = k0 < all_lo || k0 + kChunk > all_hi;
      uint32_t pf[MB][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        if (masked) {
          // masked by selection: a masked score's value, NaN or not, is dropped
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = k0 + n * 8 + lc * 2 + (e & 1);
              const bool see = key >= lo[mb][e >> 1] && key < hi[mb][e >> 1];
              c[mb][n][e] = see ? c[mb][n][e] : neg_inf();
            }
        }
        float nm[2], ref[2];
        bool grew = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(fmaxf(c[mb][0][2 * e], c[mb][0][2 * e + 1]),
                          fmaxf(c[mb][1][2 * e], c[mb][1][2 * e + 1]));
          t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
          t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
          nm[e] = fmaxf(mx[mb][e], t * a.scale_log2);
          ref[e] = nm[e] == neg_inf() ? 0.f : nm[e];
          grew = grew || nm[e] > mx[mb][e];
        }
        if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = ex2(mx[mb][e] - ref[e]);
            sum[mb][e] *= f;
            mx[mb][e] = nm[e];
#pragma unroll
            for (int n = 0; n < ND; ++n) {
              o[mb][n][2 * e] *= f;
              o[mb][n][2 * e + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[mb][n][e] = ex2(fmaf(c[mb][n][e], a.scale_log2, -ref[e >> 1]));
            sum[mb][e >> 1] += c[mb][n][e];
          }
        pf[mb][0] = pack_bf16(c[mb][0][0], c[mb][0][1]);
        pf[mb][1] = pack_bf16(c[mb][0][2], c[mb][0][3]);
        pf[mb][2] = pack_bf16(c[mb][1][0], c[mb][1][1]);
        pf[mb][3] = pack_bf16(c[mb][1][2], c[mb][1][3]);
      }
      // A zero weight does not keep an infinite or NaN value out of the product.
      // Keys outside the unit's range are zeros in the ring; keys that some of
      // the rows see are looked through, and a chunk that holds such a value is
      // summed without the matrix unit, key by key over the rows that see it.
      if (masked && rows_differ && !chunk_finite<DP>(sv)) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int k = 0; k < kChunk; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t w2 = __shfl_sync(0xFFFFFFFFu, pf[mb][(k >> 3) * 2 + e],
                                              lr * 4 + ((k & 7) >> 1));
              const float w = (k & 1) ? bf16_hi(w2) : bf16_lo(w2);
              const int key = k0 + k;
              if (key >= lo[mb][e] && key < hi[mb][e]) {
#pragma unroll
                for (int n = 0; n < ND; ++n) {
                  const uint32_t v2 = ld_shared32(sv + tile_at<DP>(k, n) + lc * 4);
                  o[mb][n][2 * e] = fmaf(w, bf16_lo(v2), o[mb][n][2 * e]);
                  o[mb][n][2 * e + 1] = fmaf(w, bf16_hi(v2), o[mb][n][2 * e + 1]);
                }
              }
            }
        __syncwarp();
        continue;
      }
#pragma unroll
      for (int n2 = 0; n2 < ND / 2; ++n2) {
        // B of two 8-column tiles: (keys 0-7, d lo), (8-15, d lo), (0-7, d hi), (8-15, d hi)
        uint32_t vf[4];
        ldmatrix4_trans(sv + tile_at<DP>(lane & 15, n2 * 2 + (lane >> 4)), vf);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          mma16816(o[mb][2 * n2], pf[mb], vf[0], vf[1]);
          mma16816(o[mb][2 * n2 + 1], pf[mb], vf[2], vf[3]);
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // ---- join the warps ----------------------------------------------------
    __syncthreads();          // every warp is done with the ring
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mb * 16 + lr + 8 * e;
        float t = sum[mb][e];
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 1);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 2);
        if (lc == 0) s_ml[warp][r] = make_float2(mx[mb][e], t);
#pragma unroll
        for (int n = 0; n < ND; ++n)
          *reinterpret_cast<float2*>(merge + (warp * TM + r) * DP + n * 8 + lc * 2) =
              make_float2(o[mb][n][2 * e], o[mb][n][2 * e + 1]);
      }
    __syncthreads();
    const bool whole = wk.whole();
    const int64_t pslot = (int64_t)blockIdx.x * 2 + wk.slot();
    for (int i = tid; i < nrows * (DP / 4); i += kRowsThreads) {
      const int r = i / (DP / 4), c4 = i - r * (DP / 4);
      float m = neg_inf();
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) m = fmaxf(m, s_ml[w][r].x);
      const float ref = m == neg_inf() ? 0.f : m;
      float l = 0.f;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float f = ex2(s_ml[w][r].x - ref);
        const float4 v = *reinterpret_cast<const float4*>(merge + (w * TM + r) * DP + c4 * 4);
        l += f * s_ml[w][r].y;
        t.x += f * v.x; t.y += f * v.y; t.z += f * v.z; t.w += f * v.w;
      }
      if (whole) {
        const int tok = div_group(a, r0 + r), head = h * a.G + (r0 + r) - tok * a.G;
        const RowEnd e = row_end(m, l, a.sinks, head);
        if (c4 * 4 < a.D) {
          uint2 w2 = make_uint2(pack_bf16(t.x * e.factor, t.y * e.factor),
                                pack_bf16(t.z * e.factor, t.w * e.factor));
          *reinterpret_cast<uint2*>(a.out + (int64_t)(s.q0 + tok) * a.out_stride +
                                    (int64_t)head * a.D + c4 * 4) = w2;
        }
        if (a.lse && c4 == 0) a.lse[(int64_t)(s.q0 + tok) * a.Hq + head] = e.lse;
      } else {
        *reinterpret_cast<float4*>(a.part_o + (pslot * TM + r) * DP + c4 * 4) = t;
        if (c4 == 0) a.part_ml[pslot * TM + r] = make_float2(m, l);
      }
    }
    if (tid == 0) unit_next<TM, TN>(a, un);
    __syncthreads();          // the merge buffer is the ring again
  }
}

// ------------------------------------------------------------------ host --
template <int DP, int MB>
static int rows_ctas() {
  // CTAs an SM holds by shared memory (227 KiB, 1 KiB reserved a CTA)
  constexpr int per = (227 * 1024) / (RowsGeo<DP, MB>::smem + 2048);
  return num_sms() * (per < 4 ? per : 4);
}

template <int DP, int MB>
static cudaError_t launch_rows(AttnArgs a, void* ws, cudaStream_t s) {
  using G = RowsGeo<DP, MB>;
  auto kern = attn_rows_kernel<DP, MB>;
  static SmemOnce once;
  cudaError_t e = once.set((const void*)kern, G::smem);
  if (e != cudaSuccess) return e;
  const int n = rows_ctas<DP, MB>();
  a.part_ml = static_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(a.part_ml + (size_t)2 * n * G::TM);
  timer_before(MOE_KERNEL_ATTN, s);
  e = launch_pdl(true, kern, dim3(n), dim3(kRowsThreads), G::smem, s, a);
  timer_after(MOE_KERNEL_ATTN, s);
  if (e != cudaSuccess) return e;
  timer_before(MOE_KERNEL_ATTN_COMBINE, s);
  e = launch_pdl(true, attn_join_kernel<G::TM, kRowsTN, DP>, dim3(n - 1), dim3(kJoinThreads), 0, s,
                 a, n);
  timer_after(MOE_KERNEL_ATTN_COMBINE, s);
  note_launches(2);
  return e;
}

template <int DP, int MB>
static size_t rows_ws() {
  return (size_t)2 * rows_ctas<DP, MB>() * RowsGeo<DP, MB>::TM * (DP + 2) * sizeof(float);
}

size_t attn_ws_bytes(int D) {
  const size_t a = D <= 64 ? rows_ws<64, 1>() : rows_ws<128, 1>();
  const size_t b = D <= 64 ? rows_ws<64, 2>() : rows_ws<128, 2>();
  const size_t t = attn_chunk_ws_bytes(D);
  const size_t ab = a > b ? a : b;
  return t > ab ? t : ab;
}

cudaError_t launch_attn(const moe_kv_cache& c, const moe_kv_batch& b, const moe_bf16* q,
                        int64_t q_stride, int Hq, float scale, int causal, int window,
                        const float* sinks, moe_bf16* out, int64_t out_stride, float* lse,
                        void* ws, int* status, cudaStream_t s) {
  AttnArgs a = {};
  a.bt = attn_batch(c, b);
  a.k = c.k; a.v = c.v; a.head_stride = c.head_stride;
  a.q = q; a.q_stride = q_stride; a.out = out; a.out_stride = out_stride;
  a.sinks = sinks; a.lse = lse;
  a.Hq = Hq; a.Hkv = c.Hkv; a.G = Hq / c.Hkv; a.D = c.D;
  a.g_recip = recip_of(a.G);
  a.scale_log2 = scale * kLog2e;
  a.causal = causal ? 1 : 0;
  // a window of the whole cache or more masks nothing
  a.window = window >= b.max_pages * c.page_size ? 0 : window;
  a.status = status;
  const int64_t rows = (int64_t)b.max_q * a.G;
  if (rows > 32 && attn_chunk_takes(c.page_size)) return launch_attn_chunk(a, c, ws, s);
  const bool small = rows <= 16;
  if (c.D <= 64) return small ? launch_rows<64, 1>(a, ws, s) : launch_rows<64, 2>(a, ws, s);
  return small ? launch_rows<128, 1>(a, ws, s) : launch_rows<128, 2>(a, ws, s);
}

}  // namespace moe
