// attn_rows.cu — attention over the paged cache for few rows per key/value
// head (decode, draft verification), and the choice between the two kernels.
//
// out = sum_j p_j v_j / sum_j p_j with p_j = exp(s_j - ref): one pass over the
// keys with a running reference and sum. With R rows over the keys the work is
// 4 R D operations for 4 D bytes of a key and value, so up to a few dozen rows
// the bound is reading the cache once. Hence: warps that never wait for each
// other, each with its own keys (a quarter of a tile), its own ring of
// asynchronous copies (24 KiB in flight a warp, two CTAs of four an SM), its own
// references, sums and accumulator, joined through shared memory once per unit.
// The products run on mma.sync (m16n8k16): its rate is far above what the copies
// feed, and it takes 16 rows where tcgen05 takes 128.
//
// A warp's step is 8 KiB of keys and values; what it costs beside the copies is
// instructions, so a row's reference is held (the maximum of its first step)
// until a score exceeds it by more than 16 in powers of two: no shuffles and no
// rescaling in the usual step; and pages of a multiple of 16 keys come by TMA, a
// box of keys an instruction of one lane, others by 16-byte copies with an
// address a key (444 instead of some 230 instructions a step).
//
// Measured with the join, L2 flushed before each run: four sequences of 65k to
// 131k keys, 32 heads to 4, D = 128, 168 us = 5.0 TB/s (145 us, 5.7 TB/s, a graph
// replayed back to back; a plain copy runs at 6.8); 64 sequences of 17 to 16k keys,
// 64 heads to 8, D = 64, 85 us = 3.8 TB/s (69 likewise). The steady state reads at 90 to 95%
// of the copy's rate; the rest is some 15 us of beginning and end: two launches,
// the schedule (3 us), the first keys (until 5 to 8 us), the parts' join. Loading
// the next unit's first keys while a unit's parts are joined changed nothing.
#include "attn.cuh"
#include "attn_join.cuh"
#include "common.cuh"
#include "internal.h"
#include "tmap.h"

#include <algorithm>

namespace moe {

constexpr float kRowsRescaleAt = 16.f;
// Keys whose sums a warp's accumulator takes (unit_next): four times as many of a
// unit's where four warps share it.
constexpr int kRowsPiece = 65536;

constexpr int kRowsThreads = 128;

// W: warps that work on a unit, 4 or 1; a block has 4 / W such groups.
template <int DP, int MB, int W>
struct RowsGeo {
  static constexpr int groups = 4 / W;
  static constexpr int TM = 16 * MB;
  static constexpr int chunk = DP == 128 ? 16 : 32;              // keys of a warp's step
  static constexpr int TN = chunk * W;
  static constexpr int row_bytes = DP * 2;
  static constexpr int stage = 2 * chunk * row_bytes;            // K and V: 8 KiB
  static constexpr int stages = 3;
  static constexpr int ring = 4 * stages * stage;
  static constexpr int q_bytes = TM * row_bytes;
  static constexpr int smem = ring + groups * q_bytes;
  static_assert(TM * DP * 4 <= stages * stage, "a warp's part is joined through its ring");
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
// Byte offset of 16-byte piece c of row r of a tile of ROWS rows: 64-element
// column blocks, each in the 128-byte swizzle TMA writes (the pieces of 8 rows
// permuted, so that ldmatrix reads 8 rows of one piece without conflicts).
template <int ROWS>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)((c >> 3) * (ROWS * 128) + r * 128 + (((c ^ r) & 7) << 4));
}

__device__ __forceinline__ uint32_t ld_shared32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// No infinity or NaN among the chunk's values (by the whole warp).
template <int DP, int KEYS>
__device__ __noinline__ bool chunk_finite(uint32_t sv) {
  bool bad = false;
#pragma unroll 4
  for (int i = 0; i < KEYS * DP / 64; ++i) {
    const uint32_t v = ld_shared32(sv + (i * 32 + (threadIdx.x & 31)) * 4);
    bad = bad || (v & 0x7F800000u) == 0x7F800000u || (v & 0x7F80u) == 0x7F80u;
  }
  return !__any_sync(0xFFFFFFFFu, bad);
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// PAGE16: pages of a multiple of 16 keys; a step's keys come in boxes of `box`
// (16, or the whole step), each in one page. Three stages a warp: with four one
// CTA an SM is left, and the sequences above take 175 and 89 us.
template <int DP, int MB, int W, bool PAGE16>
__global__ void __launch_bounds__(kRowsThreads) attn_rows_kernel(
    const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap mapK,
    const __grid_constant__ CUtensorMap mapV, int box) {
  using G = RowsGeo<DP, MB, W>;
  constexpr int TM = G::TM, TN = G::TN, S = G::stages, KC = G::chunk, NT = 32 * W;
  constexpr int ND = DP / 8;               // 8-wide column tiles of the accumulator
  constexpr int NC = DP / 8;               // 16-byte pieces of a row
  constexpr int NK = KC / 8;               // 8-key tiles of a step's scores
  constexpr int NG = KC / 16;              // 16-key groups
  constexpr int NH = DP / 64;              // column blocks
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Place pl;
  __shared__ Unit units[G::groups][2];
  __shared__ float2 s_mls[4][TM];
  __shared__ float2 s_before[G::groups][2][TM];    // of the pieces before, by turns
  __shared__ uint64_t full[4][S];
  __shared__ int s_abort;
  const int lane = threadIdx.x & 31, bwarp = threadIdx.x >> 5;
  // within the group of warps that share a unit
  const int group = bwarp / W, warp = bwarp % W, tid = threadIdx.x % NT;
  if (PAGE16 && threadIdx.x == 0) {
    for (int i = 0; i < 4 * S; ++i) mbar_init(smem_u32(&full[0][0] + i), 1);
    s_abort = 0;
    fence_mbar_init();
  }
  pdl_enter();
  locate<TM, TN, kRowsThreads, G::groups>(a, blockIdx.x * G::groups, gridDim.x * G::groups, pl,
                                          &units[0][0], 2);
  Unit* const un = units[group];
  float2(*const s_ml)[TM] = s_mls + group * W;
  auto group_sync = [&]() {
    if (W == 4) __syncthreads();
    else __syncwarp();
  };

  const uint32_t s_ring = smem_u32(smem) + bwarp * S * G::stage;
  uint8_t* const q_mem = smem + G::ring + group * G::q_bytes;
  const uint32_t s_q = smem_u32(q_mem);
  // a warp's part of the unit: in its own ring
  constexpr int kPartFloats = S * G::stage / 4;
  float* const merge = reinterpret_cast<float*>(smem + group * W * S * G::stage);
  const int lr = lane >> 2, lc = lane & 3;      // accumulator row and column pair

  volatile int never = 0;
  int used = 0, done = 0;      // ring slots filled and worked on by this warp so far
  // Where a step's keys are: lane g, its box of keys (PAGE16), or lane r, its
  // key: page and slot; slot -1: nothing to load. The page is what the table
  // says, looked at only when it is used: a lookup waits for nothing.
  struct Spot {
    int page, slot;
  };
  auto lookup = [&](const Unit& w, int j) {
    Spot p{0, -1};
    const int span = PAGE16 ? box : 1;
    const int key = (w.t0 + j) * TN + warp * KC + lane * span;
    if (j < w.nt && lane * span < KC && key + span > w.lo && key < w.hi) {
      const int pg = page_of(a.bt, key);
      p.page = a.bt.table[(int64_t)w.b * a.bt.table_stride + pg];
      p.slot = key - pg * a.bt.page_size;
    }
    return p;
  };
  // false: nothing to load, or a page outside the cache
  auto usable = [&](const Spot& p) {
    if (p.slot < 0) return false;
    if (p.page >= 0 && p.page < a.bt.n_pages) return true;
    raise_status(a.status, MOE_ERR_DEVICE_INDEX);
    return false;
  };
  // a thread's pieces of a unit's queries (rows past the unit: zeros)
  constexpr int QP = TM * NC / NT > 0 ? TM * NC / NT : 1;
  struct Pieces {
    uint4 v[QP];
  };
  auto load_q = [&](const Unit& w) {
    Pieces q;
    const int r0 = w.m * TM, nrows = min(TM, w.s.nq * a.G - r0);
#pragma unroll
    for (int i = 0; i < QP; ++i) {
      const int at = i * NT + tid, r = at / NC, c = at - r * NC;
      q.v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nrows && c * 8 < a.D) {
        const int tok = div_group(a, r0 + r), g = (r0 + r) - tok * a.G;
        q.v[i] = *reinterpret_cast<const uint4*>(a.q + (int64_t)(w.s.q0 + tok) * a.q_stride +
                                                 (int64_t)(w.h * a.G + g) * a.D + c * 8);
      }
    }
    return q;
  };

  Spot spot[S];                // of the unit's first steps
  Pieces qp;
  auto unit_loads = [&](const Unit& w) {
#pragma unroll
    for (int j = 0; j < S; ++j) spot[j] = lookup(w, j);
    qp = load_q(w);
  };
  int cur = 0;
  if (un[0].more) unit_loads(un[0]);
  while (un[cur].more) {
    const Unit wk = un[cur];
    const Seq s = wk.s;
    const int rows = s.nq * a.G;
    const int r0 = wk.m * TM;
    const int nrows = min(TM, rows - r0);
    const int h = wk.h;
    const int ntile = wk.nt;
    const int64_t head_at = (int64_t)h * a.head_stride;

    // step j of this warp: keys [first_key(j), + KC)
    auto first_key = [&](int j) { return (wk.t0 + j) * TN + warp * KC; };
    auto issue = [&](int j, Spot at) {
      if constexpr (PAGE16) {
        if (j >= ntile) return;
        const uint32_t dst = s_ring + (used % S) * G::stage;
        const uint32_t bar = smem_u32(&full[bwarp][used % S]);
        const uint32_t bytes = (uint32_t)box * 128u * (2 * NH);
        const bool some = usable(at);
        const uint32_t all = __popc(__ballot_sync(0xFFFFFFFFu, some)) * bytes;
        if (lane == 0) mbar_arrive_expect_tx(bar, all);
        __syncwarp();
        if (some) {
#pragma unroll
          for (int c = 0; c < NH; ++c) {
            const uint32_t d = dst + c * (KC * 128) + lane * box * 128;
            tma_load_4d(d, &mapK, bar, c * 64, at.slot, h, at.page);
            tma_load_4d(d + KC * G::row_bytes, &mapV, bar, c * 64, at.slot, h, at.page);
          }
        }
        ++used;
      } else {
        if (j < ntile) {
          constexpr int kRowsPer = 32 / NC;           // rows covered by one warp-wide copy
          const uint32_t dst = s_ring + (used % S) * G::stage;
          const int pc = lane % NC, pr = lane / NC;
          const int64_t mine = (int64_t)at.page * a.bt.page_stride +
                               (int64_t)at.slot * a.bt.token_stride;
          const int64_t off = usable(at) ? mine : -1;
#pragma unroll
          for (int i = 0; i < KC / kRowsPer; ++i) {
            const int r = i * kRowsPer + pr;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
            const bool in = o >= 0 && pc * 8 < a.D;
            const int64_t e = in ? o + head_at + pc * 8 : 0;
            cp_async16(dst + tile_at<KC>(r, pc), a.k + e, in);
            cp_async16(dst + KC * G::row_bytes + tile_at<KC>(r, pc), a.v + e, in);
          }
          ++used;
        }
        cp_async_commit();
      }
    };
#pragma unroll
    for (int j = 0; j < S - 1; ++j) issue(j, spot[j]);
    Spot ahead = spot[S - 1];           // the next step's, looked up a step early
#pragma unroll
    for (int i = 0; i < QP; ++i) {
      const int at = i * NT + tid, r = at / NC, c = at - r * NC;
      *reinterpret_cast<uint4*>(q_mem + tile_at<TM>(r, c)) = qp.v[i];
    }
    // the next unit, found by a thread whose warp's first copies are on their way
    if (tid == NT - 32) {
      un[cur ^ 1] = wk;
      unit_next<TM, TN>(a, un[cur ^ 1]);
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
    const bool rows_differ = wk.all_lo > wk.lo || wk.all_hi < wk.hi;

    float o[MB][ND][4];
    float mx[MB][2], sum[MB][2];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
      for (int n = 0; n < ND; ++n) o[mb][n][0] = o[mb][n][1] = o[mb][n][2] = o[mb][n][3] = 0.f;
      mx[mb][0] = mx[mb][1] = neg_inf();
      sum[mb][0] = sum[mb][1] = 0.f;
    }
    group_sync();         // the queries are in shared memory

    uint32_t qf[MB == 1 ? DP / 16 : 1][4];
    if constexpr (MB == 1) {
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
        ldmatrix4(s_q + tile_at<TM>(lane & 15, kk * 2 + (lane >> 4)), qf[kk]);
    }

#pragma unroll 1
    for (int j = 0; j < ntile; ++j) {
      issue(j + S - 1, ahead);
      ahead = lookup(wk, j + S);
      const uint32_t sk = s_ring + (done % S) * G::stage;
      const uint32_t sv = sk + KC * G::row_bytes;
      const int k0 = first_key(j);
      if constexpr (PAGE16) {
        const bool ok = mbar_wait_bounded(smem_u32(&full[bwarp][done % S]), (done / S) & 1,
                                          &s_abort, a.status);
        __syncwarp();
        if (!__all_sync(0xFFFFFFFFu, ok)) break;      // given up: reported, results void
        // values of keys out of range are what the cache or an older step left:
        // zeros, so that their zero weights give zeros
        if (k0 < wk.lo || k0 + KC > wk.hi) {
          for (int i = lane; i < KC * NC; i += 32) {
            const int key = k0 + i / NC;
            if (key < wk.lo || key >= wk.hi)
              st_shared_zero16(sv + tile_at<KC>(i / NC, i % NC));
          }
          fence_async_smem();
          __syncwarp();
        }
      } else {
        cp_async_wait<S - 1>();
        __syncwarp();
      }
      ++done;
      float c[MB][NK][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int n = 0; n < NK; ++n) c[mb][n][0] = c[mb][n][1] = c[mb][n][2] = c[mb][n][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        uint32_t q4[MB][4];
        if constexpr (MB > 1) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            ldmatrix4(s_q + tile_at<TM>(mb * 16 + (lane & 15), kk * 2 + (lane >> 4)), q4[mb]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          // B of two 8-key tiles: (keys 0-7, d lo), (0-7, d hi), (8-15, d lo), (8-15, d hi)
          uint32_t kf[4];
          ldmatrix4(sk + tile_at<KC>(g * 16 + (lane & 7) + ((lane >> 4) << 3),
                                     kk * 2 + ((lane >> 3) & 1)),
                    kf);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            const uint32_t* qa = MB == 1 ? qf[kk] : q4[mb];
            mma16816(c[mb][2 * g], qa, kf[0], kf[1]);
            mma16816(c[mb][2 * g + 1], qa, kf[2], kf[3]);
          }
        }
      }
      const bool masked = k0 < wk.all_lo || k0 + KC > wk.all_hi;
      uint32_t pf[MB][NG][4];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        if (masked) {
          // masked by selection: a masked score's value, NaN or not, is dropped
#pragma unroll
          for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = k0 + n * 8 + lc * 2 + (e & 1);
              const bool see = key >= lo[mb][e >> 1] && key < hi[mb][e >> 1];
              c[mb][n][e] = see ? c[mb][n][e] : neg_inf();
            }
        }
        float top[2];
        bool grew = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = fmaxf(c[mb][0][2 * e], c[mb][0][2 * e + 1]);
#pragma unroll
          for (int n = 1; n < NK; ++n)
            top[e] = fmaxf(top[e], fmaxf(c[mb][n][2 * e], c[mb][n][2 * e + 1]));
          grew = grew || top[e] * a.scale_log2 > mx[mb][e] + kRowsRescaleAt;
        }
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, grew), 0)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = top[e];
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2)) * a.scale_log2;
            const float nm = t > mx[mb][e] + kRowsRescaleAt ? t : mx[mb][e];
            const float f = nm == neg_inf() ? 1.f : ex2(mx[mb][e] - nm);
            mx[mb][e] = nm;
            sum[mb][e] *= f;
#pragma unroll
            for (int n = 0; n < ND; ++n) {
              o[mb][n][2 * e] *= f;
              o[mb][n][2 * e + 1] *= f;
            }
          }
        }
        const float ref[2] = {mx[mb][0] == neg_inf() ? 0.f : mx[mb][0],
                              mx[mb][1] == neg_inf() ? 0.f : mx[mb][1]};
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[mb][n][e] = ex2(fmaf(c[mb][n][e], a.scale_log2, -ref[e >> 1]));
            sum[mb][e >> 1] += c[mb][n][e];
          }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          pf[mb][g][0] = pack_bf16(c[mb][2 * g][0], c[mb][2 * g][1]);
          pf[mb][g][1] = pack_bf16(c[mb][2 * g][2], c[mb][2 * g][3]);
          pf[mb][g][2] = pack_bf16(c[mb][2 * g + 1][0], c[mb][2 * g + 1][1]);
          pf[mb][g][3] = pack_bf16(c[mb][2 * g + 1][2], c[mb][2 * g + 1][3]);
        }
      }
      // A zero weight does not keep an infinite or NaN value out of the product.
      // Keys outside the unit's range are zeros in the ring; keys that some of
      // the rows see are looked through, and a step that holds such a value is
      // summed without the matrix unit, key by key over the rows that see it.
      if (__builtin_expect(masked && rows_differ, 0) && !chunk_finite<DP, KC>(sv)) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              // the weight of (row, key) is with lane lc = key % 8 / 2 of the row
              const int src = lr * 4 + ((k & 7) >> 1);
              const uint32_t w4[2][2] = {{pf[mb][g][0], pf[mb][g][1]},
                                         {pf[mb][g][2], pf[mb][g][3]}};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t w2 = __shfl_sync(0xFFFFFFFFu, k < 8 ? w4[0][e] : w4[1][e], src);
                const float w = (k & 1) ? bf16_hi(w2) : bf16_lo(w2);
                const int key = k0 + g * 16 + k;
                const bool see = key >= lo[mb][e] && key < hi[mb][e];
#pragma unroll
                for (int n = 0; n < ND; ++n) {
                  const uint32_t v2 = ld_shared32(sv + tile_at<KC>(g * 16 + k, n) + lc * 4);
                  const float x = fmaf(w, bf16_lo(v2), o[mb][n][2 * e]);
                  const float y = fmaf(w, bf16_hi(v2), o[mb][n][2 * e + 1]);
                  o[mb][n][2 * e] = see ? x : o[mb][n][2 * e];
                  o[mb][n][2 * e + 1] = see ? y : o[mb][n][2 * e + 1];
                }
              }
            }
        __syncwarp();
        continue;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int n2 = 0; n2 < ND / 2; ++n2) {
          // B of two 8-column tiles: (keys 0-7, d lo), (8-15, d lo), (0-7, d hi), (8-15, d hi)
          uint32_t vf[4];
          ldmatrix4_trans(sv + tile_at<KC>(g * 16 + (lane & 15), n2 * 2 + (lane >> 4)), vf);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            mma16816(o[mb][2 * n2], pf[mb][g], vf[0], vf[1]);
            mma16816(o[mb][2 * n2 + 1], pf[mb][g], vf[2], vf[3]);
          }
        }
      __syncwarp();
    }
    if constexpr (PAGE16) {
      // after giving up: copies in flight land before the ring is used again
      for (; done < used; ++done)
        mbar_wait_bounded(smem_u32(&full[bwarp][done % S]), (done / S) & 1, &never, a.status);
      __syncwarp();
    } else {
      cp_async_wait<0>();
    }

    // ---- join the warps ----------------------------------------------------
    group_sync();          // every warp is done with the ring, the next unit is known
    cur ^= 1;
    if (un[cur].more) unit_loads(un[cur]);
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
          *reinterpret_cast<float2*>(merge + warp * kPartFloats + r * DP + n * 8 + lc * 2) =
              make_float2(o[mb][n][2 * e], o[mb][n][2 * e + 1]);
      }
    group_sync();
    // One row block: the unit is read once more, for registers that would be live
    // through the loop (32 single tokens, D = 128, 47.7 instead of 48.8 us; with two
    // it is the other way round, 32 drafts of 24 rows 58.9 instead of 56.0 us).
    const Unit& past = MB == 1 ? un[cur ^ 1] : wk;
    const bool whole = past.whole() && past.rest == 0;
    const int64_t pslot = ((int64_t)blockIdx.x * G::groups + group) * 2 + past.slot();
    for (int i = tid; i < nrows * (DP / 4); i += NT) {
      const int r = i / (DP / 4), c4 = i - r * (DP / 4);
      float m = neg_inf();
#pragma unroll
      for (int w = 0; w < W; ++w) m = fmaxf(m, s_ml[w][r].x);
      const float ref = m == neg_inf() ? 0.f : m;
      float l = 0.f;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = ex2(s_ml[w][r].x - ref);
        const float4 v =
            *reinterpret_cast<const float4*>(merge + w * kPartFloats + r * DP + c4 * 4);
        l += f * s_ml[w][r].y;
        t.x += f * v.x; t.y += f * v.y; t.z += f * v.z; t.w += f * v.w;
      }
      float4* const part = reinterpret_cast<float4*>(a.part_o + part_at<TM, DP>(pslot, r, c4));
      if (__builtin_expect(past.begun, 0)) {
        Part p{m, l, t};
        const float2 before = s_before[group][cur][r];
        join_part(p, before.x, before.y, *part);
        m = p.m;
        l = p.l;
        t = p.o;
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
        *part = t;
        if (c4 == 0)
          (past.rest > 0 ? s_before[group][cur ^ 1][r] : a.part_ml[pslot * TM + r]) =
              make_float2(m, l);
      }
    }
    if constexpr (PAGE16) fence_async_smem();
    group_sync();          // the merge buffer is the ring again
  }
}

// ------------------------------------------------------------------ host --
// Up to so many rows (tokens x query heads of a key head) a sequence is worked on
// by the kernel above, in one row tile of 16 or 32; more go to the chunk kernel
// where its pages allow. 64 sequences of 1000 to 3000 keys, 8 heads to a key head,
// D = 64 and 128, the kernel above and the chunk kernel: 16 rows 42 / 48 and 67 /
// 77 us, 32 rows 46 / 50 and 72 / 77 us, 40 rows 75 / 50 and 110 / 77 us.
constexpr int kFewRows = 32;
// The chunk kernel is for as much work as this, in rows x keys (what the page table
// or the window allows; where a table is far wider than the sequences need, so are
// short chunks the other kernel's) x 64 or 128: below, its beginning and its join cost
// more than the rows kernel takes, whose units are then few and short. Pages of 16, the
// kernel above and the chunk kernel, D = 64 and 128: 200 tokens over 200 keys, 8
// heads to a key head, 18 / 30 and 22 / 34 us; 300 over 900, 4 heads, 24 / 33 and
// 34 / 40; 8 x 9 over 1000 27 / 28 and 32 / 32; 16 x 9 over 1000 30 / 30 and 44 /
// 32; 200 over 2500 40 / 33 and 56 / 40.
constexpr int64_t kChunkWork = (int64_t)1 << 28;
// And for pages that TMA cannot take (no multiple of 8), where the loads are its
// bound. Pages of 13, likewise: 100 tokens over 2500 keys 30 / 46 and 44 / 62 us,
// 200 tokens 40 / 46 and 60 / 63, 400 tokens 60 / 52 and 95 / 73, 8 x 200 over 2000
// 155 / 111 and 263 / 165, 2048 over 4096 272 / 177 and 484 / 268.
constexpr int64_t kGatherWork = (int64_t)1 << 30;
// Steps a unit costs beside its tiles (1 makes the 64 sequences above 89 instead
// of 83 us, 4 changes nothing there and makes 31 tokens of D = 80 32 instead of
// 30 us), and the least steps of a stretch (between 3 and 8 no difference).
constexpr int kRowsCost = 2, kRowsLeast = 4;
// Units of at most so many tiles (512 keys at D = 128, 1024 at D = 64) are not
// cut: the second launch costs more than an even load is worth. One token over 4
// key heads, D = 128, uncut / cut: 512 keys 18 / 20 us, 1024 keys 26 / 20 us; 16
// sequences of 512 keys 20 / 22, of 1024 28 / 26; 128 of 1024 69 / 71.
constexpr int kWholeTiles = 8;
// Uncut units of at most so many keys are a warp's, not a block's, from four units
// an SM on (an SM holds eight warps): nothing to join and no one to wait for. At D =
// 64, 8 key heads, a warp's / a block's: 80 sequences of 144 keys 22 / 24 us, 128 26 /
// 28, 176 34 / 34, 320 47 / 52; of 176 keys 23 / 24, 27 / 29, 38 / 35 and 52 / 53; of
// 240 keys 24 / 25, 30 / 31, 43 / 38 and 61 / 55; 64 sequences of 112 keys 20 / 18. At
// D = 128, with 16 keys a step, a block's is never slower (320 x 256 keys 82 / 75 us).
constexpr int kWarpKeys = 192;

template <int DP, int MB, int W>
static int rows_ctas() {
  // CTAs an SM holds by shared memory (227 KiB, 1 KiB reserved a CTA)
  constexpr int per = (227 * 1024) / (RowsGeo<DP, MB, W>::smem + 2048);
  return num_sms() * (per < 4 ? per : 4);
}

template <int DP, int MB, int W, bool PAGE16>
static cudaError_t launch_rows(AttnArgs a, const moe_kv_cache& c, void* ws, cudaStream_t s) {
  using G = RowsGeo<DP, MB, W>;
  auto kern = attn_rows_kernel<DP, MB, W, PAGE16>;
  static SmemOnce once;
  cudaError_t e = once.set((const void*)kern, G::smem);
  if (e != cudaSuccess) return e;
  CUtensorMap mk = {}, mv = {};
  const int box = c.page_size % G::chunk == 0 ? G::chunk : 16;
  if (PAGE16 && (!map_kv(&mk, c.k, c, box) || !map_kv(&mv, c.v, c, box)))
    return cudaErrorInvalidValue;
  const int n = rows_ctas<DP, MB, W>();
  if (!a.whole) a.cuts = static_cast<Cut*>(ws);
  a.part_ml = reinterpret_cast<float2*>(static_cast<Cut*>(ws) + n);
  a.part_o = reinterpret_cast<float*>(a.part_ml + (size_t)2 * n * G::groups * G::TM);
  a.piece = kRowsPiece / G::chunk;
  timer_before(MOE_KERNEL_ATTN, s);
  e = launch_pdl(true, kern, dim3(n), dim3(kRowsThreads), G::smem, s, a, mk, mv, box);
  timer_after(MOE_KERNEL_ATTN, s);
  note_launches(1);
  if (e != cudaSuccess || a.whole) return e;
  timer_before(MOE_KERNEL_ATTN_COMBINE, s);
  e = launch_pdl(true, attn_join_kernel<G::TM, DP>, dim3(n - 1, 4), dim3(kJoinThreads), 0, s, a);
  timer_after(MOE_KERNEL_ATTN_COMBINE, s);
  note_launches(1);
  return e;
}

template <int DP, int MB>
static cudaError_t launch_rows(AttnArgs a, const moe_kv_cache& c, int64_t keys, void* ws,
                               cudaStream_t s) {
  a.whole = keys <= kWholeTiles * RowsGeo<DP, MB, 4>::TN ? 1 : 0;
  a.least = a.whole ? 1 : kRowsLeast;
  if constexpr (DP == 64 && MB == 1) {
    if (a.whole && keys <= kWarpKeys && c.page_size % 16 == 0 &&
        (int64_t)a.bt.B * a.Hkv >= 4 * num_sms())
      return launch_rows<DP, MB, 1, true>(a, c, ws, s);
  }
  return c.page_size % 16 == 0 ? launch_rows<DP, MB, 4, true>(a, c, ws, s)
                               : launch_rows<DP, MB, 4, false>(a, c, ws, s);
}

template <int DP, int MB, int W>
static size_t rows_ws() {
  using G = RowsGeo<DP, MB, W>;
  return (size_t)rows_ctas<DP, MB, W>() *
         (sizeof(Cut) + 2 * G::groups * G::TM * (DP + 2) * sizeof(float));
}

size_t attn_ws_bytes(int D) {
  const size_t t = attn_chunk_ws_bytes(D);
  if (D > 64) return std::max({rows_ws<128, 1, 4>(), rows_ws<128, 2, 4>(), t});
  return std::max({rows_ws<64, 1, 4>(), rows_ws<64, 2, 4>(), rows_ws<64, 1, 1>(), t});
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
  const int64_t cap = (int64_t)b.max_pages * c.page_size;
  a.window = window >= cap ? 0 : window;
  a.status = status;
  a.rows_over = 0;
  a.rows_upto = 1 << 30;
  const int64_t rows = (int64_t)b.max_q * a.G;
  const int64_t seen = (int64_t)a.window + b.max_q;
  const int64_t keys = a.window && seen < cap ? seen : cap;      // of a sequence's tokens
  const int64_t least_work = attn_chunk_boxes(c.page_size) ? kChunkWork : kGatherWork;
  const bool chunks =
      rows > kFewRows && (int64_t)b.T * Hq * keys >= least_work / (c.D <= 64 ? 64 : 128);
  // Both kernels where sequences may be of both kinds: not when all have max_q
  // tokens, nor when one is all there is.
  const bool both = chunks && b.B > 1 && b.T != (int64_t)b.B * b.max_q;
  // Single tokens are most of such a batch, and tiles of 16 rows serve them best:
  // split at 16 rows / at 32, 110 tokens of 7 heads a key head and 424 of one
  // sequence, D = 112, 138 / 148 us; 31 of 5 and 777, D = 80, 77 / 82 us.
  const int few = both && a.G <= 16 ? 16 : kFewRows;
  cudaError_t e = cudaSuccess;
  if (!chunks || both) {
    AttnArgs r = a;
    if (both) r.rows_upto = few;
    r.cost = kRowsCost;
    const bool one = (both ? few : rows) <= 16;          // a tile of 16 rows, else of 32
    if (c.D <= 64)
      e = one ? launch_rows<64, 1>(r, c, keys, ws, s) : launch_rows<64, 2>(r, c, keys, ws, s);
    else
      e = one ? launch_rows<128, 1>(r, c, keys, ws, s) : launch_rows<128, 2>(r, c, keys, ws, s);
  }
  if (e == cudaSuccess && chunks) {
    if (both) a.rows_over = few;
    // Steps a unit costs beside its tiles. Up to 128 rows tiles take as long as
    // reading them does, beyond a unit's beginning and end are four tiles' work:
    // drafts of 40 rows over 24-key pages 75 us at a cost of 1, 79 at 2, 89 at 4;
    // 4 x 4096 tokens at D = 64 654 at 4, 686 at 2; 16 prompts of 100 to 3000
    // tokens at D = 128 255 at 4, 278 at 2, 325 at 1.
    a.cost = rows <= 128 ? 1 : 4;
    e = launch_attn_chunk(a, c, ws, s);
  }
  return e;
}

}  // namespace moe
