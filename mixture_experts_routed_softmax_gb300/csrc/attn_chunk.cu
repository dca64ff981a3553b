// attn_chunk.cu — attention over the paged cache for many rows per key/value
// head (prompt chunks, prefill) on the 5th-generation tensor cores.
//
// A unit is 256 rows (two halves of 128) of one sequence and key/value head
// against its key range, in tiles of 128 keys. Per tile and half:
//   S = Q K^T      tcgen05.mma, both operands in shared memory, S in tensor memory
//   P = exp2(S * scale - max), rounded to bf16 over S's own columns (the product
//                  takes both operands in one type, V's)
//   O += P V       tcgen05.mma with P read from tensor memory
// One pass with a running reference for the exponent: a row's is the maximum of
// the first 64 keys it sees, and is only moved (O, the sum and the tile's stored
// weights rescaled) when the weights of 64 keys sum to more than 2^16: nothing
// looks for a maximum in the usual step. Weights of up to 2^16 cost no precision,
// in bf16 or in the fp32 sums, and the accumulator is next to never touched
// between products.
//
// The tensor cores and the exponentials are the two resources of like cost
// (for D = 128 four 128x128x128 products and 32 Ki exponentials a tile), so
// the halves alternate: while one half's scores are exponentiated, the other
// half's products run. Measured, L2 flushed before each run:
//   (a) 2048 tokens over 31k keys, 32 heads to 4, D = 128: 611 us, 1646 TFLOP/s,
//       85% of what a large plain product reaches; the tensor pipe is the bound;
//   (b) 4 x 4096 tokens from scratch, 64 heads to 8, D = 64: 620 us, 890 TFLOP/s,
//       46%: as many exponentials as (a) for half the products. The softmax
//       warps are the bound (some five instructions a score, every second issue
//       slot taken, the exponential unit busy 39% and the tensor pipe 37% of the
//       time).
// Choices below name their times for (a) and (b). A maximum of every score and
// the reference moved by that: 634 and 627.
//   warp 0           issues the products; owns tensor memory
//   warp 1           loads K and V tiles by TMA through a ring, one box per
//                    stretch of keys that neither a page nor a tile cuts, or by
//                    16-byte copies where that is fewer than 8 keys (then the
//                    bound: 268 instead of 108 us for 2048 tokens over 4096 keys
//                    in pages of 13, D = 128; boxes of 8 keys, pages of 24: 160,
//                    by copies 267); walks the CTA's units and hands them on
//   warp 2           the queries of a half, as soon as the unit before has had
//                    its last scores; the values of tiles that some row sees in
//                    part: out-of-range rows become zeros, and infinities and
//                    NaN are looked for
//   warp 3           D <= 64: issues S = Q K^T, warp 0 only O += P V. There an
//                    item's products take 512 cycles, less than one warp takes
//                    to issue both beside busy softmax warps on its scheduler.
//                    D > 64: nothing
//   warps 4-7, 8-11  softmax of half 0 and 1: one row per thread (the row's
//                    maximum and sum need no shuffles), the accumulator's
//                    rescale, the epilogue. (Two threads a row, 64 keys each, and
//                    so four softmax warps a scheduler: 692 and 881 when
//                    one thread a row took 634 and 675.)
#include "attn.cuh"
#include "attn_join.cuh"
#include "common.cuh"
#include "internal.h"
#include "tmap.h"

#include <type_traits>

namespace moe {

constexpr int kChunkTM = 256;
constexpr int kChunkTN = 128;
constexpr int kChunkThreads = 384;
constexpr int kMmaWarp = 0, kLoadWarp = 1, kHelpWarp = 2, kScoreWarp = 3;
constexpr float kMoveAt = 65536.f;
// Tiles whose sums one accumulator takes (unit_next): 65536 keys. Another piece
// costs what a unit's end and beginning do, some four tiles' work.
constexpr int kChunkPiece = 512;
// The least steps of a stretch: a cut costs a part's round trip. 128 tokens over
// 2500 keys, D = 128: 5 or 6 steps 42 us, 8 46 us, 12 50 us.
constexpr int kChunkLeast = 6;

template <int DP>
struct ChunkGeo {
  static constexpr int halves = DP / 64;                 // 128-byte column blocks of a row
  static constexpr int tile = kChunkTN * DP * 2;         // one K or V tile
  static constexpr int q_half = 128 * DP * 2;
  static constexpr int slots = DP == 128 ? 5 : 8;        // K and V tiles alternate
  static constexpr int smem = 2 * q_half + slots * tile + 1024;
  // Tensor memory, 512 columns: O of the two halves, and scores (the weights in
  // their place) of as many items as are left: 2 for D = 128, 3 for 64, where
  // a half's next scores so wait for it while it works on the present ones.
  static constexpr int bufs = (512 - 2 * DP) / 128;
  static constexpr uint32_t o_col0 = bufs * 128;
  // With a buffer to spare the scores need not follow the product that frees
  // theirs in one warp's order of issue: a second warp waits for its end.
  static constexpr bool split = bufs == 3;
};

// The product-issuing warp runs as one: every value an instruction takes is the
// same in all lanes (uniform registers), and one elected lane issues. A single
// lane running ahead alone costs about 90 cycles an instruction in moves to
// uniform registers, more than the 32 to 64 the product itself takes.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e != 0;
}
// A descriptor from its two halves: only the address in the low one varies.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  return ((uint64_t)hi << 32) | lo;
}
// O[tmem] (+)= P[tmem] * V[smem]
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A bounded wait whose loop is out of line: the roles' steady state has to stay
// small, or the SM spends its time fetching instructions (measured: with every
// path inline 2.5 of 7.5 cycles between a warp's instructions were fetches).
__device__ __noinline__ bool wait_slowly(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int* status) {
  return mbar_wait_bounded(bar, parity, abort_flag, status);
}
// For a whole warp: true in all lanes, or (given up) false in all. CALL: the loop
// by a call (the softmax warps, whose registers a call would need, keep it here).
template <bool CALL>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  if (__builtin_expect(__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)), 1)) return true;
  return __all_sync(0xFFFFFFFFu, CALL ? wait_slowly(bar, parity, abort_flag, status)
                                      : mbar_wait_bounded(bar, parity, abort_flag, status));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]),
        "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]),
        "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tmem_st32f(uint32_t taddr, const float* r) {
  uint32_t u[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(r[i]);
  tmem_st32(taddr, u);
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
               : "=r"(r)
               : "r"(taddr)
               : "memory");
}
// (x, y) * (a, a) + (b, b)
__device__ __forceinline__ float2 fma2(float2 x, float a, float b) {
  uint64_t r, xx, aa, bb;
  asm("mov.b64 %0, {%1, %2};" : "=l"(xx) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(aa) : "f"(a));
  asm("mov.b64 %0, {%1, %1};" : "=l"(bb) : "f"(b));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(xx), "l"(aa), "l"(bb));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  uint64_t r, xx, yy;
  asm("mov.b64 %0, {%1, %2};" : "=l"(xx) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(yy) : "f"(y.x), "f"(y.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(xx), "l"(yy));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}

// nonzero: an infinity or NaN among eight bf16 values (an exponent of all ones)
__device__ __forceinline__ uint32_t not_finite8(const uint4& v) {
  constexpr uint32_t e = 0x7F807F80u;
  return __vcmpeq2(v.x & e, e) | __vcmpeq2(v.y & e, e) | __vcmpeq2(v.z & e, e) |
         __vcmpeq2(v.w & e, e);
}

// O += P V of one tile by a warp for its 32 rows (one a lane), over the keys
// [lo, hi) of the lane's row only; P from tensor memory as the product would
// read it. Rare: a tile some rows see in part that holds an infinity or NaN.
template <int DP>
__device__ __noinline__ void add_by_hand(uint32_t t_p, uint32_t t_o, const uint8_t* vt, int k0,
                                         int lo, int hi, bool add) {
#pragma unroll 1
  for (int c = 0; c < DP; c += 32) {
    float o[32];
    tmem_ld32f(t_o + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = add ? o[i] : 0.f;
#pragma unroll 1
    for (int k = 0; k < kChunkTN; k += 2) {
      uint32_t p;
      tmem_ld1(t_p + k / 2, p);
      tmem_ld_wait();
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int key = k + kk;
        const float w = kk ? bf16_hi(p) : bf16_lo(p);
        const bool see = k0 + key >= lo && k0 + key < hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int piece = ((c & 63) >> 3) + i;
          float v[8];
          unpack8(*reinterpret_cast<const uint4*>(vt + (c >> 6) * (128 * 128) + key * 128 +
                                                  ((piece ^ (key & 7)) << 4)), v);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            o[i * 8 + q] = see ? fmaf(w, v[q], o[i * 8 + q]) : o[i * 8 + q];
        }
      }
    }
    tmem_st32f(t_o + c, o);
  }
}

// The limit of waits that may last a whole unit, which is as long as the cache:
// it counts from the last tile whose loads were issued (`issued`, of the CTA), so
// it ends a wait after kWaitLimitNs in which nothing moved, not one that is long.
struct UnitLimit {
  const volatile int* issued;
  uint64_t t0;
  int at;
  __device__ __forceinline__ explicit UnitLimit(const int* issued_)
      : issued(issued_), t0(global_ns()), at(*issued) {}
  // to be asked now and then: true to give up
  __device__ __forceinline__ bool over(volatile int* abort_flag, int* status) {
    if (*abort_flag) return true;
    const int now = *issued;
    if (now != at) {
      at = now;
      t0 = global_ns();
      return false;
    }
    if (global_ns() - t0 <= (uint64_t)kWaitLimitNs) return false;
    *abort_flag = 1;
    raise_status(status, MOE_ERR_DEVICE_TIMEOUT);
    return true;
  }
};
// Waits until `need` tiles' loads have been issued.
__device__ __forceinline__ bool issued_wait_bounded(const int* issued, int need,
                                                    volatile int* abort_flag, int* status) {
  UnitLimit limit(issued);
  for (uint32_t i = 1; *limit.issued < need; ++i) {
    __nanosleep(200);
    if ((i & 15u) == 0 && limit.over(abort_flag, status)) return false;
  }
  return true;
}
// For a warp that has time: it sleeps between its looks, so that it takes no
// issue slots from the warps it shares a scheduler with.
__device__ __forceinline__ bool mbar_doze_bounded(uint32_t bar, uint32_t parity, uint32_t ns,
                                                  const int* issued, volatile int* abort_flag,
                                                  int* status) {
  UnitLimit limit(issued);
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    __nanosleep(ns);
    if ((i & 15u) == 0 && limit.over(abort_flag, status)) return false;
  }
  return true;
}
// For a unit to be handed on: the half without rows waits for the next one while
// the other half works on its own.
__device__ __noinline__ bool unit_wait_slowly(uint32_t bar, uint32_t parity, const int* issued,
                                              volatile int* abort_flag, int* status) {
  UnitLimit limit(issued);
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i)
    if ((i & 63u) == 0 && limit.over(abort_flag, status)) return false;
  return true;
}

// A K or V tile by 16-byte copies, for pages whose keys no box can take: lane i
// has the element offsets of keys i, i + 32, .. (-1: zeros). By a whole warp.
template <int DP>
__device__ __noinline__ void gather_tile(const moe_bf16* base, uint32_t dst, int D, int64_t at0,
                                         int64_t at1, int64_t at2, int64_t at3) {
  constexpr int NC = DP / 8, kRows = 32 / NC;      // pieces of a row, rows of a copy
  const int lane = threadIdx.x & 31, pc = lane % NC, pr = lane / NC;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int64_t at = i == 0 ? at0 : i == 1 ? at1 : i == 2 ? at2 : at3;
#pragma unroll 4
    for (int k = 0; k < 32; k += kRows) {
      const int r = i * 32 + k + pr;
      const int64_t o = __shfl_sync(0xFFFFFFFFu, at, k + pr);
      const bool in = o >= 0 && pc * 8 < D;
      cp_async16(dst + (pc >> 3) * (128 * 128) + r * 128 + (((pc ^ r) & 7) << 4),
                 base + (in ? o + pc * 8 : 0), in);
    }
  }
}

// One tile's row of scores as a thread sees it: keys k0 .. k0 + 127, of which
// the row sees [lo, hi). Masked by selection: a masked score's value, NaN or
// not, is dropped.
struct RowMask {
  int lo, hi;      // less k0
  __device__ __forceinline__ float operator()(float s, int c) const {
    return c >= lo && c < hi ? s : neg_inf();
  }
};
// O of the warp's rows times a factor each
template <int DP>
__device__ __forceinline__ void scale_rows(uint32_t t_o, float f) {
#pragma unroll 1
  for (int c = 0; c < DP; c += 16) {
    uint32_t o[16];
    tmem_ld16(t_o + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    tmem_st16(t_o + c, o);
  }
  tmem_st_wait();
}
// the first n columns of stored weights (bf16 pairs) times a factor each
__device__ __forceinline__ void scale_weights(uint32_t t_p, int n, float f) {
  tmem_st_wait();
#pragma unroll 1
  for (int c = 0; c < n; c += 16) {
    uint32_t w[16];
    tmem_ld16(t_p + c, w);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16(bf16_lo(w[i]) * f, bf16_hi(w[i]) * f);
    tmem_st16(t_p + c, w);
  }
}
// The sums of a row's pieces before join the row's: O, in tensor memory, and the
// (reference, sum), which are returned.
template <int DP>
__device__ __noinline__ float2 join_before(const AttnArgs& a, uint32_t t_o, int slot, int row,
                                           float m_ref, float l) {
  const int64_t pslot = (int64_t)blockIdx.x * 2 + slot;
  const float2 before = a.part_ml[pslot * kChunkTM + row];
  const float m = fmaxf(before.x, m_ref), ref = m == neg_inf() ? 0.f : m;
  const float f = ex2(m_ref - ref), g = ex2(before.x - ref);
#pragma unroll 1
  for (int c = 0; c < DP; c += 16) {
    uint32_t o[16];
    tmem_ld16(t_o + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 b = *reinterpret_cast<const float4*>(
          a.part_o + part_at<kChunkTM, DP>(pslot, row, (c + i) / 4));
      o[i] = __float_as_uint(__uint_as_float(o[i]) * f + b.x * g);
      o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) * f + b.y * g);
      o[i + 2] = __float_as_uint(__uint_as_float(o[i + 2]) * f + b.z * g);
      o[i + 3] = __float_as_uint(__uint_as_float(o[i + 3]) * f + b.w * g);
    }
    tmem_st16(t_o + c, o);
  }
  tmem_st_wait();
  return make_float2(m, l * f + before.y * g);
}
// 64 scores to weights exp2(s * scale - ref), as bf16 pairs; their unrounded sum.
__device__ __forceinline__ float group_weights(const float* x, float scale, float ref,
                                               uint32_t* pk) {
  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < 64; c += 2) {
    float2 t = fma2(make_float2(x[c], x[c + 1]), scale, -ref);
    t = make_float2(ex2(t.x), ex2(t.y));
    acc[(c >> 1) & 1] = add2(acc[(c >> 1) & 1], t);
    pk[c / 2] = pack_bf16(t.x, t.y);
  }
  const float2 s = add2(acc[0], acc[1]);
  return s.x + s.y;
}

// Tiles [0, e0) and [e1, nt) of a unit are edge tiles: some row sees them in part.
__device__ __forceinline__ void edges(const Unit& u, int& e0, int& e1) {
  // the first tile that begins at or after all_lo, the tiles that end by all_hi
  e0 = (u.all_lo + kChunkTN - 1) / kChunkTN - u.t0;
  e0 = min(max(e0, 0), u.nt);
  e1 = u.all_hi / kChunkTN - u.t0;
  e1 = min(max(e1, e0), u.nt);
}

struct ChunkShared {
  Place pl;
  Unit unit[4];         // the CTA's units, handed on by the load warp
  uint64_t unit_full[4], unit_empty[4];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t v_seen[8];   // an edge tile's values have been looked through
  uint64_t q_ready[2], q_free[2], drain[2];
  uint64_t o_done[2][2];   // of a half, its products in turn
  uint64_t buf_free[3];    // split: the product that read the buffer has ended
  uint64_t s_full[2][3];   // of a half, its items in turn (each half waits for every one of its
                           // own, so that no phase is taken for the one after the next)
  uint64_t p_ready[3];     // of a buffer
  uint32_t tmem;
  int abort;
  int issued;           // tiles whose loads have been issued
  int q_had[2];         // of a half's queries: 0 none loaded, else 2 + the last load's parity
  int never;            // 0
  int bad[8];           // per slot: an infinity or NaN among them
};

// GATHER: pages whose keys no box can take (a kernel of its own: the other's loops
// lose 4% to where this code would put them).
template <int DP, bool GATHER>
__global__ void __launch_bounds__(kChunkThreads, 1)
    attn_chunk_kernel(const __grid_constant__ AttnArgs a,
                      const __grid_constant__ CUtensorMap mapQ,
                      const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapV, int box, int q_by_tma) {
  using G = ChunkGeo<DP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ChunkShared sh;
  pdl_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t s_q = smem_u32(smem);
  const uint32_t s_kv = s_q + 2 * G::q_half;
  uint8_t* const kv_mem = smem + 2 * G::q_half;
  volatile int* abort = &sh.abort;

  if (tid == 0) {
    for (int i = 0; i < G::slots; ++i) {
      mbar_init(smem_u32(&sh.kv_full[i]), 1);
      mbar_init(smem_u32(&sh.kv_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_seen[i]), 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(&sh.q_ready[h]), 1);
      mbar_init(smem_u32(&sh.q_free[h]), 1);
      mbar_init(smem_u32(&sh.o_done[h][0]), 1);
      mbar_init(smem_u32(&sh.o_done[h][1]), 1);
      mbar_init(smem_u32(&sh.drain[h]), 1);
    }
    for (int i = 0; i < G::bufs; ++i) {
      mbar_init(smem_u32(&sh.s_full[0][i]), 1);
      mbar_init(smem_u32(&sh.s_full[1][i]), 1);
      mbar_init(smem_u32(&sh.p_ready[i]), 4);
      mbar_init(smem_u32(&sh.buf_free[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sh.unit_full[i]), 1);
      mbar_init(smem_u32(&sh.unit_empty[i]), G::split ? 11 : 10);
    }
    sh.abort = 0;
    sh.issued = 0;
    sh.never = 0;
    sh.q_had[0] = sh.q_had[1] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  locate<kChunkTM, kChunkTN, kChunkThreads>(a, blockIdx.x, gridDim.x, sh.pl, sh.unit, 1);
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // The warp's next unit is there (false: the end, or given up); it has read it.
  auto take_unit = [&](int u, bool& ok) {
    if (!ok) return false;
    const uint32_t bar = smem_u32(&sh.unit_full[u & 3]), parity = (u >> 2) & 1;
    if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)))
      ok = __all_sync(0xFFFFFFFFu,
                      unit_wait_slowly(bar, parity, &sh.issued, abort, a.status));
    return ok && sh.unit[u & 3].more != 0;
  };
  auto give_unit = [&](int u) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.unit_empty[u & 3]));
  };
  if (warp < 4) {
    if (warp == kLoadWarp) {
      // -------------------------------------------------------------- loads --
      // lane i < nbox: the box of keys [tile + i * box, + box)
      const int nbox = kChunkTN / box;
      const uint32_t box_bytes = (uint32_t)box * 128u;
      int slot = 0;
      uint32_t phase = 0;
      int fills = 0;
      bool ok = true;
      // With copies a tile is handed on when it has landed: after the next one's
      // have been issued, or before a wait.
      int landing = -1;           // the slot not handed on yet
      auto hand_on = [&]() {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.kv_full[landing]));
        landing = -1;
      };
      auto land = [&]() {
        if (landing < 0) return;
        cp_async_wait<0>();
        hand_on();
      };
      struct Keys {
        int page[4], slot[4];     // of keys lane + 32 i; slot -1: none
      };
      auto find_keys = [&](const Unit& w, int j) {
        Keys p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = (w.t0 + j) * kChunkTN + lane + 32 * i;
          p.page[i] = 0;
          p.slot[i] = -1;
          if (j < w.nt && key >= w.lo && key < w.hi) {
            const int pg = page_of(a.bt, key);
            p.page[i] = a.bt.table[(int64_t)w.b * a.bt.table_stride + pg];
            p.slot[i] = key - pg * a.bt.page_size;
          }
        }
        return p;
      };
      for (int u = 0;; ++u) {
        // the next unit (or that there is none) for every role
        Unit& un = sh.unit[u & 3];
        if constexpr (GATHER) land();
        ok = wait_warp<true>(smem_u32(&sh.unit_empty[u & 3]), ((u >> 2) & 1) ^ 1, abort,
                             a.status);
        if (!ok) break;
        if (lane == 0) {
          if (u > 0) {
            un = sh.unit[(u - 1) & 3];
            unit_next<kChunkTM, kChunkTN>(a, un);
          }
          mbar_arrive(smem_u32(&sh.unit_full[u & 3]));
        }
        __syncwarp();
        const Unit wk = un;
        if (!wk.more) break;
        const int nt = wk.nt;
        Keys keys;
        if constexpr (GATHER) keys = find_keys(wk, 0);
        for (int j = 0; j < nt && ok; ++j) {
          if constexpr (GATHER) {
            int64_t at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              at[i] = -1;
              if (keys.slot[i] >= 0) {
                if (keys.page[i] >= 0 && keys.page[i] < a.bt.n_pages)
                  at[i] = (int64_t)keys.page[i] * a.bt.page_stride +
                          (int64_t)keys.slot[i] * a.bt.token_stride + wk.h * a.head_stride;
                else
                  raise_status(a.status, MOE_ERR_DEVICE_INDEX);
              }
            }
            keys = find_keys(wk, j + 1);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t empty = smem_u32(&sh.kv_empty[slot]);
              if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(empty, phase ^ 1u))) {
                land();
                ok = mbar_doze_bounded(empty, phase ^ 1u, 100, &sh.issued, abort, a.status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
              }
              gather_tile<DP>(kv ? a.v : a.k, s_kv + slot * G::tile, a.D, at[0], at[1], at[2],
                              at[3]);
              cp_async_commit();
              if (landing >= 0) {
                cp_async_wait<1>();
                hand_on();
              }
              landing = slot;
              ++fills;
              if (kv == 1 && lane == 0) *(volatile int*)&sh.issued = fills >> 1;
              if (++slot == G::slots) { slot = 0; phase ^= 1u; }
            }
          } else {
            const int key = (wk.t0 + j) * kChunkTN + lane * box;
            const bool mine = lane < nbox && key < wk.hi && key + box > wk.lo;
            int page = 0, pslot = 0;
            if (mine) {
              const int pg = page_of(a.bt, key);
              page = a.bt.table[(int64_t)wk.b * a.bt.table_stride + pg];
              pslot = key - pg * a.bt.page_size;
              if (page < 0 || page >= a.bt.n_pages) {
                raise_status(a.status, MOE_ERR_DEVICE_INDEX);
                page = 0;
              }
            }
            const uint32_t bytes =
                __popc(__ballot_sync(0xFFFFFFFFu, mine)) * box_bytes * (uint32_t)G::halves;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              ok = ok && mbar_doze_bounded(smem_u32(&sh.kv_empty[slot]), phase ^ 1u, 100,
                                           &sh.issued, abort, a.status);
              ok = __all_sync(0xFFFFFFFFu, ok);
              if (!ok) break;
              const uint32_t bar = smem_u32(&sh.kv_full[slot]);
              if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
              __syncwarp();
              if (mine) {
                const uint32_t dst = s_kv + slot * G::tile + lane * box_bytes;
#pragma unroll
                for (int c = 0; c < G::halves; ++c)
                  tma_load_4d(dst + c * (kChunkTN * 128),
                              kv ? (const void*)&mapV : (const void*)&mapK, bar, c * 64, pslot,
                              wk.h, page);
              }
              ++fills;
              if (kv == 1 && lane == 0) *(volatile int*)&sh.issued = fills >> 1;
              if (++slot == G::slots) { slot = 0; phase ^= 1u; }
            }
          }
        }
      }
      if constexpr (GATHER) land();
      // Copies already issued land before the CTA's shared memory goes away,
      // whether or not someone gives up: another role may do so after this warp
      // has issued its last.
      const int out = fills < G::slots ? fills : G::slots;
      volatile int never = 0;
      for (int i = 0; i < out; ++i) {
        if (--slot < 0) { slot = G::slots - 1; phase ^= 1u; }
        mbar_wait_bounded(smem_u32(&sh.kv_full[slot]), phase, &never, a.status);
      }
    } else if (warp == kMmaWarp || (G::split && warp == kScoreWarp)) {
      // ----------------------------------------------------------- products --
      constexpr uint32_t kIdQK = idesc_bf16(128, kChunkTN, 0, 0);
      constexpr uint32_t kIdPV = idesc_bf16(128, DP, 0, 1);
      const bool leader = elect_one();
      const uint32_t td = uniform(tmem);
      const uint64_t qd0 = sdesc_sw128(s_q, 16, 1024);
      const uint64_t kd0 = sdesc_sw128(s_kv, 16, 1024);
      const uint64_t vd0 = sdesc_sw128(s_kv, kChunkTN * 128, 1024);
      // Items: the (tile, half) pairs of a unit in turn; item number n of the CTA
      // has score buffer n % bufs. Scores run `bufs` items ahead of the weights.
      // This warp's own instructions are on the critical path of every item: what
      // it loops over goes through a shuffle once a unit, so that positions,
      // descriptors and branches stay in uniform registers, and positions are
      // counters that wrap.
      struct Ring {
        int at;
        uint32_t phase;
        __device__ __forceinline__ void step(int by, int n) {
          at += by;
          if (at >= n) { at -= n; phase ^= 1u; }
        }
      };
      Ring k{0, 0}, v{1, 0};            // ring slots of the next K and V tile
      Ring pb{0, 0}, sb{0, 0};          // buffers of the next weights, the next scores
      int given0 = 0, given1 = 0;       // per half: the scores' next barrier
      uint32_t done0 = 0, done1 = 0;    // per half: the product's next barrier
      uint32_t uses = 0;                // split: a bit per buffer, set once it has been used
      uint32_t units0 = 0, units1 = 0;
      uint32_t seen = 0;                // a bit per slot: the parity of its next v_seen
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = wait_warp<true>(smem_u32(bar), parity, abort, a.status) && ok;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) umma_commit(smem_u32(bar));
      };
      const uint32_t q_lo = uniform((uint32_t)qd0), q_hi = uniform((uint32_t)(qd0 >> 32));
      const uint32_t k_lo = uniform((uint32_t)kd0), v_lo = uniform((uint32_t)vd0);
      const uint32_t v_hi = uniform((uint32_t)(vd0 >> 32));

      // the scores of the next tile for half H (compile-time); last: of the unit
      auto scores = [&](auto H, bool first, bool last, bool k_done) {
        constexpr int h = decltype(H)::value;
        const uint32_t q = q_lo + h * (G::q_half >> 4);
        const uint32_t k0 = k_lo + k.at * (G::tile >> 4);
        const uint32_t d = td + sb.at * 128;
        if (first) wait(&sh.q_ready[h], (h ? units1++ : units0++) & 1);
        if constexpr (G::split) {
          // the buffer's product before: none for its first use
          if (uses >> sb.at & 1) wait(&sh.buf_free[sb.at], sb.phase ^ 1u);
          uses |= 1u << sb.at;
        }
        if (!ok) return;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            constexpr int kBlock = (128 * 128) >> 4;
            const int at = (kk >> 2) * kBlock + (kk & 3) * 2;
            umma_bf16(d, desc_of(q + at, q_hi), desc_of(k0 + at, q_hi), kIdQK, kk > 0);
          }
        }
        int& given = h ? given1 : given0;
        commit(&sh.s_full[h][given]);
        if (++given == G::bufs) given = 0;
        if (last) commit(&sh.q_free[h]);
        sb.step(1, G::bufs);
        if (k_done) {
          commit(&sh.kv_empty[k.at]);
          k.step(2, G::slots);
        }
      };
      // O of half H (+)= P V over the 16-key steps [s0, s1) of the tile
      auto product = [&](auto H, bool add, bool skip, int s0, int s1) {
        constexpr int h = decltype(H)::value;
        const uint32_t vv = v_lo + v.at * (G::tile >> 4);
        const uint32_t d = td + G::o_col0 + h * DP;
        const uint32_t p = td + pb.at * 128;
        const uint32_t ad = add ? 1u : 0u;
        wait(&sh.p_ready[pb.at], pb.phase);
        if (!ok) return;
        tc_fence_after();
        if (s1 - s0 == kChunkTN / 16) {
          if (leader && !skip) {
#pragma unroll
            for (int kk = 0; kk < kChunkTN / 16; ++kk)
              umma_ts(d, p + kk * 8, desc_of(vv + kk * (2048 >> 4), v_hi), kIdPV,
                      kk > 0 ? 1u : ad);
          }
        } else if (!skip) {
#pragma unroll 1
          for (int kk = s0; kk < s1; ++kk) {
            const uint32_t pk = uniform(p + kk * 8), vk = uniform(vv + kk * (2048 >> 4));
            const uint32_t ak = uniform(kk > s0 ? 1u : ad);
            if (leader) umma_ts(d, pk, desc_of(vk, v_hi), kIdPV, ak);
          }
        }
        uint32_t& done = h ? done1 : done0;
        commit(&sh.o_done[h][done]);
        done ^= 1u;
        if constexpr (G::split) commit(&sh.buf_free[pb.at]);
        pb.step(1, G::bufs);
      };
      using H0 = std::integral_constant<int, 0>;
      using H1 = std::integral_constant<int, 1>;

      for (int u = 0; uniform(take_unit(u, ok) ? 1u : 0u); ++u) {
        const Unit wk = sh.unit[u & 3];
        give_unit(u);
        const int nt = (int)uniform(wk.nt);
        if (nt == 0) continue;
        const bool two = uniform(wk.s.nq * a.G - wk.m * kChunkTM > 128 ? 1u : 0u) != 0;
        // tiles [0, e0) and [e1, nt) are edge tiles
        int e0 = 0, e1 = nt;
        edges(wk, e0, e1);
        e0 = (int)uniform(e0);
        e1 = (int)uniform(e1);
        if (G::split && warp == kScoreWarp) {
          for (int j = 0; j < nt && ok; ++j) {
            wait(&sh.kv_full[k.at], k.phase);
            if (ok) scores(H0{}, j == 0, j + 1 == nt, !two);
            if (two && ok) scores(H1{}, j == 0, j + 1 == nt, true);
          }
          continue;
        }
        // one warp for all: the scores of the unit's first items
        if (!G::split) {
          wait(&sh.kv_full[k.at], k.phase);
          if (ok) scores(H0{}, true, nt == 1, !two);
          if (two) {
            if (ok) scores(H1{}, true, nt == 1, true);
          } else if (nt > 1) {
            wait(&sh.kv_full[k.at], k.phase);
            if (ok) scores(H0{}, false, nt == 2, true);
          }
        }
        for (int j = 0; j < nt && ok; ++j) {
          wait(&sh.kv_full[v.at], v.phase);
          bool skip = false;
          int s0 = 0, s1 = kChunkTN / 16;
          // 16-key steps [s0, s1) of an edge tile hold the unit's keys; in the
          // others V is whatever the ring held before
          if ((j < e0 || j >= e1) && ok) {
            const int k0 = (wk.t0 + j) * kChunkTN;
            s0 = (int)uniform(max(wk.lo - k0, 0) >> 4);
            s1 = (int)uniform((min(wk.hi - k0, kChunkTN) + 15) >> 4);
            wait(&sh.v_seen[v.at], seen >> v.at & 1);
            seen ^= 1u << v.at;
            skip = uniform(sh.bad[v.at]) != 0;
          }
          // Products of one thread run in the order of issue: the new scores take
          // the buffer's place after the product has read the weights. After an
          // item: its own half's next tile; with one half, two tiles on.
          const int dj = two ? 1 : 2;
          const bool more = !G::split && j + dj < nt, last = j + dj + 1 == nt;
          if (more && ok) wait(&sh.kv_full[k.at], k.phase);
          if (ok) product(H0{}, j > 0, skip, s0, s1);
          if (more && ok) scores(H0{}, false, last, !two);
          if (two) {
            if (ok) product(H1{}, j > 0, skip, s0, s1);
            if (more && ok) scores(H1{}, false, last, true);
          }
          if (ok) commit(&sh.kv_empty[v.at]);
          v.step(2, G::slots);
        }
      }
      // every product has finished before tensor memory is freed
      uint64_t* const drain = &sh.drain[warp == kMmaWarp ? 0 : 1];
      commit(drain);
      volatile int never = 0;
      mbar_wait_bounded(smem_u32(drain), 0, &never, a.status);
      __syncwarp();
    } else if (warp == kHelpWarp) {
      // ------------------------------------------------ queries, edge values --
      constexpr int NC = DP / 8;            // 16-byte pieces of a row
      int vslot = 1, gone = 0;              // gone: tiles gone by
      uint32_t vphase = 0, units = 0;     // units: two bits a half
      bool ok = true;
      for (int u = 0; take_unit(u, ok); ++u) {
        const Unit wk = sh.unit[u & 3];
        give_unit(u);
        const int nt = wk.nt;
        if (nt == 0) continue;
        int e0, e1;
        edges(wk, e0, e1);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int r0 = wk.m * kChunkTM + half * 128;
          const int nrows = wk.s.nq * a.G - r0;
          if (nrows <= 0) break;
          // 0: no unit of the half so far; else 2 + the parity of the last one's end
          const uint32_t had = units >> (2 * half) & 3;
          if (had)
            ok = ok && mbar_doze_bounded(smem_u32(&sh.q_free[half]), had & 1, 200, &sh.issued,
                                         abort, a.status);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          if (lane == 0) sh.q_had[half] = had == 2 ? 3 : 2;
          units = (units & ~(3u << (2 * half))) | ((had == 2 ? 3u : 2u) << (2 * half));
          const uint32_t bar = smem_u32(&sh.q_ready[half]);
          const uint32_t dst = s_q + half * G::q_half;
          if (q_by_tma) {
            // G heads x 128 / G tokens; rows past the sequence are other tokens'
            // queries or zeros, and what comes of them is dropped
            if (lane == 0) {
              mbar_arrive_expect_tx(bar, G::q_half);
#pragma unroll
              for (int c = 0; c < G::halves; ++c)
                tma_load_3d(dst + c * (128 * 128), &mapQ, bar, c * 64, wk.h * a.G,
                            wk.s.q0 + div_group(a, r0));
            }
            __syncwarp();
          } else {
            // four rows a lane
#pragma unroll 1
            for (int r = lane; r < 128; r += 32) {
              const int rr = r0 + min(r, nrows - 1);
              const int tok = div_group(a, rr), g = rr - tok * a.G;
              const moe_bf16* src = a.q + (int64_t)(wk.s.q0 + tok) * a.q_stride +
                                    (int64_t)(wk.h * a.G + g) * a.D;
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                const bool in = c * 8 < a.D;
                cp_async16(dst + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           src + (in ? c * 8 : 0), in);
              }
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
          }
        }
        for (int j = 0; j < nt; ++j) {
          if (j < e0 || j >= e1) {
            // the tiles between are not waited for, so first the loads must have
            // come to this one: a barrier's parity tells one round of the ring
            // from the next, not from the one after
            ok = issued_wait_bounded(&sh.issued, gone + 1, abort, a.status) &&
                 mbar_wait_bounded(smem_u32(&sh.kv_full[vslot]), vphase, abort, a.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            const int k0 = (wk.t0 + j) * kChunkTN;
            uint8_t* const vt = kv_mem + vslot * G::tile;
            // Zeros: the rows out of range in the first and last 16-key step that
            // the product takes. Looked through: the rows that only some see.
            const int v0 = max(wk.lo - k0, 0), v1 = min(wk.hi - k0, kChunkTN);
            const int f0 = min(max(wk.all_lo - k0, v0), v1), f1 = max(min(wk.all_hi - k0, v1), f0);
            auto piece = [&](int i) {      // piece i % NC of key row i / NC
              const int row = i / NC, c = i - row * NC;
              return reinterpret_cast<uint4*>(vt + (c >> 3) * (128 * 128) + row * 128 +
                                              (((c ^ row) & 7) << 4));
            };
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
            for (int i = (v0 & ~15) * NC + lane; i < v0 * NC; i += 32) *piece(i) = zero;
#pragma unroll 1
            for (int i = v1 * NC + lane; i < ((v1 + 15) & ~15) * NC; i += 32) *piece(i) = zero;
            uint32_t bad = 0;
#pragma unroll 4
            for (int i = v0 * NC + lane; i < f0 * NC; i += 32) bad |= not_finite8(*piece(i));
#pragma unroll 4
            for (int i = f1 * NC + lane; i < v1 * NC; i += 32) bad |= not_finite8(*piece(i));
            fence_async_smem();
            const int any = __any_sync(0xFFFFFFFFu, bad != 0);
            if (lane == 0) {
              sh.bad[vslot] = any;
              mbar_arrive(smem_u32(&sh.v_seen[vslot]));
            }
            __syncwarp();
          }
          ++gone;
          vslot += 2;
          if (vslot >= G::slots) { vslot -= G::slots; vphase ^= 1u; }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax --
    const int half = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;             // of the half
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_o = t_lane + G::o_col0 + half * DP;
    uint32_t item0 = 0;               // as the product warp counts
    int tile0 = 0;
    uint32_t mine = 0;                // this half's items so far
    uint32_t seen = 0;
    bool ok = true;
    for (int u = 0; take_unit(u, ok); ++u) {
      const Unit wk = sh.unit[u & 3];
      give_unit(u);
      const Seq s = wk.s;
      const int r0 = wk.m * kChunkTM + half * 128;
      const int left = s.nq * a.G - wk.m * kChunkTM;
      const int nh = left > 128 ? 2 : 1;
      const int nrows = min(128, left - half * 128);
      const int nt = wk.nt, t0 = wk.t0;
      int e0, e1;
      edges(wk, e0, e1);
      const uint32_t first_item = item0 + half;
      const int first_tile = tile0;
      item0 += nt * nh;
      tile0 += nt;
      if (nrows <= 0) {               // the half has no rows: its tiles go by
        for (int j = 0; j < nt; ++j)
          if (j < e0 || j >= e1) seen ^= 1u << ((2 * (first_tile + j) + 1) % G::slots);
        continue;
      }
      const int r = r0 + min(row, nrows - 1);
      const int tok = div_group(a, r), head = wk.h * a.G + (r - tok * a.G);
      const int64_t grow = s.q0 + tok;
      const bool real = row < nrows;
      float m_ref = neg_inf(), l = 0.f;
      if (nt > 0) {
        const int lo = key_lo(a, s, tok), hi = real ? key_hi(a, s, tok) : 0;
        // keys every row of the warp sees: [warp_lo, warp_hi)
        const int w0 = r0 + min((warp & 3) * 32, nrows - 1);
        const int w1 = r0 + min((warp & 3) * 32 + 31, nrows - 1);
        const int warp_lo = key_lo(a, s, div_group(a, w1)),
                  warp_hi = key_hi(a, s, div_group(a, w0));

        for (int j = 0; j < nt; ++j) {
          const int k0 = (t0 + j) * kChunkTN;
          const uint32_t n = first_item + j * nh;
          const int buf = n % G::bufs;
          const uint32_t t_s = t_lane + buf * 128;
          ok = ok && wait_warp<false>(smem_u32(&sh.s_full[half][mine % G::bufs]),
                                      (mine / G::bufs) & 1, abort, a.status);
          if (!ok) break;
          tc_fence_after();
          // the half's product before this one has ended, for who is to change O
          // (the two before it have: their buffers hold later scores)
          auto o_is_done = [&]() {
            ok = ok && wait_warp<false>(smem_u32(&sh.o_done[half][(mine - 1) & 1]),
                                 ((mine - 1) >> 1) & 1, abort, a.status);
            tc_fence_after();
          };
          // In groups of 64 keys; a group's weights take the place of scores already
          // read. The loop is kept rolled, and the group's code there once, for the
          // instruction cache ((a) and (b) before sums replaced the maxima: this form
          // 634 and 628, all 128 keys in line 661 and 894, groups of 32 730 and 700, a
          // second copy of the weights' code 632 and 644).
          const bool masked = k0 + kChunkTN > warp_hi || k0 < warp_lo;
          const RowMask mask{lo - k0, hi - k0};
#pragma unroll 1
          for (int g = 0; g < 4;) {             // g: in 32 keys
            float x[64];
            tmem_ld32f(t_s + g * 32, x);
            tmem_ld32f(t_s + g * 32 + 32, x + 32);
            tmem_ld_wait();
            if (__builtin_expect(masked, 0)) {
#pragma unroll
              for (int c = 0; c < 64; ++c) x[c] = mask(x[c], g * 32 + c);
            }
            uint32_t pk[32];
            const float sum =
                group_weights(x, a.scale_log2, m_ref == neg_inf() ? 0.f : m_ref, pk);
            // Infinite and NaN sums come here as well; a reference that is the group's
            // maximum does not move again, so they are stored the second time.
            const bool check = real && (m_ref == neg_inf() || !(sum <= kMoveAt));
            if (__builtin_expect(__any_sync(0xFFFFFFFFu, check), 0)) {
              float top = x[0];
#pragma unroll
              for (int c = 1; c < 63; c += 2) top = max3(top, x[c], x[c + 1]);
              top = fmaxf(top, x[63]) * a.scale_log2;
              const bool grew = check && top > m_ref;
              if (__any_sync(0xFFFFFFFFu, grew)) {
                const float nm = grew ? top : m_ref;
                const float f = nm == neg_inf() ? 1.f : ex2(m_ref - nm);
                m_ref = nm;
                l *= f;
                scale_weights(t_s, g * 16, f);
                if (j > 0) {
                  o_is_done();
                  scale_rows<DP>(t_o, f);
                }
                continue;        // once more: no score of the group is above now
              }
            }
            l += sum;
            tmem_st32(t_s + g * 16, pk);
            g += 2;
          }
          tmem_st_wait();
          if (__builtin_expect(j < e0 || j >= e1, 0)) {
            // A zero weight does not keep an infinite or NaN value out of the
            // product: a tile that some row sees in part and that holds one is not
            // multiplied; its P V is added here, key by key over the rows that see it.
            const int t = first_tile + j, vslot = (2 * t + 1) % G::slots;
            ok = ok && wait_warp<false>(smem_u32(&sh.v_seen[vslot]), seen >> vslot & 1, abort,
                                        a.status);
            seen ^= 1u << vslot;
            const bool by_hand = ok && sh.bad[vslot] != 0;
            if (__any_sync(0xFFFFFFFFu, by_hand)) {
              ok = ok && wait_warp<false>(smem_u32(&sh.kv_full[vslot]),
                                          ((2 * t + 1) / G::slots) & 1, abort, a.status);
              if (j > 0) o_is_done();
              __syncwarp();
              add_by_hand<DP>(t_s, t_o, kv_mem + vslot * G::tile, k0, lo, hi, j > 0);
              tmem_st_wait();
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.p_ready[buf]));
          ++mine;
        }
        // the last two products in turn: a parity tells a barrier's latest phase
        // only from the one before
        for (uint32_t i = mine > 1 ? mine - 2 : 0; i < mine && ok; ++i)
          ok = wait_warp<false>(smem_u32(&sh.o_done[half][i & 1]), (i >> 1) & 1, abort, a.status);
        if (!ok) break;
        tc_fence_after();
        if (__builtin_expect(wk.begun, 0)) {
          const float2 ml = join_before<DP>(a, t_o, wk.slot(), half * 128 + row, m_ref, l);
          m_ref = ml.x;
          l = ml.y;
        }
      }
      // ---- the unit's rows: final, or this CTA's part (so far) ---------------
      const bool whole = wk.whole() && wk.rest == 0;
      RowEnd e{1.f, 0.f};
      if (whole) e = row_end(m_ref, l, a.sinks, head);
      const int64_t pslot = (int64_t)blockIdx.x * 2 + wk.slot();
      moe_bf16* const dst = a.out + grow * a.out_stride + (int64_t)head * a.D;
#pragma unroll 1
      for (int c = 0; c < DP; c += 32) {
        float o[32];
        if (nt > 0) {
          tmem_ld32f(t_o + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (real && whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = o[i * 8 + q] * e.factor;
            if (c + i * 8 < a.D) *reinterpret_cast<uint4*>(dst + c + i * 8) = pack8(v);
          }
        } else if (real) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(
                a.part_o + part_at<kChunkTM, DP>(pslot, half * 128 + row, c / 4 + i)) =
                make_float4(o[i * 4], o[i * 4 + 1], o[i * 4 + 2], o[i * 4 + 3]);
        }
        __syncwarp();      // the next load is the whole warp's
      }
      if (real) {
        if (!whole) a.part_ml[pslot * kChunkTM + half * 128 + row] = make_float2(m_ref, l);
        else if (a.lse) a.lse[grow * a.Hq + head] = e.lse;
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // after giving up: queries already asked for land before the CTA's shared memory
  // goes away (waited for in the helper's own branch: 689 instead of 644 us a
  // 4 x 4096-token prefill, by where the code then lies)
  if (*abort && q_by_tma && tid < 2 && sh.q_had[tid])
    wait_slowly(smem_u32(&sh.q_ready[tid]), sh.q_had[tid] & 1, &sh.never, a.status);
  __syncwarp();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host --
static int kv_box(int page_size) {      // keys that neither a page nor a tile cuts
  int b = kChunkTN;
  while (page_size % b) b >>= 1;
  return b;
}

bool attn_chunk_boxes(int page_size) { return page_size % 8 == 0; }

size_t attn_chunk_ws_bytes(int D) {
  const int DP = D <= 64 ? 64 : 128;
  return (size_t)num_sms() * (sizeof(Cut) + 2 * kChunkTM * (DP + 2) * sizeof(float));
}

template <int DP, bool GATHER>
static cudaError_t launch_chunk(AttnArgs a, const moe_kv_cache& c, void* ws, cudaStream_t s) {
  using G = ChunkGeo<DP>;
  CUtensorMap mk = {}, mv = {};
  const int box = GATHER ? kChunkTN : kv_box(c.page_size);
  if (!GATHER && (!map_kv(&mk, c.k, c, box) || !map_kv(&mv, c.v, c, box)))
    return cudaErrorInvalidValue;
  // a half's 128 rows are whole tokens when G divides 128
  const int by_tma = 128 % a.G == 0 ? 1 : 0;
  CUtensorMap mq = mk;
  if (by_tma && !map_heads(&mq, a.q, a.D, a.Hq, a.bt.T, a.q_stride, a.G, 128 / a.G))
    return cudaErrorInvalidValue;
  auto kern = attn_chunk_kernel<DP, GATHER>;
  static SmemOnce once;
  cudaError_t e = once.set((const void*)kern, G::smem);
  if (e != cudaSuccess) return e;
  const int n = num_sms();
  a.least = kChunkLeast;
  a.piece = kChunkPiece;
  a.cuts = static_cast<Cut*>(ws);
  a.part_ml = reinterpret_cast<float2*>(a.cuts + n);
  a.part_o = reinterpret_cast<float*>(a.part_ml + (size_t)2 * n * kChunkTM);
  timer_before(MOE_KERNEL_ATTN, s);
  e = launch_pdl(true, kern, dim3(n), dim3(kChunkThreads), G::smem, s, a, mq, mk, mv, box,
                 by_tma);
  timer_after(MOE_KERNEL_ATTN, s);
  if (e != cudaSuccess) return e;
  timer_before(MOE_KERNEL_ATTN_COMBINE, s);
  e = launch_pdl(true, attn_join_kernel<kChunkTM, DP>, dim3(n - 1, 16), dim3(kJoinThreads), 0, s,
                 a);
  timer_after(MOE_KERNEL_ATTN_COMBINE, s);
  note_launches(2);
  return e;
}

cudaError_t launch_attn_chunk(const AttnArgs& a, const moe_kv_cache& c, void* ws,
                              cudaStream_t s) {
  if (!attn_chunk_boxes(c.page_size))
    return c.D <= 64 ? launch_chunk<64, true>(a, c, ws, s) : launch_chunk<128, true>(a, c, ws, s);
  return c.D <= 64 ? launch_chunk<64, false>(a, c, ws, s) : launch_chunk<128, false>(a, c, ws, s);
}

}  // namespace moe
