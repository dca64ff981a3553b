// attn_chunk.cu — attention over the paged cache for many rows per key/value
// head (prompt chunks, prefill) on the 5th-generation tensor cores.
//
// A unit is 256 rows (two halves of 128) of one sequence and key/value head
// against its key range, in tiles of 128 keys. Per tile and half:
//   S = Q K^T      tcgen05.mma, both operands in shared memory, S in tensor memory
//   P = exp2(S * scale - max), rounded to bf16 over S's own columns
//   O += P V       tcgen05.mma with P read from tensor memory
// One pass with a running maximum: a row's reference maximum is only moved
// (and O rescaled in tensor memory) when it grew by more than 2^8, so the
// accumulator is touched a few times a unit instead of once a tile; weights of
// up to 2^8 cost no precision, in bf16 or in the fp32 sums.
//
// The tensor cores and the exponentials are the two resources of like cost
// (for D = 128 four 128x128x128 products and 32 Ki exponentials a tile), so
// the halves alternate: while one half's scores are exponentiated, the other
// half's products run.
//   warps 0-3, 4-7   softmax of half 0 and 1: one row per thread (the row's
//                    maximum and sum need no shuffles), the accumulator's
//                    rescale, the epilogue, and loading the half's queries
//   warp 8           issues the products (one thread); owns tensor memory
//   warp 9           loads K and V tiles by TMA through a ring, one box per
//                    stretch of keys that neither a page nor a tile cuts
#include "attn.cuh"
#include "attn_join.cuh"
#include "common.cuh"
#include "internal.h"
#include "tmap.h"

namespace moe {

constexpr int kChunkTM = 256;
constexpr int kChunkTN = 128;
constexpr int kChunkThreads = 384;    // warps 10 and 11 only give up their registers
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr float kRescaleAt = 8.f;

template <int DP>
struct ChunkGeo {
  static constexpr int halves = DP / 64;                 // 128-byte column blocks of a row
  static constexpr int tile = kChunkTN * DP * 2;         // one K or V tile
  static constexpr int q_half = 128 * DP * 2;
  static constexpr int slots = DP == 128 ? 5 : 8;        // K and V tiles alternate
  static constexpr int smem = 2 * q_half + slots * tile + 1024;
  static constexpr uint32_t s_col0 = 0;                  // S (and P) of half h: h * 128
  static constexpr uint32_t o_col0 = 256;                // O of half h: 256 + h * DP
};

// The product-issuing warp runs as one: every value an instruction takes is the
// same in all lanes (uniform registers), and one elected lane issues. A single
// lane running ahead alone costs about 90 cycles an instruction in moves to
// uniform registers, more than the 32 to 64 the product itself takes.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(e));
  return e;
}
// A descriptor from its two halves: only the address in the low one varies.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  return ((uint64_t)hi << 32) | lo;
}
// S[tmem] (+)= Q[smem] * K[smem]^T, by the elected lane
__device__ __forceinline__ void umma_ss(uint32_t leader, uint32_t d_tmem, uint64_t adesc,
                                        uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// O[tmem] (+)= P[tmem] * V[smem]
__device__ __forceinline__ void umma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                        uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void umma_commit_by(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(
          bar),
      "r"(leader)
      : "memory");
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
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
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

// no infinity or NaN among eight bf16 values
__device__ __forceinline__ bool finite8(const uint4& v) {
  bool bad = false;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bad = bad || (w[i] & 0x7F800000u) == 0x7F800000u || (w[i] & 0x7F80u) == 0x7F80u;
  return !bad;
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
    for (int k = 0; k < kChunkTN; k += 16) {
      uint32_t p[8];
      tmem_ld8(t_p + k / 2, p);
      tmem_ld_wait();
#pragma unroll
      for (int kk = 0; kk < 16; ++kk) {
        const int key = k + kk;
        const float w = (kk & 1) ? bf16_hi(p[kk >> 1]) : bf16_lo(p[kk >> 1]);
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

// A warpgroup's registers a thread. 384 threads start with 168 each (64512);
// the softmax warpgroups hold 128 scores and their packed weights at once:
// 2 x 128 x 200 + 128 x 88 = 62464.
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct ChunkShared {
  Place pl;
  uint64_t kv_full[8], kv_empty[8];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_done[2], drain;
  uint32_t tmem;
  int abort;
  uint64_t looked[2];   // the half's warps have looked through a tile's values
  int bad[2][2][4];     // what each of them found (two tiles in turn)
  int by_hand[2];       // they have added this tile's P V themselves
};

template <int DP>
__global__ void __launch_bounds__(kChunkThreads, 1)
    attn_chunk_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap mapK,
                      const __grid_constant__ CUtensorMap mapV, int box) {
  using G = ChunkGeo<DP>;
  using TL = Tiling<kChunkTM, kChunkTN>;
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
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(smem_u32(&sh.q_ready[h]), 4);
      mbar_init(smem_u32(&sh.s_full[h]), 1);
      mbar_init(smem_u32(&sh.p_ready[h]), 4);
      mbar_init(smem_u32(&sh.o_done[h]), 1);
      mbar_init(smem_u32(&sh.looked[h]), 4);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool work = locate<kChunkTM, kChunkTN, kChunkThreads>(a, blockIdx.x, gridDim.x, sh.pl);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp >= 8) {
    regs_down<88>();
    if (work && warp == kLoadWarp) {
      // -------------------------------------------------------------- loads --
      // lane i < nbox: the box of keys [tile + i * box, + box)
      const int nbox = kChunkTN / box;
      const uint32_t box_bytes = (uint32_t)box * 128u;
      int slot = 0;
      uint32_t phase = 0;
      int fills = 0;
      bool ok = true;
      for (Walk<kChunkTM, kChunkTN> wk(a, sh.pl, blockIdx.x, gridDim.x); wk.more() && ok;
           wk.next()) {
        const int nt = wk.sp.nt > 0 ? wk.take : 0;
        for (int j = 0; j < nt && ok; ++j) {
          const int key = (wk.sp.t0 + wk.off + j) * kChunkTN + lane * box;
          const bool mine = lane < nbox && key < wk.sp.hi && key + box > wk.sp.lo;
          int page = 0, pslot = 0;
          if (mine) {
            const int pg = key / a.bt.page_size;
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
            ok = ok && mbar_wait_bounded(smem_u32(&sh.kv_empty[slot]), phase ^ 1u, abort, a.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint32_t bar = smem_u32(&sh.kv_full[slot]);
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (mine) {
              const uint32_t dst = s_kv + slot * G::tile + lane * box_bytes;
#pragma unroll
              for (int c = 0; c < G::halves; ++c)
                tma_load_4d(dst + c * (kChunkTN * 128), kv ? (const void*)&mapV : (const void*)&mapK,
                            bar, c * 64, pslot, wk.h, page);
            }
            ++fills;
            if (++slot == G::slots) { slot = 0; phase ^= 1u; }
          }
        }
      }
      if (*abort) {
        // copies already issued land before the CTA's shared memory goes away
        const int out = fills < G::slots ? fills : G::slots;
        volatile int never = 0;
        for (int i = 0; i < out; ++i) {
          if (--slot < 0) { slot = G::slots - 1; phase ^= 1u; }
          mbar_wait_bounded(smem_u32(&sh.kv_full[slot]), phase, &never, a.status);
        }
      }
    } else if (work && warp == kMmaWarp) {
      // ----------------------------------------------------------- products --
      constexpr uint32_t kIdQK = idesc_bf16(128, kChunkTN, 0, 0);
      constexpr uint32_t kIdPV = idesc_bf16(128, DP, 0, 1);
      const uint32_t leader = elect_one();
      const uint32_t td = uniform(tmem);
      const uint64_t qd0 = sdesc_sw128(s_q, 16, 1024);
      const uint64_t kd0 = sdesc_sw128(s_kv, 16, 1024);
      const uint64_t vd0 = sdesc_sw128(s_kv, kChunkTN * 128, 1024);
      int kslot = 0;                    // ring slot of the next K tile
      uint32_t kphase = 0;
      uint32_t units[2] = {0, 0}, tiles[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait_bounded(smem_u32(bar), parity, abort, a.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
        return ok;
      };
      auto commit = [&](uint64_t* bar) { umma_commit_by(leader, smem_u32(bar)); };
      auto qk = [&](int h, int slot) {
        const uint32_t q = uniform((uint32_t)qd0 + h * (G::q_half >> 4));
        const uint32_t k = uniform((uint32_t)kd0 + slot * (G::tile >> 4));
        const uint32_t hi = uniform((uint32_t)(kd0 >> 32));
        const uint32_t d = uniform(td + G::s_col0 + h * 128);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          constexpr int kBlock = (128 * 128) >> 4;
          const int at = (kk >> 2) * kBlock + (kk & 3) * 2;
          umma_ss(leader, d, desc_of(q + at, hi), desc_of(k + at, hi), kIdQK, kk > 0);
        }
        commit(&sh.s_full[h]);
      };
      auto pv = [&](int h, int slot, bool first) {
        const uint32_t v = uniform((uint32_t)vd0 + slot * (G::tile >> 4));
        const uint32_t hi = uniform((uint32_t)(vd0 >> 32));
        const uint32_t d = uniform(td + G::o_col0 + h * DP);
        const uint32_t p = uniform(td + G::s_col0 + h * 128);
        const uint32_t add = uniform(first ? 0u : 1u);
#pragma unroll
        for (int kk = 0; kk < kChunkTN / 16; ++kk)
          umma_ts(leader, d, p + kk * 8, desc_of(v + kk * (2048 >> 4), hi), kIdPV,
                  kk > 0 ? 1u : add);
      };
      for (Walk<kChunkTM, kChunkTN> wk(a, sh.pl, blockIdx.x, gridDim.x); wk.more() && ok;
           wk.next()) {
        const int nt = wk.sp.nt > 0 ? wk.take : 0;
        if (nt == 0) continue;
        const int nh = wk.s.nq * a.G - wk.m * kChunkTM > 128 ? 2 : 1;
        auto step = [&]() { if (++kslot == G::slots) { kslot = 0; kphase ^= 1u; } };
        // the first tile's scores
        if (!wait(&sh.kv_full[kslot], kphase)) break;
        for (int h = 0; h < nh; ++h) {
          if (!wait(&sh.q_ready[h], units[h] & 1)) break;
          ++units[h];
          tc_fence_after();
          qk(h, kslot);
        }
        if (!ok) break;
        commit(&sh.kv_empty[kslot]);
        step();
        for (int j = 0; j < nt; ++j) {
          const int vslot = kslot;
          if (!wait(&sh.kv_full[vslot], kphase)) break;
          step();
          const bool more = j + 1 < nt;
          const int nkslot = kslot;
          if (more && !wait(&sh.kv_full[nkslot], kphase)) break;
          for (int h = 0; h < nh; ++h) {
            if (!wait(&sh.p_ready[h], tiles[h] & 1)) break;
            ++tiles[h];
            tc_fence_after();
            // products of one thread run in the order of issue: the next scores
            // overwrite P's columns after this product has read them
            const bool skip = *(volatile int*)&sh.by_hand[h];
            if (!__any_sync(0xFFFFFFFFu, skip)) pv(h, vslot, j == 0);
            if (more) qk(h, nkslot);
            else commit(&sh.o_done[h]);
          }
          if (!ok) break;
          commit(&sh.kv_empty[vslot]);
          if (more) {
            commit(&sh.kv_empty[nkslot]);
            step();
          }
        }
      }
      // every product has finished before tensor memory is freed
      commit(&sh.drain);
      volatile int never = 0;
      mbar_wait_bounded(smem_u32(&sh.drain), 0, &never, a.status);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax --
    regs_up<200>();
    const int half = warp >> 2;
    const int row = (warp & 3) * 32 + lane;             // of the half
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = t_lane + G::s_col0 + half * 128;
    const uint32_t t_o = t_lane + G::o_col0 + half * DP;
    uint8_t* const q_mem = smem + half * G::q_half;
    int vslot = 1;                    // ring slot of the tile's V (K's is the one before)
    uint32_t vphase = 0;
    uint32_t tiles = 0, ends = 0, looks = 0;
    bool ok = true;
    auto vstep = [&]() {
      vslot += 2;
      if (vslot >= G::slots) { vslot -= G::slots; vphase ^= 1u; }
    };
    Walk<kChunkTM, kChunkTN> wk(a, sh.pl, blockIdx.x, gridDim.x, work);
    for (; wk.more() && ok; wk.next()) {
      const Seq s = wk.s;
      const int r0 = wk.m * kChunkTM + half * 128;
      const int nrows = min(128, s.nq * a.G - r0);
      const int nt = wk.sp.nt > 0 ? wk.take : 0;
      if (nrows <= 0) {               // the half has no rows: its tiles go by
        for (int j = 0; j < nt; ++j) vstep();
        continue;
      }
      const int r = r0 + min(row, nrows - 1);
      const int tok = r / a.G, head = wk.h * a.G + (r - tok * a.G);
      const int64_t grow = s.q0 + tok;
      const bool real = row < nrows;
      float m_ref = neg_inf(), l = 0.f;
      if (nt > 0) {
        // ---- queries: one row per thread, in the 128-byte swizzle ------------
        const uint4* src =
            reinterpret_cast<const uint4*>(a.q + grow * a.q_stride + (int64_t)head * a.D);
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (real && c * 8 < a.D) v = src[c];
          *reinterpret_cast<uint4*>(q_mem + (c >> 3) * (128 * 128) + row * 128 +
                                    (((c & 7) ^ (row & 7)) << 4)) = v;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.q_ready[half]));

        const int lo = key_lo(a, s, tok), hi = real ? key_hi(a, s, tok) : 0;
        // keys every row of the half sees: [all_lo, all_hi); of the warp alike
        const int all_lo = key_lo(a, s, (r0 + nrows - 1) / a.G), all_hi = key_hi(a, s, r0 / a.G);
        const int w0 = r0 + min((warp & 3) * 32, nrows - 1);
        const int w1 = r0 + min((warp & 3) * 32 + 31, nrows - 1);
        const int warp_lo = key_lo(a, s, w1 / a.G), warp_hi = key_hi(a, s, w0 / a.G);

        for (int j = 0; j < nt; ++j) {
          const int k0 = (wk.sp.t0 + wk.off + j) * kChunkTN;
          ok = ok && mbar_wait_bounded(smem_u32(&sh.s_full[half]), tiles & 1, abort, a.status);
          if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
          ++tiles;
          tc_fence_after();
          float sc[128];
          tmem_ld32f(t_s, sc);
          tmem_ld32f(t_s + 32, sc + 32);
          tmem_ld32f(t_s + 64, sc + 64);
          tmem_ld32f(t_s + 96, sc + 96);
          tmem_ld_wait();
          if (k0 < warp_lo || k0 + kChunkTN > warp_hi) {
            // masked by selection: a masked score's value, NaN or not, is dropped
#pragma unroll
            for (int c = 0; c < 128; ++c)
              sc[c] = (k0 + c >= lo && k0 + c < hi) ? sc[c] : neg_inf();
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = fmaxf(sc[2 * i], sc[2 * i + 1]);
#pragma unroll
          for (int c = 8; c < 128; c += 2)
            mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], sc[c], sc[c + 1]);
          const float m2 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
          const bool grew = m2 > m_ref + kRescaleAt;      // true for the first key a row sees
          if (__any_sync(0xFFFFFFFFu, grew)) {
            const float nm = grew ? m2 : m_ref;
            const float f = nm == neg_inf() ? 1.f : ex2(m_ref - nm);
            m_ref = nm;
            l *= f;
            if (j > 0) {
              // the scores' barrier stands for every product issued before them
#pragma unroll 1
              for (int c = 0; c < DP; c += 32) {
                float o[32];
                tmem_ld32f(t_o + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] *= f;
                tmem_st32f(t_o + c, o);
              }
            }
          }
          const float ref = m_ref == neg_inf() ? 0.f : m_ref;
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
#pragma unroll
          for (int c0 = 0; c0 < 128; c0 += 64) {
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              float2 t = fma2(make_float2(sc[c0 + c], sc[c0 + c + 1]), a.scale_log2, -ref);
              t = make_float2(ex2(t.x), ex2(t.y));
              acc[(c >> 1) & 3] = add2(acc[(c >> 1) & 3], t);
              pk[c / 2] = pack_bf16(t.x, t.y);
            }
            tmem_st32(t_s + c0 / 2, pk);
          }
          acc[0] = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
          l += acc[0].x + acc[0].y;
          // A zero weight does not keep an infinite or NaN value out of the product.
          // V rows outside the unit's keys hold whatever the cache holds there:
          // they become zeros. In a tile that some of the half's rows see only in
          // part, the values are looked through; should one not be finite, the
          // half's warps add the tile's P V to O themselves, key by key over the
          // rows that see it, and the product is not issued.
          const bool ragged = k0 < wk.sp.lo || k0 + kChunkTN > wk.sp.hi;
          const bool differ = max(k0, wk.sp.lo) < all_lo || min(k0 + kChunkTN, wk.sp.hi) > all_hi;
          bool by_hand = false;
          if (ragged || differ) {
            ok = ok && mbar_wait_bounded(smem_u32(&sh.kv_full[vslot]), vphase, abort, a.status);
            uint8_t* const vt = kv_mem + vslot * G::tile;
            // one key row per thread, its 16-byte pieces in an order of its own
            // (no two of 8 lanes on the same banks)
            const bool in = k0 + row >= wk.sp.lo && k0 + row < wk.sp.hi;
            bool bad = false;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) {
              uint4* p = reinterpret_cast<uint4*>(vt + (c >> 3) * (128 * 128) + row * 128 +
                                                  (((c + row) & 7) << 4));
              if (!in) *p = make_uint4(0u, 0u, 0u, 0u);
              else if (differ) bad = bad || !finite8(*p);
            }
            fence_async_smem();
            if (differ) {
              const int at = looks & 1;
              sh.bad[half][at][warp & 3] = __any_sync(0xFFFFFFFFu, bad);
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&sh.looked[half]));
              ok = ok && mbar_wait_bounded(smem_u32(&sh.looked[half]), looks & 1, abort, a.status);
              ++looks;
              const volatile int* f = sh.bad[half][at];
              by_hand = (f[0] | f[1] | f[2] | f[3]) != 0;
              __syncwarp();
            }
            if (by_hand) {
              tmem_st_wait();
              add_by_hand<DP>(t_s, t_o, vt, k0, lo, hi, j > 0);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            *(volatile int*)&sh.by_hand[half] = by_hand;
            mbar_arrive(smem_u32(&sh.p_ready[half]));
          }
          vstep();
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        ok = mbar_wait_bounded(smem_u32(&sh.o_done[half]), ends & 1, abort, a.status);
        ++ends;
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
      }
      // ---- the unit's rows: final, or this CTA's part ------------------------
      const bool whole = wk.whole();
      RowEnd e{1.f, 0.f};
      if (whole) e = row_end(m_ref, l, a.sinks, head);
      moe_bf16* const dst = a.out + grow * a.out_stride + (int64_t)head * a.D;
      const int64_t prow = ((int64_t)blockIdx.x * 2 + wk.slot()) * kChunkTM + half * 128 + row;
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
            *reinterpret_cast<float4*>(a.part_o + prow * DP + c + i * 4) =
                make_float4(o[i * 4], o[i * 4 + 1], o[i * 4 + 2], o[i * 4 + 3]);
        }
        __syncwarp();      // the next load is the whole warp's
      }
      if (real) {
        if (!whole) a.part_ml[prow] = make_float2(m_ref, l);
        else if (a.lse) a.lse[grow * a.Hq + head] = e.lse;
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ host --
static int kv_box(int page_size) {      // keys that neither a page nor a tile cuts
  int b = kChunkTN;
  while (page_size % b) b >>= 1;
  return b;
}

bool attn_chunk_takes(int page_size) { return page_size % 8 == 0; }

size_t attn_chunk_ws_bytes(int D) {
  const int DP = D <= 64 ? 64 : 128;
  return (size_t)2 * num_sms() * kChunkTM * (DP + 2) * sizeof(float);
}

template <int DP>
static cudaError_t launch_chunk(AttnArgs a, const moe_kv_cache& c, void* ws, cudaStream_t s) {
  using G = ChunkGeo<DP>;
  CUtensorMap mk, mv;
  const int box = kv_box(c.page_size);
  if (!map_kv(&mk, c.k, c, box) || !map_kv(&mv, c.v, c, box)) return cudaErrorInvalidValue;
  auto kern = attn_chunk_kernel<DP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::smem);
  if (e != cudaSuccess) return e;
  const int n = num_sms();
  a.part_ml = static_cast<float2*>(ws);
  a.part_o = reinterpret_cast<float*>(a.part_ml + (size_t)2 * n * kChunkTM);
  timer_before(MOE_KERNEL_ATTN, s);
  e = launch_pdl(true, kern, dim3(n), dim3(kChunkThreads), G::smem, s, a, mk, mv, box);
  timer_after(MOE_KERNEL_ATTN, s);
  if (e != cudaSuccess) return e;
  timer_before(MOE_KERNEL_ATTN_COMBINE, s);
  e = launch_pdl(true, attn_join_kernel<kChunkTM, kChunkTN, DP>, dim3(n - 1, 8),
                 dim3(kJoinThreads), 0, s, a, n);
  timer_after(MOE_KERNEL_ATTN_COMBINE, s);
  note_launches(2);
  return e;
}

cudaError_t launch_attn_chunk(const AttnArgs& a, const moe_kv_cache& c, void* ws,
                              cudaStream_t s) {
  return c.D <= 64 ? launch_chunk<64>(a, c, ws, s) : launch_chunk<128>(a, c, ws, s);
}

}  // namespace moe
