// w4_tiles.cu — products of many rows with 4-bit weights (layout: w4.cuh) on the
// 5th-generation tensor cores: a linear layer, and the experts' gate/up and down
// products over the padded expert-grouped layout (permute.cu).
//
//   D[n, r] += W^T[n, k] x^T[k, r]
// Two blocks of a cluster work on 128 columns n each of the same rows of x, by products of both
// (cta_group::2, M = 256). The weights are the A operand, 256 k a stage; up to 256 rows of x
// are the B operand, N = their number rounded up to 16, half of them in either block. A
// lives in tensor memory: eight warps take four 512-byte tiles of codes each a stage, turn them
// into bf16 code * scale in registers (W4Decoder), and store it as the 16x256b shape, whose
// lanes hold just what a lane's codes are. So the bf16 weights never pass through shared memory,
// whose bandwidth the products' B operand needs, and the codes are decoded once for 256
// rows. code * scale is rounded to bf16 there; scales of few bits (moe_w4_quantise's) make
// it exact.
//
// What bounds it (a stage, cycles): decoding about 1000, most of it on the pipe of the logical
// operations; the products 8 N, some 500 at least to issue. With few
// rows decoding and the hand-over of a stage of A between warps and blocks add up: 16 rows of
// 4096 x 38912 take 26 us, where reading the codes takes 13. With 512 rows 92 us, 92% of the
// rate of a large bf16 product. Measured on the way there: products of one block each, the
// rows of x multicast to both: 98 us at 512 rows, 45 at 160 (now 37), the rows came in at 50 bytes a
// cycle and SM whatever else was left out; sixteen decoding warps of two tiles each: 128 rows 36.6
// us, eight 35.6.
//
// The 128 columns: two runs of 64, of gate and up or of one matrix. Sixteen columns of each
// make up a warp's 32 lanes of tensor memory, so that gate and up of a column meet by a shuffle.
//
// Roles (20 warps): 0 loads rows of x by TMA, 128 k a stage, 256 where rows are few; 3 streams the
// codes and scales, contiguous pieces of 64 columns by 256 rows, by bulk copies; 4-11 the eight
// above; 1 of the first block issues the products; 12-19 take the finished tile from tensor
// memory (a thread a column). Tensor memory: 256 columns of accumulators (two tiles of up to 128
// rows, so that one is taken out while the next is summed, or one of more), two stages of 128
// columns of A. The first block's barriers of x, of A and of emptied accumulators count both
// blocks' arrivals. Every wait is bounded.
//
// An expert's rows are cut into equal chunks of at most 256; tiles of one run of columns
// follow one another, so that its codes are in L2 for the next chunk.
#include <mutex>

#include "tmap.h"
#include "w4.cuh"

namespace moe {

enum class TileMode { Linear, GateUp, Down };

constexpr int kTileRows = 256;              // rows of x a tile, at most
constexpr int kXStages = 5;                 // of x: 128 k of 128 rows a block, 256 of 64
constexpr int kXBytes = kTileRows * 128;
constexpr int kAStages = 2;                 // of A in tensor memory: 256 k of 128 columns
constexpr int kCStages = 3;                 // of codes: 256 k
constexpr int kCSteps = 4;                  // (in 64 k)
constexpr int kCBytes = 8 * kCSteps * kW4Tile;
constexpr int kSBytes = 2048;               // and their scales, at most
constexpr int kDecWarp0 = 4, kDecWarps = 8, kOutWarp0 = 12, kOutWarps = 8;
constexpr int kTileThreads = 32 * (kOutWarp0 + kOutWarps);
constexpr int kAccCols = 256;               // accumulators: two halves of 128 columns
constexpr int kTileSmem = 1024 + kXStages * kXBytes + kCStages * (kCBytes + kSBytes) +
                          8 * (kMaxExperts + 2) + 512;

struct TileArgs {
  const uint8_t* codes[2];
  const moe_bf16* scales[2];
  int K, N, E;
  const int64_t* offsets;      // NULL: one matrix, T rows
  int64_t T;
  ActParams act;
  void* out;
  int64_t out_stride;
  int out_fp32;
  int splits;                  // Linear: K in so many runs of stages, partial sums in fp32 to
  float* part;                 // part [splits][T][N] where there are several
  int* status;
};

__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem] of both blocks, B's rows half in either
__device__ __forceinline__ void umma_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// a box into this block, counted on a barrier of either (a shared::cluster address)
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void* map, uint32_t bar,
                                                 int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// An arrival at a barrier of either block (a shared::cluster address) that hands over tensor
// memory alone: the warp's accesses there are over (tcgen05.wait) and nothing in
// ordinary memory goes with them, so it needs no release to the cluster, which took 1150 cycles
// a stage (64 rows of 4096 x 38912 47 us).
__device__ __forceinline__ void arrive_for_tmem(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
// untiled copy: 16-byte aligned addresses, size a multiple of 16
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// A bounded wait of one lane that sleeps in the barrier (10 us at a time) instead of taking
// issue slots from the warps that decode; false as mbar_wait_bounded.
static __device__ __noinline__ bool wait_asleep(uint32_t bar, uint32_t parity,
                                                volatile int* abort_flag, int* status) {
  const uint64_t t0 = global_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(10000u)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > (uint64_t)kWaitLimitNs) {
      *abort_flag = 1;
      raise_status(status, MOE_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
}
// For a whole warp: true in all lanes, or (given up) false in all. The loop is out of
// line: the roles' steady state has to stay small.
static __device__ __noinline__ bool wait_slowly_w4(uint32_t bar, uint32_t parity,
                                                   volatile int* abort_flag, int* status) {
  __syncwarp();
  return __all_sync(0xFFFFFFFFu, wait_asleep(bar, parity, abort_flag, status));
}
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                         int* status) {
  // (a phase once seen complete by one lane is complete for every lane that asks later)
  if (__builtin_expect(__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)), 1)) return true;
  return wait_slowly_w4(bar, parity, abort_flag, status);
}
// The same for the warps that wait a whole tile long: they look now and then.
__device__ __forceinline__ bool wait_patiently(uint32_t bar, uint32_t parity,
                                               volatile int* abort_flag, int* status) {
  for (int i = 0; i < 100; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    __nanosleep(200);
  }
  return wait_slowly_w4(bar, parity, abort_flag, status);
}

template <bool B>
struct Bool {
  static constexpr bool value = B;
};

struct Tile {
  int e, n0, rows;
  int kb0, kb1;               // its steps of 64 k
  int sp;
  int64_t m0;
  // the products' columns; of the half of them that a block loads: rows, boxes of 32, and
  // steps of 64 k that fit a stage of x
  __device__ __forceinline__ int cols() const { return (rows + 15) & ~15; }
  __device__ __forceinline__ int half() const { return cols() / 2; }
  __device__ __forceinline__ int boxes() const { return (half() + 31) / 32; }
  __device__ __forceinline__ int per_stage() const { return boxes() > 2 ? 2 : kCSteps; }
};

template <TileMode M, bool FP4, int GPS>
__global__ void __launch_bounds__(kTileThreads, 1)
    w4_tiles_kernel(const __grid_constant__ CUtensorMap mapX, const TileArgs a) {
  pdl_enter();
  constexpr int kWide = M == TileMode::GateUp ? 64 : 128;    // columns n a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint8_t* s_codes = smem + kXStages * kXBytes;
  uint8_t* s_scales = s_codes + kCStages * kCBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_scales + kCStages * kSBytes);
  int* tstart = reinterpret_cast<int*>(bars + 40);
  const uint32_t bar0 = smem_u32(bars);
  auto x_full = [&](int s) { return bar0 + 8u * s; };
  auto x_empty = [&](int s) { return bar0 + 8u * (kXStages + s); };
  auto a_full = [&](int s) { return bar0 + 8u * (2 * kXStages + s); };
  auto a_empty = [&](int s) { return bar0 + 8u * (2 * kXStages + kAStages + s); };
  auto c_full = [&](int s) { return bar0 + 8u * (2 * kXStages + 2 * kAStages + s); };
  auto c_empty = [&](int s) { return bar0 + 8u * (2 * kXStages + 2 * kAStages + kCStages + s); };
  const uint32_t acc_full = bar0 + 8u * (2 * kXStages + 2 * kAStages + 2 * kCStages);
  const uint32_t acc_empty = acc_full + 16, drain = acc_full + 32;       // of either half
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 36);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  static_assert(2 * kXStages + 2 * kAStages + 2 * kCStages + 5 <= 36, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(x_full(s), 1);
      mbar_init(x_empty(s), 1);
    }
    for (int s = 0; s < kAStages; ++s) {
      mbar_init(a_full(s), 2 * kDecWarps);           // of both blocks
      mbar_init(a_empty(s), 1);
    }
    for (int s = 0; s < kCStages; ++s) {
      mbar_init(c_full(s), 1);
      mbar_init(c_empty(s), kDecWarps);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(acc_full + 8 * h, 1);
      mbar_init(acc_empty + 8 * h, 2 * kOutWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapX);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(s_tmem), 512);
    tmem_relinquish_pair();
  }
  const int nN = (a.N + 2 * kWide - 1) / (2 * kWide);         // pairs of tiles
  const int rank = (int)cluster_ctarank(), first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  // tstart[e]: pairs of tiles before expert e; rstart[e]: rows
  int* rstart = tstart + a.E + 1;
  for (int e = threadIdx.x; e < a.E; e += kTileThreads) {
    const int r0 = a.offsets ? (int)a.offsets[e] : 0;
    const int r1 = a.offsets ? (int)a.offsets[e + 1] : (int)a.T;
    rstart[e] = r0;
    if (e == a.E - 1) rstart[a.E] = r1;
    tstart[e + 1] = (r1 - r0 + kTileRows - 1) / kTileRows * nN * a.splits;
  }
  __syncthreads();
  if (warp == 3) {
    int run = 0;
    for (int b = 0; b < a.E; b += 32) {
      const int e = b + lane;
      int v = e < a.E ? tstart[e + 1] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += o;
      }
      if (e < a.E) tstart[e + 1] = run + v;
      run += __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (lane == 0) tstart[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                            // the other block's barriers are there
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int total = tstart[a.E];
  const int kbs = w4_kblocks(a.K), steps = w4_steps(a.K), nbs = w4_nblocks(a.N);

  // whether an expert's scales (of run `half`) take the short form
  auto plain_of = [&](int e, int half) {
    const moe_bf16* p = M == TileMode::GateUp && half ? a.scales[1] : a.scales[0];
    return reinterpret_cast<const uint32_t*>(p + w4_flags_at(a.E, a.K, a.N, 128 / GPS))[e] == 0u;
  };
  auto tile_at = [&](int i) {
    int lo = 0, hi = a.E;                   // the last expert with tstart[lo] <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tstart[mid] <= i) lo = mid; else hi = mid;
    }
    Tile t;
    t.e = lo;
    const int L = rstart[lo + 1] - rstart[lo], chunks = (L + kTileRows - 1) / kTileRows;
    const int size = ((L + 15) / 16 + chunks - 1) / chunks * 16;
    int at = i - tstart[lo];
    t.sp = 0;
    t.kb0 = 0;
    t.kb1 = kbs;
    if (M == TileMode::Linear && a.splits > 1) {
      // whole stages of kCSteps, as even as they go
      const int all = (kbs + kCSteps - 1) / kCSteps;
      t.sp = at % a.splits;
      at /= a.splits;
      t.kb0 = all * t.sp / a.splits * kCSteps;
      t.kb1 = min(kbs, all * (t.sp + 1) / a.splits * kCSteps);
    }
    const int c = at % chunks;
    t.n0 = (at / chunks * 2 + rank) * kWide;
    t.rows = min(size, L - c * size);       // (chunks of up to sixteen sixteens: none is empty)
    t.m0 = rstart[lo] + (int64_t)c * size;
    return t;
  };

  if (warp == 0) {
    // ------------------------------------------------------------- rows of x --
    const bool leader = elect_one();
    const uint32_t x0 = uniform(smem_u32(smem)), full0 = uniform(mapa_shared(bar0, 0));
    int s = 0, fills = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = first; i < total && ok; i += stride) {
      const Tile t = tile_at(i);
      const int boxes = uniform(t.boxes()), per = uniform(t.per_stage());
      const int m0 = uniform((int)t.m0 + rank * t.half());
      for (int ks = t.kb0; ks < t.kb1; ks += per) {
        if (!wait_all(x_empty(s), ph ^ 1u, s_abort, a.status)) {
          ok = false;
          break;
        }
        const uint32_t full = full0 + 8u * s;
        uint32_t dst = x0 + s * kXBytes;
        const int n = min(per, t.kb1 - ks);
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(x_full(s), 2 * n * boxes * 4096);
          for (int k = ks; k < ks + n; ++k)
            for (int b = 0; b < boxes; ++b, dst += 4096)
              tma_load_3d_pair(dst, &mapX, full, k * 64, 0, m0 + 32 * b);
        }
        ++fills;
        if (++s == kXStages) { s = 0; ph ^= 1u; }
      }
    }
    // copies already issued land before the block's shared memory goes away; the second
    // block's are counted in the first, so after a wait that gave up it lets time pass instead
    volatile int never = 0;
    if (rank == 0) {
      for (int n = fills < kXStages ? fills : kXStages; n > 0; --n) {
        if (--s < 0) { s = kXStages - 1; ph ^= 1u; }
        mbar_wait_bounded(x_full(s), ph, &never, a.status);
      }
    } else if (!ok) {
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 200000ull) {
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------ codes and scales --
    // a piece of either run a stage: 64 columns by 256 rows of codes, their scales
    const bool leader = elect_one();
    const uint32_t codes_s = uniform(smem_u32(s_codes)), scales_s = uniform(smem_u32(s_scales));
    const uint32_t full0 = uniform(c_full(0));
    int s = 0, fills = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = first; i < total && ok; i += stride) {
      const Tile t = tile_at(i);
      const int64_t ec = t.e * w4_codes_per_expert(a.K, a.N);
      const int64_t es = t.e * w4_scales_per_expert(a.K, a.N, 128 / GPS);
      // A run of 64 columns is the first or second half of a block of 128, whose tiles of
      // 256 rows lie together: cb of its cw tiles, the first at tile c0 of them.
      int cb[2], c0[2], cw[2];
      const uint8_t* csrc[2];
      const moe_bf16* ssrc[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int nb = t.n0 / 16 + (M == TileMode::GateUp ? 0 : 4 * m);
        const int mat = M == TileMode::GateUp ? m : 0;
        c0[m] = uniform(nb & 7);
        cw[m] = uniform(min(8, nbs - (nb & ~7)));
        cb[m] = uniform(max(0, min(4, nbs - nb)));
        csrc[m] = a.codes[mat] + ec + ((int64_t)(nb & ~7) * kbs + t.kb0 * cw[m]) * kW4Tile;
        ssrc[m] =
            a.scales[mat] + es + ((int64_t)(nb & ~7) * steps + t.kb0 / 2 * cw[m]) * 16 * GPS;
      }
      for (int ks = t.kb0; ks < t.kb1; ks += kCSteps) {
        if (!wait_all(c_empty(s), ph ^ 1u, s_abort, a.status)) {
          ok = false;
          break;
        }
        const int n = t.kb1 - ks < kCSteps ? t.kb1 - ks : kCSteps;
        const uint32_t cbytes = n * kW4Tile, sbytes = (n + 1) / 2 * 32 * GPS;
        const uint32_t full = full0 + 8u * s;
        if (leader) {
          mbar_arrive_expect_tx(full, (cb[0] + cb[1]) * (cbytes + sbytes));
#pragma unroll
          for (int m = 0; m < 2; ++m)
            if (cb[m]) {
              bulk_load(codes_s + s * kCBytes + m * (kCBytes / 2), csrc[m] + c0[m] * cbytes,
                        cb[m] * cbytes, full);
              bulk_load(scales_s + s * kSBytes + m * (kSBytes / 2),
                        ssrc[m] + c0[m] * sbytes / 2, cb[m] * sbytes, full);
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          csrc[m] += cw[m] * cbytes;
          ssrc[m] += cw[m] * sbytes / 2;
        }
        ++fills;
        if (++s == kCStages) { s = 0; ph ^= 1u; }
      }
    }
    volatile int never = 0;
    for (int n = fills < kCStages ? fills : kCStages; n > 0; --n) {
      if (--s < 0) { s = kCStages - 1; ph ^= 1u; }
      mbar_wait_bounded(c_full(s), ph, &never, a.status);
    }
  } else if (warp >= kDecWarp0 && warp < kOutWarp0) {
    // ------------------------------------------------------- codes into bf16 --
    // A stage's stores to tensor memory are waited for when the first values of the next
    // are ready, so that their latency is not the warp's own.
    const int q = warp & 3, half = (warp - kDecWarp0) >> 2;
    const int g = lane >> 2;
    const uint32_t dst0 = tmem + ((uint32_t)(32 * q + 16 * half) << 16) + kAccCols;
    const uint8_t* codes0 = s_codes + half * (kCBytes / 2) + 16 * lane;
    const uint8_t* scales0 =
        s_scales + half * (kSBytes / 2) + g * 4 * GPS;
    const uint32_t full0 = mapa_shared(a_full(0), 0), empty0 = a_empty(0);
    const W4Decoder<FP4> decode;
    int s = 0, cs = 0;
    uint32_t ph = 0, cph = 0;
    bool ok = true, before = false;          // before: the other stage's stores are under way
    auto stored = [&]() {
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_for_tmem(full0 + 8u * (s ^ 1));
    };
    static_assert(kAStages == 2, "the other stage");
    for (int i = first; i < total && ok; i += stride) {
      const Tile t = tile_at(i);
      const bool plain = plain_of(t.e, half);
      // All of the tile's stages of 256 rows, four tiles of codes a warp. (Where the last rows
      // are fewer, some warps decode what lies there; no product reads it.)
      auto stages = [&](auto P) {
        constexpr bool PLAIN = decltype(P)::value;
        for (int ks = t.kb0; ks < t.kb1; ks += kCSteps) {
          if (!wait_all(c_full(cs), cph, s_abort, a.status)) return false;
          const int n = t.kb1 - ks < kCSteps ? t.kb1 - ks : kCSteps;
          const uint8_t* cp = codes0 + cs * kCBytes + q * n * kW4Tile;
          const uint8_t* sp = scales0 + cs * kSBytes + q * ((n + 1) / 2) * 32 * GPS;
#pragma unroll
          for (int sub = 0; sub < 4; ++sub) {
            const uint4 c = *reinterpret_cast<const uint4*>(cp + sub * kW4Tile);
            uint32_t sw[2];                       // of the 64 rows' runs of 32
            const uint8_t* at = sp + (sub >> 1) * 32 * GPS + (sub & 1) * GPS * 2;
            if (GPS == 4) {
              const uint2 v = *reinterpret_cast<const uint2*>(at);
              sw[0] = v.x;
              sw[1] = v.y;
            } else {
              sw[0] = sw[1] = *reinterpret_cast<const uint32_t*>(GPS == 2 ? at : sp + (sub >> 1) * 32);
            }
            uint32_t r[16];
            const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t p[4];
              const uint32_t lo = __byte_perm(sw[j >> 1], 0, 0x1010);
              const uint32_t hi = __byte_perm(sw[j >> 1], 0, 0x3232);
              if (PLAIN)
                decode.scaled(word[j], decode.template factor<0>(lo), decode.template factor<1>(hi),
                              p);
              else
                decode.general(word[j], lo, hi, p);
              r[4 * j + 0] = p[0];
              r[4 * j + 1] = p[2];
              r[4 * j + 2] = p[1];
              r[4 * j + 3] = p[3];
            }
            if (sub == 0) {
              if (before) stored();
              before = false;
              if (!wait_all(empty0 + 8u * s, ph ^ 1u, s_abort, a.status)) return false;
              tc_fence_after();
            }
            tmem_st_16x256b_x4(dst0 + 128 * s + 32 * sub, r);
          }
          before = true;
          s ^= 1;
          if (s == 0) ph ^= 1u;
          if (lane == 0) mbar_arrive(c_empty(cs));
          __syncwarp();
          if (++cs == kCStages) { cs = 0; cph ^= 1u; }
        }
        return true;
      };
      ok = plain ? stages(Bool<true>()) : stages(Bool<false>());
    }
    if (before) stored();
  } else if (warp == 1 && rank == 0) {
    // -------------------------------------------------------------- products --
    // Addresses and descriptors go through a shuffle once, so that they stay in uniform
    // registers: issued by a lane of a divergent branch, a step's eight products took
    // that lane 840 cycles, longer than the decoding.
    const bool leader = elect_one();
    const uint32_t td = uniform(tmem), bars_u = uniform(bar0);
    const uint64_t bd0 = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint32_t b_lo = uniform((uint32_t)bd0), b_hi = uniform((uint32_t)(bd0 >> 32));
    int s = 0, xs = 0, h = 0;
    uint32_t ph = 0, xph = 0, used = 0;      // used: a bit a half of the accumulators, its phase
    bool ok = true;
    for (int i = first; i < total && ok; i += stride) {
      const Tile t = tile_at(i);
      const int N = uniform(t.cols()), per = uniform(t.per_stage());
      const uint32_t step_b = uniform(t.boxes() * (4096 >> 4));
      if (N > 128) {                         // both halves, from the first column on
        h = 0;
        if (!wait_all(acc_empty + 8, (used >> 1 & 1u) ^ 1u, s_abort, a.status)) break;
        used ^= 2u;
      }
      if (!wait_all(acc_empty + 8 * h, (used >> h & 1u) ^ 1u, s_abort, a.status)) break;
      used ^= 1u << h;
      const uint32_t idesc = idesc_bf16(256, N, 0, 0), d = td + 128 * h;
      for (int ks = t.kb0; ks < t.kb1; ks += kCSteps) {
        if (!wait_all(a_full(s), ph, s_abort, a.status)) {
          ok = false;
          break;
        }
        const int n = t.kb1 - ks < kCSteps ? t.kb1 - ks : kCSteps;
        for (int k2 = 0; k2 < n; k2 += per) {
          if (!wait_all(x_full(xs), xph, s_abort, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int m = min(per, n - k2);
          uint32_t at = td + kAccCols + 128 * s + 32 * k2, b = b_lo + xs * (kXBytes >> 4);
          if (leader) {
            for (int j = 0; j < m; ++j, at += 32, b += step_b) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_tmem_a(d, at + 8 * kk, ((uint64_t)b_hi << 32) | (b + kk * (32 >> 4)), idesc,
                            ks + k2 + j > t.kb0 || kk > 0);
            }
            umma_commit_pair(bars_u + 8u * (kXStages + xs), 3);          // x_empty
          }
          if (++xs == kXStages) { xs = 0; xph ^= 1u; }
        }
        if (!ok) break;
        if (leader) umma_commit_pair(bars_u + 8u * (2 * kXStages + kAStages + s), 3);   // a_empty
        if (++s == kAStages) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if (leader) umma_commit_pair(acc_full + 8 * h, 3);
      h = N > 128 ? 0 : h ^ 1;
    }
    // every product has ended before tensor memory is freed
    if (leader) {
      umma_commit_pair(drain, 3);
      volatile int never = 0;
      mbar_wait_bounded(drain, 0, &never, a.status);
    }
  } else if (warp == 1) {
    // the first block's products read and write this one's memory
    volatile int never = 0;
    mbar_wait_bounded(drain, 0, &never, a.status);
  } else if (warp >= kOutWarp0) {
    // --------------------------------------------------------------- results --
    const int q = warp & 3, part = (warp - kOutWarp0) >> 2;
    const uint32_t at = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t given_back = mapa_shared(acc_empty, 0);
    // this lane's column: of the first run (lanes 0-15) or the second
    const bool second = lane >= 16;
    const int col = 16 * q + (lane & 15) + (M != TileMode::GateUp && second ? 64 : 0);
    uint32_t seen = 0;                       // a bit a half: its phase
    int h = 0;
    for (int i = first; i < total; i += stride) {
      const Tile t = tile_at(i);
      const bool wide = t.rows > 128;
      if (wide) h = 0;
      if (!wait_patiently(acc_full + 8 * h, seen >> h & 1u, s_abort, a.status)) break;
      seen ^= 1u << h;
      tc_fence_after();
      const int n = t.n0 + col;
      const float unit = plain_of(t.e, second) ? W4Decoder<FP4>::kScaled : 1.f;
      bool half0 = true;                     // the first 128 columns are still to be given back
      for (int c0 = 16 * part; c0 < t.rows; c0 += 32) {
        uint32_t v[16];
        tmem_ld16(at + 128 * h + c0, v);
        tmem_ld_wait();
        const int64_t stride = M == TileMode::Linear && a.splits > 1 ? a.N : a.out_stride;
        const int64_t first_at = (t.m0 + c0) * stride + n;
        const int here = n < a.N ? t.rows - c0 : 0;          // rows of these sixteen
        if (M == TileMode::GateUp) {
          // of two rows the lower lanes, which hold gates, take the first, the upper ones,
          // which hold the same columns' ups, the second
          moe_bf16* o = static_cast<moe_bf16*>(a.out) + first_at + second * a.out_stride;
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const float mine0 = __uint_as_float(v[c]) * unit, mine1 = __uint_as_float(v[c + 1]) * unit;
            const float got = __shfl_xor_sync(0xFFFFFFFFu, second ? mine0 : mine1, 16);
            const float y = gated(second ? got : mine0, second ? mine1 : got, a.act);
            if (c + second < here) *o = __bfloat16_as_ushort(__float2bfloat16_rn(y));
            o += 2 * a.out_stride;
          }
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float f = __uint_as_float(v[c]) * unit;
            const int64_t o = first_at + c * stride;
            if (c < here) {
              if (M == TileMode::Linear && a.splits > 1)
                a.part[t.sp * a.T * a.N + o] = f;
              else if (M == TileMode::Down || a.out_fp32)
                static_cast<float*>(a.out)[o] = f;
              else
                static_cast<moe_bf16*>(a.out)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(f));
            }
          }
        }
        if (wide && c0 + 32 >= 128 && half0) {
          half0 = false;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_for_tmem(given_back);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (half0) arrive_for_tmem(given_back + 8 * h);
        if (wide) arrive_for_tmem(given_back + 8);
      }
      h = wide ? 0 : h ^ 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                            // no copy or arrival for this block is still to come
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

// -------------------------------------------------------------------- host --
template <TileMode M, bool FP4, int GPS>
static cudaError_t run_tiles(const CUtensorMap& x, const TileArgs& a, bool pdl, cudaStream_t s) {
  const auto kernel = w4_tiles_kernel<M, FP4, GPS>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // as launch_pdl
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // as many clusters as the device holds at a time (a device's blocks are asked for once)
  static int clusters[64] = {};
  static std::mutex mu;
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!clusters[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3((unsigned)(num_sms() & ~1));
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = num_sms() / 2;
      }
      clusters[dev] = n;
    }
    n = clusters[dev];
  }
  cfg.gridDim = dim3((unsigned)(2 * n));
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, x, a);
}

template <TileMode M>
static cudaError_t tiles(const TileArgs& a, const moe_w4& w, const moe_bf16* x, int64_t rows,
                         int64_t stride, bool pdl, cudaStream_t s) {
  CUtensorMap map;
  if (!map_heads(&map, x, a.K, 1, rows, stride, 1, 32)) return cudaErrorInvalidValue;
  const int gps = w4_gps(w.group);
  timer_before(MOE_KERNEL_W4_TILES, s);
  cudaError_t e;
  if (w.kind == MOE_W4_FP4)
    e = gps == 4   ? run_tiles<M, true, 4>(map, a, pdl, s)
        : gps == 2 ? run_tiles<M, true, 2>(map, a, pdl, s)
                   : run_tiles<M, true, 1>(map, a, pdl, s);
  else
    e = gps == 4   ? run_tiles<M, false, 4>(map, a, pdl, s)
        : gps == 2 ? run_tiles<M, false, 2>(map, a, pdl, s)
                   : run_tiles<M, false, 1>(map, a, pdl, s);
  note_launches(1);
  timer_after(MOE_KERNEL_W4_TILES, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// y = the splits' partial sums in order
__global__ void __launch_bounds__(256) w4_join_kernel(const float* __restrict__ part, int splits,
                                                      int64_t T, int N, void* __restrict__ y,
                                                      int64_t stride, int fp32) {
  pdl_enter();
  const int64_t n4 = T * N / 4;               // N is a multiple of 8
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n4) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = 0; j < splits; ++j) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(part) + j * n4 + i);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  const int64_t t = 4 * i / N, n = 4 * i - t * N;
  if (fp32) {
    float* o = static_cast<float*>(y) + t * stride + n;
    o[0] = s.x; o[1] = s.y; o[2] = s.z; o[3] = s.w;
  } else {
    const uint32_t a = pack_bf16(s.x, s.y), b = pack_bf16(s.z, s.w);
    moe_bf16* o = static_cast<moe_bf16*>(y) + t * stride + n;
    o[0] = (moe_bf16)a; o[1] = (moe_bf16)(a >> 16); o[2] = (moe_bf16)b; o[3] = (moe_bf16)(b >> 16);
  }
}

// Runs of K: as many as fill the device once, of at least two stages each (4096 x 2880, 40
// rows: 12 pairs of tiles for 76 clusters, 14.5 us in one run, 11.2 in six; 8192 x 8192, 256
// rows: 32 pairs, 44 us and 30 in two; each before the products of two blocks).
int w4_linear_splits(int64_t T, int K, int N) {
  const int64_t pairs = (int64_t)((N + 255) / 256) * ((T + kTileRows - 1) / kTileRows);
  const int64_t stages = (w4_kblocks(K) + kCSteps - 1) / kCSteps;
  int64_t s = num_sms() / 2 / pairs;
  if (s > stages / 2) s = stages / 2;
  if (s > 8) s = 8;
  return s < 2 ? 1 : (int)s;
}

cudaError_t launch_w4_linear_tiles(const moe_w4& w, const moe_bf16* x, int64_t x_stride, int64_t T,
                                   void* y, int64_t y_stride, int y_fp32, float* part, int* status,
                                   cudaStream_t s) {
  TileArgs a{};
  a.codes[0] = w.codes;
  a.scales[0] = w.scales;
  a.K = w.K;
  a.N = w.N;
  a.E = 1;
  a.T = T;
  a.out = y;
  a.out_stride = y_stride;
  a.out_fp32 = y_fp32;
  a.splits = w4_linear_splits(T, w.K, w.N);
  a.part = part;
  a.status = status;
  cudaError_t e = tiles<TileMode::Linear>(a, w, x, T, x_stride, pdl_for_tokens(T), s);
  if (e == cudaSuccess && a.splits > 1) {
    e = launch_pdl(pdl_for_tokens(T), w4_join_kernel, dim3((unsigned)((T * w.N / 4 + 255) / 256)),
                   dim3(256), 0, s, part, a.splits, T, w.N, y, y_stride, y_fp32);
    note_launches(1);
  }
  return e;
}

cudaError_t launch_w4_experts_tiles(const W4Experts& q, const moe_bf16* xp, const int64_t* offsets,
                                    int64_t R_cap, moe_bf16* A, float* yp, int* status,
                                    cudaStream_t s) {
  const bool pdl = pdl_for_tokens(q.T);
  TileArgs a{};
  a.codes[0] = q.gate->codes;
  a.codes[1] = q.up->codes;
  a.scales[0] = q.gate->scales;
  a.scales[1] = q.up->scales;
  a.K = q.d;
  a.N = q.f;
  a.E = q.E + q.S;
  a.offsets = offsets;
  a.act = q.act;
  a.out = A;
  a.out_stride = q.f;
  a.splits = 1;
  a.status = status;
  cudaError_t e = tiles<TileMode::GateUp>(a, *q.gate, xp, R_cap, q.d, pdl, s);
  a.codes[0] = q.down->codes;
  a.scales[0] = q.down->scales;
  a.K = q.f;
  a.N = q.d;
  a.out = yp;
  a.out_stride = q.d;
  if (e == cudaSuccess) e = tiles<TileMode::Down>(a, *q.down, A, R_cap, q.f, pdl, s);
  return e;
}

}  // namespace moe
