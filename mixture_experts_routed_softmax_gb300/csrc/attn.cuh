// attn.cuh — what the attention kernels share: the batch, the mask as a key
// range per row, and the schedule that cuts the batch's work evenly.
//
// Work units. The G query heads of one key/value head and the n_q new tokens
// of a sequence are n_q * G rows over the same keys: row r is token r / G,
// head h * G + r % G. A unit is (sequence b, head h, row tile m of TM rows);
// its keys are one range (the union of its rows' masks), cut into tiles of TN.
// Units in the order (b, h, m) laid end to end, one step a tile and `cost` steps
// more a unit (beginning and ending one takes about that long), make a line;
// each of n CTAs takes an n-th of it. Every CTA so has the same work
// whatever the lengths, and writes at most two partial results: the unit it
// enters in the middle (slot 0) and the unit it begins and does not end (slot
// 1). A boundary in a unit's first `cost` or last `snap` steps moves to its
// beginning or end: `cost` in long stretches, where it saves a part, one step
// in short ones, where evenness is worth more (kLongStretch). A second launch
// joins the parts of each cut unit in order, so results do not depend on timing.
#pragma once

#include <atomic>

#include "common.cuh"

namespace moe {

constexpr int kAttnMaxD = 128;
constexpr int kAttnMaxKeys = 1 << 30;
// Stretches of so many steps are long. Moving ends by `cost` steps everywhere: 777
// tokens over 2500 keys (8 steps a CTA) 54 us; by one step everywhere: 4 x 2000
// tokens with a window of 512 (66 steps) 159 us; by this rule 50 and 151 us (64
// for the limit: 158 us; 16: 150 us).
constexpr int kLongStretch = 32;

struct AttnBatch {
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t table_stride;
  int64_t n_pages, page_stride, token_stride;
  int T, B, max_pages, page_size;
  uint32_t page_recip;
};

// Divisions by sizes known at run time: the product with ceil(2^32 / d), whose
// high half is the quotient or one more for any 32-bit dividend below 2^31.
// recip 0 stands for d = 1.
inline uint32_t recip_of(int d) {
  return d == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + d - 1) / d);
}
__device__ __forceinline__ int divide_by(int n, int d, uint32_t recip) {
  const uint32_t q = __umulhi((uint32_t)n, recip);
  return recip == 0 ? n : (int)(q * (uint32_t)d > (uint32_t)n ? q - 1 : q);
}
__device__ __forceinline__ int page_of(const AttnBatch& b, int key) {
  return divide_by(key, b.page_size, b.page_recip);
}

inline AttnBatch attn_batch(const moe_kv_cache& c, const moe_kv_batch& b) {
  return AttnBatch{b.cu_q, b.kv_len, b.page_table, b.table_stride, c.n_pages, c.page_stride,
                   c.token_stride, (int)b.T, b.B, b.max_pages, c.page_size, recip_of(c.page_size)};
}

struct AttnArgs {
  AttnBatch bt;
  const moe_bf16* k;
  const moe_bf16* v;
  int64_t head_stride;
  const moe_bf16* q;
  moe_bf16* out;
  int64_t q_stride, out_stride;
  const float* sinks;
  float* lse;
  int Hq, Hkv, G, D;
  uint32_t g_recip;
  float scale_log2;      // scale * log2(e): scores and maxima are kept in powers of two
  int causal, window;    // window 0: none
  int rows_over, rows_upto;   // sequences with rows in (rows_over, rows_upto] take part
  int whole;             // units are not cut: a CTA takes those that begin in its stretch
  int cost;              // steps a unit takes beside its tiles
  int least;             // a stretch has at least so many steps
  int piece;             // tiles whose sums one accumulator takes (unit_next)
  struct Cut* cuts;      // [CTAs] the cut in front of each
  float* part_o;         // [2 * CTAs (or groups)][TM][DP] unnormalised partial outputs
  float2* part_ml;       // [2 * CTAs (or groups)][TM] their (max, sum)
  int* status;
};

__device__ __forceinline__ int div_group(const AttnArgs& a, int row) {
  return divide_by(row, a.G, a.g_recip);
}

// ------------------------------------------------------------- the batch --
// The sequence row t belongs to: the number of sequences that end at or
// before t. Called by a whole warp; 32 ends are looked at a step. -1: none.
__device__ __forceinline__ int find_sequence(const int32_t* cu_q, int B, int t, int lane) {
  int lo = 0, end = B;      // the answer lies in [lo, end]
  while (lo < end) {
    const int step = (end - lo + 31) >> 5;
    const int64_t last = (int64_t)lo + (int64_t)(lane + 1) * step - 1;
    const bool past = last < end && cu_q[last + 1] <= t;
    const int full = __popc(__ballot_sync(0xFFFFFFFFu, past));
    lo += full * step;
    // the first group not wholly past: its last sequence is known to end later
    if (full < 32 && lo + step - 1 < end) end = lo + step - 1;
    if (step == 1) break;
  }
  return lo < B ? lo : -1;
}

struct Seq {
  int q0, nq, n;     // first row, new tokens, keys
};
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  const int s = a.bt.cu_q[b], e = a.bt.cu_q[b + 1];
  int n = a.bt.kv_len[b];
  const int cap = a.bt.max_pages * a.bt.page_size;
  Seq q{s, e - s, n};
  const bool bad_rows = s < 0 || e < s || e > a.bt.T;
  if (bad_rows || n < 0 || n > cap) raise_status(a.status, MOE_ERR_DEVICE_INDEX);
  q.n = min(max(n, 0), cap);
  if (bad_rows) q.nq = 0;
  const int rows = q.nq * a.G;
  if (rows <= a.rows_over || rows > a.rows_upto) q.nq = 0;
  return q;
}

// ---------------------------------------------------------------- the mask --
// Token i of a sequence sees keys [key_lo, key_hi).
__device__ __forceinline__ int key_hi(const AttnArgs& a, const Seq& s, int i) {
  if (!a.causal) return s.n;
  const int c = s.n - s.nq + i;
  return c < 0 ? 0 : c + 1;       // c < n always
}
__device__ __forceinline__ int key_lo(const AttnArgs& a, const Seq& s, int i) {
  if (a.window == 0) return 0;
  const int c = s.n - s.nq + i - a.window + 1;
  return c < 0 ? 0 : c;
}

template <int TM, int TN>
struct Tiling {
  static __device__ __forceinline__ int row_tiles(const AttnArgs& a, const Seq& s) {
    return (s.nq * a.G + TM - 1) / TM;
  }
  // key range and tiles of row tile m
  struct Span {
    int lo, hi, t0, nt;
  };
  static __device__ __forceinline__ Span span(const AttnArgs& a, const Seq& s, int m) {
    const int rows = s.nq * a.G;
    const int r0 = m * TM;
    const int r1 = min(r0 + TM, rows) - 1;
    Span p;
    p.lo = key_lo(a, s, div_group(a, r0));
    p.hi = key_hi(a, s, div_group(a, r1));
    if (p.hi <= p.lo) {
      p.lo = p.hi = p.t0 = p.nt = 0;
    } else {
      p.t0 = p.lo / TN;
      p.nt = (p.hi + TN - 1) / TN - p.t0;
    }
    return p;
  }
  static __device__ __forceinline__ int weight(const AttnArgs& a, const Seq& s, int m) {
    return span(a, s, m).nt + a.cost;
  }
};

// ------------------------------------------------------------ the schedule --
// All of it runs once a unit or less and is kept out of line: what a warp's
// steady state executes has to fit the instruction cache.
// a / b of values that nearly always fit 32 bits
static __device__ __noinline__ long long divide_long(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (__builtin_expect(((a | b) >> 32) == 0, 1)) return (long long)((uint32_t)a / (uint32_t)b);
  return divide_long(a, b);
}
struct Line {               // the line of steps, cut for n CTAs (or fewer, of a least length)
  long long total, per;     // per = total / n; the first `rem` CTAs take one more
  int n, rem;
  __device__ __forceinline__ Line(long long total_, int ctas, int least)
      : total(total_), per(divide(total_, ctas)), n(ctas) {
    if (per < least) {
      n = max(1, (int)divide(total, least));
      per = divide(total, n);
    }
    rem = (int)(total - per * n);
  }
  __device__ __forceinline__ long long start(int cta) const {
    return cta >= n ? total : per * cta + (cta < rem ? cta : rem);
  }
};
struct Place {              // locate's, in shared memory
  long long warp_sum[32];
  struct {
    long long in_seq, x0, x1, prev, per;
    int rem, tall;          // tall: the sequence found has several row tiles
  } at[4];                  // of each stretch of the block
};
// What a join block needs of the cut in front of a CTA: a unit's rows and the
// CTAs first .. last - 1 that have parts of it. first < 0: no cut to join there.
struct alignas(32) Cut {
  int q0, r0, nrows, h, first, last, pad[2];
};

// A unit of a CTA's stretch, in shared memory: written by one thread, read by
// those that work on it.
struct Unit {
  long long to_end;    // steps from the unit's first to the end of the stretch
  Seq s;
  int more;            // 0: the stretch has no further unit
  int snap;
  int b, h, m, nm;
  int w, off, stop;    // the unit's steps; this CTA has [off, stop) of them
  int lo, hi;          // the keys of its rows
  int all_lo, all_hi;  // those every row sees
  int t0, nt;          // tiles: the first, and this CTA's number of them (of the piece)
  int begun, rest;     // pieces of the CTA's part: whether one came before, tiles that follow

  __device__ __forceinline__ bool whole() const { return off == 0 && stop == w; }
  __device__ __forceinline__ int slot() const { return off > 0 ? 0 : 1; }
};

// Steps of one head of the sequence of each lane (0 for nq = 0). A lane with
// many row tiles gets its warp's help.
template <int TM, int TN>
__device__ __forceinline__ long long head_weight(const AttnArgs& a, const Seq& s) {
  using TL = Tiling<TM, TN>;
  const int lane = threadIdx.x & 31;
  const int nm = s.nq > 0 ? TL::row_tiles(a, s) : 0;
  long long w = 0;
  if (nm == 1) w = TL::weight(a, s, 0);
  uint32_t big = __ballot_sync(0xFFFFFFFFu, nm > 1);
  while (big) {
    const int src = __ffs(big) - 1;
    big &= big - 1;
    Seq t;
    t.q0 = 0;
    t.nq = __shfl_sync(0xFFFFFFFFu, s.nq, src);
    t.n = __shfl_sync(0xFFFFFFFFu, s.n, src);
    const int tm = __shfl_sync(0xFFFFFFFFu, nm, src);
    long long part = 0;
    for (int m = lane; m < tm; m += 32) part += TL::weight(a, t, m);
#pragma unroll
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
    if (lane == src) w = part;
  }
  return w;
}

// The unit (u.s, u.h, u.m) from step u.off on, for as far as the stretch goes.
template <int TM, int TN>
__device__ __forceinline__ void unit_set(const AttnArgs& a, Unit& u) {
  const typename Tiling<TM, TN>::Span sp = Tiling<TM, TN>::span(a, u.s, u.m);
  u.w = sp.nt + a.cost;
  u.stop = u.w;
  if (!a.whole && u.to_end < u.w) {
    const int e = (int)u.to_end;
    if (e <= a.cost) {
      u.more = 0;
      return;
    }
    if (u.w - e > u.snap) u.stop = e;
  }
  u.more = 1;
  u.lo = sp.lo;
  u.hi = sp.hi;
  const int rows = u.s.nq * a.G;
  u.all_lo = key_lo(a, u.s, div_group(a, min(u.m * TM + TM, rows) - 1));
  u.all_hi = key_hi(a, u.s, div_group(a, u.m * TM));
  const int begin = max(u.off - a.cost, 0), nt = max(u.stop - a.cost, 0) - begin;
  u.t0 = sp.t0 + begin;
  u.nt = min(nt, a.piece);
  u.rest = nt - u.nt;
  u.begun = 0;
}
// The next unit, or the next piece of a long one. The matrix units cut what they add
// to an accumulator at its last place, by up to 2^-23 of the sum each time, and this
// adds up: a mean of values of one sign came out 0.5% low after 2^16 steps of 16
// keys in one accumulator, 2.6% after 2^18. So a unit is worked on in pieces of
// `piece` tiles; a piece's sums go where the CTA's part of the unit would, and the
// next one's join them in fp32.
template <int TM, int TN>
__device__ __forceinline__ void unit_next(const AttnArgs& a, Unit& u) {
  if (u.rest > 0) {
    u.t0 += u.nt;
    u.nt = min(u.rest, a.piece);
    u.rest -= u.nt;
    u.begun = 1;
    return;
  }
  u.to_end -= u.w;
  u.more = 0;
  if (u.stop < u.w || u.to_end <= 0) return;
  u.off = 0;
  if (++u.m == u.nm) {
    u.m = 0;
    if (++u.h == a.Hkv) {
      u.h = 0;
      int nm = 0, b = u.b;
      Seq s{0, 0, 0};
      while (nm == 0 && ++b < a.bt.B) {
        s = load_seq(a, b);
        nm = Tiling<TM, TN>::row_tiles(a, s);
      }
      if (nm == 0) return;      // lengths that changed under the kernel
      u.b = b;
      u.s = s;
      u.nm = nm;
    }
  }
  unit_set<TM, TN>(a, u);
}
// The stretch's first unit, from the unit (u.s, b, h, m, nm) its first step x0
// lies in, `off` steps into it; and the cut in front of the stretch.
template <int TM, int TN>
__device__ __noinline__ void unit_first(const AttnArgs& a, const Place& place, int k, int cta,
                                        int off, Unit& u) {
  const auto& pl = place.at[k];
  Cut c{0, 0, 0, 0, -1, 0, {0, 0}};
  const long long unit0 = pl.x0 - off;
  u.to_end = pl.x1 - unit0;
  u.rest = 0;
  u.w = u.stop = Tiling<TM, TN>::weight(a, u.s, u.m);
  const bool at_begin = a.whole ? off == 0 : off <= a.cost;
  const bool at_end = a.whole || u.w - off <= u.snap;
  if (at_begin) {
    u.off = 0;
    unit_set<TM, TN>(a, u);
  } else if (at_end) {
    unit_next<TM, TN>(a, u);
  } else {
    u.off = off;
    if (pl.prev - unit0 <= a.cost) {
      // the first cut of its unit; the last part is that of the CTA that has the
      // step the end's boundary is measured from
      const long long y = unit0 + u.w - u.snap - 1, big = (long long)pl.rem * (pl.per + 1);
      c.first = cta - 1;
      c.last = 1 + (int)(y < big ? divide(y, pl.per + 1) : pl.rem + divide(y - big, pl.per));
      c.q0 = u.s.q0;
      c.h = u.h;
      c.r0 = u.m * TM;
      c.nrows = min(TM, u.s.nq * a.G - c.r0);
    }
    unit_set<TM, TN>(a, u);
  }
  if (a.cuts) a.cuts[cta] = c;
}

// Stretches cta .. cta + K - 1 of `n` (one a CTA, or one a warp of its own units):
// the first unit of stretch cta + k into u[k * pitch], and the cut in front of it
// into a.cuts. By the whole block of NT threads; ends with a barrier.
template <int TM, int TN, int NT, int K = 1>
__device__ __noinline__ void locate(const AttnArgs& a, int cta, int n, Place& pl, Unit* us,
                                    int pitch) {
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.bt.B;
  // The line's length, then the sequence that holds the CTA's first step. Up to
  // NT sequences, one a thread, the second pass looks at what the first has; the
  // thread that finds a sequence of one row tile has all the unit takes.
  Seq s{0, 0, 0};
  long long total = 0, hw = 0, inc = 0, before = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += NT) {
      const int b = b0 + tid;
      if (pass == 0 || B > NT) {
        s = Seq{0, 0, 0};
        if (b < B) s = load_seq(a, b);
        hw = head_weight<TM, TN>(a, s);
        inc = hw * a.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
          if (lane >= o) inc += up;
        }
        __syncthreads();
        if (lane == 31) pl.warp_sum[warp] = inc;
        __syncthreads();
        before = 0;
        long long all = 0;
#pragma unroll 1
        for (int i = 0; i < NW; ++i) {
          const long long v = pl.warp_sum[i];
          if (i < warp) before += v;
          all += v;
        }
        total = base + all;
      }
      if (pass == 1) {
        const long long hi = base + before + inc, lo = hi - hw * a.Hkv;
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
          const long long x0 = pl.at[k].x0;
          if (x0 < lo || x0 >= hi) continue;
          Unit& u = us[k * pitch];
          u.s = s;
          u.b = b;
          u.nm = Tiling<TM, TN>::row_tiles(a, s);
          u.h = (int)divide(x0 - lo, hw);
          pl.at[k].in_seq = x0 - lo - u.h * hw;
          pl.at[k].tall = u.nm > 1;
          if (u.nm == 1) {
            u.m = 0;
            unit_first<TM, TN>(a, pl, k, cta + k, (int)pl.at[k].in_seq, u);
          }
        }
      }
      base = total;
    }
    if (pass == 0) {
      const Line ln(total, n, a.least);
      if (tid < K) {
        auto& at = pl.at[tid];
        const int c = cta + tid;
        at.x0 = ln.start(c);
        at.x1 = ln.start(c + 1);
        at.prev = c > 0 ? ln.start(c - 1) : 0;
        at.per = ln.per;
        at.rem = ln.rem;
        at.tall = 0;
        us[tid * pitch].more = 0;
        us[tid * pitch].snap = ln.per >= kLongStretch ? a.cost : 1;
        // a start at the line's end: no steps
        if (at.x0 >= total && a.cuts) a.cuts[c] = Cut{0, 0, 0, 0, -1, 0, {0, 0}};
      }
      __syncthreads();
      if (pl.at[0].x0 >= total) return;      // nor for the stretches after it
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    if (!pl.at[k].tall) continue;
    if (warp == 0) {
      // which of the sequence's row tiles
      Unit& u = us[k * pitch];
      const Seq t = u.s;
      const int nm = u.nm;
      long long rem = pl.at[k].in_seq;
#pragma unroll 1
      for (int m0 = 0; m0 < nm; m0 += 32) {
        const int m = m0 + lane;
        const int w = m < nm ? Tiling<TM, TN>::weight(a, t, m) : 0;
        long long run = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long up = __shfl_up_sync(0xFFFFFFFFu, run, o);
          if (lane >= o) run += up;
        }
        const bool here = rem >= run - w && rem < run;
        if (here) {
          u.m = m;
          unit_first<TM, TN>(a, pl, k, cta + k, (int)(rem - (run - w)), u);
        }
        if (__any_sync(0xFFFFFFFFu, here)) break;
        rem -= __shfl_sync(0xFFFFFFFFu, run, 31);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------- asynchronous copies --
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
  const int n = full ? 16 : 0;       // 0: the destination is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ host --
// Raises a kernel's shared-memory limit on the current device, once per device.
struct SmemOnce {
  std::atomic<uint64_t> done{0};
  cudaError_t set(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_release);
    return e;
  }
};

// ------------------------------------------------------------- arithmetic --
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float neg_inf() { return __int_as_float((int)0xFF800000); }
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kLog2e = 1.44269504088896340736f;

// A row's (max, sum) with its sink joined, the factor its accumulator takes and
// its log-sum-exp. A row without keys (l = 0) gets factor 0.
struct RowEnd {
  float factor, lse;
};
__device__ __forceinline__ RowEnd row_end(float m, float l, const float* sinks, int head) {
  float f = 1.f;
  if (sinks) {
    const float s2 = sinks[head] * kLog2e;
    const float mt = fmaxf(m, s2);
    const float ref = mt == neg_inf() ? 0.f : mt;
    f = ex2(m - ref);
    l = l * f + ex2(s2 - ref);
    m = mt;
  }
  RowEnd e;
  e.factor = l == 0.f ? 0.f : f / l;
  e.lse = l == 0.f ? neg_inf() : m * kLn2 + logf(l);
  return e;
}

// attn_chunk.cu
bool attn_chunk_boxes(int page_size);      // keys by TMA; else by 16-byte copies
size_t attn_chunk_ws_bytes(int D);
cudaError_t launch_attn_chunk(const AttnArgs& a, const moe_kv_cache& c, void* ws, cudaStream_t s);

}  // namespace moe
