// w4_rows.cu — products of a few rows with 4-bit weights (layout: w4.cuh): one
// linear layer, and the experts' gate/up and down products of a few tokens.
//
//   out[r, n] = sum_k x[r, k] value(code[k, n]) scale[k / group, n]
//
// Bound by reading the codes (half a byte a weight). Each weight is read once and
// used for 8 NT rows: the codes are the A operand of m16n8k16 products, 16 columns n
// by 16 k straight from 16-byte loads without shared memory (w4.cuh), the rows of x are
// the B operand, eight rows a product. The values go in exactly (int4's as 2^-13 of them, given
// back at the end: a scale times 2^13 would leave fp32's range from 2^115 on); a group's partial
// sum is multiplied by its scale in fp32, so any scale is exact too.
//
// A block of eight warps takes RB blocks of 16 columns (of one matrix, or of gate
// and up together) of one expert, for all of that expert's rows, 8 NT at a time;
// its warps share the steps of 128 k, and their sums meet in shared memory in warp
// order. There is no list of rows made beforehand: a block looks through the
// tokens' choices itself (up to kRowsMaxPairs of them), which costs less than a launch.
#include "w4.cuh"

namespace moe {

constexpr int kRowWarps = 8;
constexpr int kRowThreads = 32 * kRowWarps;

enum class RowsMode { Linear, GateUp, Down };

struct RowsArgs {
  const uint8_t* codes[2];
  const moe_bf16* scales[2];
  int K, N;
  const moe_bf16* x;
  int64_t x_stride;
  const int32_t* idx;         // [T*k] chosen experts; NULL: one matrix, every row
  int64_t T;
  int k, E, S;
  int by_pair;                // blockIdx.y: a pair (works if it is its expert's first), or an expert
  ActParams act;
  void* out;                  // bf16 A [pairs, N]; fp32 Yp [pairs, N]; y [T, N]
  int64_t out_stride;
  int out_fp32;
  int64_t lo;                 // 0, or where A's second halves stand behind the first (in elements)
  int* status;
};

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The rows of expert e among the choices, in ascending order, into list; returns how
// many. Every thread of the block calls it; P <= kRowsMaxPairs.
__device__ __forceinline__ int list_rows(const int32_t* __restrict__ idx, int P, int E, int e,
                                         int* list, int* warp_n, bool check, int* status) {
  constexpr int kSegs = kRowsMaxPairs / kRowThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = (P + kRowThreads - 1) / kRowThreads;     // ballots a warp takes
  uint32_t found[kSegs];
  int n = 0;
#pragma unroll
  for (int i = 0; i < kSegs; ++i) {
    found[i] = 0;
    if (i < seg) {
      const int p = (warp * seg + i) * 32 + lane;
      const int id = p < P ? idx[p] : -2;
      if (check && p < P && (id < 0 || id >= E)) raise_status(status, MOE_ERR_DEVICE_INDEX);
      found[i] = __ballot_sync(0xFFFFFFFFu, p < P && id == e);
      n += __popc(found[i]);
    }
  }
  if (lane == 0) warp_n[warp] = n;
  __syncthreads();
  int at = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    const int c = warp_n[w];
    if (w < warp) at += c;
    total += c;
  }
#pragma unroll
  for (int i = 0; i < kSegs; ++i) {
    if (i < seg) {
      if ((found[i] >> lane) & 1u)
        list[at + __popc(found[i] & ((1u << lane) - 1u))] = (warp * seg + i) * 32 + lane;
      at += __popc(found[i]);
    }
  }
  __syncthreads();
  return total;
}

// Blocks an SM that registers are cut for. A linear layer's few blocks want the loads of
// several steps on their way (one row of 8192 x 8192: 13.8 -> 12.1 us, of 2048 x 2048 3.2 -> 2.5);
// the experts' many want more of them at a time (the same bound took 16 tokens through
// 128 experts from 69 to 100 us), as the compiler cuts them, but two blocks of gate and up at
// least (one: 16 tokens 78 -> 96 us, 64 tokens 116 -> 144).
constexpr int rows_blocks(RowsMode m, int nt, int rb) {
  return m == RowsMode::Linear && nt == 1   ? (rb == 2 ? 3 : 1)
         : m == RowsMode::GateUp && nt == 1 && rb == 2 ? 2
                                                       : 0;
}

template <RowsMode M, bool FP4, int GPS, int NT, int RB>
__global__ void __launch_bounds__(kRowThreads, rows_blocks(M, NT, RB)) w4_rows_kernel(RowsArgs a) {
  constexpr int MATS = M == RowsMode::GateUp ? 2 : 1;
  constexpr int R = RB * MATS;                 // 16-column tiles a warp works on
  constexpr int CP = 8 * NT + 2;               // padded columns of the sums in shared memory
  extern __shared__ float red[];               // [warps][R][16][CP]
  __shared__ int list[M == RowsMode::Linear ? 1 : kRowsMaxPairs];
  __shared__ int warp_n[kRowWarps];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  int e = 0;
  int64_t rows = a.T;
  const int64_t P = a.T * a.k;
  int64_t shared_base = 0;                     // of a shared expert: the pair of token 0
  bool shared = M == RowsMode::Linear;
  if (M != RowsMode::Linear) {
    const int y = blockIdx.y, routed = a.by_pair ? (int)P : a.E;
    if (y >= routed) {
      e = a.E + y - routed;
      shared = true;
      shared_base = P + (int64_t)(y - routed) * a.T;
    } else {
      e = a.by_pair ? a.idx[y] : y;
      if (e < 0 || e >= a.E) {
        if (threadIdx.x == 0) raise_status(a.status, MOE_ERR_DEVICE_INDEX);
        return;
      }
      rows = list_rows(a.idx, (int)P, a.E, e, list, warp_n, y == 0 && blockIdx.x == 0, a.status);
      if (rows == 0 || (a.by_pair && list[0] != y)) return;
    }
  }
  const W4Decoder<FP4> decode;
  const int kbs = w4_kblocks(a.K), steps = w4_steps(a.K);
  const int nb0 = blockIdx.x * RB, nbs = w4_nblocks(a.N);
  const uint8_t* codes[MATS];
  const moe_bf16* scales[MATS];
#pragma unroll
  for (int m = 0; m < MATS; ++m) {
    codes[m] = a.codes[m] + e * w4_codes_per_expert(a.K, a.N) + 16 * lane;
    scales[m] = a.scales[m] + e * w4_scales_per_expert(a.K, a.N, 128 / GPS) + 2 * GPS * g;
  }
  // Down: a row of A as one or two columns of the product (divided by, not shifted by: the same
  // with shifts got other registers, and 16 tokens through 128 experts took 87 us instead of 71)
  const int per = M == RowsMode::Down && a.lo ? 2 : 1;
  rows *= per;
  for (int64_t r0 = 0; r0 < rows; r0 += 8 * NT) {
    const moe_bf16* xr[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int64_t r = r0 + 8 * nt + g;
      xr[nt] = nullptr;
      if (r < rows) {
        int64_t row = r;
        if (M == RowsMode::GateUp && !shared) row = list[r] / a.k;
        if (M == RowsMode::Down) row = shared ? shared_base + r / per : list[r / per];
        xr[nt] = a.x + row * a.x_stride;
        if (M == RowsMode::Down && (r & (per - 1))) xr[nt] += a.lo;
      }
    }
    float acc[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        acc[r][nt][0] = acc[r][nt][1] = acc[r][nt][2] = acc[r][nt][3] = 0.f;
    for (int step = warp; step < steps; step += kRowWarps) {
      uint4 cw[R][2];
      uint32_t sw[R][GPS];
      const bool second = 2 * step + 1 < kbs;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int nb = nb0 + r / MATS, m = r % MATS;
        const uint32_t zero = FP4 ? 0u : 0x88888888u;
        cw[r][0] = cw[r][1] = make_uint4(zero, zero, zero, zero);
#pragma unroll
        for (int q = 0; q < GPS; ++q) sw[r][q] = 0u;
        if (nb < nbs) {
          const uint8_t* src = codes[m] + w4_tile_at(nb, 2 * step, nbs, kbs);
          cw[r][0] = ldg_stream(src);
          if (second) cw[r][1] = ldg_stream(src + kW4Tile);
          const uint32_t* sp = reinterpret_cast<const uint32_t*>(
              scales[m] + w4_scales_at(nb, step, nbs, steps, GPS));
          if (GPS == 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(sp));
            sw[r][0] = v.x; sw[r][1 % GPS] = v.y; sw[r][2 % GPS] = v.z; sw[r][3 % GPS] = v.w;
          } else if (GPS == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp));
            sw[r][0] = v.x; sw[r][1 % GPS] = v.y;
          } else {
            sw[r][0] = __ldg(sp);
          }
        }
      }
      uint2 xv[NT][8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const int k = 128 * step + 16 * h + 4 * t;
          xv[nt][h] = make_uint2(0u, 0u);
          if (xr[nt] && k < a.K) xv[nt][h] = *reinterpret_cast<const uint2*>(xr[nt] + k);
        }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float part[NT][4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (h % (4 / GPS) == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              part[nt][0] = part[nt][1] = part[nt][2] = part[nt][3] = 0.f;
          }
          const uint4 c = cw[r][h >> 1];
          uint32_t av[4];
          decode.values((h & 1) ? c.z : c.x, av);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(part[nt], av, xv[nt][2 * h].x, xv[nt][2 * h].y);
          decode.values((h & 1) ? c.w : c.y, av);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(part[nt], av, xv[nt][2 * h + 1].x, xv[nt][2 * h + 1].y);
          if (h % (4 / GPS) == 4 / GPS - 1) {
            const uint32_t s = sw[r][h / (4 / GPS)];
            const float lo = bf16_lo(s), hi = bf16_hi(s);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              acc[r][nt][0] = fmaf(lo, part[nt][0], acc[r][nt][0]);
              acc[r][nt][1] = fmaf(lo, part[nt][1], acc[r][nt][1]);
              acc[r][nt][2] = fmaf(hi, part[nt][2], acc[r][nt][2]);
              acc[r][nt][3] = fmaf(hi, part[nt][3], acc[r][nt][3]);
            }
          }
        }
      }
    }
    // the warps' sums
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* o = red + ((warp * R + r) * 16 + g) * CP + 8 * nt + 2 * t;
        *reinterpret_cast<float2*>(o) = make_float2(acc[r][nt][0], acc[r][nt][1]);
        *reinterpret_cast<float2*>(o + 8 * CP) = make_float2(acc[r][nt][2], acc[r][nt][3]);
      }
    __syncthreads();
    const int here = (int)(rows - r0 < 8 * NT ? rows - r0 : 8 * NT);
    for (int o = threadIdx.x; o < RB * 16 * (here / per); o += kRowThreads) {
      const int nl = o % (RB * 16), c = o / (RB * 16) * per;
      const int n = nb0 * 16 + nl;
      if (n >= a.N) continue;
      float sum[MATS];
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        sum[m] = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w)
          sum[m] += red[((w * R + (nl / 16) * MATS + m) * 16 + nl % 16) * CP + c];
        if (per == 2) {
#pragma unroll
          for (int w = 0; w < kRowWarps; ++w)
            sum[m] += red[((w * R + (nl / 16) * MATS + m) * 16 + nl % 16) * CP + c + 1];
        }
        sum[m] *= decode.kUnit;
      }
      const int64_t r = (r0 + c) / per;
      if (M == RowsMode::Linear) {
        const int64_t at = r * a.out_stride + n;
        if (a.out_fp32)
          static_cast<float*>(a.out)[at] = sum[0];
        else
          static_cast<moe_bf16*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(sum[0]));
      } else {
        const int64_t at = (shared ? shared_base + r : (int64_t)list[r]) * a.N + n;
        if (M == RowsMode::GateUp) {
          const float v = gated(sum[0], sum[MATS - 1], a.act);
          const __nv_bfloat16 hi = __float2bfloat16_rn(v);
          static_cast<moe_bf16*>(a.out)[at] = __bfloat16_as_ushort(hi);
          // (what is not finite has no rest)
          if (a.lo) {
            const float rest = v - __bfloat162float(hi);
            static_cast<moe_bf16*>(a.out)[at + a.lo] =
                __bfloat16_as_ushort(__float2bfloat16_rn(rest - rest == 0.f ? rest : 0.f));
          }
        } else {
          static_cast<float*>(a.out)[at] = sum[0];
        }
      }
    }
    __syncthreads();
  }
}

// One token's down products and their weighted sum over its experts in one go: a block takes
// 16 columns of all of them, its warps the steps of 128 k of expert after expert, four
// at a time so that 4 KB a warp are on their way. y [d], rows A by slot (k choices, S shared).
template <bool FP4, int GPS>
__global__ void __launch_bounds__(kRowThreads) w4_token_kernel(RowsArgs a,
                                                               const float* __restrict__ w) {
  constexpr int U = 4;
  __shared__ float red[kRowWarps][16];
  __shared__ int expert[32];
  __shared__ float weight[32];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int slots = a.k + a.S;
  if (threadIdx.x < slots) {
    const int j = threadIdx.x;
    const int id = j < a.k ? a.idx[j] : a.E + j - a.k;
    // (an id out of range is reported by the gate/up products; its weight, which may be
    // anything, does not meet the sum)
    const bool out = j < a.k && (id < 0 || id >= a.E);
    expert[j] = out ? -1 : id;
    weight[j] = out ? 0.f : j < a.k ? w[j] : 1.f;
  }
  __syncthreads();
  const W4Decoder<FP4> decode;
  const int kbs = w4_kblocks(a.K), steps = w4_steps(a.K), nbs = w4_nblocks(a.N), nb = blockIdx.x;
  float acc[4] = {};
  for (int u0 = warp * U; u0 < slots * steps; u0 += kRowWarps * U) {
    uint4 cw[U][2];
    uint32_t sw[U][GPS];
    uint2 xv[U][8];
    float f[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int slot = min((u0 + i) / steps, slots - 1), step = (u0 + i) - slot * steps;
      const int id = step < steps ? expert[slot] : -1;
      f[i] = weight[slot];
      const uint32_t zero = FP4 ? 0u : 0x88888888u;
      cw[i][0] = cw[i][1] = make_uint4(zero, zero, zero, zero);
#pragma unroll
      for (int q = 0; q < GPS; ++q) sw[i][q] = 0u;
      if (id >= 0) {
        const uint8_t* src = a.codes[0] + id * w4_codes_per_expert(a.K, a.N) +
                             w4_tile_at(nb, 2 * step, nbs, kbs) + 16 * lane;
        cw[i][0] = ldg_stream(src);
        if (2 * step + 1 < kbs) cw[i][1] = ldg_stream(src + kW4Tile);
        const uint32_t* sp = reinterpret_cast<const uint32_t*>(
            a.scales[0] + id * w4_scales_per_expert(a.K, a.N, 128 / GPS) +
            w4_scales_at(nb, step, nbs, steps, GPS) + 2 * GPS * g);
#pragma unroll
        for (int q = 0; q < GPS; ++q) sw[i][q] = __ldg(sp + q);
      }
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const int k = 128 * step + 16 * h + 4 * t;
        xv[i][h] = make_uint2(0u, 0u);
        // columns 0 and 1 of the product's B operand, the others stay zeros
        if (id >= 0 && g < 2 && k < a.K)
          xv[i][h] = *reinterpret_cast<const uint2*>(a.x + slot * a.x_stride + g * a.lo + k);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float part[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        if (h % (4 / GPS) == 0) part[0] = part[1] = part[2] = part[3] = 0.f;
        const uint4 c = cw[i][h >> 1];
        uint32_t av[4];
        decode.values((h & 1) ? c.z : c.x, av);
        mma16816(part, av, xv[i][2 * h].x, xv[i][2 * h].y);
        decode.values((h & 1) ? c.w : c.y, av);
        mma16816(part, av, xv[i][2 * h + 1].x, xv[i][2 * h + 1].y);
        if (h % (4 / GPS) == 4 / GPS - 1) {
          const uint32_t s = sw[i][h / (4 / GPS)];
          acc[0] = fmaf(f[i], bf16_lo(s) * (part[0] + part[1]), acc[0]);
          acc[2] = fmaf(f[i], bf16_hi(s) * (part[2] + part[3]), acc[2]);
        }
      }
    }
  }
  if (t == 0) {                              // columns 0 and 1: this token
    red[warp][g] = acc[0];
    red[warp][g + 8] = acc[2];
  }
  __syncthreads();
  const int n = nb * 16 + (int)threadIdx.x;
  if (threadIdx.x < 16 && n < a.N) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) sum += red[i][threadIdx.x];
    static_cast<moe_bf16*>(a.out)[n] = __bfloat16_as_ushort(__float2bfloat16_rn(sum * decode.kUnit));
  }
}

// y[t] = sum_j w[t, j] Yp[t k + j] + the shared experts' rows, in slot order; a pair
// whose expert is out of range is left out. A warp takes 256 columns of a token.
__global__ void __launch_bounds__(256) w4_combine_kernel(
    const float* __restrict__ yp, const int32_t* __restrict__ idx, const float* __restrict__ w,
    int64_t T, int k, int E, int S, int d, moe_bf16* __restrict__ y) {
  pdl_enter();
  const int lane = threadIdx.x & 31, nv = d / 8, nchunk = (nv + 31) / 32;
  const int64_t wid = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  if (wid >= T * nchunk) return;
  const int64_t t = wid / nchunk;
  const int v = (int)(wid - t * nchunk) * 32 + lane;
  int ok = 0;
  float wj = 1.f;
  if (lane < k) {
    const int e = idx[t * k + lane];
    ok = e >= 0 && e < E;
    wj = w[t * k + lane];
  } else if (lane < k + S) {
    ok = 1;
  }
  float acc[8] = {};
#pragma unroll 4
  for (int j = 0; j < k + S; ++j) {
    const int okj = __shfl_sync(0xFFFFFFFFu, ok, j);
    const float f = __shfl_sync(0xFFFFFFFFu, wj, j);
    if (!okj || v >= nv) continue;
    const int64_t row = j < k ? t * k + j : T * k + (int64_t)(j - k) * T + t;
    const float4* src = reinterpret_cast<const float4*>(yp + row * d) + 2 * v;
    const float4 p = src[0], q = src[1];
    acc[0] = fmaf(f, p.x, acc[0]); acc[1] = fmaf(f, p.y, acc[1]);
    acc[2] = fmaf(f, p.z, acc[2]); acc[3] = fmaf(f, p.w, acc[3]);
    acc[4] = fmaf(f, q.x, acc[4]); acc[5] = fmaf(f, q.y, acc[5]);
    acc[6] = fmaf(f, q.z, acc[6]); acc[7] = fmaf(f, q.w, acc[7]);
  }
  if (v < nv) reinterpret_cast<uint4*>(y + t * d)[v] = pack8(acc);
}

// -------------------------------------------------------------------- host --
template <RowsMode M, bool FP4, int GPS, int NT, int RB>
static cudaError_t run_rows(const RowsArgs& a, int units, cudaStream_t s) {
  constexpr int MATS = M == RowsMode::GateUp ? 2 : 1;
  constexpr size_t smem = (size_t)kRowWarps * RB * MATS * 16 * (8 * NT + 2) * sizeof(float);
  const auto kernel = w4_rows_kernel<M, FP4, GPS, NT, RB>;
  if (smem > 40 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int gx = (w4_nblocks(a.N) + RB - 1) / RB;
  return launch_pdl(true, kernel, dim3(gx, units), dim3(kRowThreads), smem, s, a);
}

// Blocks of 16 columns a block takes (RB): as many as leave two blocks an SM, since the rows of
// x are loaded once for all of them; fewer for small matrices (2880 x 5120, one row: 7.9 us
// with four always, 6.4 so).
template <RowsMode M, bool FP4, int GPS, int NT, int RB>
static cudaError_t run_rows_rb(const RowsArgs& a, int units, cudaStream_t s) {
  if constexpr (RB > 1) {
    if ((int64_t)((w4_nblocks(a.N) + RB - 1) / RB) * units < 2 * num_sms())
      return run_rows_rb<M, FP4, GPS, NT, RB / 2>(a, units, s);
  }
  return run_rows<M, FP4, GPS, NT, RB>(a, units, s);
}

template <RowsMode M, bool FP4, int GPS>
static cudaError_t run_rows_nt(const RowsArgs& a, int units, int nt, cudaStream_t s) {
  constexpr int RB = M == RowsMode::GateUp ? 2 : 4;
  return nt <= 1   ? run_rows_rb<M, FP4, GPS, 1, M == RowsMode::Linear ? 2 : RB>(a, units, s)
         : nt <= 2 ? run_rows_rb<M, FP4, GPS, 2, RB>(a, units, s)
                   : run_rows_rb<M, FP4, GPS, 4, RB / 2>(a, units, s);
}

template <RowsMode M>
static cudaError_t rows(const RowsArgs& a, const moe_w4& w, int units, int nt, cudaStream_t s) {
  const int gps = w4_gps(w.group);
  if (w.kind == MOE_W4_FP4)
    return gps == 4   ? run_rows_nt<M, true, 4>(a, units, nt, s)
           : gps == 2 ? run_rows_nt<M, true, 2>(a, units, nt, s)
                      : run_rows_nt<M, true, 1>(a, units, nt, s);
  return gps == 4   ? run_rows_nt<M, false, 4>(a, units, nt, s)
         : gps == 2 ? run_rows_nt<M, false, 2>(a, units, nt, s)
                    : run_rows_nt<M, false, 1>(a, units, nt, s);
}

// Eight rows a product: 8, 16 or 32 rows at once, as many as an expert gets on
// average and half as many again.
static int tiles_for(double rows_per_expert, int64_t most) {
  const double want = 1.5 * rows_per_expert;
  const int64_t n = want < (double)most ? (int64_t)want : most;
  return n <= 8 ? 1 : n <= 16 ? 2 : 4;
}

cudaError_t launch_w4_linear_rows(const moe_w4& w, const moe_bf16* x, int64_t x_stride, int64_t T,
                                  void* y, int64_t y_stride, int y_fp32, int* status,
                                  cudaStream_t s) {
  RowsArgs a{};
  a.codes[0] = w.codes;
  a.scales[0] = w.scales;
  a.K = w.K;
  a.N = w.N;
  a.x = x;
  a.x_stride = x_stride;
  a.T = T;
  a.k = 1;
  a.out = y;
  a.out_stride = y_stride;
  a.out_fp32 = y_fp32;
  a.status = status;
  timer_before(MOE_KERNEL_W4_ROWS, s);
  const cudaError_t e = rows<RowsMode::Linear>(a, w, 1, T <= 8 ? 1 : T <= 16 ? 2 : 4, s);
  note_launches(1);
  timer_after(MOE_KERNEL_W4_ROWS, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

static cudaError_t launch_w4_combine(const W4Experts& q, const float* yp, moe_bf16* y, cudaStream_t s) {
  timer_before(MOE_KERNEL_COMBINE, s);
  const int64_t warps = q.T * (((int64_t)q.d / 8 + 31) / 32);
  const cudaError_t e =
      launch_pdl(pdl_for_tokens(q.T), w4_combine_kernel, dim3((unsigned)((warps + 7) / 8)),
                 dim3(256), 0, s, yp, q.topk_idx, q.topk_w, q.T, q.k, q.E, q.S, q.d, y);
  note_launches(1);
  timer_after(MOE_KERNEL_COMBINE, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_w4_experts_rows(const W4Experts& q, moe_bf16* A, int64_t A_lo, float* yp,
                                   moe_bf16* y, int* status, cudaStream_t s) {
  const int64_t P = q.T * q.k;
  RowsArgs a{};
  a.codes[0] = q.gate->codes;
  a.codes[1] = q.up->codes;
  a.scales[0] = q.gate->scales;
  a.scales[1] = q.up->scales;
  a.K = q.d;
  a.N = q.f;
  a.x = q.x;
  a.x_stride = q.d;
  a.idx = q.topk_idx;
  a.T = q.T;
  a.k = q.k;
  a.E = q.E;
  a.S = q.S;
  a.by_pair = P < q.E;
  a.act = q.act;
  a.out = A;
  a.lo = A_lo;
  a.status = status;
  const int units = (int)(a.by_pair ? P : q.E) + q.S;
  const int nt = tiles_for((double)P / q.E, q.T);
  timer_before(MOE_KERNEL_W4_ROWS, s);
  cudaError_t e = rows<RowsMode::GateUp>(a, *q.gate, units, nt, s);
  a.codes[0] = q.down->codes;
  a.scales[0] = q.down->scales;
  a.K = q.f;
  a.N = q.d;
  a.x = A;
  a.x_stride = q.f;
  a.out = yp;
  if (q.T == 1) {
    // one token: no rows of single experts, no launch to add them up (one of 128 experts
    // of 2048 x 768, top-8: 15.4 us with both, 11.5 so)
    a.out = y;
    const int gps = w4_gps(q.down->group);
    const auto kernel = q.down->kind == MOE_W4_FP4
                            ? (gps == 4   ? w4_token_kernel<true, 4>
                               : gps == 2 ? w4_token_kernel<true, 2>
                                          : w4_token_kernel<true, 1>)
                            : (gps == 4   ? w4_token_kernel<false, 4>
                               : gps == 2 ? w4_token_kernel<false, 2>
                                          : w4_token_kernel<false, 1>);
    if (e == cudaSuccess)
      e = launch_pdl(true, kernel, dim3(w4_nblocks(q.d)), dim3(kRowThreads), 0, s, a, q.topk_w);
  } else if (e == cudaSuccess) {
    const int per = A_lo ? 2 : 1;
    e = rows<RowsMode::Down>(a, *q.down, units, tiles_for((double)per * P / q.E, per * q.T), s);
  }
  note_launches(2);
  timer_after(MOE_KERNEL_W4_ROWS, s);
  if (e == cudaSuccess && q.T > 1) e = launch_w4_combine(q, yp, y, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
