// select.cu — the router's choice of experts from its logits, and the gradient
// of that choice's weights.
//
//   s   = softmax(l) over the experts, or sigmoid(l)
//   c   = s + balance                       (the choice value; balance moves the choice only)
//   groups of E / n_groups neighbouring experts rank by the sum of their
//   group_rank (1 or 2) largest c; the topk_groups first ones stay
//   S   = the k largest c among them, in descending order, ties to the lower index
//   w_j = scale s_j, or scale s_j / sum_S s  (renormalise)
//
// Without a balance (and without sums of two) the order of c is the order of l,
// which needs no score at all: the choice is exact. Otherwise it is made from
// fp32 scores whose error has a bound (kErr*, below); a token where two values
// that decide lie nearer to one another than that bound is decided again from
// scores in 64 bits. So the choice does not hang on how fp32 rounds: it is
// that of 64-bit scores for every token (about one in 300 takes the second
// look at 256 experts, top-8 with a balance).
//
// Gradient of L by the logits, g_j = dL/dw_j (the choice itself is piecewise
// constant, and balance gets none):
//   renormalise:  h_j = w_j (g_j - sum_i q_i g_i), q = w / scale  (to log s_j)
//                 softmax: dl_j = h_j;  sigmoid: dl_j = h_j (1 - s_j);  0 elsewhere
//   otherwise:    sigmoid: dl_j = scale g_j s_j (1 - s_j), 0 elsewhere
//                 softmax: dl_e = scale p_e ([e in S] g_e - sum_j p_j g_j), every e
//
// One warp a token, lane i holds experts i*NV .. i*NV + NV - 1, so the lowest lane
// with a value holds its lowest index. Both are bound by memory in floor (4 bytes
// a logit), by the rounds of the top-k in practice.
#include "common.cuh"
#include "internal.h"
#include "topk.cuh"

namespace moe {

constexpr int kSelWarps = 4;

struct SelArgs {
  int E, k;
  int sigmoid, n_groups, topk_groups, group_rank, renorm;
  float scale;
  const float* balance;
};

// ------------------------------------------------------------- score errors --
// Bounds of a choice value's error, relative to the largest score or value of the
// row, in units of 2^-24 (half an fp32 step). Sigmoid, 1 / (1 + e): expf within 2 steps, 1 + e, the
// quotient and the added balance half a step each: 7 halves. Softmax, e / Z: the
// argument's rounding moves e by at most |x| e^x < 0.4 halves of the largest, expf
// 4 halves, the same again for the terms of Z, Z's NV + 5 additions one half each,
// the quotient and the balance one each. A rank of two adds a rounding of its own:
// the groups' border asks for three times a pair's distance instead of twice.
template <int NV>
__device__ __forceinline__ float score_err(bool sigmoid) {
  return (sigmoid ? 8.f : (float)(NV + 5 + 12)) * 5.9604645e-8f;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
  return v;
}
template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// a larger float is a larger key, and every float's key is > 0
__device__ __forceinline__ uint32_t sort_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);      // -0 ranks as 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// A logit that is -inf or NaN: the expert is masked. It has score 0 and is
// chosen (in index order) only where fewer than k others remain.
__device__ __forceinline__ bool masked(float l) { return !(l > -INFINITY); }

// exp(l - m) with m the largest logit: 1 where both are infinite
__device__ __forceinline__ float exp_below(float l, float m) {
  return masked(l) ? 0.f : l == m ? 1.f : expf(l - m);
}
__device__ __forceinline__ double exp_below(float l, double m) {
  return masked(l) ? 0.0 : (double)l == m ? 1.0 : exp((double)l - m);
}
__device__ __forceinline__ float sigmoid_of(float l, float) { return 1.0f / (1.0f + expf(-l)); }
__device__ __forceinline__ double sigmoid_of(float l, double) {
  return 1.0 / (1.0 + exp(-(double)l));
}

template <int NV>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, bool vec,
                                         float* l) {
  if (NV >= 4 && vec) {
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = lane * NV + i;
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) v = *reinterpret_cast<const float4*>(row + e);
      l[i] = v.x;
      if (i + 1 < NV) l[i + 1] = v.y;
      if (i + 2 < NV) l[i + 2] = v.z;
      if (i + 3 < NV) l[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane * NV + i;
      l[i] = e < E ? row[e] : -INFINITY;
    }
  }
}

// Ranks of the groups from the choice values in the warp's row (R: float or
// double), kept groups as one bit a lane's expert: bit i of the result says that
// expert lane*NV + i is in a kept group. tight: two groups at the border are nearer
// than `err`. A group ranks by its unmasked members alone; one without any
// ranks last.
template <int NV, typename R>
__device__ __forceinline__ uint32_t keep_groups(const SelArgs& a, int lane, const R* row, R* rank,
                                                R err, bool* tight) {
  const int gs = a.E / a.n_groups;
  const R none = -(R)INFINITY;
  for (int g = lane; g < a.n_groups; g += 32) {
    R b0 = none, b1 = none;
    for (int i = 0; i < gs; ++i) {
      const R c = row[g * gs + i];
      if (c > b0) {
        b1 = b0;
        b0 = c;
      } else if (c > b1) {
        b1 = c;
      }
    }
    rank[g] = a.group_rank == 2 && b1 > none ? b0 + b1 : b0;
  }
  __syncwarp();
  // how many groups come before each; the border's two neighbours
  R low = (R)INFINITY, high = none;
  uint64_t kept = 0;                      // bit i: group lane + 32 i (up to 2048 groups)
  for (int g = lane, i = 0; g < a.n_groups; g += 32, ++i) {
    const R v = rank[g];
    int before = 0;
    for (int h = 0; h < a.n_groups; ++h) before += rank[h] > v || (rank[h] == v && h < g);
    if (before < a.topk_groups) {
      kept |= (uint64_t)1 << i;
      if (v < low) low = v;
    } else if (v > high) {
      high = v;
    }
  }
  __syncwarp();
  for (int g = lane, i = 0; g < a.n_groups; g += 32, ++i)
    rank[g] = (kept >> i) & 1 ? (R)1 : (R)0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const R ol = __shfl_xor_sync(0xFFFFFFFFu, low, off);
    const R oh = __shfl_xor_sync(0xFFFFFFFFu, high, off);
    if (ol < low) low = ol;
    if (oh > high) high = oh;
  }
  __syncwarp();
  *tight = high > none && !(low - high > err);
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    if (e < a.E && rank[e / gs] > (R)0) bits |= 1u << i;
  }
  __syncwarp();
  return bits;
}

// The choice from scores in 64 bits, for the tokens whose fp32 scores leave it open.
// Returns slot `lane`'s expert (lanes < k).
template <int NV>
__device__ __noinline__ int choose_64(const SelArgs& a, const float* __restrict__ lrow, int lane,
                                      bool vec, double* row) {
  float l[NV];
  load_row<NV>(lrow, a.E, lane, vec, l);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) m = masked(l[i]) ? m : fmaxf(m, l[i]);
  m = warp_max(m);
  double c[NV], z = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    c[i] = masked(l[i]) ? 0.0
                        : a.sigmoid ? sigmoid_of(l[i], 0.0) : exp_below(l[i], (double)m);
    z += c[i];
  }
  z = a.sigmoid ? 1.0 : warp_sum(z);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    c[i] = c[i] / z + (a.balance && e < a.E ? (double)__ldg(a.balance + e) : 0.0);
    if (masked(l[i]) || c[i] != c[i]) c[i] = -(double)INFINITY;
  }
  uint32_t open = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane * NV + i < a.E) open |= 1u << i;
  if (a.n_groups > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane * NV + i < a.E) row[lane * NV + i] = c[i];
    __syncwarp();
    bool tight;
    open &= keep_groups<NV, double>(a, lane, row, row + a.E, 0.0, &tight);
  }
  int my_e = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = 0.0;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (((open >> i) & 1u) && (at == 0x7FFFFFFF || c[i] > best)) {
        best = c[i];
        at = lane * NV + i;
      }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double ob = __shfl_xor_sync(0xFFFFFFFFu, best, off);
      const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, off);
      if (oa != 0x7FFFFFFF && (at == 0x7FFFFFFF || ob > best || (ob == best && oa < at))) {
        best = ob;
        at = oa;
      }
    }
    if (at / NV == lane) open &= ~(1u << (at % NV));
    if (lane == j) my_e = at;
  }
  return my_e;
}

// One token: lrow its logits (global or shared), row: the warp's 2E doubles of
// shared memory (groups or second looks; lrow may not lie in it). Writes idx and w.
template <int NV>
__device__ __forceinline__ void select_warp(const SelArgs& a, const float* lrow, bool vec,
                                            const int32_t* __restrict__ forced, int lane,
                                            double* row, int32_t* __restrict__ idx_out,
                                            float* __restrict__ w_out, int* status) {
  float l[NV];
  load_row<NV>(lrow, a.E, lane, vec, l);
  // softmax scores: the largest logit and the denominator, where something needs them
  const bool direct = !a.balance && (a.n_groups == 1 || a.group_rank == 1);
  float m = 0.f, z = 1.f;
  float e[NV] = {};
  if (!a.sigmoid && (!direct || !a.renorm)) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = masked(l[i]) ? m : fmaxf(m, l[i]);
    m = warp_max(m);
    z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      e[i] = exp_below(l[i], m);
      z += e[i];
    }
    z = warp_sum(z);
  }
  int my_e = 0;
  if (forced) {
    if (lane < a.k) my_e = forced[lane];
  } else {
    // choice values as sort keys; 0: no expert, or one that is taken
    uint32_t key[NV];
    float top = 0.f;                      // the largest magnitude among scores and values
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ex = lane * NV + i;
      float c = l[i];
      if (!direct && ex < a.E && !masked(c)) {
        const float s = a.sigmoid ? sigmoid_of(c, 0.f) : e[i] / z;
        c = a.balance ? s + __ldg(a.balance + ex) : s;
        top = fmaxf(top, fmaxf(s, fabsf(c)));
      }
      if (masked(l[i]) || c != c) c = -INFINITY;
      key[i] = ex < a.E ? sort_key(c) : 0u;
    }
    bool open = false;                    // the fp32 scores leave the choice open
    float err = 0.f;
    // (and scores below fp32's normal range, which have fewer bits, stay open)
    if (!direct) err = 2.f * score_err<NV>(a.sigmoid) * warp_max(top) + 1e-37f;
    if (a.n_groups > 1) {
      float* frow = reinterpret_cast<float*>(row);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (lane * NV + i < a.E) frow[lane * NV + i] = key_value(key[i]);
      __syncwarp();
      const uint32_t keep = keep_groups<NV, float>(a, lane, frow, frow + a.E, 3.f * err, &open);
      open = open && !direct;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (!((keep >> i) & 1u)) key[i] = 0u;
    }
    float before = 0.f;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) mine = mine > key[i] ? mine : key[i];
    const int rounds = direct ? a.k : a.k + 1;   // one more value than is taken: the border
    for (int j = 0; j < rounds; ++j) {
      const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, mine);
      if (best == 0u) break;
      if (!direct) {
        // neighbours in the order have to be further apart than their errors (masked
        // experts, all -inf, go by their index)
        const float v = key_value(best);
        if (j > 0 && v > -INFINITY && !(before - v > err)) open = true;
        before = v;
      }
      if (j == a.k) break;
      const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, mine == best)) - 1;
      int at = 0;
      if (lane == owner) {
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
          if (key[i] == best) at = i;
        mine = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i == at) key[i] = 0u;
          mine = mine > key[i] ? mine : key[i];
        }
      }
      at = __shfl_sync(0xFFFFFFFFu, at, owner);
      if (lane == j) my_e = owner * NV + at;
    }
    if (open) my_e = choose_64<NV>(a, lrow, lane, vec, row);
  }
  // the weights of the slots
  const bool slot = lane < a.k;
  const bool valid = slot && my_e >= 0 && my_e < a.E;
  if (slot && !valid) raise_status(status, MOE_ERR_DEVICE_INDEX);
  const float lj = valid ? lrow[my_e] : -INFINITY;
  const bool dead = masked(lj);
  float s;
  if (!a.renorm) {
    s = dead ? 0.f : a.sigmoid ? sigmoid_of(lj, 0.f) : exp_below(lj, m) / z;
  } else {
    // scores up to a common factor e^-r that the quotient drops: r the largest
    // chosen logit, for sigmoids only where it is below 0, so that tiny scores
    // keep their ratios
    float r = warp_max(dead ? -INFINITY : lj);
    if (a.sigmoid) r = fminf(r, 0.f);
    s = dead ? 0.f
             : !a.sigmoid ? exp_below(lj, r)
                          : lj >= 0.f ? sigmoid_of(lj, 0.f) : expf(lj - r) / (1.0f + expf(lj));
    const float sum = warp_sum(s);
    s = sum > 0.f ? s / sum : 0.f;
  }
  if (slot) {
    idx_out[lane] = my_e;
    w_out[lane] = a.scale * s;
  }
}

template <int NV>
__global__ void __launch_bounds__(32 * kSelWarps) select_kernel(
    SelArgs a, const float* __restrict__ logits, const int32_t* __restrict__ forced, int64_t T,
    bool vec, int row_doubles, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
    int* status) {
  pdl_enter();
  extern __shared__ double sel_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kSelWarps + warp;
  if (t >= T) return;
  select_warp<NV>(a, logits + t * a.E, vec, forced ? forced + t * a.k : nullptr, lane,
                  sel_rows + (size_t)warp * row_doubles, topk_idx + t * a.k, topk_w + t * a.k,
                  status);
}

static SelArgs sel_args(const moe_router& r) {
  return SelArgs{r.E,           r.k,          r.score == MOE_SCORE_SIGMOID, r.n_groups,
                 r.topk_groups, r.group_rank, r.renormalise,                r.scale,
                 r.balance};
}

// choose_64 and the groups' ranks need 2E values of the warp's row
static int sel_row_doubles(const moe_router& r) { return r.n_groups > 1 ? 2 * r.E : 0; }

template <int NV>
static cudaError_t run_select(const moe_router& r, const float* logits, const int32_t* forced,
                              int64_t T, int32_t* topk_idx, float* topk_w, int* status,
                              cudaStream_t s) {
  const int rd = sel_row_doubles(r);
  const size_t smem = (size_t)kSelWarps * rd * sizeof(double);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        select_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const bool vec = r.E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0;
  return launch_pdl(pdl_for_tokens(T), select_kernel<NV>,
                    dim3((unsigned)((T + kSelWarps - 1) / kSelWarps)), dim3(32 * kSelWarps), smem,
                    s, sel_args(r), logits, forced, T, vec, rd, topk_idx, topk_w, status);
}

cudaError_t launch_select(const moe_router& r, const float* logits, const int32_t* forced,
                          int64_t T, int32_t* topk_idx, float* topk_w, int* status,
                          cudaStream_t s) {
  timer_before(MOE_KERNEL_SELECT, s);
  const int nv = (r.E + 31) / 32;
  const auto run = nv <= 1   ? run_select<1>
                   : nv <= 2 ? run_select<2>
                   : nv <= 4 ? run_select<4>
                   : nv <= 8 ? run_select<8>
                   : nv <= 16 ? run_select<16>
                              : run_select<kMaxExperts / 32>;
  const cudaError_t e = run(r, logits, forced, T, topk_idx, topk_w, status, s);
  note_launches(1);
  timer_after(MOE_KERNEL_SELECT, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// A few tokens from the router's row-slice partials (route.cu): one block a token adds
// the slices in order, writes the logits, and its first warp chooses.
template <int NV>
__global__ void __launch_bounds__(256) select_small_kernel(
    SelArgs a, const float* __restrict__ part, int ns, int64_t T, const float* __restrict__ bias,
    const int32_t* __restrict__ forced, float* __restrict__ logits,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, int* status) {
  pdl_enter();
  extern __shared__ double sel_rows[];
  __shared__ __align__(16) float lrow[kMaxExperts];
  const int64_t t = blockIdx.x;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    const float sum = router_small_sum(part, ns, T, t, a.E, e) + (bias ? bias[e] : 0.f);
    lrow[e] = sum;
    logits[t * a.E + e] = sum;
  }
  __syncthreads();
  if (threadIdx.x < 32)
    select_warp<NV>(a, lrow, a.E % 4 == 0, forced ? forced + t * a.k : nullptr, threadIdx.x,
                    sel_rows, topk_idx + t * a.k, topk_w + t * a.k, status);
}

template <int NV>
static cudaError_t run_select_small(const moe_router& r, const float* part, int ns, int64_t T,
                                    const float* bias, const int32_t* forced, float* logits,
                                    int32_t* topk_idx, float* topk_w, int* status,
                                    cudaStream_t s) {
  return launch_pdl(true, select_small_kernel<NV>, dim3((unsigned)T), dim3(256),
                    (size_t)sel_row_doubles(r) * sizeof(double), s, sel_args(r), part, ns, T, bias,
                    forced, logits, topk_idx, topk_w, status);
}

cudaError_t launch_select_small(const moe_router& r, const float* part, int ns, int64_t T,
                                const float* bias, const int32_t* forced, float* logits,
                                int32_t* topk_idx, float* topk_w, int* status, cudaStream_t s) {
  timer_before(MOE_KERNEL_SELECT, s);
  const int nv = (r.E + 31) / 32;
  const auto run = nv <= 1   ? run_select_small<1>
                   : nv <= 2 ? run_select_small<2>
                   : nv <= 4 ? run_select_small<4>
                   : nv <= 8 ? run_select_small<8>
                   : nv <= 16 ? run_select_small<16>
                              : run_select_small<kMaxExperts / 32>;
  const cudaError_t e = run(r, part, ns, T, bias, forced, logits, topk_idx, topk_w, status, s);
  note_launches(1);
  timer_after(MOE_KERNEL_SELECT, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------- gradient --
// One warp a token. The chosen slots' gradients are worked out a lane each; the
// row is written whole (zeros, or every expert's term for unnormalised softmax
// scores), and then the chosen entries. Slots that name one expert twice
// (a caller's own choice) add up in slot order.
template <int NV>
__global__ void __launch_bounds__(32 * kSelWarps) select_bwd_kernel(
    SelArgs a, const float* __restrict__ d_topk_w, const float* __restrict__ logits,
    const int32_t* __restrict__ topk_idx, int64_t T, int accumulate, bool vec,
    float* __restrict__ d_logits, int* status) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kSelWarps + warp;
  if (t >= T) return;
  const float* lrow = logits + t * a.E;
  float* drow = d_logits + t * a.E;
  const bool dense = !a.sigmoid && !a.renorm;
  const bool slot = lane < a.k;
  int my_e = slot ? topk_idx[t * a.k + lane] : -1;
  float g = slot ? a.scale * d_topk_w[t * a.k + lane] : 0.f;
  if (slot && (my_e < 0 || my_e >= a.E)) {
    raise_status(status, MOE_ERR_DEVICE_INDEX);
    my_e = -1;
  }
  const float lj = my_e >= 0 ? __ldg(lrow + my_e) : -INFINITY;
  const bool dead = masked(lj);
  if (dead) g = 0.f;                      // its weight is 0 whatever the others do
  float l[NV];
  float m = -INFINITY, z = 0.f;
  if (dense) {
    load_row<NV>(lrow, a.E, lane, vec, l);
#pragma unroll
    for (int i = 0; i < NV; ++i) m = masked(l[i]) ? m : fmaxf(m, l[i]);
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < NV; ++i) z += exp_below(l[i], m);
    z = warp_sum(z);
  }
  float dl = 0.f, inner = 0.f;
  if (a.renorm) {
    float r = warp_max(lj);
    if (a.sigmoid) r = fminf(r, 0.f);
    float q = dead ? 0.f
                   : !a.sigmoid ? exp_below(lj, r)
                                : lj >= 0.f ? sigmoid_of(lj, 0.f) : expf(lj - r) / (1.0f + expf(lj));
    const float sum = warp_sum(q);
    q = sum > 0.f ? q / sum : 0.f;
    inner = warp_sum(q * g);
    dl = q * (g - inner);
    if (a.sigmoid) dl = dead ? 0.f : dl * sigmoid_of(-lj, 0.f);     // 1 - s, without its cancellation
  } else if (a.sigmoid) {
    dl = dead ? 0.f : g * sigmoid_of(lj, 0.f) * sigmoid_of(-lj, 0.f);
  } else {
    const float p = dead ? 0.f : exp_below(lj, m) / z;
    inner = warp_sum(p * g);
    dl = p * g;                           // the chosen entry's own term; - p_e inner for every e
  }
  // one lane an expert: the first slot that names it takes the others' terms
  bool writes = my_e >= 0;
  float add = dl;
  if (__any_sync(0xFFFFFFFFu, my_e >= 0)) {
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, my_e);
    const bool first = (same & ((1u << lane) - 1u)) == 0;
    if (__any_sync(0xFFFFFFFFu, writes && !first)) {
      add = 0.f;
      for (int j = 0; j < a.k; ++j) {
        const float dj = __shfl_sync(0xFFFFFFFFu, dl, j);
        if ((same >> j) & 1u) add += dj;
      }
      writes = writes && first;
    }
  }
  if (dense) {
    const float p = dead ? 0.f : exp_below(lj, m) / z;
    add -= p * inner;
    const float gz = z > 0.f ? inner / z : 0.f;
    if (NV >= 4 && vec) {
#pragma unroll
      for (int i = 0; i + 3 < NV; i += 4) {
        const int e = lane * NV + i;
        if (e >= a.E) continue;
        float4 v = make_float4(-exp_below(l[i], m) * gz, -exp_below(l[i + 1], m) * gz,
                               -exp_below(l[i + 2], m) * gz, -exp_below(l[i + 3], m) * gz);
        float4* dst = reinterpret_cast<float4*>(drow + e);
        if (accumulate) {
          const float4 o = *dst;
          v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
        }
        *dst = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane * NV + i;
        if (e < a.E) drow[e] = (accumulate ? drow[e] : 0.f) - exp_below(l[i], m) * gz;
      }
    }
    // the chosen entries get p g on top of that
    __syncwarp();
    if (writes) {
      if (accumulate) {
        drow[my_e] += add + p * inner;
      } else {
        drow[my_e] = add;
      }
    }
    return;
  }
  if (!accumulate) {
    if (vec) {
      for (int e = 4 * lane; e < a.E; e += 128)
        *reinterpret_cast<float4*>(drow + e) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int e = lane; e < a.E; e += 32) drow[e] = 0.f;
    }
    __syncwarp();
    if (writes) drow[my_e] = add;
  } else if (writes) {
    drow[my_e] += add;
  }
}

template <int NV>
static cudaError_t run_select_bwd(const moe_router& r, const float* dw, const float* logits,
                                  const int32_t* idx, int64_t T, int accumulate, float* d_logits,
                                  int* status, cudaStream_t s) {
  const bool vec = r.E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 &&
                   (reinterpret_cast<uintptr_t>(d_logits) & 15u) == 0;
  return launch_pdl(pdl_for_tokens(T), select_bwd_kernel<NV>,
                    dim3((unsigned)((T + kSelWarps - 1) / kSelWarps)), dim3(32 * kSelWarps), 0, s,
                    sel_args(r), dw, logits, idx, T, accumulate, vec, d_logits, status);
}

cudaError_t launch_select_bwd(const moe_router& r, const float* d_topk_w, const float* logits,
                              const int32_t* topk_idx, int64_t T, int accumulate, float* d_logits,
                              int* status, cudaStream_t s) {
  timer_before(MOE_KERNEL_SELECT_BWD, s);
  const int nv = (r.E + 31) / 32;
  const auto run = nv <= 1   ? run_select_bwd<1>
                   : nv <= 2 ? run_select_bwd<2>
                   : nv <= 4 ? run_select_bwd<4>
                   : nv <= 8 ? run_select_bwd<8>
                   : nv <= 16 ? run_select_bwd<16>
                              : run_select_bwd<kMaxExperts / 32>;
  const cudaError_t e = run(r, d_topk_w, logits, topk_idx, T, accumulate, d_logits, status, s);
  note_launches(1);
  timer_after(MOE_KERNEL_SELECT_BWD, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
