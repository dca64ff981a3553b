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
// Without a balance (and without sums of two that decide) the order of c is the order of l,
// which needs no score at all: the choice is exact. Otherwise it is made from
// fp32 scores whose error has a bound (score_err, below); a token where two values
// that decide lie nearer to one another than that bound is decided again from
// scores in 64 bits (softmax: to 2^-39 of the largest). So the choice does not hang on how
// fp32 rounds: it is that of 64-bit scores for every token (about one in 200 takes the second
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
// a logit), in practice by instruction issue, some 1050 a token at 256 experts in 8 groups
// (16384 such tokens: 25 us; the floor is 2.6). Eight blocks an SM (64 registers) took 22 to 25 us
// there, seven 25 to 27.
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
// Bounds of a score's error, relative to the largest score of the row, in units of
// 2^-24 (half an fp32 step). Sigmoid, s = 1 / (1 + e) with __expf (e = exp(-l), within
// 2 + 1.173 |l| steps) and __fdividef (2 steps): e's error counts (1 - s) of s, 1 + e's one
// half, the quotient's four. s (1 - s) (4 + 2.35 |l|) is below 1.6 everywhere, so 3.2 of the
// largest score where that is over 1/2; below, s (4 + 2.35 |l|) grows with l and is 4 + 2.35 |m|
// of the largest score at most, m the largest logit (and one more for that score's own
// rounding): 10 + 2.4 max(0, -m). Softmax, e (1 / Z): the argument's rounding
// moves e by at most |x| e^x < 0.4 halves of the largest, expf 4 halves. Z: expf's 4 again, its NV + 5
// additions one half each, and of the arguments' roundings, which may all go one way, sum |x| e^x / Z:
// at most f with f e^(f + 1) = E - 1 (one expert far above equal others), 4.5 for 1024 experts. The
// inverse and the product one each: NV + 20. The balance's addition is a half of the value itself
// (border_err).
template <int NV>
__device__ __forceinline__ float score_err(bool sigmoid, float m) {
  return (sigmoid ? 10.f + 2.4f * fmaxf(0.f, -m) : (float)(NV + 20)) * 5.9604645e-8f;
}
// how far apart two values near v have to be to be told apart (and scores below
// fp32's normal range, which have fewer bits, never are)
__device__ __forceinline__ float border_err(float score, float v) {
  return 2.f * score + 2.3841858e-7f * fabsf(v) + 1e-37f;
}

// A group's rank is a sum of two values, each rounded on its own, whose signs may differ: what it is
// off by goes by what it is a sum of, not by itself.
__device__ __forceinline__ float rank_size(const SelArgs& a, float c0, float c1) {
  return a.group_rank == 2 && c1 > -INFINITY ? fabsf(c0) + fabsf(c1) : 0.f;
}
// How far apart two groups' ranks near v have to be: both carry the error of two scores, and half
// a step each of either value and of their sum, 2 2^-24 of `size` (the largest rank_size); border_err
// allows it four.
__device__ __forceinline__ float rank_err(float score, float v, float size) {
  return 2.f * border_err(score, fmaxf(fabsf(v), size));
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

// Sort keys: a larger number is a larger key, and every number's key is > 0 (0: no
// expert, or one that is taken). Key by type: 32 bits of a float, 64 of a double.
typedef unsigned long long u64;
__device__ __forceinline__ uint32_t sort_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);      // -0 ranks as 0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}
__device__ __forceinline__ u64 sort_key(double v) {
  const u64 b = (u64)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}
__device__ __forceinline__ double key_value(u64 key) {
  return __longlong_as_double((long long)((key >> 63) ? (key & ~(1ull << 63)) : ~key));
}
__device__ __forceinline__ uint32_t warp_max_key(uint32_t v) {
  return __reduce_max_sync(0xFFFFFFFFu, v);
}
__device__ __forceinline__ u64 warp_max_key(u64 v) {
  const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(v >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (u64)hi << 32 | lo;
}

// A logit that is -inf or NaN (NaN is read as -inf): the expert is masked. It has
// score 0 and is chosen (in index order) only where fewer than k others remain.
__device__ __forceinline__ bool masked(float l) { return !(l > -INFINITY); }

// exp(l - m) with m the largest logit: 1 where both are infinite
__device__ __forceinline__ float exp_below(float l, float m) {
  return masked(l) ? 0.f : l == m ? 1.f : expf(l - m);
}
__device__ __forceinline__ float sigmoid_of(float l) { return 1.0f / (1.0f + expf(-l)); }
// to the choice alone (score_err); 0 below 2^-126
__device__ __forceinline__ float sigmoid_near(float l) {
  return __fdividef(1.0f, 1.0f + __expf(-l));
}

// score times e^-r (sigmoid: r = 0 wherever l >= 0)
__device__ __forceinline__ float renorm_score(bool sigmoid, float l, float r) {
  const float e = l == r ? 1.f : expf(l - r);
  const float q = sigmoid ? (l >= 0.f ? 1.f : e) / (1.f + expf(-fabsf(l))) : e;
  return masked(l) ? 0.f : q;
}

template <int NV>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, bool vec, float* l) {
  if (NV >= 4 && vec) {
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = lane * NV + i;
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) v = *reinterpret_cast<const float4*>(row + e);
      l[i] = fmaxf(v.x, -INFINITY);
      if (i + 1 < NV) l[i + 1] = fmaxf(v.y, -INFINITY);
      if (i + 2 < NV) l[i + 2] = fmaxf(v.z, -INFINITY);
      if (i + 3 < NV) l[i + 3] = fmaxf(v.w, -INFINITY);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane * NV + i;
      l[i] = e < E ? fmaxf(row[e], -INFINITY) : -INFINITY;
    }
  }
}

// -------------------------------------------------------------- the k largest --
// Descending order over the lanes (a bitonic network); equal keys by index.
template <typename K>
__device__ __forceinline__ void sort_lanes(K& key, int& at, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int off = size >> 1; off > 0; off >>= 1) {
      const K ok = __shfl_xor_sync(0xFFFFFFFFu, key, off);
      const int oa = __shfl_xor_sync(0xFFFFFFFFu, at, off);
      const bool mine = key > ok || (key == ok && at < oa);       // mine comes first
      const bool first = ((lane & off) == 0) == ((lane & size) == 0 || size == 32);
      if (mine != first) {
        key = ok;
        at = oa;
      }
    }
}
// The same order for one key a lane that stand in shared memory too (n of them, zeros up to
// the next multiple of four), lanes in index order: a lane counts the larger ones, which takes
// a third of the network's instructions.
__device__ __forceinline__ int rank_among(uint32_t key, int n, const uint32_t* keys, int lane) {
  int r = 0;
  for (int j = 0; j < n; j += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(keys + j);
    r += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
  }
  return r + __popc(__match_any_sync(0xFFFFFFFFu, key) & ((1u << lane) - 1u));
}

// The `need` <= 33 largest keys in order, ties to the lower expert: lane j gets the j-th's
// key and expert (key 0: there are no more), *last the 33rd's key.
// The need-th largest of the lanes' own largest is a floor for the need-th largest of
// all (found by as many warp maxima; lanes with equal keys leave together, which only lowers
// it): what reaches it (or floor_of(it), somewhat lower) is seldom more than 32 keys, which
// meet in shared memory (`meet`, 32 entries) and are sorted, a key a lane: true, the lanes
// hold every key of at least floor_of(the need-th). With more of them (ties, masked
// rows, need = 33) the keys are taken one by one: false.
template <int NV, typename F>
__device__ __forceinline__ bool largest(uint32_t* key, int need, int lane, uint32_t* meet_key,
                                        int* meet_at, F floor_of, uint32_t* out, int* at_out,
                                        uint32_t* last) {
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) mine = max(mine, key[i]);
  *last = 0;
  if (NV == 1) {
    *out = key[0];
    *at_out = lane;
    if (need <= 32) {
      meet_key[lane] = key[0];
      __syncwarp();
      const int r = rank_among(key[0], 32, meet_key, lane);
      __syncwarp();
      meet_key[r] = key[0];
      meet_at[r] = lane;
      __syncwarp();
      *out = meet_key[lane];
      *at_out = meet_at[lane];
      return true;
    }
  } else if (need <= 32) {
    uint32_t tau = 0, rest = mine;
    for (int j = 0; j < need; ++j) {
      tau = warp_max_key(rest);
      if (rest == tau) rest = 0;
    }
    const uint32_t floor = tau ? floor_of(tau) : 1u;
    uint32_t take = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) take |= (key[i] >= floor ? 1u : 0u) << i;
    int n = __popc(take);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, n, off);
      if (lane >= off) n += o;
    }
    const int total = __shfl_sync(0xFFFFFFFFu, n, 31);
    if (total <= 32) {
      int p = n - __popc(take);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((take >> i) & 1u) {
          meet_key[p] = key[i];
          meet_at[p] = lane * NV + i;
          ++p;
        }
      if (lane >= total) meet_key[lane] = 0;
      __syncwarp();
      const uint32_t k0 = meet_key[lane];
      const int a0 = lane < total ? meet_at[lane] : 0x7FFFFFFF;
      const int r = rank_among(k0, total, meet_key, lane);
      __syncwarp();
      meet_key[r] = k0;
      meet_at[r] = a0;
      __syncwarp();
      *out = meet_key[lane];
      *at_out = meet_at[lane];
      return true;
    }
  }
  *out = 0;
  *at_out = 0x7FFFFFFF;
  for (int j = 0; j < need; ++j) {
    const uint32_t best = warp_max_key(mine);
    if (best == 0) break;
    const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, mine == best)) - 1;
    int at = 0;
    if (lane == owner) {
#pragma unroll
      for (int i = NV - 1; i >= 0; --i)
        if (key[i] == best) at = i;
      mine = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i == at) key[i] = 0;
        mine = max(mine, key[i]);
      }
    }
    at = __shfl_sync(0xFFFFFFFFu, at, owner);
    if (j == 32) {
      *last = best;
    } else if (lane == j) {
      *out = best;
      *at_out = owner * NV + at;
    }
  }
  return false;
}

// ------------------------------------------------------------- second looks --
// Tokens whose fp32 scores leave the choice open are looked at again in 64 bits:
// about one in some hundred, but a call of many tokens ends with one of them, so
// what counts is how long a warp takes on its own. A double operation takes it some
// 50 cycles here, so only what stands near a border gets a 64-bit score, a value a
// lane, and a softmax's exponentials are pairs of fp32 (8192 tokens of 512 experts: 16.6 us
// without a second look, 24.7 with them in double arithmetic, 18.7 in pairs).

// 2^(j / 32) as a pair: an fp32 number and the rest
__device__ const float2 kExp2_32[32] = {
    {1.0f, 0.0f}, {1.0218971967697144f, -4.811559861650494e-08f},
    {1.0442737340927124f, 4.8334701574503924e-08f}, {1.0671404600143433f, -5.9337519786595294e-08f},
    {1.0905077457427979f, -1.3077539939843064e-08f}, {1.114386796951294f, -5.435540018083884e-08f},
    {1.1387885808944702f, 5.386222312608879e-08f}, {1.1637248992919922f, -4.051441493402308e-08f},
    {1.1892070770263672f, 3.797635272917432e-08f}, {1.215247392654419f, -3.267394887984665e-08f},
    {1.2418577671051025f, 4.496838101886169e-08f}, {1.2690509557724f, 1.419333317542737e-09f},
    {1.2968395948410034f, -4.018999533172973e-08f}, {1.3252366781234741f, -3.496373324196611e-08f},
    {1.3542555570602417f, -1.0123349269974824e-08f}, {1.3839099407196045f, -5.875577357983275e-08f},
    {1.4142135381698608f, 2.4203234971764687e-08f}, {1.4451807737350464f, 3.324199937537742e-08f},
    {1.4768261909484863f, -4.500898853621038e-08f}, {1.5091644525527954f, -2.4959373234878512e-08f},
    {1.5422108173370361f, 8.070904833346049e-09f}, {1.5759809017181396f, -5.661025426206834e-08f},
    {1.610490322113037f, 9.836217174097328e-09f}, {1.6457555294036865f, -5.124972091152813e-08f},
    {1.6817928552627563f, -2.4755326677450284e-08f}, {1.7186193466186523f, -4.8496175963919086e-08f},
    {1.7562521696090698f, -9.235770370707996e-09f}, {1.7947090864181519f, -1.141504490931311e-08f},
    {1.8340080976486206f, -1.1239277952768134e-08f}, {1.8741676807403564f, -4.663005626071026e-08f},
    {1.9152065515518188f, 9.845328108326612e-09f}, {1.9571441411972046f, -1.7021804410433106e-08f}};
// the lane's own entry; every lane of the warp calls exp_pair together
__device__ __forceinline__ float2 exp_table(int lane) { return kExp2_32[lane]; }

// exp(l - m) for finite l <= m, to 2^-42 of itself, as hi + lo (a table-driven exponential as in
// Tang, ACM TOMS 1989, with Cody and Waite's reduction): 2^(k / 32) from the table times
// 1 + r + r^2 / 2 + .. r^5 / 120 (the rest below 2^-48), r = l - m - k log(2) / 32, |r| <=
// log(2) / 64. log(2) / 32 is three numbers, k times the first of 12 bits is exact; sums and
// products keep their roundings' errors (Knuth's two-sum, Dekker's pairs) down to the
// terms of 2^-20. Below -42 (where hi would leave the normal range with what follows) the
// caller takes something else.
__device__ __forceinline__ float2 exp_pair(float l, float m, float2 table) {
  const float xh = __fsub_rn(l, m), xb = __fsub_rn(xh, l);
  const float xl = __fsub_rn(__fsub_rn(l, __fsub_rn(xh, xb)), __fadd_rn(m, xb));
  const float kf = rintf(fmaxf(xh, -43.f) * 46.166241f);               // 32 / log(2)
  const int k = (int)kf;
  const float r0 = fmaf(-kf, 2839.f / 131072.f, xh);
  const float ph = __fmul_rn(kf, 9.983182280848268e-07f), pl = fmaf(kf, 9.983182280848268e-07f, -ph);
  const float r1 = __fsub_rn(r0, ph), rb = __fsub_rn(r1, r0);
  const float re = __fsub_rn(__fsub_rn(r0, __fsub_rn(r1, rb)), __fadd_rn(ph, rb));
  const float r2 = __fadd_rn(xl, __fsub_rn(re, fmaf(kf, 5.14560928046269e-14f, pl)));
  const float rh = __fadd_rn(r1, r2), rz = __fsub_rn(rh, r1);
  const float rl = __fadd_rn(__fsub_rn(r1, __fsub_rn(rh, rz)), __fsub_rn(r2, rz));
  const float sq = __fmul_rn(rh, rh), sl = fmaf(rh + rh, rl, fmaf(rh, rh, -sq));
  const float p = fmaf(rh, fmaf(rh, 1.f / 120, 1.f / 24), 1.f / 6);
  const float low = fmaf(__fmul_rn(rh, sq), p, fmaf(0.5f, sl, rl));
  const float h = 0.5f * sq, uh = __fadd_rn(rh, h);
  const float ul = __fadd_rn(__fsub_rn(h, __fsub_rn(uh, rh)), low);
  const float th = __shfl_sync(0xFFFFFFFFu, table.x, k & 31);
  const float tl = __shfl_sync(0xFFFFFFFFu, table.y, k & 31);
  const float q = __fmul_rn(th, uh), ql = fmaf(th, uh, -q);
  const float eh = __fadd_rn(th, q);
  const float el = __fadd_rn(__fsub_rn(q, __fsub_rn(eh, th)),
                             __fadd_rn(__fadd_rn(ql, tl), fmaf(th, ul, tl * uh)));
  const float unit = __int_as_float(((k >> 5) + 127) << 23);
  return make_float2(eh * unit, el * unit);
}

// Sum of exp(l - m) over the row, to 2^-40. Terms below 2^-60 of the largest are left out.
static __device__ __noinline__ double denominator_64(const float* lrow, int E, int lane, float m,
                                                     float2 table) {
  float zh = 0.f, zl = 0.f;
#pragma unroll 4
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const float l = e < E ? fmaxf(lrow[e], -INFINITY) : -INFINITY;
    const bool one = l == m, in = l - m > -42.f;         // (both infinite: 1)
    float2 v = exp_pair(in ? l : 0.f, in ? m : 0.f, table);
    if (!in || one) v = make_float2(one ? 1.f : 0.f, 0.f);
    const float s = __fadd_rn(zh, v.x), b = __fsub_rn(s, zh);
    zl += __fadd_rn(__fsub_rn(zh, __fsub_rn(s, b)), __fsub_rn(v.x, b)) + v.y;
    zh = s;
  }
  return warp_sum((double)zh + (double)zl);
}

struct Row64 {          // what a 64-bit choice value needs
  const float* lrow;
  float m;              // softmax: the largest logit, and the denominator's inverse
  double rz;
  float2 table;
};
__device__ __forceinline__ Row64 row_64(const SelArgs& a, const float* lrow, int lane, float m) {
  const float2 table = exp_table(lane);
  return Row64{lrow, m, a.sigmoid || masked(m) ? 1.0 : 1.0 / denominator_64(lrow, a.E, lane, m, table),
               table};
}
// the sort key of expert e's choice value, or 0 for e < 0; every lane of the warp calls it
static __device__ __noinline__ u64 key_64(const SelArgs& a, Row64 r, int e) {
  const float l = e >= 0 ? r.lrow[e] : -INFINITY;
  double c;
  if (a.sigmoid) {
    c = 1.0 / (1.0 + exp(-(double)l));
  } else {
    const bool one = l == r.m, in = l - r.m > -42.f;
    const float2 v = exp_pair(in && !one ? l : 0.f, in && !one ? r.m : 0.f, r.table);
    c = (double)v.x + (double)v.y;
    if (!in && !one && !masked(l)) c = exp((double)l - (double)r.m);
    c *= r.rz;
  }
  const u64 none = sort_key(-(double)INFINITY);
  if (e < 0) return 0ull;
  if (masked(l)) return none;
  if (a.balance) c += (double)__ldg(a.balance + e);
  return c == c ? sort_key(c) : none;
}

// The groups' border: `rank` is this lane's group's rank in fp32 (lanes L * g hold group
// g's, n_groups <= 32), sure and kept by the fp32 ranks or in question. Those in question are
// ranked again. Returns whether this lane's group stays.
static __device__ __noinline__ bool settle_groups(const SelArgs& a, Row64 r, int lane, int L,
                                           bool question, bool sure) {
  const int gs = a.E / a.n_groups;
  const u64 none = sort_key(-(double)INFINITY);
  const uint32_t heads = L == 32 ? 1u : (uint32_t)(0xFFFFFFFFu / ((1u << L) - 1u));   // bits 0, L, 2L ..
  const uint32_t asked = __ballot_sync(0xFFFFFFFFu, question) & heads;
  int room = a.topk_groups - __popc(__ballot_sync(0xFFFFFFFFu, sure) & heads);
  u64 mine = 0;
  for (uint32_t todo = asked; todo; todo &= todo - 1) {
    const int g = (__ffs(todo) - 1) / L;
    u64 b0 = none, b1 = none;
    for (int i0 = 0; i0 < gs; i0 += 32) {
      const u64 v = key_64(a, r, i0 + lane < gs ? g * gs + i0 + lane : -1), c = v ? v : none;
      const u64 top = warp_max_key(c);
      const bool first = lane == __ffs(__ballot_sync(0xFFFFFFFFu, c == top)) - 1;
      const u64 next = warp_max_key(first ? none : c);
      const u64 lo = top < b0 ? top : b0;
      b0 = top > b0 ? top : b0;
      b1 = lo > b1 ? lo : b1;
      b1 = next > b1 ? next : b1;
    }
    const u64 rank =
        a.group_rank == 2 && b1 > none ? sort_key(key_value(b0) + key_value(b1)) : b0;
    if (lane / L == g) mine = rank;
  }
  bool stays = sure;
  const int g = lane / L;
  int before = 0;
  for (uint32_t todo = asked; todo; todo &= todo - 1) {
    const int h = (__ffs(todo) - 1) / L;
    const u64 o = __shfl_sync(0xFFFFFFFFu, mine, h * L);
    before += o > mine || (o == mine && h < g);
  }
  if (question && before < room) stays = true;
  return stays;
}

// The whole choice in 64 bits, for what the above do not take: more than 32 values near
// a border (equal logits), groups that are no whole lanes. In loops, for short code.
// Returns slot `lane`'s expert (lanes < k). row: E keys and, with groups, E more.
static __device__ __noinline__ int choose_64(const SelArgs& a, Row64 r, int lane, u64* row) {
  const u64 none = sort_key(-(double)INFINITY);
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const u64 c = key_64(a, r, e0 + lane < a.E ? e0 + lane : -1);
    if (e0 + lane < a.E) row[e0 + lane] = c;
  }
  __syncwarp();
  if (a.n_groups > 1) {
    const int gs = a.E / a.n_groups;
    u64* rank = row + a.E;
    for (int g = lane; g < a.n_groups; g += 32) {
      u64 b0 = none, b1 = none;
      for (int i = 0; i < gs; ++i) {
        const u64 c = row[g * gs + i];
        const u64 lo = c < b0 ? c : b0;
        b0 = c > b0 ? c : b0;
        b1 = lo > b1 ? lo : b1;
      }
      rank[g] = a.group_rank == 2 && b1 > none ? sort_key(key_value(b0) + key_value(b1)) : b0;
    }
    __syncwarp();
    for (int g = lane; g < a.n_groups; g += 32) {
      int before = 0;
      for (int h = 0; h < a.n_groups; ++h)
        before += rank[h] > rank[g] || (rank[h] == rank[g] && h < g);
      if (before >= a.topk_groups)
        for (int i = 0; i < gs; ++i) row[g * gs + i] = 0;
    }
    __syncwarp();
  }
  int my_e = 0;
  for (int j = 0; j < a.k; ++j) {
    u64 best = 0;
    int at = 0x7FFFFFFF;
    for (int e = lane; e < a.E; e += 32) {
      const u64 c = row[e];
      if (c > best) {
        best = c;
        at = e;
      }
    }
    const u64 top = warp_max_key(best);
    const int first = __reduce_min_sync(0xFFFFFFFFu, best == top ? at : 0x7FFFFFFF);
    if (at == first) row[first] = 0;
    if (lane == j) my_e = first;
    __syncwarp();
  }
  return my_e;
}

// ------------------------------------------------------------------- groups --
// Which experts of this lane are in groups that stay (bit i: expert lane*NV + i), from
// their keys. A group ranks by its unmasked members alone; one without any ranks last.
// Where a group is a power of two of whole lanes its two largest meet by shuffles, and
// groups that fp32 cannot tell apart at the border are settled here; otherwise through the
// warp's row in shared memory, a lane a group, and *open says that they could not be told apart.
template <int NV>
__device__ __forceinline__ uint32_t keep_groups(const SelArgs& a, int lane, const uint32_t* key,
                                                const float* lrow, float m, bool direct, float top,
                                                double* row, bool* open) {
  const int gs = a.E / a.n_groups;
  const uint32_t none = sort_key(-INFINITY);
  auto rank_of = [&](uint32_t b0, uint32_t b1) {
    return a.group_rank == 2 && b1 > none ? sort_key(key_value(b0) + key_value(b1)) : b0;
  };
  *open = false;
  const int L = gs / NV;
  if (gs % NV == 0 && L <= 32 && (L & (L - 1)) == 0) {
    uint32_t b0 = none, b1 = none;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t c = max(key[i], none);
      b1 = max(b1, min(c, b0));
      b0 = max(b0, c);
    }
    for (int off = 1; off < L; off <<= 1) {
      const uint32_t o0 = __shfl_xor_sync(0xFFFFFFFFu, b0, off);
      const uint32_t o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, off);
      b1 = max(max(b1, o1), min(b0, o0));
      b0 = max(b0, o0);
    }
    const uint32_t rank = rank_of(b0, b1);
    const bool real = lane * NV < a.E;
    bool stays = false;
    uint32_t rest = real ? rank : 0u, low = 0u;
    for (int j = 0; j < a.topk_groups; ++j) {          // the first lane that has it is a head
      low = warp_max_key(rest);
      const int head = __ffs(__ballot_sync(0xFFFFFFFFu, rest == low)) - 1;
      if (((lane ^ head) & -L) == 0) {
        stays = true;
        rest = 0u;
      }
    }
    if (!direct) {
      const float lv = key_value(low);
      const uint32_t high = warp_max_key(rest);
      const float size = rank_size(a, key_value(b0), key_value(b1));
      const float hv = key_value(high),
                  err = rank_err(top, hv, __uint_as_float(warp_max_key(__float_as_uint(size))));
      if (high != 0u && hv > -INFINITY && !(lv - hv > err)) {
        const float v = key_value(rank);
        const bool sure = real && v - hv > err, out = !real || lv - v > err;
        stays = settle_groups(a, row_64(a, lrow, lane, m), lane, L, !sure && !out, sure);
      }
    }
    return stays ? ~0u : 0u;
  }
  uint32_t* crow = reinterpret_cast<uint32_t*>(row);
  uint32_t* rank = crow + a.E;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane * NV + i < a.E) crow[lane * NV + i] = key[i];
  __syncwarp();
  float size = 0.f;
  for (int g = lane; g < a.n_groups; g += 32) {
    uint32_t b0 = none, b1 = none;
    for (int i = 0; i < gs; ++i) {
      const uint32_t c = max(crow[g * gs + i], none);
      b1 = max(b1, min(c, b0));
      b0 = max(b0, c);
    }
    rank[g] = rank_of(b0, b1);
    size = fmaxf(size, rank_size(a, key_value(b0), key_value(b1)));
  }
  __syncwarp();
  uint32_t lo = ~0u, hi = 0u, kept = 0u;   // bit i: group lane + 32 i (up to 1024 groups)
  for (int g = lane, i = 0; g < a.n_groups; g += 32, ++i) {
    const uint32_t v = rank[g];
    int before = 0;
    for (int h = 0; h < a.n_groups; ++h) before += rank[h] > v || (rank[h] == v && h < g);
    if (before < a.topk_groups) {
      kept |= 1u << i;
      lo = min(lo, v);
    } else {
      hi = max(hi, v);
    }
  }
  __syncwarp();
  for (int g = lane, i = 0; g < a.n_groups; g += 32, ++i) rank[g] = (kept >> i) & 1u;
  const float lv = key_value(__reduce_min_sync(0xFFFFFFFFu, lo));
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  const float hv = key_value(hi);
  size = __uint_as_float(warp_max_key(__float_as_uint(size)));
  *open = !direct && hi != 0u && hv > -INFINITY && !(lv - hv > rank_err(top, hv, size));
  __syncwarp();
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane * NV + i;
    if (e < a.E && rank[e / gs]) bits |= 1u << i;
  }
  __syncwarp();
  return bits;
}

// One token: lrow its logits (global or shared), row: the warp's E (2E with groups)
// doubles of shared memory, meet: 32 keys and experts. Writes idx and w.
template <int NV>
__device__ __forceinline__ void select_warp(const SelArgs& a, const float* lrow, bool vec,
                                            const int32_t* __restrict__ forced, int lane,
                                            double* row, uint32_t* meet_key, int* meet_at,
                                            int32_t* __restrict__ idx_out,
                                            float* __restrict__ w_out, int* status) {
  const bool direct = !a.balance && (a.n_groups == 1 || a.group_rank == 1);
  float l[NV];
  load_row<NV>(lrow, a.E, lane, vec, l);
  // the largest logit and the softmax's denominator, where something needs them
  float m = 0.f, rz = 1.f;
  float s[NV] = {};
  if (!direct || !(a.sigmoid || a.renorm)) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
  }
  if (!a.sigmoid && (!direct || !a.renorm)) {
    float z = 0.f;
    if (m == INFINITY) {
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = l[i] == m ? 1.f : 0.f;
    } else {
      const float mm = masked(m) ? 0.f : m;            // all masked: exp(-inf) = 0
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = expf(l[i] - mm);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) z += s[i];
    z = warp_sum(z);
    rz = z > 0.f ? 1.0f / z : 0.f;
  }
  int my_e = 0;
  if (forced) {
    if (lane < a.k) my_e = forced[lane];
  } else {
    uint32_t key[NV];                     // of the choice values
    float top = 0.f;                      // a score's largest error
    if (direct) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = lane * NV + i < a.E ? sort_key(l[i]) : 0u;
    } else {
      top = masked(m) ? 0.f : score_err<NV>(a.sigmoid, m) * (a.sigmoid ? sigmoid_near(m) : rz);
      float bal[NV] = {};
      if (a.balance) {
        if (NV >= 4 && a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.balance) & 15u) == 0) {
#pragma unroll
          for (int i = 0; i + 3 < NV; i += 4)
            if (lane * NV + i < a.E) {
              const float4 b = __ldg(reinterpret_cast<const float4*>(a.balance + lane * NV + i));
              bal[i] = b.x; bal[i + 1] = b.y; bal[i + 2] = b.z; bal[i + 3] = b.w;
            }
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (lane * NV + i < a.E) bal[i] = __ldg(a.balance + lane * NV + i);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float c = (a.sigmoid ? sigmoid_near(l[i]) : s[i] * rz) + bal[i];
        const uint32_t kc = sort_key(masked(l[i]) || c != c ? -INFINITY : c);
        key[i] = lane * NV + i < a.E ? kc : 0u;
      }
    }
    bool open = false;                    // the fp32 scores leave the choice open
    if (a.n_groups > 1) {
      const uint32_t keep = keep_groups<NV>(a, lane, key, lrow, m, direct, top, row, &open);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (!((keep >> i) & 1u)) key[i] = 0u;
    }
    // one value more than is taken: the border
    const int need = direct ? a.k : a.k + 1;
    uint32_t out, last;
    const bool all = largest<NV>(
        key, need, lane, meet_key, meet_at,
        [&](uint32_t tau) {
          const float v = key_value(tau);
          return direct || !(v > -INFINITY) ? tau : sort_key(v - border_err(top, v));
        },
        &out, &my_e, &last);
    if (!direct) {
      // neighbours in the order have to be further apart than their errors (masked
      // experts, all -inf, go by their index)
      uint32_t next = __shfl_down_sync(0xFFFFFFFFu, out, 1);
      if (lane == 31) next = last;
      const float v = key_value(out), nv = key_value(next);
      const bool near = lane < a.k && next != 0u && nv > -INFINITY &&
                        !(v - nv > border_err(top, nv));
      const bool any = __any_sync(0xFFFFFFFFu, near);
      if (any || open) {
        const Row64 r = row_64(a, lrow, lane, m);
        if (all && !open) {
          u64 k64 = key_64(a, r, out ? my_e : -1);
          sort_lanes(k64, my_e, lane);
        } else {
          my_e = choose_64(a, r, lane, reinterpret_cast<u64*>(row));
        }
      }
    }
  }
  // the weights of the slots
  const bool slot = lane < a.k;
  const bool valid = slot && my_e >= 0 && my_e < a.E;
  if (slot && !valid) raise_status(status, MOE_ERR_DEVICE_INDEX);
  const float lj = valid ? fmaxf(lrow[my_e], -INFINITY) : -INFINITY;
  const bool dead = masked(lj);
  float sj;
  if (!a.renorm) {
    sj = dead ? 0.f : a.sigmoid ? sigmoid_of(lj) : exp_below(lj, m) * rz;
  } else {
    // scores up to a common factor e^-r that the quotient drops: r the largest
    // chosen logit, for sigmoids only where it is below 0, so that tiny scores
    // keep their ratios
    float r = warp_max(lj);
    if (a.sigmoid) r = fminf(r, 0.f);
    sj = renorm_score(a.sigmoid, lj, r);
    const float sum = warp_sum(sj);
    sj = sum > 0.f ? sj / sum : 0.f;
  }
  if (slot) {
    idx_out[lane] = my_e;
    w_out[lane] = a.scale * sj;
  }
}

template <int NV>
__global__ void __launch_bounds__(32 * kSelWarps, NV <= 8 ? 8 : 1) select_kernel(
    const __grid_constant__ SelArgs a, const float* __restrict__ logits, const int32_t* __restrict__ forced, int64_t T,
    bool vec, int row_doubles, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
    int* status) {
  pdl_enter();
  extern __shared__ double sel_rows[];
  __shared__ __align__(16) uint32_t meet_key[kSelWarps][32];
  __shared__ int meet_at[kSelWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kSelWarps + warp;
  if (t >= T) return;
  select_warp<NV>(a, logits + t * a.E, vec, forced ? forced + t * a.k : nullptr, lane,
                  sel_rows + (size_t)warp * row_doubles, meet_key[warp], meet_at[warp],
                  topk_idx + t * a.k, topk_w + t * a.k, status);
}

static SelArgs sel_args(const moe_router& r) {
  // (groups that all stay decide nothing)
  return SelArgs{r.E,           r.k,          r.score == MOE_SCORE_SIGMOID,
                 r.topk_groups == r.n_groups ? 1 : r.n_groups,
                 r.topk_groups, r.group_rank, r.renormalise,                r.scale,
                 r.balance};
}

// a second look and groups need E or 2E values of the warp's row
static int sel_row_doubles(const moe_router& r) {
  return r.n_groups > 1 ? 2 * r.E : r.balance ? r.E : 0;
}

template <int NV>
static cudaError_t run_select(const moe_router& r, const float* logits, const int32_t* forced,
                              int64_t T, int32_t* topk_idx, float* topk_w, int* status,
                              cudaStream_t s) {
  const int rd = sel_row_doubles(r);
  const size_t smem = (size_t)kSelWarps * rd * sizeof(double);
  if (smem > 40 * 1024) {                   // (with the kernel's own, 48 KB need no leave)
    // (the most that this instance takes, in every call: another thread's call with fewer experts
    // does not lower it)
    const cudaError_t e =
        cudaFuncSetAttribute(select_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSelWarps * 2 * 32 * NV * (int)sizeof(double));
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
    const __grid_constant__ SelArgs a, const float* __restrict__ part, int ns, int64_t T, const float* __restrict__ bias,
    const int32_t* __restrict__ forced, float* __restrict__ logits,
    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w, int* status) {
  pdl_enter();
  extern __shared__ double sel_rows[];
  __shared__ __align__(16) float lrow[kMaxExperts];
  __shared__ __align__(16) uint32_t meet_key[32];
  __shared__ int meet_at[32];
  const int64_t t = blockIdx.x;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    const float sum = router_small_sum(part, ns, T, t, a.E, e) + (bias ? bias[e] : 0.f);
    lrow[e] = sum;
    logits[t * a.E + e] = sum;
  }
  __syncthreads();
  if (threadIdx.x < 32)
    select_warp<NV>(a, lrow, a.E % 4 == 0, forced ? forced + t * a.k : nullptr, threadIdx.x,
                    sel_rows, meet_key, meet_at, topk_idx + t * a.k, topk_w + t * a.k, status);
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
// Slots that name one expert twice (a caller's own choice) add up in slot order. A slot
// whose expert is masked has weight 0 whatever the others do, so it has no gradient.
//
// Where only the chosen entries get any (all but raw softmax scores) the loads, first idx, then
// the logits there, are what a warp waits for: a slot a lane, 32 / SLOTS tokens a warp, and
// the zeros of the tokens' rows on their way before (16384 tokens of 256 experts, top-8:
// a token a warp and the zeros last 12.3 us, this 8.5).
template <int SLOTS>
__global__ void __launch_bounds__(32 * kSelWarps) select_bwd_chosen_kernel(
    const __grid_constant__ SelArgs a, const float* __restrict__ d_topk_w,
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx, int64_t T,
    int accumulate, bool vec, float* __restrict__ d_logits, int* status) {
  pdl_enter();
  constexpr int TOKENS = 32 / SLOTS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = ((int64_t)blockIdx.x * kSelWarps + warp) * TOKENS;
  if (t0 >= T) return;
  const int seg = lane / SLOTS, j = lane % SLOTS;
  const int64_t t = t0 + seg;
  const bool slot = j < a.k && t < T;
  int my_e = slot ? __ldg(topk_idx + t * a.k + j) : -1;
  float g = slot ? __ldg(d_topk_w + t * a.k + j) : 0.f;
  if (!accumulate) {
    float* rows = d_logits + t0 * a.E;
    const int n = (int)(T - t0 < TOKENS ? T - t0 : TOKENS) * a.E;
    if (vec) {
      for (int i = 4 * lane; i < n; i += 128)
        *reinterpret_cast<float4*>(rows + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int i = lane; i < n; i += 32) rows[i] = 0.f;
    }
  }
  if (slot && (my_e < 0 || my_e >= a.E)) {
    raise_status(status, MOE_ERR_DEVICE_INDEX);
    my_e = -1;
  }
  const float l = my_e >= 0 ? __ldg(logits + t * a.E + my_e) : -INFINITY;
  if (masked(l)) g = 0.f;
  auto sum = [](float v) {
#pragma unroll
    for (int off = SLOTS / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
  };
  float dl;
  if (a.renorm) {
    float r = fmaxf(l, -INFINITY);
#pragma unroll
    for (int off = SLOTS / 2; off > 0; off >>= 1)
      r = fmaxf(r, __shfl_xor_sync(0xFFFFFFFFu, r, off));
    // A constant on all of g changes nothing: less the g of the largest score, whose q may be
    // nearly all of the sum, so that what is left there is not the difference of equal numbers.
    const uint32_t is_top = __ballot_sync(0xFFFFFFFFu, l == r) >> (seg * SLOTS);
    g = (g - __shfl_sync(0xFFFFFFFFu, g, seg * SLOTS + ((__ffs(is_top) - 1) & (SLOTS - 1)))) *
        a.scale;
    if (a.sigmoid) r = fminf(r, 0.f);
    float q = renorm_score(a.sigmoid, l, r);
    const float total = sum(q);
    q = total > 0.f ? q / total : 0.f;
    dl = q * (g - sum(q * g));
    if (a.sigmoid) dl *= sigmoid_of(-l);                      // 1 - s, without its cancellation
  } else {
    dl = g * a.scale * sigmoid_of(l) * sigmoid_of(-l);
  }
  if (masked(l)) dl = 0.f;
  // one lane an expert: the first slot that names it takes the others' terms
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, seg << 16 | (my_e & 0xFFFF));
  const bool first = (same & ((1u << lane) - 1u)) == 0;
  float add = dl;
  if (__any_sync(0xFFFFFFFFu, my_e >= 0 && !first)) {
    add = 0.f;
    for (int i = 0; i < a.k; ++i) {
      const float di = __shfl_sync(0xFFFFFFFFu, dl, seg * SLOTS + i);
      if ((same >> (seg * SLOTS + i)) & 1u) add += di;
    }
  }
  __syncwarp();
  if (my_e >= 0 && first) {
    float* dst = d_logits + t * a.E + my_e;
    *dst = accumulate ? *dst + add : add;
  }
}

// Raw softmax scores: a warp a token, every expert's - p_e (sum_j p_j g_j) written, then the
// chosen entries with their own, p_e (g_e - sum_j p_j g_j). Where a chosen expert * has more than half
// of the row these are differences of nearly equal numbers; a constant on every expert's g (0 where
// it is not chosen) changes nothing, so there they are, less g_*,
//   p_e ((g_e - g_*) - (sum_{chosen, not *} p_j g_j - g_* sum_{not *} p)).
template <int NV>
__global__ void __launch_bounds__(32 * kSelWarps) select_bwd_kernel(
    const __grid_constant__ SelArgs a, const float* __restrict__ d_topk_w,
    const float* __restrict__ logits, const int32_t* __restrict__ topk_idx, int64_t T,
    int accumulate, bool vec, float* __restrict__ d_logits, int* status) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kSelWarps + warp;
  if (t >= T) return;
  const float* lrow = logits + t * a.E;
  float* drow = d_logits + t * a.E;
  const bool slot = lane < a.k;
  int my_e = slot ? topk_idx[t * a.k + lane] : -1;
  float g = slot ? d_topk_w[t * a.k + lane] : 0.f;
  if (slot && (my_e < 0 || my_e >= a.E)) {
    raise_status(status, MOE_ERR_DEVICE_INDEX);
    my_e = -1;
  }
  const float lj = my_e >= 0 ? __ldg(lrow + my_e) : -INFINITY;
  const bool dead = masked(lj);
  if (dead) g = 0.f;
  float l[NV];
  float m = -INFINITY, z = 0.f;
  load_row<NV>(lrow, a.E, lane, vec, l);
#pragma unroll
  for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    l[i] = exp_below(l[i], m);            // from here on the terms themselves
    z += l[i];
  }
  z = warp_sum(z);
  const float p = dead ? 0.f : exp_below(lj, m) / z;
  const float inner = a.scale * warp_sum(p * g);
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, my_e);
  const bool first = (same & ((1u << lane) - 1u)) == 0;
  // the g of all the slots that name this lane's expert
  if (__any_sync(0xFFFFFFFFu, my_e >= 0 && !first)) {
    float all = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const float gj = __shfl_sync(0xFFFFFFFFu, g, j);
      if ((same >> j) & 1u) all += gj;
    }
    g = all;
  }
  float own = a.scale * (p * g) - p * inner;
  const uint32_t most = __ballot_sync(0xFFFFFFFFu, p > 0.5f);
  if (most) {
    const int star = __shfl_sync(0xFFFFFFFFu, my_e, __ffs(most) - 1);
    const float gs = __shfl_sync(0xFFFFFFFFu, g, __ffs(most) - 1);
    float others = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) others += lane * NV + i == star ? 0.f : l[i];
    others = warp_sum(others) / z;
    const float rest = warp_sum(first && my_e >= 0 && my_e != star ? p * g : 0.f) - gs * others;
    own = a.scale * (p * ((g - gs) - rest));
  }
  const float before = accumulate && my_e >= 0 ? drow[my_e] : 0.f;
  __syncwarp();
  const float gz = z > 0.f ? inner / z : 0.f;
  if (NV >= 4 && vec) {
#pragma unroll
    for (int i = 0; i + 3 < NV; i += 4) {
      const int e = lane * NV + i;
      if (e >= a.E) continue;
      float4 v = make_float4(-l[i] * gz, -l[i + 1] * gz, -l[i + 2] * gz, -l[i + 3] * gz);
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
      if (e < a.E) drow[e] = (accumulate ? drow[e] : 0.f) - l[i] * gz;
    }
  }
  __syncwarp();
  if (my_e >= 0 && first) drow[my_e] = before + own;
}

// NV: logits a lane, or CHOSEN: lanes a token
template <int NV, bool CHOSEN>
static cudaError_t run_select_bwd(const moe_router& r, const float* dw, const float* logits,
                                  const int32_t* idx, int64_t T, int accumulate, float* d_logits,
                                  int* status, cudaStream_t s) {
  const bool vec = r.E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 &&
                   (reinterpret_cast<uintptr_t>(d_logits) & 15u) == 0;
  const int tokens = kSelWarps * (CHOSEN ? 32 / NV : 1);           // a block
  const dim3 grid((unsigned)((T + tokens - 1) / tokens)), block(32 * kSelWarps);
  if constexpr (CHOSEN)
    return launch_pdl(pdl_for_tokens(T), select_bwd_chosen_kernel<NV>, grid, block, 0, s,
                      sel_args(r), dw, logits, idx, T, accumulate, vec, d_logits, status);
  else
    return launch_pdl(pdl_for_tokens(T), select_bwd_kernel<NV>, grid, block, 0, s, sel_args(r), dw,
                      logits, idx, T, accumulate, vec, d_logits, status);
}

cudaError_t launch_select_bwd(const moe_router& r, const float* d_topk_w, const float* logits,
                              const int32_t* topk_idx, int64_t T, int accumulate, float* d_logits,
                              int* status, cudaStream_t s) {
  timer_before(MOE_KERNEL_SELECT_BWD, s);
  const int nv = (r.E + 31) / 32;
  const auto run = r.score == MOE_SCORE_SIGMOID || r.renormalise
                       ? (r.k <= 4    ? run_select_bwd<4, true>
                          : r.k <= 8  ? run_select_bwd<8, true>
                          : r.k <= 16 ? run_select_bwd<16, true>
                                      : run_select_bwd<32, true>)
                   : nv <= 1  ? run_select_bwd<1, false>
                   : nv <= 2  ? run_select_bwd<2, false>
                   : nv <= 4  ? run_select_bwd<4, false>
                   : nv <= 8  ? run_select_bwd<8, false>
                   : nv <= 16 ? run_select_bwd<16, false>
                              : run_select_bwd<kMaxExperts / 32, false>;
  const cudaError_t e = run(r, d_topk_w, logits, topk_idx, T, accumulate, d_logits, status, s);
  note_launches(1);
  timer_after(MOE_KERNEL_SELECT_BWD, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
