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
// fp32 scores whose error has a bound (score_err, below); a token where two values
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
// Bounds of a score's error, relative to the largest score of the row, in units of
// 2^-24 (half an fp32 step). Sigmoid, 1 / (1 + e): expf within 2 steps, 1 + e and the
// quotient half a step each: 6 halves. Softmax, e (1 / Z): the argument's rounding
// moves e by at most |x| e^x < 0.4 halves of the largest, expf 4 halves, the same again
// for the terms of Z, Z's NV + 5 additions one half each, its inverse and the product one
// each. The balance's addition is a half of the value itself (border_err).
template <int NV>
__device__ __forceinline__ float score_err(bool sigmoid) {
  return (sigmoid ? 6.f : (float)(NV + 5 + 11)) * 5.9604645e-8f;
}
// how far apart two values near v have to be to be told apart (and scores below
// fp32's normal range, which have fewer bits, never are)
__device__ __forceinline__ float border_err(float score, float v) {
  return 2.f * score + 2.3841858e-7f * fabsf(v) + 1e-37f;
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
template <typename K>
__device__ __forceinline__ K sort_lane_keys(K key, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int off = size >> 1; off > 0; off >>= 1) {
      const K ok = __shfl_xor_sync(0xFFFFFFFFu, key, off);
      const bool first = ((lane & off) == 0) == ((lane & size) == 0 || size == 32);
      key = (key > ok) == first ? key : ok;
    }
  return key;
}

// The `need` <= 33 largest keys in order, ties to the lower expert: lane j gets the j-th's
// key and expert (key 0: there are no more), *last the 33rd's key.
// The need-th largest of the lanes' own largest is a floor for the need-th largest of
// all: what reaches it (or floor_of(it), somewhat lower) is seldom more than 32 keys, which
// meet in shared memory (`meet`, 32 entries) and are sorted, a key a lane: true, the lanes
// hold every key of at least floor_of(the need-th). With more of them (ties, masked
// rows, need = 33) the keys are taken one by one: false.
template <int NV, typename K, typename F>
__device__ __forceinline__ bool largest(K* key, int need, int lane, K* meet_key, int* meet_at,
                                        F floor_of, K* out, int* at_out, K* last) {
  K mine = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) mine = key[i] > mine ? key[i] : mine;
  *last = 0;
  if (NV == 1) {
    *out = key[0];
    *at_out = lane;
    if (need <= 32) {
      sort_lanes(*out, *at_out, lane);
      return true;
    }
  } else if (need <= 32) {
    const K tau = __shfl_sync(0xFFFFFFFFu, sort_lane_keys(mine, lane), need - 1);
    const K floor = tau ? floor_of(tau) : (K)1;
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
      __syncwarp();
      *out = lane < total ? meet_key[lane] : (K)0;
      *at_out = lane < total ? meet_at[lane] : 0x7FFFFFFF;
      __syncwarp();
      sort_lanes(*out, *at_out, lane);
      return true;
    }
  }
  *out = 0;
  *at_out = 0x7FFFFFFF;
  for (int j = 0; j < need; ++j) {
    const K best = warp_max_key(mine);
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
        mine = key[i] > mine ? key[i] : mine;
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
// lane; the softmax's denominator, which needs every expert's, is summed from
// exponentials of a dozen operations (whole row in 64 bits with exp() and a division an
// expert: 22 us at the end of a call at 512 experts).

// 2^(j / 32)
__device__ const double kExp2_32[32] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002};

// sum of exp(l - m) over the row, to 2^-46: 2^(k / 32) from a table (lane j holds 2^(j / 32))
// times the Taylor series of the rest r, |r| <= log(2) / 64 (r^6 / 720 < 2^-48; k times the
// rounding of log(2) / 32 < 2^-47). Terms below
// 2^-60 of the largest are left out.
static __device__ __noinline__ double denominator_64(const float* lrow, int E, int lane, float m) {
  const double tab = kExp2_32[lane], md = (double)m;
  double z = 0.0;
#pragma unroll 4
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const float l = e < E ? fmaxf(lrow[e], -INFINITY) : -INFINITY;
    const bool in = l - m > -42.f || l == m;             // (both infinite: 1)
    const float kf = in && l != m ? rintf((l - m) * 46.166241f) : 0.f;   // 32 / log(2)
    const double x = in && l != m ? (double)l - md : 0.0;
    const int k = (int)kf;
    const double r = fma((double)kf, -0.021660849392498290, x);          // log(2) / 32
    const double t = __shfl_sync(0xFFFFFFFFu, tab, k & 31);
    double q = fma(r, 1.0 / 120, 1.0 / 24);
    q = fma(q, r, 1.0 / 6);
    q = fma(q, r, 0.5);
    q = fma(q, r, 1.0);
    q = fma(q, r, 1.0);
    const double v = q * __longlong_as_double(__double_as_longlong(t) + ((long long)(k >> 5) << 52));
    z += in ? v : 0.0;
  }
  return warp_sum(z);
}

struct Row64 {          // what a 64-bit choice value needs
  const float* lrow;
  float m;              // softmax: the largest logit, and the denominator
  double z;
};
__device__ __forceinline__ Row64 row_64(const SelArgs& a, const float* lrow, int lane, float m) {
  return Row64{lrow, m, a.sigmoid || masked(m) ? 1.0 : denominator_64(lrow, a.E, lane, m)};
}
// the sort key of expert e's choice value
static __device__ __noinline__ u64 key_64(const SelArgs& a, const Row64& r, int e) {
  const float l = r.lrow[e];
  const u64 none = sort_key(-(double)INFINITY);
  if (masked(l)) return none;
  const double v = exp(a.sigmoid ? -(double)l : l == r.m ? 0.0 : (double)l - (double)r.m);
  double c = a.sigmoid ? 1.0 / (1.0 + v) : v / r.z;
  if (a.balance) c += (double)__ldg(a.balance + e);
  return c == c ? sort_key(c) : none;
}

// The groups' border: `rank` is this lane's group's rank in fp32 (lanes L * g hold group
// g's, n_groups <= 32), sure and kept by the fp32 ranks or in question. Those in question are
// ranked again. Returns whether this lane's group stays.
static __device__ __noinline__ bool settle_groups(const SelArgs& a, const Row64& r, int lane, int L,
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
      const u64 c = i0 + lane < gs ? key_64(a, r, g * gs + i0 + lane) : none;
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
static __device__ __noinline__ int choose_64(const SelArgs& a, const Row64& r, int lane, u64* row) {
  const u64 none = sort_key(-(double)INFINITY);
  for (int e = lane; e < a.E; e += 32) row[e] = key_64(a, r, e);
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
    const int g = lane / L;
    int before = 0;
    for (int h = 0; h < a.n_groups; ++h) {
      const uint32_t r = __shfl_sync(0xFFFFFFFFu, rank, h * L);
      before += r > rank || (r == rank && h < g);
    }
    const bool real = g < a.n_groups;
    bool stays = real && before < a.topk_groups;
    if (!direct) {
      // ranks of two carry two errors
      const float lv = key_value(__reduce_min_sync(0xFFFFFFFFu, stays ? rank : ~0u));
      const uint32_t high = __reduce_max_sync(0xFFFFFFFFu, real && !stays ? rank : 0u);
      const float hv = key_value(high), err = 2.f * border_err(top, hv);
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
  for (int g = lane; g < a.n_groups; g += 32) {
    uint32_t b0 = none, b1 = none;
    for (int i = 0; i < gs; ++i) {
      const uint32_t c = max(crow[g * gs + i], none);
      b1 = max(b1, min(c, b0));
      b0 = max(b0, c);
    }
    rank[g] = rank_of(b0, b1);
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
  *open = !direct && hi != 0u && hv > -INFINITY && !(lv - hv > 2.f * border_err(top, hv));
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
      top = score_err<NV>(a.sigmoid) * (a.sigmoid ? masked(m) ? 0.f : sigmoid_of(m) : rz);
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
        const float c = (a.sigmoid ? sigmoid_of(l[i]) : s[i] * rz) + bal[i];
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
    const bool all = largest<NV, uint32_t>(
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
          u64 k64 = out ? key_64(a, r, my_e) : 0ull;
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
    sj = dead ? 0.f
              : !a.sigmoid ? exp_below(lj, r)
                           : lj >= 0.f ? sigmoid_of(lj) : expf(lj - r) / (1.0f + expf(lj));
    const float sum = warp_sum(sj);
    sj = sum > 0.f ? sj / sum : 0.f;
  }
  if (slot) {
    idx_out[lane] = my_e;
    w_out[lane] = a.scale * sj;
  }
}

template <int NV>
__global__ void __launch_bounds__(32 * kSelWarps) select_kernel(
    SelArgs a, const float* __restrict__ logits, const int32_t* __restrict__ forced, int64_t T,
    bool vec, int row_doubles, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
    int* status) {
  pdl_enter();
  extern __shared__ double sel_rows[];
  __shared__ uint32_t meet_key[kSelWarps][32];
  __shared__ int meet_at[kSelWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kSelWarps + warp;
  if (t >= T) return;
  select_warp<NV>(a, logits + t * a.E, vec, forced ? forced + t * a.k : nullptr, lane,
                  sel_rows + (size_t)warp * row_doubles, meet_key[warp], meet_at[warp],
                  topk_idx + t * a.k, topk_w + t * a.k, status);
}

static SelArgs sel_args(const moe_router& r) {
  return SelArgs{r.E,           r.k,          r.score == MOE_SCORE_SIGMOID, r.n_groups,
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
  __shared__ uint32_t meet_key[32];
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
                                : lj >= 0.f ? sigmoid_of(lj) : expf(lj - r) / (1.0f + expf(lj));
    const float sum = warp_sum(q);
    q = sum > 0.f ? q / sum : 0.f;
    inner = warp_sum(q * g);
    dl = q * (g - inner);
    if (a.sigmoid) dl = dead ? 0.f : dl * sigmoid_of(-lj);     // 1 - s, without its cancellation
  } else if (a.sigmoid) {
    dl = dead ? 0.f : g * sigmoid_of(lj) * sigmoid_of(-lj);
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
