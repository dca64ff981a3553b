// api_w4.cu — the C ABI of the 4-bit weights (include/moe.h): argument checks,
// then the launches.
#include "internal.h"
#include "w4.cuh"

using namespace moe;

static bool on(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
static int cuda_code(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
static size_t al256w(size_t b) { return (b + 255) & ~(size_t)255; }

static int check_dims(int E, int K, int N) {
  if (E <= 0 || K <= 0 || N <= 0) return MOE_ERR_ARG;
  if (E > kMaxExperts || K % 8 != 0 || N % 8 != 0 || K > 65536 || N > 65536)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }
static int check_w4(const moe_w4* w) {
  if (!w || !w->codes || !w->scales || !on(w->codes, 16) || !on(w->scales, 16)) return MOE_ERR_ARG;
  if (w->kind != MOE_W4_INT4 && w->kind != MOE_W4_FP4) return MOE_ERR_ARG;
  if (!group_ok(w->group)) return MOE_ERR_ARG;
  return check_dims(w->E, w->K, w->N);
}
static int check_T(int64_t T) {
  return T < 0 ? MOE_ERR_ARG : T >= ((int64_t)1 << 26) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// Few rows go through the rows kernel (w4_rows.cu), many through tensor memory
// (w4_tiles.cu). The rows kernel takes 32 rows at a time, K over a block's warps; small matrices
// leave it few blocks. Measured, rows against tiles: 8192 x 8192, 8 rows 14.5 against 16 us, 16
// rows 26 against 16; 4096 x 2880, 16 rows 7.6 against 10.3, 32 rows 13.3 against 10.3; 2048 x
// 2048, 64 rows 9.4 against 8.9; 4096 x 512, 32 rows 7.6 against 9.5, 64 rows 14.1 against 10.1;
// 1024 x 1024, 64 rows 5.6 against 8.0, 128 rows 10.2 against 9.0; 128 x 128, 64 rows 3.2 against
// 4.8, 128 rows 5.5 against 5.6, 2048 rows 75 against 7.6. Experts, int4 in groups of 32, by rows an expert on average: 2048 x 768, top-8 of
// 128, 2 rows 90 against 110 us, 4 122 against 127, 8 231 against 139; 2880 x 2880, top-4 of 32, 4
// rows 130 against 140 us, 8 217 against 157; 2560 x 640, top-10 of 512, 640 pairs 310 against 294,
// 1280 pairs 439 against 377 (a block of the rows kernel looks through all of them). All without
// shared experts, which get every token and are not counted: 64 tokens, top-8 of 128 of 2048 x 768,
// 119 us with none, 154 with one.
static bool linear_by_tiles(int64_t T, int K, int N) {
  return T > 8 && (T > 96 || T * K > 180000 || (double)T * K * N > 3.4e8);
}
static bool experts_by_tiles(int64_t T, int k, int E) {
  return T * k > kRowsMaxPairs || T * k > (int64_t)4 * E;
}

// A as two bf16 numbers, its rounding and the rest of it: two columns of the rows kernel's down
// products, which have columns to spare where an expert gets few rows (with it y is off by its own
// rounding alone, 0.0017 of its size, else by 0.0024). Up to a row an expert on average it costs
// 3% at most (16 tokens, top-8 of 128 experts: 71 against 69 us); at two 8%, at four 36%.
static bool split_A(int64_t T, int k, int E) {
  return !experts_by_tiles(T, k, E) && T * k <= E;
}

// The workspace of the experts' forward.
struct ExpertWs {
  size_t A, yp, xp, counts, offsets, dst_row, src_pair, permute, total;
  int64_t R_cap;
};
constexpr int kTileAlign = 16;
static ExpertWs expert_ws(int64_t T, int k, int E, int S, int d, int f) {
  ExpertWs w{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += al256w(bytes);
    return was;
  };
  const bool tiles = experts_by_tiles(T, k, E);
  w.R_cap = T * (k + S) + (tiles ? (int64_t)(E + S) * (kTileAlign - 1) : 0);
  w.A = take((size_t)w.R_cap * f * (split_A(T, k, E) ? 4 : 2));
  w.yp = take((size_t)w.R_cap * d * 4);
  if (tiles) {
    w.xp = take((size_t)w.R_cap * d * 2);
    w.counts = take((size_t)(E + S) * 4);
    w.offsets = take((size_t)(E + S + 1) * 8);
    w.dst_row = take((size_t)T * (k + S) * 4);
    w.src_pair = take((size_t)w.R_cap * 4);
    w.permute = take(permute_ws_bytes(T, k, E));
  }
  w.total = at;
  return w;
}

extern "C" {

size_t moe_w4_codes_bytes(int E, int K, int N) {
  return check_dims(E, K, N) ? 0 : (size_t)E * w4_codes_per_expert(K, N);
}
size_t moe_w4_scales_bytes(int E, int K, int N, int group) {
  return check_dims(E, K, N) || !group_ok(group)
             ? 0
             : w4_flags_at(E, K, N, group) * sizeof(moe_bf16) + ((size_t)E * 4 + 15) / 16 * 16;
}

int moe_w4_quantise(const moe_w4* w, const moe_bf16* src, moe_stream_t stream) {
  const int rc = check_w4(w);
  if (rc) return rc;
  if (!src || !on(src, 16)) return MOE_ERR_ARG;
  return cuda_code(launch_w4_pack(*w, src, nullptr, nullptr,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

int moe_w4_pack(const moe_w4* w, const uint8_t* codes, const moe_bf16* scales,
                moe_stream_t stream) {
  const int rc = check_w4(w);
  if (rc) return rc;
  if (!codes || !scales || !on(codes, 8) || !on(scales, 2)) return MOE_ERR_ARG;
  return cuda_code(launch_w4_pack(*w, nullptr, codes, scales,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

int moe_w4_dequantise(const moe_w4* w, moe_bf16* dst, moe_stream_t stream) {
  const int rc = check_w4(w);
  if (rc) return rc;
  if (!dst || !on(dst, 16)) return MOE_ERR_ARG;
  return cuda_code(launch_w4_unpack(*w, dst, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_w4_linear_workspace_size(const moe_w4* w, int64_t T) {
  if (!w || check_dims(w->E, w->K, w->N) || check_T(T) || !linear_by_tiles(T, w->K, w->N)) return 0;
  const int n = w4_linear_splits(T, w->K, w->N);
  return n > 1 ? (size_t)n * T * w->N * sizeof(float) : 0;
}

int moe_w4_linear(const moe_w4* w, const moe_bf16* x, int64_t x_stride, int64_t T, void* y,
                  int64_t y_stride, int y_fp32, void* ws, size_t ws_bytes, moe_stream_t stream) {
  int rc = check_w4(w);
  if (!rc) rc = check_T(T);
  if (rc) return rc;
  if (w->E != 1) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !y || !on(x, 16) || !on(y, y_fp32 ? 4 : 2)) return MOE_ERR_ARG;
  if (x_stride < w->K || x_stride % 8 != 0 || y_stride < w->N) return MOE_ERR_ARG;
  const size_t need = moe_w4_linear_workspace_size(w, T);
  if (need && (!ws || ws_bytes < need || !on(ws, 256))) return MOE_ERR_ARG;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return cuda_code(linear_by_tiles(T, w->K, w->N)
                       ? launch_w4_linear_tiles(*w, x, x_stride, T, y, y_stride, y_fp32,
                                                static_cast<float*>(ws), st, s)
                       : launch_w4_linear_rows(*w, x, x_stride, T, y, y_stride, y_fp32, st, s));
}

size_t moe_expert_fwd_w4_workspace_size(int64_t T, int k, int E, int S, int d, int f) {
  if (check_T(T) || T == 0 || k <= 0 || k > E || S < 0 || k + S > kMaxTopK ||
      check_dims(E + S, d, f))
    return 0;
  return expert_ws(T, k, E, S, d, f).total;
}

int moe_expert_fwd_w4(const moe_w4* gate, const moe_w4* up, const moe_w4* down,
                      const moe_swiglu* act, const moe_bf16* x, const int32_t* topk_idx,
                      const float* topk_w, int64_t T, int k, int E, int S, moe_bf16* y, void* ws,
                      size_t ws_bytes, moe_stream_t stream) {
  int rc = check_w4(gate);
  if (!rc) rc = check_w4(up);
  if (!rc) rc = check_w4(down);
  if (!rc) rc = check_T(T);
  if (rc) return rc;
  if (k <= 0 || E <= 0 || k > E || S < 0) return MOE_ERR_ARG;
  if (k + S > kMaxTopK) return MOE_ERR_UNSUPPORTED;
  const int d = gate->K, f = gate->N;
  if (gate->E != E + S || up->E != E + S || down->E != E + S || up->K != d || up->N != f ||
      down->K != f || down->N != d)
    return MOE_ERR_ARG;
  if (up->kind != gate->kind || up->group != gate->group) return MOE_ERR_ARG;
  W4Experts q{};
  if (!act) {
    q.act = ActParams{INFINITY, 1.0f, 0.0f};
  } else {
    if (!(act->limit > 0.0f) || act->alpha != act->alpha || act->up_offset != act->up_offset)
      return MOE_ERR_ARG;
    q.act = ActParams{act->limit, act->alpha, act->up_offset};
  }
  if (T == 0) return MOE_OK;
  if (!x || !topk_idx || !topk_w || !y || !on(x, 16) || !on(y, 16)) return MOE_ERR_ARG;
  if (!ws || !on(ws, 256) || ws_bytes < moe_expert_fwd_w4_workspace_size(T, k, E, S, d, f))
    return MOE_ERR_ARG;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  q.gate = gate;
  q.up = up;
  q.down = down;
  q.k = k;
  q.E = E;
  q.S = S;
  q.d = d;
  q.f = f;
  q.T = T;
  q.x = x;
  q.topk_idx = topk_idx;
  q.topk_w = topk_w;
  const ExpertWs w = expert_ws(T, k, E, S, d, f);
  if (w.R_cap >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  char* p = static_cast<char*>(ws);
  moe_bf16* A = reinterpret_cast<moe_bf16*>(p + w.A);
  float* yp = reinterpret_cast<float*>(p + w.yp);
  if (!experts_by_tiles(T, k, E)) {
    const int64_t lo = split_A(T, k, E) ? w.R_cap * f : 0;
    return cuda_code(launch_w4_experts_rows(q, A, lo, yp, y, st, s));
  }
  moe_bf16* xp = reinterpret_cast<moe_bf16*>(p + w.xp);
  int64_t* offsets = reinterpret_cast<int64_t*>(p + w.offsets);
  int32_t* dst_row = reinterpret_cast<int32_t*>(p + w.dst_row);
  cudaError_t e = launch_permute(topk_idx, T, k, E, S, kTileAlign, x, d, w.R_cap,
                                 reinterpret_cast<int32_t*>(p + w.counts), offsets, dst_row,
                                 reinterpret_cast<int32_t*>(p + w.src_pair), xp, p + w.permute, st,
                                 s);
  if (e == cudaSuccess) e = launch_w4_experts_tiles(q, xp, offsets, w.R_cap, A, yp, st, s);
  if (e == cudaSuccess) e = launch_combine(yp, dst_row, topk_w, T, k, S, d, y, s);
  return cuda_code(e);
}

}  // extern "C"
