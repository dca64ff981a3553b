// api_router.cu — the C ABI of the scored router (include/moe.h): argument
// checks, then the launches.
#include <cmath>

#include "common.cuh"
#include "internal.h"

using namespace moe;

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
static int cuda_code(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

static int check_router(const moe_router* r) {
  if (!r || r->E <= 0 || r->k <= 0 || r->k > r->E) return MOE_ERR_ARG;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_ARG;
  if (r->n_groups < 1 || r->E % r->n_groups != 0) return MOE_ERR_ARG;
  if (r->topk_groups < 1 || r->topk_groups > r->n_groups) return MOE_ERR_ARG;
  if (r->group_rank != 1 && r->group_rank != 2) return MOE_ERR_ARG;
  if (r->k > (int64_t)r->topk_groups * (r->E / r->n_groups)) return MOE_ERR_ARG;
  if (!std::isfinite(r->scale) || !aligned4(r->balance)) return MOE_ERR_ARG;
  if (r->E > kMaxExperts || r->k > kMaxTopK) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static int check_T(int64_t T) {
  return T < 0 ? MOE_ERR_ARG : T >= ((int64_t)1 << 31) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

extern "C" {

int moe_select(const moe_router* router, const float* logits, const int32_t* forced_idx, int64_t T,
               int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  int rc = check_router(router);
  if (!rc) rc = check_T(T);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_ARG;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  return cuda_code(launch_select(*router, logits, forced_idx, T, topk_idx, topk_w, st,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

int moe_select_bwd(const moe_router* router, const float* d_topk_w, const float* logits,
                   const int32_t* topk_idx, int64_t T, int accumulate, float* d_logits,
                   moe_stream_t stream) {
  int rc = check_router(router);
  if (!rc) rc = check_T(T);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!d_topk_w || !logits || !topk_idx || !d_logits || d_logits == logits) return MOE_ERR_ARG;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  return cuda_code(launch_select_bwd(*router, d_topk_w, logits, topk_idx, T, accumulate, d_logits,
                                     st, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_route_scored(const moe_router* router, const moe_bf16* x, const float* w_router,
                     const float* bias, const int32_t* forced_idx, int64_t T, int d,
                     float* logits, int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                     moe_stream_t stream) {
  int rc = check_router(router);
  if (!rc) rc = check_T(T);
  if (!rc && d <= 0) rc = MOE_ERR_ARG;
  if (!rc && d % 8 != 0) rc = MOE_ERR_UNSUPPORTED;
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!w_router || !x || !logits || !topk_idx || !topk_w || !aligned16(x)) return MOE_ERR_ARG;
  const int E = router->E;
  if (!ws || ws_bytes < route_ws_bytes(T, d, E) || !aligned256(ws)) return MOE_ERR_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  if (route_is_small(T)) {
    int ns = 0;
    cudaError_t e = launch_router_small_partial(x, w_router, T, d, E, ws, &ns, s);
    if (e == cudaSuccess)
      e = launch_select_small(*router, static_cast<const float*>(ws), ns, T, bias, forced_idx,
                              logits, topk_idx, topk_w, st, s);
    return cuda_code(e);
  }
  cudaError_t e = launch_router_logits(x, w_router, bias, T, d, E, logits, ws, st, s);
  if (e == cudaSuccess)
    e = launch_select(*router, logits, forced_idx, T, topk_idx, topk_w, st, s);
  return cuda_code(e);
}

size_t moe_logits_bwd_workspace_size(int64_t T, int d, int E, int dense) {
  if (check_T(T) || d <= 0 || E <= 0 || d % 8 != 0 || E > kMaxExperts) return 0;
  return logits_bwd_ws_bytes(T, d, E, dense);
}

int moe_logits_bwd(const float* d_logits, const float* w_router, const moe_bf16* x, int64_t T,
                   int d, int E, int dense, int k, int S, moe_bf16* dx_inout, const float* dxp,
                   const int32_t* dst_row, float* dw_router, float* dbias, void* ws,
                   size_t ws_bytes, moe_stream_t stream) {
  int rc = check_T(T);
  if (rc) return rc;
  if (d <= 0 || E <= 0 || k < 0 || S < 0 || !w_router || !dw_router) return MOE_ERR_ARG;
  if (E > kMaxExperts || k + S > kMaxTopK || d % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!d_logits || !x || !dx_inout)) return MOE_ERR_ARG;
  if (dxp && ((T > 0 && !dst_row) || !aligned16(dxp))) return MOE_ERR_ARG;
  if (!aligned16(x) || !aligned16(dx_inout)) return MOE_ERR_ARG;
  if (!ws || ws_bytes < logits_bwd_ws_bytes(T, d, E, dense) || !aligned256(ws)) return MOE_ERR_ARG;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  return cuda_code(launch_logits_bwd(d_logits, w_router, x, T, d, E, dense, k, S, dx_inout, dxp,
                                     dst_row, dw_router, dbias, ws, st,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
