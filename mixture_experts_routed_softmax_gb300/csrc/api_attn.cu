// api_attn.cu — the C ABI of the attention operators (include/moe.h): argument
// checks, then the launches.
#include <cmath>

#include "attn.cuh"
#include "internal.h"

using namespace moe;

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static int cuda_code(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// a [T, H, D] view: 16-byte aligned, the token stride a multiple of 8 and >= H*D
static int check_view(const void* p, int64_t stride, int64_t H, int D) {
  if (!p || !aligned16(p)) return MOE_ERR_ARG;
  if (stride < H * D || stride % 8 != 0) return MOE_ERR_ARG;
  return MOE_OK;
}
static int check_head_dim(int D) {
  if (D <= 0) return MOE_ERR_ARG;
  return D % 8 != 0 || D > kAttnMaxD ? MOE_ERR_UNSUPPORTED : MOE_OK;
}
static int check_tokens(int64_t T, int64_t H) {
  if (T < 0 || H <= 0) return MOE_ERR_ARG;
  if (T >= ((int64_t)1 << 30) || H > 65536 || T * H > ((int64_t)1 << 30))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static int check_rotary(const moe_rotary* r, int D) {
  if (!r->turns || r->rd < 2 || r->rd > D || r->rd % 2 != 0) return MOE_ERR_ARG;
  if (r->n_axes < 1 || r->n_axes > 8 || !std::isfinite(r->scale)) return MOE_ERR_ARG;
  return MOE_OK;
}
static int check_cache(const moe_kv_cache* c) {
  if (!c || !c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return MOE_ERR_ARG;
  if (c->n_pages <= 0 || c->page_size <= 0 || c->Hkv <= 0) return MOE_ERR_ARG;
  if (c->page_stride <= 0 || c->head_stride <= 0 || c->token_stride <= 0 ||
      c->page_stride % 8 != 0 || c->head_stride % 8 != 0 || c->token_stride % 8 != 0)
    return MOE_ERR_ARG;
  if (c->head_stride < c->D || c->token_stride < c->D) return MOE_ERR_ARG;
  if (c->n_pages >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  return check_head_dim(c->D);
}
static int check_batch(const moe_kv_cache* c, const moe_kv_batch* b) {
  if (!b || b->T < 0 || b->B < 0 || b->max_q < 0 || b->max_pages < 0) return MOE_ERR_ARG;
  if (b->table_stride < b->max_pages) return MOE_ERR_ARG;
  if (b->B > 0 && (!b->cu_q || !b->kv_len)) return MOE_ERR_ARG;
  if (b->B > 0 && b->max_pages > 0 && !b->page_table) return MOE_ERR_ARG;
  if ((int64_t)b->max_pages * c->page_size > kAttnMaxKeys) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

extern "C" {

int moe_rope(const moe_rotary* rot, const int32_t* pos, int64_t T, int D, int transpose,
             const moe_bf16* q, int64_t q_stride, int Hq, moe_bf16* q_out, int64_t qo_stride,
             const moe_bf16* k, int64_t k_stride, int Hk, moe_bf16* k_out, int64_t ko_stride,
             moe_stream_t stream) {
  if (!rot) return MOE_ERR_ARG;
  int rc = check_head_dim(D);
  if (!rc) rc = check_rotary(rot, D);
  if (!rc && k && Hk <= 0) rc = MOE_ERR_ARG;
  if (!rc) rc = Hq <= 0 ? MOE_ERR_ARG : check_tokens(T, (int64_t)Hq + (k ? Hk : 0));
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  if (!pos) return MOE_ERR_ARG;
  rc = check_view(q, q_stride, Hq, D);
  if (!rc) rc = check_view(q_out, qo_stride, Hq, D);
  if (!rc && k) rc = check_view(k, k_stride, Hk, D);
  if (!rc && k) rc = check_view(k_out, ko_stride, Hk, D);
  if (rc) return rc;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  return cuda_code(launch_rope(rot, pos, T, D, transpose, q, q_stride, Hq, q_out, qo_stride, k,
                               k_stride, Hk, k_out, ko_stride, st,
                               reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv_append(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_rotary* rot,
                  const int32_t* pos, const moe_bf16* k, int64_t k_stride, const moe_bf16* v,
                  int64_t v_stride, const moe_bf16* q, int64_t q_stride, int Hq, moe_bf16* q_out,
                  int64_t qo_stride, moe_stream_t stream) {
  int rc = check_cache(cache);
  if (!rc) rc = check_batch(cache, batch);
  if (!rc && rot) rc = check_rotary(rot, cache->D);
  if (!rc && q && Hq <= 0) rc = MOE_ERR_ARG;
  if (!rc) rc = check_tokens(batch->T, (int64_t)cache->Hkv + (q ? Hq : 0));
  if (rc) return rc;
  if (batch->T == 0) return MOE_OK;
  rc = check_view(k, k_stride, cache->Hkv, cache->D);
  if (!rc) rc = check_view(v, v_stride, cache->Hkv, cache->D);
  if (!rc && q) rc = check_view(q, q_stride, Hq, cache->D);
  if (!rc && q) rc = check_view(q_out, qo_stride, Hq, cache->D);
  if (rc) return rc;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  return cuda_code(launch_kv_append(*cache, *batch, rot, pos, k, k_stride, v, v_stride, q,
                                    q_stride, Hq, q_out, qo_stride, st,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_attn_paged_workspace_size(int Hq, int Hkv, int D) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || check_head_dim(D) != MOE_OK) return 0;
  return attn_ws_bytes(D);
}

int moe_attn_paged(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_bf16* q,
                   int64_t q_stride, int Hq, float scale, int causal, int window,
                   const float* sinks, moe_bf16* out, int64_t out_stride, float* lse, void* ws,
                   size_t ws_bytes, moe_stream_t stream) {
  int rc = check_cache(cache);
  if (!rc) rc = check_batch(cache, batch);
  if (rc) return rc;
  if (Hq <= 0 || Hq % cache->Hkv != 0 || window < 0) return MOE_ERR_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return MOE_ERR_ARG;
  rc = check_tokens(batch->T, Hq);
  if (rc) return rc;
  if (batch->T == 0 || batch->B == 0) return MOE_OK;
  rc = check_view(q, q_stride, Hq, cache->D);
  if (!rc) rc = check_view(out, out_stride, Hq, cache->D);
  if (rc) return rc;
  if (!ws || ws_bytes < attn_ws_bytes(cache->D) || (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ARG;
  int* st = device_status_ptr();
  if (!st) return MOE_ERR_CUDA;
  return cuda_code(launch_attn(*cache, *batch, q, q_stride, Hq, scale, causal, window, sinks, out,
                               out_stride, lse, ws, st, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
