// logits_bwd.cu — from the gradient of the router's logits to those of its
// weight, its bias and the layer's input: with logits = x W_r + b,
//   dW_r = x^T dl      db = column sums of dl      dx (+)= dl W_r^T
// dx also takes the permute's transpose when dXp is given, in the same pass.
//
// dW_r runs on the tensor cores as in the softmax router's backward: dl is split
// exactly into three bf16 parts side by side, and products of bf16 values are
// exact in fp32. For dx there are two forms. Rows with a few entries
// (renormalised or sigmoid scores: the chosen experts) gather those rows of
// W_r^T, k d fp32 products a token. Dense rows go through the tensor cores: the
// first two parts of dl (16 significant bits; dx itself keeps 8) against the three
// parts of W_r^T. Measured at 8192 tokens of 512 experts, d = 2560: 203 us with 10 entries a
// row, 395 dense (the bytes alone take 22 us at the copy's rate); 16384 tokens of 256, d = 2048: 192
// with 8 entries, 385 dense.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {

static inline size_t al256l(size_t b) { return (b + 255) & ~(size_t)255; }
static inline int round8l(int v) { return (v + 7) & ~7; }

constexpr int kBiasRows = 128;      // rows a block sums for db
constexpr int kTokWarps = 4;

struct LogitsBwdWs {
  size_t dl3, dl2, wt, part, bias, total;
  int sp_w, sp_x;
};
static LogitsBwdWs logits_bwd_ws(int64_t T, int d, int E, bool dense) {
  LogitsBwdWs w{};
  const int E8 = round8l(E), N3 = 3 * E8;
  w.sp_w = router_wgrad_ksplit(T, d, N3);
  w.sp_x = dense && T > 0 ? router_ksplit(T, 2 * E8, d) : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += al256l(bytes);
    return was;
  };
  w.dl3 = take((size_t)T * N3 * 2);
  w.dl2 = take(dense ? (size_t)T * 2 * E8 * 2 : 0);
  w.wt = take(dense ? (size_t)3 * 2 * E8 * d * 2 : (size_t)E * d * 4);
  w.bias = take((size_t)((T + kBiasRows - 1) / kBiasRows) * E * 4);
  // the two products' partials, one after the other
  w.part = take(std::max((size_t)w.sp_w * d * N3 * 4, (size_t)w.sp_x * T * d * 4));
  w.total = at;
  return w;
}
size_t logits_bwd_ws_bytes(int64_t T, int d, int E, int dense) {
  return logits_bwd_ws(T, d, E, dense != 0).total;
}

// dl [T, E] -> its three bf16 parts side by side (columns >= E are zeros), and
// for the dense form the first two of them
__global__ void __launch_bounds__(256) split_dl_kernel(const float* __restrict__ dl, int64_t T,
                                                       int E, int E8, moe_bf16* __restrict__ dl3,
                                                       moe_bf16* __restrict__ dl2) {
  pdl_enter();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= T * E8) return;
  const int64_t t = i / E8;
  const int e = (int)(i - t * E8);
  const float v = e < E ? dl[t * E + e] : 0.f;
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  const float r1 = v - __bfloat162float(hi);
  const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
  const __nv_bfloat16 lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
  moe_bf16* row = dl3 + t * 3 * E8 + e;
  row[0] = __bfloat16_as_ushort(hi);
  row[E8] = __bfloat16_as_ushort(mid);
  row[2 * E8] = __bfloat16_as_ushort(lo);
  if (dl2) {
    dl2[t * 2 * E8 + e] = __bfloat16_as_ushort(hi);
    dl2[t * 2 * E8 + E8 + e] = __bfloat16_as_ushort(mid);
  }
}

// db's partial sums: block (chunk, column block) adds its rows, eight row lanes in
// row order each, then the lanes in order
__global__ void __launch_bounds__(256) bias_part_kernel(const float* __restrict__ dl, int64_t T,
                                                        int E, float* __restrict__ part) {
  pdl_enter();
  __shared__ float sums[8][32];
  const int e = blockIdx.y * 32 + threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.x * kBiasRows;
  float a = 0.f;
#pragma unroll 4
  for (int i = threadIdx.y; i < kBiasRows; i += 8)
    if (e < E && r0 + i < T) a += dl[(r0 + i) * E + e];
  sums[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && e < E) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
    part[(int64_t)blockIdx.x * E + e] = s;
  }
}

// W_r [d, E] -> W_r^T: fp32 [E, d], or (planes) its three bf16 parts, each
// [2 E8, d] with the matrix twice below one another, rows >= E zeros
__global__ void transpose_wr_kernel(const float* __restrict__ wr, int d, int E, int E8,
                                    float* __restrict__ out, moe_bf16* __restrict__ planes) {
  pdl_enter();
  __shared__ float tile[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  for (int i = threadIdx.y; i < 32; i += 8) {
    const int r = blockIdx.y * 32 + i;
    tile[i][threadIdx.x] = (r < d && c < E) ? wr[(int64_t)r * E + c] : 0.f;
  }
  __syncthreads();
  const int r2 = blockIdx.y * 32 + threadIdx.x;
  for (int i = threadIdx.y; i < 32; i += 8) {
    const int c2 = blockIdx.x * 32 + i;
    if (r2 >= d || c2 >= (planes ? E8 : E)) continue;
    const float v = tile[threadIdx.x][i];
    if (!planes) {
      out[(int64_t)c2 * d + r2] = v;
      continue;
    }
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    const float r1 = v - __bfloat162float(hi);
    const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
    const __nv_bfloat16 lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
    const int64_t plane = (int64_t)2 * E8 * d, at = (int64_t)c2 * d + r2, twin = (int64_t)E8 * d;
    planes[at] = planes[at + twin] = __bfloat16_as_ushort(hi);
    planes[plane + at] = planes[plane + at + twin] = __bfloat16_as_ushort(mid);
    planes[2 * plane + at] = planes[2 * plane + at + twin] = __bfloat16_as_ushort(lo);
  }
}

// One warp a token: dx[t] (old dx, or the sum of the token's dXp rows) plus the
// router's term: the sum over the row's non-zero entries of dl_e W_r[:, e]
// (entries gathered into shared memory once, any number of them), or the chunks'
// partials of the dense product in order. fp32, rounded to bf16 once.
__global__ void __launch_bounds__(32 * kTokWarps) logits_dx_kernel(
    const float* __restrict__ dl, const float* __restrict__ wrT, const float* __restrict__ part,
    int ksplit, int64_t T, int d, int E, int k, int S, moe_bf16* __restrict__ dx,
    const float* __restrict__ dxp, const int32_t* __restrict__ dst_row) {
  pdl_enter();
  extern __shared__ float2 entries[];        // [kTokWarps][E]: value, expert
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kTokWarps + warp;
  if (t >= T) return;
  float2* mine = entries + (size_t)warp * E;
  int n = 0;
  if (!part) {
    for (int e0 = 0; e0 < E; e0 += 32) {
      const float v = e0 + lane < E ? __ldg(dl + t * E + e0 + lane) : 0.f;
      const uint32_t some = __ballot_sync(0xFFFFFFFFu, v != 0.f);
      if (v != 0.f)
        mine[n + __popc(some & ((1u << lane) - 1u))] = make_float2(v, __int_as_float(e0 + lane));
      n += __popc(some);
    }
    __syncwarp();
  }
  const int slots = k + S;
  int r = -1;
  if (dxp) {
    if (lane < k) r = dst_row[t * k + lane];
    else if (lane < slots) r = dst_row[T * k + (int64_t)(lane - k) * T + t];
  }
  moe_bf16* dxr = dx + t * d;
  for (int c0 = 0; c0 < d; c0 += 256) {      // every lane runs along: the shuffles need the warp
    const int c = c0 + lane * 8;
    const bool in = c < d;
    float acc[8] = {};
    auto add8 = [&](const float* src, float f) {
      const float4 p = __ldg(reinterpret_cast<const float4*>(src));
      const float4 q = __ldg(reinterpret_cast<const float4*>(src) + 1);
      acc[0] = fmaf(f, p.x, acc[0]); acc[1] = fmaf(f, p.y, acc[1]);
      acc[2] = fmaf(f, p.z, acc[2]); acc[3] = fmaf(f, p.w, acc[3]);
      acc[4] = fmaf(f, q.x, acc[4]); acc[5] = fmaf(f, q.y, acc[5]);
      acc[6] = fmaf(f, q.z, acc[6]); acc[7] = fmaf(f, q.w, acc[7]);
    };
    if (dxp) {
#pragma unroll 4
      for (int j = 0; j < slots; ++j) {
        const int rj = __shfl_sync(0xFFFFFFFFu, r, j);
        if (in && rj >= 0) add8(dxp + (int64_t)rj * d + c, 1.f);
      }
    } else if (in) {
      unpack8(*reinterpret_cast<const uint4*>(dxr + c), acc);
    }
    if (!in) continue;
    if (part) {
      for (int sp = 0; sp < ksplit; ++sp) add8(part + ((int64_t)sp * T + t) * d + c, 1.f);
    } else {
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const float2 en = mine[j];
        add8(wrT + (int64_t)__float_as_int(en.y) * d + c, en.x);
      }
    }
    *reinterpret_cast<uint4*>(dxr + c) = pack8(acc);
  }
}

// blockIdx.y == 0: dW_r[i, e] = the K chunks' partials, in order, of the three
// parts' columns; blockIdx.y == 1: db[e] = the chunks' sums in order
__global__ void __launch_bounds__(256) logits_reduce_kernel(
    const float* __restrict__ part, int ksplit, int d, int E, int E8,
    const float* __restrict__ bias_part, int chunks, float* __restrict__ dw_router,
    float* __restrict__ dbias) {
  pdl_enter();
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (blockIdx.y == 0) {
    if (idx >= (int64_t)d * E) return;
    const int i = (int)(idx / E), e = (int)(idx % E);
    const int N3 = 3 * E8;
    float a = 0.f;
    for (int s = 0; s < ksplit; ++s) {
      const float* q = part + ((int64_t)s * d + i) * N3 + e;
      a += q[0] + q[E8] + q[2 * E8];
    }
    dw_router[idx] = a;
  } else if (idx < E) {
    float a = 0.f;
    for (int c = 0; c < chunks; ++c) a += bias_part[(int64_t)c * E + idx];
    dbias[idx] = a;
  }
}

cudaError_t launch_logits_bwd(const float* d_logits, const float* w_router, const moe_bf16* x,
                              int64_t T, int d, int E, int dense, int k, int S, moe_bf16* dx,
                              const float* dxp, const int32_t* dst_row, float* dw_router,
                              float* dbias, void* ws, int* status, cudaStream_t s) {
  const LogitsBwdWs w = logits_bwd_ws(T, d, E, dense != 0);
  const int E8 = round8l(E), N3 = 3 * E8;
  char* p = static_cast<char*>(ws);
  moe_bf16* dl3 = reinterpret_cast<moe_bf16*>(p + w.dl3);
  moe_bf16* dl2 = dense ? reinterpret_cast<moe_bf16*>(p + w.dl2) : nullptr;
  float* wrT = dense ? nullptr : reinterpret_cast<float*>(p + w.wt);
  moe_bf16* planes = dense ? reinterpret_cast<moe_bf16*>(p + w.wt) : nullptr;
  float* bias_part = reinterpret_cast<float*>(p + w.bias);
  float* part = reinterpret_cast<float*>(p + w.part);
  const int chunks = (int)((T + kBiasRows - 1) / kBiasRows);
  const bool pdl = pdl_for_tokens(T);
  cudaError_t err = cudaSuccess;
  timer_before(MOE_KERNEL_LOGITS_BWD, s);
  auto note = [&](cudaError_t e) {
    if (err == cudaSuccess) err = e;
    note_launches(1);
  };
  if (T > 0) {
    note(launch_pdl(pdl, transpose_wr_kernel, dim3((E8 + 31) / 32, (d + 31) / 32), dim3(32, 8), 0, s,
                    w_router, d, E, E8, wrT, planes));
    note(launch_pdl(pdl, split_dl_kernel, dim3((unsigned)((T * E8 + 255) / 256)), dim3(256), 0, s,
                    d_logits, T, E, E8, dl3, dl2));
    if (dbias)
      note(launch_pdl(pdl, bias_part_kernel, dim3(chunks, (E + 31) / 32), dim3(32, 8), 0, s,
                      d_logits, T, E, bias_part));
    if (dense && err == cudaSuccess)
      err = launch_router_gemm(dl2, planes, nullptr, T, 2 * E8, d, d, w.sp_x, part, status, s);
    const size_t smem = dense ? 0 : (size_t)kTokWarps * E * sizeof(float2);
    note(launch_pdl(pdl, logits_dx_kernel, dim3((unsigned)((T + kTokWarps - 1) / kTokWarps)),
                    dim3(32 * kTokWarps), smem, s, d_logits, wrT, dense ? part : nullptr, w.sp_x,
                    T, d, E, k, S, dx, dxp, dst_row));
  }
  if (err == cudaSuccess) err = launch_router_wgrad_gemm(x, dl3, T, d, N3, w.sp_w, part, status, s);
  if (err == cudaSuccess) {
    const int64_t n = std::max<int64_t>((int64_t)d * E, E);
    note(launch_pdl(pdl, logits_reduce_kernel, dim3((unsigned)((n + 255) / 256), dbias ? 2 : 1),
                    dim3(256), 0, s, part, w.sp_w, d, E, E8, bias_part, chunks, dw_router, dbias));
  }
  timer_after(MOE_KERNEL_LOGITS_BWD, s);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace moe
