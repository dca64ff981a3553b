// tmap.h — tensor maps that files beside gemm.cu build through its driver entry point.
#pragma once

#include <cuda.h>

#include "../../include/moe.h"

namespace moe {

// Keys or values (at `ptr`) of a paged cache: axes (D, slot, head, page), boxes
// of 64 elements x `slots` slots of one page and head, 128-byte swizzle;
// elements past D read as zeros.
bool map_kv(CUtensorMap* m, const void* ptr, const moe_kv_cache& c, int slots);

// A [T, H, D] view with packed heads, tokens `stride` elements apart: axes
// (D, head, token), boxes of 64 elements x `heads` x `tokens`, 128-byte swizzle.
bool map_heads(CUtensorMap* m, const void* ptr, int D, int H, int64_t T, int64_t stride,
               int heads, int tokens);

}  // namespace moe
