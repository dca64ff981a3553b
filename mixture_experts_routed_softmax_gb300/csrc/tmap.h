// tmap.h — tensor maps that files beside gemm.cu build through its driver entry point.
#pragma once

#include <cuda.h>

#include "../../include/moe.h"

namespace moe {

// Keys or values (at `ptr`) of a paged cache: axes (D, slot, head, page), boxes
// of 64 elements x `slots` slots of one page and head, 128-byte swizzle;
// elements past D read as zeros.
bool map_kv(CUtensorMap* m, const void* ptr, const moe_kv_cache& c, int slots);

}  // namespace moe
