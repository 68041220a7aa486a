// api_internal.h -- what the two files of C entry points share.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "moe.h"

namespace moe {

moe_status check_shape(const moe_shape* shape);
int device_sms();
// Bytes, row-major [outer, inner]; box [box_outer x 128], 128-byte swizzle.
bool map_bytes(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_outer);

// bf16 [outer, mid, inner] in boxes of 64 x 64, bytes [outer, mid, inner] in
// boxes of 128 x 128, both with the 128-byte swizzle.
bool map_bf16_tiles(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t mid, uint64_t outer);
bool map_byte_tiles(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t mid, uint64_t outer);

}  // namespace moe
