// Host helpers shared by the entry-point files (abi.cpp, attn_abi.cpp).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "dense_types.h"

namespace glora {

// Set this host thread's error text and return `code`; ok() clears it and returns LORA_OK.
int fail(int code, const char* fmt, ...);
int ok();
int cuda_fail(int err, const char* what);
int device_sm_count_or(int fallback);

// A BF16 tensor map of `rank` (2 or 3) dimensions, innermost first: extents in elements, strides of the
// outer dimensions in bytes, the box, with the given swizzle. Returns a lora_status.
int encode_bf16_map(TensorMapBytes* out, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                    const uint32_t* box, CUtensorMapSwizzle swz, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace glora
