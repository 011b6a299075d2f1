// Host helpers shared by the entry-point files (abi.cpp, attn_abi.cpp).
#pragma once

#include <stdint.h>

namespace glora {

// Set this host thread's error text and return `code`; ok() clears it and returns LORA_OK.
int fail(int code, const char* fmt, ...);
int ok();
int cuda_fail(int err, const char* what);
int device_sm_count_or(int fallback);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace glora
