// lora_attn_decode_window's kernels (attn_decode.cuh): a translation unit of their own, compiled beside the others.
#include "attn_decode.cuh"

namespace glora {

int launch_decode_window(const DecodeArgs& a, void* stream) { return launch_any<true>(a, stream); }

}  // namespace glora
