// lora_attn_decode's kernels (attn_decode.cuh).
#include "attn_decode.cuh"

namespace glora {

int launch_decode(const DecodeArgs& a, void* stream) { return launch_any<false>(a, stream); }

}  // namespace glora
