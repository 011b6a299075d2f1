// lora_attn_decode_window's kernels: those of attn_decode.cu with a window.
#define GLORA_DECODE_WINDOW
#include "attn_decode.cu"
