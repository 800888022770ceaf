// The split-K kernel's instantiations over E4M3 pools with a scale per
// (block, kv head) for bf16 q, compiled apart from decode.cu's so the
// translation units build in parallel.  Everything else lives in decode.cu.
#define PA_DECODE_SCALED_UNIT __nv_bfloat16
#include "decode.cu"
