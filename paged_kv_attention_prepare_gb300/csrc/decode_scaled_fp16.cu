// As decode_scaled.cu, for fp16 q.
#define PA_DECODE_SCALED_UNIT __half
#include "decode.cu"
