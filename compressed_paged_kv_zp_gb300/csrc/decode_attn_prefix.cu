// decode_attn_prefix.cu -- the decode of decode_attn.cu for the tokens behind a
// shared prefix (zp_prefix_decode_attn): the same main kernels, whose
// records one kernel joins with the prefix's.
#define ZP_DECODE_PREFIX 1
#include "decode_attn.cu"
