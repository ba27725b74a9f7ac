// decode_attn_prefix.cu -- the decode of decode_attn.cu for the tokens behind a
// shared prefix (zp_prefix_decode_attn): the same kernels with every sequence's
// softmax starting from its prefix's record.
#define ZP_DECODE_PREFIX 1
#include "decode_attn.cu"
