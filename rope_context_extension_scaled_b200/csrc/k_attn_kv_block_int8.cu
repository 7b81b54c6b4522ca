// Few-row attention over the block-scaled KV cache, int8 codes.
#define RCX_KB_KIND 0
#define RCX_KB_NAME int8
#include "k_attn_kv_block.inc"
