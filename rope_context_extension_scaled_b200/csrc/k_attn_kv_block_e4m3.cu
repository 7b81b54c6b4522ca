// Few-row attention over the block-scaled KV cache, e4m3 codes.
#define RCX_KB_KIND 1
#define RCX_KB_NAME e4m3
#include "k_attn_kv_block.inc"
