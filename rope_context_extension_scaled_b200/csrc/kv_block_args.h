// Launch parameters of the block-scaled KV cache kernels (kv_block.cuh,
// attn_kv_block.cuh, attn_kv_block_tc.cuh).
#pragma once
#include "common.cuh"

namespace rcx {

// Pools of codes (1 byte each; strides in bytes between blocks, tokens and
// heads), scales [n_blocks, Hkv] and the table [B, width] of a cache.
struct KvBlockView {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t k_sb, k_sn, k_sh, v_sb, v_sn, v_sh;
  const int32_t* table;
  int64_t t_sb;
  int n_blocks, block_log2, Hkv;
  int cap;                          // tokens a table row holds: width << block_log2
};

struct KvAppendArgs {
  View4 k, v;                       // new tokens [B, N, Hkv, d]
  KvBlockView c;
  const int64_t *start, *count;     // [B]; count may be null (N each)
  int N, d_log2, b0;
};

struct KvReadArgs {
  View4 k, v;                       // outputs [B, n, Hkv, d]
  KvBlockView c;
  const int64_t* len;               // [B]
  int n, d_log2, b0;
  int wide;                         // output rows are 32-byte aligned
};

struct KvAttnArgs {
  View4 q, o;                       // [B, N, Hq, d]
  float* lse;                       // [B, Hq, N] or null
  int64_t lse_sb, lse_sh;
  KvBlockView c;
  const int64_t *start, *count;
  int B, N, G, b0;                  // B sequences from sequence b0 on
  // by G, Hkv, n_rt and N (direct): a walk makes a dozen divisions on its way to the first load
  FastDiv div_g, div_hkv, div_nrt, div_n;
  int window, n_sink;               // window 0 = none
  float scale_log2;                 // log2(e) / (sqrt(d) * t)
  int o_bf16;
  int o_wide;                       // rows of o are 32-byte aligned
  int rows_item;                    // rows (token, head of the group) an item holds
  int n_rt;                         // items a (sequence, KV head) has at most
  int n_cta;                        // CTAs the key tiles (direct: items) are dealt to
  int min_tiles;                    // key tiles a CTA takes at least
  int start_tiles;                  // tiles' worth of time that beginning an item costs
  int direct;                       // items are not cut: no partials, no merge
  float* part_o;                    // [n_cta, 2, rows_item, d]: partials of items that several CTAs share
  float* part_lse;                  // [n_cta, 2, rows_item]
  int* prefix;                      // [B * n_rt + 2] first key tile of each (sequence, row tile); pieces of an item
  uint8_t* img;                     // tiles converted before the launch, or null
  float* img_vref;                  // [B, Hkv] V scale their V tiles are relative to
  int img_tiles;                    // tiles a sequence and head has room for
  float k_unscale, v_unscale;       // factors of the converted K and V values
  int64_t inject_spins;             // test hook of the tensor-core kernel
};

}  // namespace rcx
