// Launchers of the tensor-core attention over the block-scaled KV cache
// (attn_kv_block_tc.cuh) and of the merge of partials (attn_kv_block.cuh).
#include <algorithm>
#include "launch.h"
#include "attn_kv_block_tc.cuh"

namespace rcx {

template <int D, int KIND>
static int kb_tc_launch(const KvAttnArgs& a, cudaStream_t stream) {
  auto kern = attn_kv_block_tc_kernel<D, KIND>;
  if (allow_smem(kern, BtSmem<D>::total)) return RCX_ERR_CUDA;
  kern<<<a.n_cta, kBtThreads, BtSmem<D>::total, stream>>>(a);
  return launch_status();
}

// K and V tiles of a.img (a.k_unscale, a.v_unscale: what they are to be multiplied by).
template <int D, int KIND>
static int kb_expand(KvAttnArgs& a, cudaStream_t stream) {
  LaunchScope scope(RCX_KERNEL_DECODE, stream);
  a.k_unscale = KIND == 1 ? kE4m3Unscale : 1.f;
  a.v_unscale = a.k_unscale / kBtVUp<KIND>;
  kv_block_vmax_kernel<<<dim3((unsigned)a.c.Hkv, (unsigned)a.B), 256, 0, stream>>>(a);
  const int st = launch_status();
  if (st) return st;
  kv_block_expand_kernel<D, KIND><<<dim3((unsigned)a.img_tiles, (unsigned)a.c.Hkv, (unsigned)a.B), 256, 0, stream>>>(a);
  return launch_status();
}

int attn_kv_block_tc_launch(const KvAttnArgs& args, int kind, cudaStream_t stream) {
  KvAttnArgs a = args;
  if (a.img) {
    const int st = a.q.D == 64 ? (kind == 0 ? kb_expand<64, 0>(a, stream) : kb_expand<64, 1>(a, stream))
                               : (kind == 0 ? kb_expand<128, 0>(a, stream) : kb_expand<128, 1>(a, stream));
    if (st) return st;
    LaunchScope scope(RCX_KERNEL_ATTN_TC, stream);
    return a.q.D == 64 ? kb_tc_launch<64, 2>(a, stream) : kb_tc_launch<128, 2>(a, stream);
  }
  LaunchScope scope(RCX_KERNEL_ATTN_TC, stream);
  if (a.q.D == 64) return kind == 0 ? kb_tc_launch<64, 0>(a, stream) : kb_tc_launch<64, 1>(a, stream);
  return kind == 0 ? kb_tc_launch<128, 0>(a, stream) : kb_tc_launch<128, 1>(a, stream);
}

// Where items are small and CTAs many times as many, so are a row's partials: eight
// warps share them.  Otherwise a warp takes a row, with as many CTAs an item as
// fill the GPU once (256 rows in 5 to 18 pieces: 41 us an attention call with eight
// warps a row, 35 so).
int attn_kv_block_merge_launch(const KvAttnArgs& a, cudaStream_t stream) {
  LaunchScope scope(RCX_KERNEL_DECODE, stream);
  const int64_t items = (int64_t)a.B * a.n_rt * a.c.Hkv;
  const bool many = a.rows_item <= kKvFewItemRows && items * 16 <= a.n_cta;
  const int rows = std::min(a.N * a.G, a.rows_item);
  const int z = many ? rows : (int)std::min<int64_t>((rows + 7) / 8, std::max<int64_t>(4, 8 * sm_count() / items));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.n_rt), (unsigned)a.c.Hkv, (unsigned)z);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  auto kern = a.q.D == 64 ? (many ? attn_kv_block_merge_kernel<64, 8> : attn_kv_block_merge_kernel<64, 1>)
                          : (many ? attn_kv_block_merge_kernel<128, 8> : attn_kv_block_merge_kernel<128, 1>);
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
    launch_status();
    return RCX_ERR_CUDA;
  }
  return launch_status();
}

int status_exchange_attn_kv_block_tc(cudaStream_t stream, int* status) { return device_status_exchange(stream, status); }

}  // namespace rcx
