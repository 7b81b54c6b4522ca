// Launchers of the block-scaled KV cache's append and read kernels (kv_block.cuh).
#include "launch.h"
#include "kv_block.cuh"

namespace rcx {

static_assert(kKrThreads * kKrPieces == kKvReadPerCta, "pieces per CTA");

int kv_block_append_launch(const KvAppendArgs& a, int dtype, int kind, dim3 grid, int block, cudaStream_t stream) {
  LaunchScope scope(RCX_KERNEL_DECODE, stream);
  if (dtype == RCX_BF16) {
    if (kind == 0) kv_block_append_kernel<__nv_bfloat16, 0><<<grid, block, 0, stream>>>(a);
    else kv_block_append_kernel<__nv_bfloat16, 1><<<grid, block, 0, stream>>>(a);
  } else {
    if (kind == 0) kv_block_append_kernel<float, 0><<<grid, block, 0, stream>>>(a);
    else kv_block_append_kernel<float, 1><<<grid, block, 0, stream>>>(a);
  }
  return launch_status();
}

int kv_block_read_launch(const KvReadArgs& a, int dtype, int kind, dim3 grid, cudaStream_t stream) {
  LaunchScope scope(RCX_KERNEL_DECODE, stream);
  if (dtype == RCX_BF16) {
    if (kind == 0) kv_block_read_kernel<__nv_bfloat16, 0><<<grid, kKrThreads, 0, stream>>>(a);
    else kv_block_read_kernel<__nv_bfloat16, 1><<<grid, kKrThreads, 0, stream>>>(a);
  } else {
    if (kind == 0) kv_block_read_kernel<float, 0><<<grid, kKrThreads, 0, stream>>>(a);
    else kv_block_read_kernel<float, 1><<<grid, kKrThreads, 0, stream>>>(a);
  }
  return launch_status();
}

int status_exchange_kv_block(cudaStream_t stream, int* status) { return device_status_exchange(stream, status); }

}  // namespace rcx
