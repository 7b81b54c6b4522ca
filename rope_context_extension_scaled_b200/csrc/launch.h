// Host-side interface between the C-ABI translation unit (rcx_api.cu) and the
// kernel translation units (k_*.cu), which are compiled separately and in
// parallel.  Each k_*.cu file holds one family of kernels and the functions
// that launch them; rcx_api.cu holds argument checking, planning and the C
// entry points.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/rcx.h"

namespace rcx {

struct AttnArgs;
struct RopeArgs;
struct MergeArgs;
struct DecodeArgs;
struct QuantArgs;
struct RopeAxesArgs;
struct KvAppendArgs;
struct KvReadArgs;
struct KvAttnArgs;

// Counts a launch of `kind` (rcx_kernel_kind); with timing on, records CUDA
// events around it on `stream`.  Defined in rcx_api.cu.
class LaunchScope {
 public:
  LaunchScope(int kind, cudaStream_t stream);
  ~LaunchScope();
  LaunchScope(const LaunchScope&) = delete;
  LaunchScope& operator=(const LaunchScope&) = delete;

 private:
  int kind_;
  cudaStream_t stream_;
  cudaEvent_t start_ = nullptr, stop_ = nullptr;
};

int sm_count();            // SMs of the current device (read once)
int launch_status();       // RCX_OK, or RCX_ERR_CUDA after printing the launch error

// Opt a kernel into more than 48 KB of dynamic shared memory.
template <typename K>
inline int allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess
             ? RCX_OK
             : RCX_ERR_CUDA;
}

// ---- k_rope.cu
int rope_apply_launch(const RopeArgs& a, int dtype, int grid, int block, cudaStream_t stream);

int rope_axes_launch(const RopeAxesArgs& a, int dtype, dim3 grid, int block, cudaStream_t stream);

// ---- k_merge.cu
int merge_launch(const MergeArgs& a, int out_dtype, int grid, cudaStream_t stream);

// ---- k_attn_simt_*.cu (one unit per input/output dtype pair)
int attn_simt_launch_f32_f32(const AttnArgs& a, cudaStream_t stream);
int attn_simt_launch_f32_bf16(const AttnArgs& a, cudaStream_t stream);
int attn_simt_launch_bf16_f32(const AttnArgs& a, cudaStream_t stream);
int attn_simt_launch_bf16_bf16(const AttnArgs& a, cudaStream_t stream);

// ---- k_attn_tc.cu
int attn_tc_launch(const AttnArgs& a, const rcx_tensor& q, const rcx_tensor& k, const rcx_tensor& v,
                   const rcx_tensor& o, cudaStream_t stream);
void attn_tc_set_inject(int64_t spins);
int64_t attn_tc_inject();

// ---- k_decode.cu
int decode_launch(const DecodeArgs& a, int G, bool tensor_core, dim3 grid, cudaStream_t stream);
int decode_i8_launch(const DecodeArgs& a, int G, const float* k_scale, const float* v_scale, dim3 grid,
                     cudaStream_t stream);
int decode_combine_launch(const DecodeArgs& a, int out_dtype, int grid, cudaStream_t stream);
// rows16: bf16 rows and code rows both 16-byte aligned (eight-lanes-per-row kernel)
int quantize_i8_launch(const QuantArgs& a, bool rows16, int grid, cudaStream_t stream);

// ---- k_kv_block.cu, k_attn_kv_block_*.cu (kind: 0 int8, 1 e4m3 codes)
int kv_block_append_launch(const KvAppendArgs& a, int dtype, int kind, dim3 grid, int block, cudaStream_t stream);
int kv_block_read_launch(const KvReadArgs& a, int dtype, int kind, dim3 grid, cudaStream_t stream);
// Rows (tokens x heads of a group) up to which the mma.sync kernel runs.  Its time
// and the tcgen05 kernel's, d = 128, over 512 and 8192 tokens: 64 rows (8 sequences
// of 4 heads) 19 and 60 us against 21 and 58, 96 rows 19 and 74 against 22 and 59.
constexpr int kKvFewRows = 64;
constexpr int kKvFewItemRows = 32;     // rows of an item of it, at most
constexpr int kKvFewTile = 32;         // its key tile
constexpr int kKvFewWarps = 4;         // warps of its CTA, a tile each
// Resident CTAs for head dim D and nt columns of 8 rows.  Registers allow four at
// d = 64 with one column (a 4096-token window over 24 sequences 43 -> 41 us), two
// elsewhere; three at d = 128 would need a two-stage ring (no faster).
constexpr int kv_few_ctas(int D, int nt) { return D == 64 && nt == 1 ? 4 : 2; }
constexpr int kKvFewStages = 3;        // of 32-key tiles in flight a warp
constexpr int kKvFewMinTiles = 4;      // tiles a CTA takes at least
constexpr int kKvFewStartTiles = 24;   // beginning an item costs a CTA as much as so many tiles
constexpr int kKvFewMergeTiles = 6;    // what a scan and a merge cost, in tile times (see kv_attn_impl)
constexpr int kKvTcRows = 256;         // rows of an item of the tcgen05 kernel, and its key tile
constexpr int kKvTcTile = 128;
// Rows of a sequence from which its tiles are converted once, before the launch,
// where they fit kKvPreBytes (two bytes a code).  Without and with it, 8 heads,
// d = 128: 2048 rows over 8192 tokens 143 and 126 us, 4000 rows 247 and 189 us,
// 32,768 rows over 32,768 tokens 5.6 and 3.8 ms; 1024 rows 76 and 79 us.
constexpr int kKvPreRows = 2048;
constexpr int64_t kKvPreBytes = int64_t(1) << 30;
constexpr int kKvTcMinTiles = 3;
constexpr int kKvTcStartTiles = 4;
constexpr int kKvTcMergeTiles = 6;
constexpr int kKvMaxSlice = 4096;      // sequences a launch takes
constexpr int kKvReadPerCta = 256;     // 16-code pieces a CTA of the read kernel takes
int attn_kv_block_launch_int8(const KvAttnArgs& a, cudaStream_t stream);
int attn_kv_block_launch_e4m3(const KvAttnArgs& a, cudaStream_t stream);
int attn_kv_block_tc_launch(const KvAttnArgs& a, int kind, cudaStream_t stream);
int attn_kv_block_merge_launch(const KvAttnArgs& a, cudaStream_t stream);

// Device status words: every translation unit whose kernels have bounded
// waits keeps its own word; these read one into *status and clear it
// (stream-ordered, synchronising `stream`).
int status_exchange_attn_tc(cudaStream_t stream, int* status);
int status_exchange_rope(cudaStream_t stream, int* status);
int status_exchange_kv_block(cudaStream_t stream, int* status);
int status_exchange_attn_kv_block_int8(cudaStream_t stream, int* status);
int status_exchange_attn_kv_block_e4m3(cudaStream_t stream, int* status);
int status_exchange_attn_kv_block_tc(cudaStream_t stream, int* status);

}  // namespace rcx
