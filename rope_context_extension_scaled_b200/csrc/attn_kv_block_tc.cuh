// Tensor-core (tcgen05 / TMEM) attention of many query rows (drafts and prompt
// chunks) over a block-scaled 8-bit paged KV cache, d = 64 or 128.
//
// Mathematics, mask and fp16 operands as in attn_kv_block.cuh: exact fp16 codes
// and power-of-two scaled queries, so S is the fp32 sum of exact products; P as
// 2^7 p in fp16.  Compute-bound for prompt chunks.
//
// One CTA per SM, walking its segments of the shared line of key tiles
// (kv_block_plan.cuh).  An item is 256 rows (token, head of the group) of one
// KV head, two slots of 128 that share every K/V tile; flattening tokens and
// heads fills the MMA's 128 rows at any group size.  512 threads:
//   warps 0-3   softmax, Q load and epilogue of slot 0 (a thread per row)
//   warps 4-7   the same of slot 1 (idle when an item has at most 128 rows)
//   warps 8-11  converters: codes in shared memory -> fp16, stored as
//               128B-swizzled K and V tiles (two stages)
//   warp  12    MMA issuer and TMEM owner
//   warp  13    producer: follows the table, copies the next tile's codes to
//               shared memory (bulk copies of 16 tokens, or of a token where
//               those are not contiguous) and works out its scales, so the
//               cache is read as it is stored and never copied whole
//   (14, 15 zero the rows of tokens past a sequence's count, in direct launches)
// The softmax threads hold a row of S: registers move to them from the other
// warpgroups (setmaxnreg; 2 x 200, 72 and 40 a thread are the launch's 65,536),
// and each warp's place in the walk over segments is kept in shared memory.
// TMEM: S0 | S1 | O0 | O1, 128 columns each.  P overwrites the first half of its
// S; O += P V takes P from TMEM.
//  * d order: a word's codes leave codes4_to_h2 in the order 0, 2, 1, 3.  Q is
//    stored in the same order, and O's columns are put back in the epilogue.
//  * K scales multiply S in the softmax, one factor per 16 columns, inside the
//    multiply-add that the exponential needs anyway.  V scales go into the fp16
//    V tile as ratio to a reference (one half-precision product per pair of codes
//    in the converters, which have the time; 11 bits beside the 8 of a bf16
//    output).  The reference is the largest scale of the keys that the item's rows
//    see (KIND 2: that any row sees), with some headroom as it grows tile by tile.
//    16 keys whose scale is below 2^-14 of it take the rest as a power of two 2^lv
//    that the weights carry (v_part): the row's running reference m is the largest
//    x + lv, in units of the V reference (so m falls by log2 of its growth), weights
//    are 2^(x + lv - m), and their sum takes 2^-lv back.  So a row keeps fp16's
//    range for the scales it sees, whatever the others; lv = 0 nearly always.
//    A non-finite V scale counts as zero there and marks its 16 keys; a row
//    that sees a marked key ends as NaN, and no other row does.
// Converting a tile in every item that sees it is right for few row tiles; the
// conversion then costs a third of the softmax's issue slots.  For many (2048
// rows a sequence and more, kv_attn_impl) the tiles are converted once, before
// the launch, into images of the swizzled shared-memory tiles (kv_block_expand),
// and the producer copies those (KIND 2, no converters).
// Every mbarrier wait is bounded, as in attn_tc.cuh.
#pragma once
#include <type_traits>
#include "attn_tc.cuh"
#include "attn_kv_block.cuh"

namespace rcx {

constexpr int kBtM = 128;                       // rows per slot
constexpr int kBtN = kKvTcTile;                 // keys per tile
constexpr int kBtLogN = 7;
static_assert(1 << kBtLogN == kBtN && 2 * kBtM == kKvTcRows, "tile");
constexpr int kBtThreads = 512;
template <int KIND>
struct BtRegs {                                 // registers a thread after the split
  static constexpr int softmax = KIND == 2 ? 216 : 200, conv = KIND == 2 ? 40 : 72, mma = 40;
  static_assert(128 * (2 * softmax + conv + mma) <= 512 * 128, "registers of the launch");
};
constexpr int kBtConv = 8;                      // first converter warp
constexpr int kBtMma = 12;
constexpr int kBtProd = 13;
constexpr int kBtWalkers = 14;                  // warps that walk the segments
constexpr int kBtStages = 2;
constexpr int kBtMeta = 8;                      // ring of per-tile scales
constexpr uint32_t kBtHalf = kBtM * 128;        // 128 rows x 64 fp16, one swizzled block

// The fp16 V tile holds value * this / (256 for e4m3) / (largest V scale): at
// most 127 * 2^8 or 1.75 * 2^15, as far from fp16's subnormals as it goes.
// KIND: 0 int8, 1 e4m3 codes, 2 tiles converted before the launch.
template <int KIND>
constexpr float kBtVUp = KIND == 0 ? 256.f : 32768.f;

struct BtMeta {
  float ks[8];                                  // K scale of each 16 keys
  uint32_t ratio[8];                            // V scale / (vref 2^lv) * kBtVUp, an fp16 pair
  int8_t lv[8];                                 // of each 16 keys
  int rare;                                     // kBtWide where a lv is not 0, and the two below; 0 nearly always
  float vref;                                   // V scales' reference
};

constexpr int kBtBad = 0xff;                    // 16-key groups with a non-finite V scale
constexpr int kBtWide = 0x100;
constexpr int kBtGrown = 16;                    // from this bit on: log2 of vref's growth

// V scale s relative to vref (inv: its inverse): ratio 2^lv, lv = 0 down to a ratio
// of 2^-14, and 2^-90 at least.  0 for scales that are not finite, and lv = -90 for
// zero, so that such keys do not raise a row's reference.
struct VPart {
  float ratio;
  int lv;
};
__device__ __forceinline__ VPart v_part(float s, float vref, float inv) {
  if (!(s >= 0x1p-126f && s < INFINITY)) return {0.f, s < 0x1p-126f ? -90 : 0};
  const int lv = max(-90, min(0, ((__float_as_int(s) - __float_as_int(vref)) >> 23) + 14));
  return {s * (inv * __int_as_float((127 - lv) << 23)), lv};
}

// A warp's place in the walk (e, off, x: see SegWalk) and its current segment.
struct BtSeg {
  int e, off, x, x0, x1, even;
  int ok;                                       // a segment is there
  int b, hk, r0, rows, start;
  KeySpan span;
  int u0, n, slot, whole;
};

// Next segment of the calling warp: one lane walks, all read.
__device__ __forceinline__ bool bt_next(BtSeg* g, const KvAttnArgs& a, int lane) {
  __syncwarp();                                 // the old segment has been read
  if (lane == 0) {
    SegWalk w;
    w.e = g->e; w.off = g->off; w.x = g->x; w.x0 = g->x0; w.x1 = g->x1; w.even = g->even;
    w.fresh = false;
    g->ok = w.next<kBtLogN>(a);
    if (g->ok) {
      g->e = w.e; g->off = w.off; g->x = w.x;
      g->b = w.t.b; g->hk = w.hk; g->r0 = w.t.r0; g->rows = w.t.rows; g->start = w.t.start;
      g->span = w.t.span;
      g->u0 = w.u0; g->n = w.u1 - w.u0; g->slot = w.slot(); g->whole = w.whole();
    }
  }
  __syncwarp();
  return g->ok;
}

template <int D>
struct BtSmem {
  static constexpr uint32_t tile = kBtHalf * (D / 64);
  static constexpr uint32_t q = 0;
  static constexpr uint32_t k = q + 2 * tile;
  static constexpr uint32_t v = k + kBtStages * tile;
  static constexpr uint32_t raw = v + kBtStages * tile;            // codes of the next K and V tile
  static constexpr uint32_t bar = raw + 2 * kBtN * D;
  static constexpr uint32_t meta = bar + 256;
  static constexpr uint32_t seg = meta + kBtMeta * sizeof(BtMeta);
  static constexpr uint32_t total = seg + kBtWalkers * sizeof(BtSeg) + 1024;   // + alignment slack
};

// kind::f16 descriptor: fp16 A and B, fp32 accumulator, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(bool b_mn_major, int n) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kBtM >> 4) << 24);
}

// Bulk copy of `bytes` (16-byte aligned on both sides, a multiple of 16) that
// completes on mbarrier `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Packed fp32 arithmetic: two values an instruction.
__device__ __forceinline__ void mul2(float& a, float& b, float f) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(f));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(c), "f"(d));
}

// A warp's arrival for what its lanes stored to shared memory for the MMAs.
__device__ __forceinline__ void warp_arrive_stored(uint32_t bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// Blocks that the window hides from every row of a sequence: [sinks, first).
struct HiddenBlocks {
  int sinks, first;
  __device__ __forceinline__ bool has(int j) const { return j >= sinks && j < first; }
};
__device__ __forceinline__ HiddenBlocks hidden_blocks(const KvAttnArgs& a, int start) {
  const int lb = a.c.block_log2, lo = a.window > 0 ? max(0, start + 1 - a.window) : 0;
  return {(min(a.n_sink, lo) + (1 << lb) - 1) >> lb, lo >> lb};
}

// Largest finite V scale of each sequence's visible blocks and KV head (the vref
// of KIND 2).  One CTA each.
static __global__ void __launch_bounds__(256) kv_block_vmax_kernel(const KvAttnArgs a) {
  __shared__ uint32_t sm[8];
  const int hk = blockIdx.x, b = a.b0 + blockIdx.y;
  const SeqRange s = seq_range(a.start, a.count, b, a.N, a.c.cap);
  const int blocks = s.n > 0 ? (s.start + s.n - 1 >> a.c.block_log2) + 1 : 0;
  const HiddenBlocks hidden = hidden_blocks(a, s.start);
  uint32_t m = 0;
#pragma unroll 4
  for (int j = threadIdx.x; j < blocks; j += 256) {
    if (hidden.has(j)) continue;
    int e = a.c.table[b * a.c.t_sb + j];
    if ((unsigned)e >= (unsigned)a.c.n_blocks) e = 0;            // reported by the kernels that read it
    const float v = a.c.vs[(int64_t)e * a.c.Hkv + hk];
    if (v >= 0x1p-126f && v < INFINITY) m = max(m, __float_as_uint(v));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) m = max(m, sm[i]);
    a.img_vref[(int64_t)blockIdx.y * a.c.Hkv + hk] = __uint_as_float(m);
  }
}

// Images of the swizzled fp16 K and V tiles of 128 keys, once per tile that a row
// sees: [sequence, KV head, tile, K | V].  One CTA of 256 threads each; bound by
// HBM (a byte in, two out).  Blocks of the tile that no row sees are zeros: vref
// does not cover their scales, and a V beyond fp16 would make NaN of its weight 0.
template <int D, int KIND>
static __global__ void __launch_bounds__(256) kv_block_expand_kernel(const KvAttnArgs a) {
  constexpr int kPieces = D / 16;
  constexpr uint32_t kTile = BtSmem<D>::tile;
  const KvBlockView& kv = a.c;
  const int t = blockIdx.x, hk = blockIdx.y, bl = blockIdx.z, b = a.b0 + bl;
  const SeqRange s = seq_range(a.start, a.count, b, a.N, kv.cap);
  const int hi = s.start + s.n;
  if (s.n == 0 || t * kBtN >= hi) return;
  const int lo = a.window > 0 ? max(0, s.start + 1 - a.window) : 0;
  if ((t + 1) * kBtN <= lo && t * kBtN >= min(a.n_sink, lo)) return;
  const float vref = a.img_vref[(int64_t)bl * kv.Hkv + hk], inv = vref > 0.f ? 1.f / vref : 0.f;
  const HiddenBlocks hidden = hidden_blocks(a, s.start);
  uint8_t* img = a.img + (((int64_t)bl * kv.Hkv + hk) * a.img_tiles + t) * 2 * kTile;
#pragma unroll 4
  for (int i = threadIdx.x; i < kBtN * kPieces; i += 256) {
    const int row = i / kPieces, pc = i % kPieces, key = t * kBtN + row;
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    float sv = 0.f;
    if (key < hi && !hidden.has(key >> kv.block_log2)) {
      const int e = max(0, checked_block(kv, b, key >> kv.block_log2));      // a bad entry reads as block 0
      const int64_t r = key & ((1 << kv.block_log2) - 1);
      x = __ldcs(reinterpret_cast<const uint4*>(kv.k + e * kv.k_sb + r * kv.k_sn + hk * kv.k_sh + pc * 16));
      y = __ldcs(reinterpret_cast<const uint4*>(kv.v + e * kv.v_sb + r * kv.v_sn + hk * kv.v_sh + pc * 16));
      sv = kv.vs[(int64_t)e * kv.Hkv + hk];
    }
    const __half2 rh = __float2half2_rn(v_part(sv, vref, inv).ratio * kBtVUp<KIND>);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
    uint32_t h[8], g[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      codes4_to_h2<KIND>(xw[e], h[2 * e], h[2 * e + 1]);
      codes4_to_h2<KIND>(yw[e], g[2 * e], g[2 * e + 1]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&g[e]), rh);
      g[e] = *reinterpret_cast<const uint32_t*>(&z);
    }
    const uint32_t at = (pc >> 2) * kBtHalf + row * 128, c0 = ((2 * (pc & 3)) ^ (row & 7)) * 16, c1 = c0 ^ 16;
    *reinterpret_cast<uint4*>(img + at + c0) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(img + at + c1) = make_uint4(h[4], h[5], h[6], h[7]);
    *reinterpret_cast<uint4*>(img + kTile + at + c0) = make_uint4(g[0], g[1], g[2], g[3]);
    *reinterpret_cast<uint4*>(img + kTile + at + c1) = make_uint4(g[4], g[5], g[6], g[7]);
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(kBtThreads, 1) attn_kv_block_tc_kernel(const __grid_constant__ KvAttnArgs a) {
  using L = BtSmem<D>;
  static_assert(L::total <= 227 * 1024, "shared memory of a CTA");
  constexpr int kPieces = D / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar0 = sbase + L::bar;
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  enum {
    B_QREADY = 0,                     // [2] Q rows of the slot stored (one arrival a warp)
    B_KFULL = 2,                      // [stages] (one arrival a warp)
    B_KEMPTY = B_KFULL + kBtStages,
    B_VFULL = B_KEMPTY + kBtStages,
    B_VEMPTY = B_VFULL + kBtStages,
    B_SFULL = B_VEMPTY + kBtStages,   // [2]
    B_PREADY = B_SFULL + 2,           // [2] (one arrival a warp)
    B_OFINAL = B_PREADY + 2,          // [2]
    B_META = B_OFINAL + 2,            // [ring] scales of a tile written
    B_RFULL = B_META + kBtMeta,       // [K, V] codes of a tile landed
    B_REMPTY = B_RFULL + 2,           // [K, V] they have been read (one arrival a warp)
    B_DRAIN = B_REMPTY + 2,
    B_NEVER,
    B_COUNT
  };
  static_assert(8 * B_COUNT + 16 <= 256, "barrier area");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::bar + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::bar + 8 * B_COUNT + 8);
  BtMeta* meta = reinterpret_cast<BtMeta*>(smem + L::meta);
  BtSeg* segs_all = reinterpret_cast<BtSeg*>(smem + L::seg);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      uint32_t cnt = 1;
      if (i < 2 || (i >= B_KFULL && i < B_KFULL + kBtStages) || (i >= B_VFULL && i < B_VFULL + kBtStages) ||
          i == B_PREADY || i == B_PREADY + 1 || i == B_REMPTY || i == B_REMPTY + 1)
        cnt = KIND == 2 && i >= B_KFULL && i < B_PREADY ? 1 : 4;
      mbar_init(BAR(i), cnt);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    const PlanStart p = plan_start<kBtLogN>(a, blockIdx.x, lane);
    if (lane < kBtWalkers) {
      BtSeg* g = segs_all + lane;
      g->e = p.e; g->off = p.off; g->x = g->x0 = p.x0; g->x1 = p.x1; g->even = p.even;
    }
  }
  if (warp == kBtMma) tmem_alloc(smem_addr(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  auto tS = [&](int s) { return tmem + 128u * (uint32_t)s; };
  auto tO = [&](int s) { return tmem + 256u + 128u * (uint32_t)s; };
  auto warp_wait = [&](int b, uint32_t par) { return __all_sync(0xffffffffu, mbar_wait(BAR(b), par, abort_flag)); };
  BtSeg* const w = segs_all + min(warp, kBtWalkers - 1);
  bool ok = true;

  if (warp >= kBtMma) {
    regs_down<BtRegs<KIND>::mma>();
    if (warp == kBtMma) {
    // ================================================================ MMA issuer
    constexpr uint32_t id_qk = idesc_f16(false, kBtN);
    constexpr uint32_t id_pv = idesc_f16(true, D);
    const uint32_t d_hi = (uint32_t)(sw128_desc(sbase, 16, 1024) >> 32);
    const uint32_t q_lo = (uint32_t)sw128_desc(sbase + L::q, 16, 1024);
    const uint32_t k_lo = (uint32_t)sw128_desc(sbase + L::k, 16, 1024);
    const uint32_t v_lo = (uint32_t)sw128_desc(sbase + L::v, kBtHalf, 1024);
    auto issue_s = [&](int s, int st) {
      const uint32_t a0 = q_lo + s * (L::tile >> 4), b0 = k_lo + st * (L::tile >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * kBtHalf + (kk % 4) * 32) >> 4;
        umma_ss_e(tS(s), a0 + off, b0 + off, d_hi, id_qk, kk > 0);
      }
    };
    auto issue_pv = [&](int s, int st, bool first_tile) {
      const uint32_t b0 = v_lo + st * (L::tile >> 4);
#pragma unroll
      for (int kk = 0; kk < kBtN / 16; ++kk)
        umma_ts_e(tO(s), tS(s) + kk * 8, b0 + kk * (2048 >> 4), d_hi, id_pv, (!first_tile || kk > 0) ? 1u : 0u);
    };
    if (a.inject_spins > 0) {
      // test hook: a wait that nothing ends
      bool got = false;
      if (lane == 0) {
        for (int64_t i = 0; i < a.inject_spins && !got; ++i) got = mbar_test(BAR(B_NEVER), 0);
        if (!got) {
          *abort_flag = 1;
          record_device_error(RCX_ERR_DEVICE_TIMEOUT);
        }
      }
      ok = __shfl_sync(0xffffffffu, got ? 1 : 0, 0) != 0;
    }
    int jg = 0, js[2] = {0, 0}, segs[2] = {0, 0};   // tiles so far (all, per slot), segments per slot
    while (ok && bt_next(w, a, lane)) {
      const int n = w->n;
      const int ns = w->rows > kBtM ? 2 : 1;
      for (int s = 0; s < ns && ok; ++s) ok = warp_wait(B_QREADY + s, segs[s] & 1);
      if (!ok) break;
      {
        const int st0 = jg % kBtStages;
        if (!(ok = warp_wait(B_KFULL + st0, (jg / kBtStages) & 1))) break;
        tc_fence_after();
        for (int s = 0; s < ns; ++s) {
          issue_s(s, st0);
          umma_commit_e(BAR(B_SFULL + s));
        }
        umma_commit_e(BAR(B_KEMPTY + st0));
      }
      for (int j = 0; ok && j < n; ++j) {
        const int g = jg + j;
        const int st = g % kBtStages, st1 = (g + 1) % kBtStages;
        const bool last = j == n - 1;
        if (!(ok = warp_wait(B_VFULL + st, (g / kBtStages) & 1))) break;
        for (int s = 0; s < ns; ++s) {
          if (!(ok = warp_wait(B_PREADY + s, (js[s] + j) & 1))) break;
          tc_fence_after();
          issue_pv(s, st, j == 0);
          if (last) umma_commit_e(BAR(B_OFINAL + s));
          if (s == ns - 1) umma_commit_e(BAR(B_VEMPTY + st));
          if (!last) {
            if (s == 0) {
              if (!(ok = warp_wait(B_KFULL + st1, ((g + 1) / kBtStages) & 1))) break;
              tc_fence_after();
            }
            issue_s(s, st1);
            umma_commit_e(BAR(B_SFULL + s));
            if (s == ns - 1) umma_commit_e(BAR(B_KEMPTY + st1));
          }
        }
      }
      jg += n;
      for (int s = 0; s < ns; ++s) {
        js[s] += n;
        ++segs[s];
      }
    }
    // all MMAs issued complete before TMEM is released
    umma_commit_e(BAR(B_DRAIN));
    if (lane == 0) mbar_wait(BAR(B_DRAIN), 0, abort_flag, 100000000ull, false);
    __syncwarp();
    } else if (warp == kBtProd) {
    // ================================================================ producer
    const KvBlockView& kv = a.c;
    const int lb = kv.block_log2, bmask = (1 << lb) - 1;
    const uint32_t raw = sbase + L::raw;
    (void)raw;
    int jg = 0, sent[2] = {0, 0};                 // tiles; K and V tiles whose copies were issued
    int hidden = 0;                               // keys up to here, sinks apart, are outside every row's window
    // whether a row of the item sees one of the 16 keys i = lane % 8 of tile u
    auto seen = [&](int u, int u1) {
      const int key = (w->span.tile(u) << kBtLogN) + 16 * (lane & 7);
      return u < u1 && key < w->span.hi && (key + 15 > hidden || key < a.n_sink);
    };
    // lane i < 8: block of 16-key group i of tile u (0 where no row sees it)
    auto load_phys = [&](int u, int u1) {
      int e = 0;
      if (u < u1) {
        const int key = (w->span.tile(u) << kBtLogN) + 16 * (lane & 7);
        if (seen(u, u1)) {
          e = kv.table[(int64_t)w->b * kv.t_sb + (key >> lb)];
          if ((unsigned)e >= (unsigned)kv.n_blocks) {
            record_device_error(RCX_ERR_DEVICE_INDEX);
            e = 0;
          }
        }
      }
      return e;
    };
    // lanes 0-7 K, 8-15 V scale of the groups of tile u with blocks ph
    auto load_scale = [&](int u, int u1, int ph) {
      float sc = 0.f;
      if (lane < 16 && seen(u, u1))
        sc = (lane < 8 ? kv.ks : kv.vs)[(int64_t)ph * kv.Hkv + w->hk];
      return sc;
    };
    // codes of tile u's keys in the sequence -> raw rows; what stands in the other
    // rows converts to finite numbers too, and their weights are zero.  (KIND 2:
    // the tile's image -> its stage.)
    auto copy_codes = [&](int u, int ph, int isv) {
      if constexpr (KIND == 2) {
        const int st = jg % kBtStages;
        if (lane == 0) {
          const uint32_t bar = BAR((isv ? B_VFULL : B_KFULL) + st);
          const int64_t tile = ((int64_t)(w->b - a.b0) * kv.Hkv + w->hk) * a.img_tiles + w->span.tile(u);
          mbar_expect_tx(bar, L::tile);
          bulk_load(sbase + (isv ? L::v : L::k) + st * L::tile, a.img + (2 * tile + isv) * L::tile, L::tile, bar);
        }
      } else {
        const uint8_t* base = isv ? kv.v + w->hk * kv.v_sh : kv.k + w->hk * kv.k_sh;
        const int64_t sb = isv ? kv.v_sb : kv.k_sb, sn = isv ? kv.v_sn : kv.k_sn;
        const uint32_t dst = raw + isv * kBtN * D, bar = BAR(B_RFULL + isv);
        const int key0 = w->span.tile(u) << kBtLogN;
        const int rows = min(w->span.hi - key0, kBtN);
        const int64_t off = ph * sb + ((key0 + 16 * (lane & 7)) & bmask) * sn;     // of the lane's group
        if (lane == 0) mbar_expect_tx(bar, rows * D);
        __syncwarp();
        if (sn == D) {
          const int n = min(rows - 16 * lane, 16);
          if (lane < 8 && n > 0) bulk_load(dst + 16 * lane * D, base + off, n * D, bar);
        } else {
          for (int i = 0; i < kBtN / 32; ++i) {
            const int r = 32 * i + lane;
            const int64_t o = __shfl_sync(0xffffffffu, off, r >> 4) + (r & 15) * sn;
            if (r < rows) bulk_load(dst + r * D, base + o, D, bar);
          }
        }
      }
      ++sent[isv];
    };
    // until K's (V's) place for tile jg is free
    auto wait_place = [&](int isv) {
      if constexpr (KIND == 2) return warp_wait((isv ? B_VEMPTY : B_KEMPTY) + jg % kBtStages, ((jg / kBtStages) & 1) ^ 1);
      else return warp_wait(B_REMPTY + isv, (jg & 1) ^ 1);
    };
    while (ok && bt_next(w, a, lane)) {
      const int u0 = w->u0, u1 = u0 + w->n;
      hidden = a.window > 0 ? w->start + (int)fast_div(w->r0, a.div_g) - a.window : -1;
      int ph = load_phys(u0, u1), ph_next = load_phys(u0 + 1, u1);
      float sc = load_scale(u0, u1, ph);
      float vref = 0.f, inv = 0.f;
      if constexpr (KIND == 2) {
        vref = a.img_vref[(int64_t)(w->b - a.b0) * kv.Hkv + w->hk];
        inv = vref > 0.f ? 1.f / vref : 0.f;
      }
      for (int u = u0; u < u1; ++u, ++jg) {
        const int ph_next2 = load_phys(u + 2, u1);
        const float sc_next = load_scale(u + 1, u1, ph_next);
        if (!(ok = wait_place(0))) break;
        copy_codes(u, ph, 0);
        // V scales (lanes 8-15 hold the groups'): the first one that is not zero times a
        // power of two is their reference, at least twice the largest where it begins or
        // grows, so that it seldom does
        const bool is_v = lane >= 8 && lane < 16;
        const bool bad = is_v && !(fabsf(sc) < INFINITY);
        const uint32_t vbad = (__ballot_sync(0xffffffffu, bad) >> 8) & 0xffu;
        int grown = 0;
        if constexpr (KIND != 2) {
          const bool counts = is_v && !bad && sc >= 0x1p-126f;
          const int top = (int)__reduce_max_sync(0xffffffffu, counts ? __float_as_uint(sc) : 0u);
          if (top > __float_as_int(vref)) {
            const bool first = vref == 0.f;
            if (first) {
              vref = __shfl_sync(0xffffffffu, sc, __ffs(__ballot_sync(0xffffffffu, counts)) - 1);
              inv = 1.f / vref;
            }
            const int k = max(0, min(((top - __float_as_int(vref) + 0x7fffff) >> 23) + 1, 251 - (__float_as_int(vref) >> 23)));
            vref = __int_as_float(__float_as_int(vref) + (k << 23));
            inv = __int_as_float(__float_as_int(inv) - (k << 23));
            grown = first ? 0 : k;               // (nothing but zeros so far: O is 0)
          }
        }
        VPart part = v_part(sc, vref, inv);
        if (!is_v || !seen(u, u1)) part = {0.f, 0};
        const bool wide = __any_sync(0xffffffffu, part.lv != 0);
        // the slot's last reader was the softmax of tile jg - 8: the copies above waited
        // for K of jg - 1 to be read, so K of jg - 2 stands in its stage and S of jg - 4
        // is done, which came after both slots' weights of jg - 5 (KIND 2: for S of
        // jg - 2, after their weights of jg - 3)
        BtMeta* mt = meta + jg % kBtMeta;
        if (lane < 8) mt->ks[lane] = sc;
        if (is_v) {
          mt->ratio[lane - 8] = f2_to_h2(part.ratio * kBtVUp<KIND>, part.ratio * kBtVUp<KIND>);
          mt->lv[lane - 8] = (int8_t)part.lv;
        }
        if (lane == 0) {
          mt->rare = (grown << kBtGrown) | (wide ? kBtWide : 0) | (int)vbad;
          mt->vref = vref;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_META + jg % kBtMeta));
        if (!(ok = wait_place(1))) break;
        copy_codes(u, ph, 1);                     // its arrival also publishes the ratios
        ph = ph_next;
        ph_next = ph_next2;
        sc = sc_next;
      }
    }
    if (*abort_flag && lane == 0)                 // copies in flight land before the CTA ends
      for (int i = 0; i < 2; ++i) {
        if constexpr (KIND == 2) {
          for (int n = max(0, sent[i] - kBtStages); n < sent[i]; ++n)
            mbar_wait(BAR((i ? B_VFULL : B_KFULL) + n % kBtStages), (n / kBtStages) & 1, abort_flag, 100000000ull, false);
        } else if (sent[i]) {
          mbar_wait(BAR(B_RFULL + i), (sent[i] - 1) & 1, abort_flag, 100000000ull, false);
        }
      }
    __syncwarp();
    } else if (a.direct) {
      empty_rows<D>(a, warp - kBtProd - 1, 2, lane);
    }
  } else if (warp >= kBtConv) {
    // ================================================================ converters
    regs_down<BtRegs<KIND>::conv>();
    const int tid = threadIdx.x - kBtConv * 32;
    constexpr int kRows = 128 / kPieces;          // key rows the 128 threads cover at once
    // Piece pc of key rows i * kRows + pr.  Eight lanes take the pieces of one half
    // of a row and of the other half of the next: their 16-byte reads, and their
    // stores into the swizzled tile, fall into eight different bank groups.
    const int pr = D == 128 ? (warp - kBtConv) * 4 + ((lane >> 2) & 1) + ((lane >> 4) << 1) : tid / 4;
    const int pc = D == 128 ? (lane & 3) + (((lane >> 3) ^ (lane >> 2)) & 1) * 4 : tid % 4;
    // a piece of 16 codes becomes the two 16-byte chunks 2 (pc % 4), + 1 of its row;
    // row % 8 does not change with i
    const uint32_t dst0 = (pc >> 2) * kBtHalf + pr * 128 + (((2 * (pc & 3)) ^ (pr & 7)) * 16);
    const uint4* raw_k = reinterpret_cast<const uint4*>(smem + L::raw + pr * D + pc * 16);
    const uint4* raw_v = raw_k + kBtN * D / 16;
    auto store_tile = [&](uint32_t tile_off, const uint4* raw, const uint32_t* ratios, auto scaled) {
      uint8_t* dst = smem + tile_off + dst0;
      uint8_t* dst1 = smem + tile_off + (dst0 ^ 16);
#pragma unroll 2
      for (int i = 0; i < kPieces; ++i) {
        const uint4 x = raw[i * kRows * D / 16];
        const uint32_t wv[4] = {x.x, x.y, x.z, x.w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) codes4_to_h2<KIND == 2 ? 0 : KIND>(wv[e], h[2 * e], h[2 * e + 1]);
        if constexpr (decltype(scaled)::value) {
          const uint32_t rb = ratios[(i * kRows + pr) >> 4];
          const __half2 rh = *reinterpret_cast<const __half2*>(&rb);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[e]), rh);
            h[e] = *reinterpret_cast<const uint32_t*>(&y);
          }
        }
        *reinterpret_cast<uint4*>(dst + i * kRows * 128) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(dst1 + i * kRows * 128) = make_uint4(h[4], h[5], h[6], h[7]);
      }
    };
    int jg = 0;
    while (KIND != 2 && ok && bt_next(w, a, lane)) {
      const int end = jg + w->n;
      for (; jg < end; ++jg) {
        const int st = jg % kBtStages;
        const uint32_t par = ((jg / kBtStages) & 1) ^ 1;
        if (!(ok = warp_wait(B_KEMPTY + st, par) && warp_wait(B_RFULL, jg & 1))) break;
        store_tile(L::k + st * L::tile, raw_k, nullptr, std::false_type{});
        warp_arrive_stored(BAR(B_KFULL + st), lane);
        if (lane == 0) mbar_arrive(BAR(B_REMPTY));
        if (!(ok = warp_wait(B_VEMPTY + st, par) && warp_wait(B_RFULL + 1, jg & 1))) break;
        store_tile(L::v + st * L::tile, raw_v, meta[jg % kBtMeta].ratio, std::true_type{});
        warp_arrive_stored(BAR(B_VFULL + st), lane);
        if (lane == 0) mbar_arrive(BAR(B_REMPTY + 1));
      }
    }
  } else {
    // ================================================================ softmax + epilogue
    regs_up<BtRegs<KIND>::softmax>();
    const int s = warp / 4;                     // slot of this warpgroup
    const int q4 = warp % 4;                    // TMEM lane quarter
    const int r = q4 * 32 + lane;               // row within the slot
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    int jg = 0, js = 0, segs = 0;
    // the slot's row of this thread in the current segment
    int gi = 0, full_hi = 0, full_lo = 0;
    float fac = 0.f;
    // what the epilogue of the segment before needs
    bool pending = false, whole = false, row_ok = false;
    float inv = 0.f;
    int64_t prow = 0, off = 0;
    auto row_of = [&]() { return w->r0 + min(s * kBtM + r, w->rows - 1); };   // rows behind the last repeat it
    // next segment with rows of this slot, and its Q rows: power-of-two scaled fp16
    // in shared memory.  The buffer is free: the slot's last OFINAL came after every
    // S MMA that read it.
    auto next_rows = [&]() {
      bool have = bt_next(w, a, lane);
      while (have && s * kBtM >= w->rows) {
        jg += w->n;
        have = bt_next(w, a, lane);
      }
      if (!have) return false;
      const int rr = row_of(), tok = (int)fast_div(rr, a.div_g), hq = w->hk * a.G + rr - tok * a.G;
      gi = w->start + tok;
      // tiles of keys full_lo < key0 <= full_hi, and sink tiles, need no mask for the slot's rows
      full_hi = w->start + (int)fast_div(w->r0 + s * kBtM, a.div_g) + 1 - kBtN;
      full_lo =
          a.window == 0 ? -1 : w->start + (int)fast_div(w->r0 + min((s + 1) * kBtM, w->rows) - 1, a.div_g) - a.window;
      const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q.ptr) + (int64_t)w->b * a.q.sb +
                                                       (int64_t)tok * a.q.sn + (int64_t)hq * a.q.sh);
      uint4 x[D / 8];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) x[i] = qp[i];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t wv[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = max(mx, max(wv[e] & 0x7fff0000u, (wv[e] << 16) & 0x7fff0000u));
      }
      float up, down;
      row_pow2(mx, up, down);
      fac = down * a.scale_log2 * (KIND == 2 ? a.k_unscale : KIND == 1 ? kE4m3Unscale : 1.f);
      uint8_t* qrow = smem + L::q + s * L::tile + r * 128;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const float2 f0 = bf2_to_f2(x[i].x), f1 = bf2_to_f2(x[i].y), f2 = bf2_to_f2(x[i].z), f3 = bf2_to_f2(x[i].w);
        const uint4 h = make_uint4(f2_to_h2(f0.x * up, f1.x * up), f2_to_h2(f0.y * up, f1.y * up),
                                   f2_to_h2(f2.x * up, f3.x * up), f2_to_h2(f2.y * up, f3.y * up));
        *reinterpret_cast<uint4*>(qrow + (i >> 3) * kBtHalf + (((i & 7) ^ (r & 7)) * 16)) = h;
      }
      warp_arrive_stored(BAR(B_QREADY + s), lane);
      return true;
    };
    while (ok) {
      const bool have = next_rows();            // its first S MMAs run beside the stores below
      if (pending) {
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          uint32_t o[32];
          tmem_ld32(tO(s) + lane_off + cb * 32, o);
          tmem_wait_ld<32>(o);
          if (row_ok) {
            float y[32];
#pragma unroll
            for (int c = 0; c < 32; c += 4) {     // columns hold dims 0, 2, 1, 3 of each four
              y[c] = __uint_as_float(o[c]) * inv;
              y[c + 1] = __uint_as_float(o[c + 2]) * inv;
              y[c + 2] = __uint_as_float(o[c + 1]) * inv;
              y[c + 3] = __uint_as_float(o[c + 3]) * inv;
            }
            if (!whole) {
#pragma unroll
              for (int c = 0; c < 32; c += 8) store_32b(a.part_o + prow * D + 32 * cb + c, reinterpret_cast<uint32_t*>(y) + c);
            } else if (a.o_bf16 && a.o_wide) {
              uint32_t h[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) h[c] = f2_to_bf2(y[2 * c], y[2 * c + 1]);
              __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.o.ptr) + off + 32 * cb;
              store_32b(op, h);
              store_32b(op + 16, h + 8);
            } else {
#pragma unroll
              for (int c = 0; c < 32; c += 4) store_o4(a, off + 32 * cb + c, make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]));
            }
          }
        }
        tc_fence_before();                      // O is read before the slot's next weights are announced
        pending = false;
      }
      if (!have) break;
      const int n = w->n;
      float m_used = -INFINITY, l = 0.f, vref = 0.f, poison = 0.f;
      for (int j = 0; j < n; ++j) {
        const int g = jg + j;
        // S first: its phases are counted per slot, and once tile g's S is there the
        // ring's barrier stands at tile g (a slot that sat out segments would take an
        // older phase of equal parity for it)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(BAR(B_SFULL + s), (js + j) & 1, abort_flag) &&
                                               mbar_wait(BAR(B_META + g % kBtMeta), (g / kBtMeta) & 1, abort_flag))))
          break;
        tc_fence_after();
        float x[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(tS(s) + lane_off + 32 * i, reinterpret_cast<uint32_t*>(x) + 32 * i);
        const BtMeta* mt = meta + g % kBtMeta;
        const int key0 = w->span.tile(w->u0 + j) << kBtLogN;
        const bool full = (key0 <= full_hi) && (key0 > full_lo || key0 + kBtN <= a.n_sink);
        tmem_wait_ld<128>(reinterpret_cast<uint32_t*>(x));
        // logits in log2 units: the product is rounded here, once, so that the row
        // maximum below is one of them and the winner's weight is 2^0 exactly
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float f = mt->ks[q] * fac;
#pragma unroll
          for (int c = 16 * q; c < 16 * q + 16; c += 2) mul2(x[c], x[c + 1], f);
        }
        if (!full) {
          const int lim = gi - key0;            // columns up to here are the row's past
          if (a.window == 0) {
#pragma unroll
            for (int c = 0; c < kBtN; ++c)
              if (c > lim) x[c] = -INFINITY;
          } else {
            const int win_lo = gi - a.window - key0, snk = a.n_sink - 1 - key0;
#pragma unroll
            for (int c = 0; c < kBtN; ++c)
              if (c > lim || (c <= win_lo && c > snk)) x[c] = -INFINITY;
          }
        }
        float of = 1.f;                         // O's factor
        const int rare = mt->rare;
        if (__builtin_expect(rare != 0, 0)) {
          if (rare & kBtBad) {                  // NaN for the rows that see a marked key
            for (int c = 0; c < kBtN; ++c)
              if (((rare >> (c >> 4)) & 1) && key0 + c <= gi &&
                  (a.window == 0 || key0 + c > gi - a.window || key0 + c < a.n_sink))
                poison = __uint_as_float(0x7fffffffu);
          }
          if (rare & kBtWide) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float e = (float)mt->lv[q];
#pragma unroll
              for (int c = 16 * q; c < 16 * q + 16; ++c) x[c] += e;
            }
          }
          // m in units of the new reference; where l would pass 2^96, O takes the rest
          const int by = rare >> kBtGrown, sh = max(0, min(by, 96 + 127 - (int)(__float_as_uint(l) >> 23)));
          m_used -= (float)sh;
          if (l > 0.f) l *= __int_as_float((127 + sh) << 23);
          of = by - sh > 126 ? 0.f : __int_as_float((127 - by + sh) << 23);
        }
        float m8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) m8[u] = fmaxf(x[2 * u], x[2 * u + 1]);
#pragma unroll
        for (int c = 16; c < kBtN; c += 16) {
#pragma unroll
          for (int u = 0; u < 8; ++u) m8[u] = fmax3(m8[u], x[c + 2 * u], x[c + 2 * u + 1]);
        }
        const float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
        const float m_new = fmaxf(m_used, mx);
        const bool need = m_new > m_used + kLazyRescale;
        vref = mt->vref;
        if (need) {
          const float alpha = fast_exp2(m_used - m_new);   // 0 when m_used = -inf
          m_used = m_new;
          l *= alpha;
          of *= alpha;
        }
        const float mref = kKbUp - (m_used == -INFINITY ? 0.f : m_used);
        // weights, packed in pairs, over the columns of S as they are made
        float l2[2] = {0.f, 0.f};
        if (__builtin_expect(rare & kBtWide, 0)) {   // l's terms, without 2^lv
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            float t = 0.f;
#pragma unroll
            for (int c = 16 * q; c < 16 * q + 16; ++c) t += fast_exp2(x[c] + mref);
            l += t * __int_as_float((127 - mt->lv[q]) << 23);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pc[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = 32 * q + 2 * i;
            add2(x[c], x[c + 1], mref, mref);
            x[c] = fast_exp2(x[c]);
            x[c + 1] = fast_exp2(x[c + 1]);
            add2(l2[0], l2[1], x[c], x[c + 1]);
            pc[i] = f2_to_h2(x[c], x[c + 1]);
          }
          tmem_st16(tS(s) + lane_off + 16 * q, pc);
        }
        if (!(rare & kBtWide)) l += l2[0] + l2[1];
        if (__any_sync(0xffffffffu, of != 1.f) && j > 0) {
#pragma unroll 1
          for (int cb = 0; cb < D / 32; ++cb) {
            uint32_t o[32];
            tmem_ld32(tO(s) + lane_off + cb * 32, o);
            tmem_wait_ld<32>(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * of);
            tmem_st32(tO(s) + lane_off + cb * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_PREADY + s));
      }
      if (!ok) break;

      // ---- epilogue: O / l -> the output row, or a partial for the merge
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(BAR(B_OFINAL + s), segs & 1, abort_flag)))) break;
      tc_fence_after();
      const int rr = row_of(), tok = (int)fast_div(rr, a.div_g), hq = w->hk * a.G + rr - tok * a.G;
      whole = w->whole;
      row_ok = s * kBtM + r < w->rows;
      const float lse = l == 0.f ? -INFINITY : (m_used - kKbUp + log2f(l)) * 0.69314718055994530942f;
      inv = (l == 0.f ? 0.f : vref * (KIND == 2 ? a.v_unscale : (KIND == 1 ? kE4m3Unscale : 1.f) / kBtVUp<KIND>) / l) + poison;
      prow = ((int64_t)blockIdx.x * 2 + w->slot) * a.rows_item + s * kBtM + r;
      off = (int64_t)w->b * a.o.sb + (int64_t)tok * a.o.sn + (int64_t)hq * a.o.sh;
      if (row_ok) {
        if (!whole) a.part_lse[prow] = lse;
        else if (a.lse) a.lse[(int64_t)w->b * a.lse_sb + hq * a.lse_sh + tok] = lse;
      }
      jg += n;
      js += n;
      ++segs;
      pending = true;
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kBtMma) tmem_dealloc(tmem, 512);
}

}  // namespace rcx
