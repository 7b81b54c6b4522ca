// Attention of few query rows (one token, or some drafted tokens, of each
// sequence; items of at most 32 rows) over a block-scaled 8-bit paged KV cache, and the merge of partials.
//
// Key j of KV head h stands for k_code[j] * k_scale[block(j), h] (and likewise
// V).  For every row:  x_j = (q . k_code_j) * k_scale * log2(e) / (sqrt(d) t),
// p_j = 2^(x_j - m), O = sum p_j v_code_j v_scale / sum p_j, LSE = ln 2 (m +
// log2 sum p_j).  Memory-bound: every code and scale a row sees is read once
// per item, that is for up to 32 rows of a (sequence, KV head) together.
//
// A warp takes 32-key tiles through a ring of cp.async stages and computes, per
// 16 keys, S^T = K Q^T and O^T += V^T P^T on fp16 MMAs (m16n8k16, fp32
// accumulators) with the keys (then the head dim) as MMA rows and the query
// rows as the 8-wide columns, so no MMA row is padding.
//  * Codes become exact fp16 by bit arithmetic (codes4_to_h2).  Each query row
//    is scaled by a power of two to at most 2^15 and is then exact in fp16 too
//    (down to 2^-28 of its largest element), so S is the fp32 sum of exact
//    products: the logits carry no operand rounding.
//  * The d order inside a dot product is free: lane (g, c) takes the 16-byte
//    pieces c and c + 4 of key rows g and g + 8, and Q is laid out to match.
//  * V^T comes from ldmatrix.trans over 16-bit elements (two dims of one key).
//  * The block scale of K multiplies S per 16 keys (blocks are 16 tokens or
//    more); that of V multiplies P as ratio to vref, which follows the scales up
//    and, past 2^-4 of it, down again (not below 2^-80 of the largest), O changing
//    with it in fp32.  So P's range is spent on weights, whatever scales other rows
//    see.  P is held as 2^7 p in fp16 (p <= 2^8 between moves of m): weights down
//    to 2^-28 of the largest keep their place; 11 bits of P against 8 of a bf16
//    output.
//  * 16 keys that no row of the item sees are not read, nor is their table entry.
//  * m moves only when a logit passes it by 2^8: most tiles need no shuffle
//    and no rescale of O.
// Table entries and scales come 16 tiles at a time, one per lane, a batch ahead.
#pragma once
#include "launch.h"
#include "kv_int8.cuh"
#include "kv_block_plan.cuh"

namespace rcx {

constexpr int kKbWarps = kKvFewWarps;
constexpr int kKbKeys = kKvFewTile;             // keys per tile
constexpr float kKbLazy = 8.f;                  // log2 units a logit may pass m
constexpr float kKbUp = 7.f;                    // P is held times 2^7

template <int D>
constexpr int kb_stage_bytes = 2 * kKbKeys * D;
template <int D, int NT>
constexpr int kb_smem_bytes = kKbWarps * kKvFewStages * kb_stage_bytes<D> + NT * (D / 16) * 32 * 8 + NT * 8 * 4;

// 16-byte piece p of key row r sits at piece p ^ kb_swz(r): conflict-free for
// the 8-row ldmatrix reads and for the quarter-warp reads of two rows.
template <int D>
__device__ __forceinline__ int kb_swz(int r) {
  return D == 128 ? ((r & 1) << 2) | ((r >> 1) & 3) : (r >> 1) & 3;
}

// Power of two that brings a row of largest |element| `bits` (bf16 bits << 16)
// into [2^14, 2^15), and its inverse; a row with infinities or NaN stays.
__device__ __forceinline__ void row_pow2(uint32_t bits, float& up, float& down) {
  const int eb = (int)(bits >> 23);
  const int f = eb == 255 ? 127 : min(252, 268 - eb);
  up = __uint_as_float((uint32_t)f << 23);
  down = __uint_as_float((uint32_t)(254 - f) << 23);
}

// Reference of the V scales: the first scale that is not zero times a power of two,
// so that moving it is exact, and scales that are all alike are exact too.  Keys
// of scales lo .. hi (positive) move it to hi or just above where hi passes it or
// lo falls below 2^-4 of it, but not below 2^-80 of the largest so far.
struct VRef {
  float v, inv, top;
  __device__ __forceinline__ bool holds(float lo, float hi) const { return hi <= v && lo * 16.f >= v; }
  __device__ __forceinline__ void begin(float s) {
    if (v > 0.f) return;
    v = top = fmaxf(s, 0x1p-126f);
    inv = 1.f / v;
  }
  // what O is to be multiplied by
  __device__ __forceinline__ float move(float hi) {
    const int want = __float_as_int(fminf(fmaxf(fmaxf(hi, top * 0x1p-80f), 0x1p-126f), 0x1p125f));
    const int k = (want - __float_as_int(v) + 0x7fffff) >> 23;     // least k with v 2^k >= want
    v = __int_as_float(__float_as_int(v) + (k << 23));
    inv = __int_as_float(__float_as_int(inv) - (k << 23));
    top = fmaxf(top, v);
    return k > 126 ? 0.f : __int_as_float((127 - k) << 23);
  }
  __device__ __forceinline__ float follow(float s) {
    if (!(s > 0.f)) return 1.f;                  // zero or NaN
    begin(s);
    return holds(s, s) ? 1.f : move(s);
  }
};

template <int D, int NT, int KIND>
__global__ void __launch_bounds__(kKbWarps * 32, kv_few_ctas(D, NT)) attn_kv_block_kernel(const KvAttnArgs a) {
  constexpr int LOGT = 5;
  static_assert(1 << LOGT == kKbKeys, "tile");
  constexpr int kChunks = D / 16;               // 16-dim MMA steps
  constexpr int kStage = kb_stage_bytes<D>;
  constexpr int kKbStages = kKvFewStages;
  constexpr int kTile = kKbKeys * D;
  constexpr int kPieces = D / 16;               // 16-byte pieces per key row
  constexpr int kRowsPerCopy = 32 / kPieces;    // key rows one warp-wide 16-byte copy covers
  constexpr bool kQRegs = NT <= 2;
  extern __shared__ __align__(128) uint8_t kb_smem[];
  __shared__ float sm_m[kKbWarps][NT * 8], sm_l[kKbWarps][NT * 8];
  __shared__ PlanStart sm_plan;
  uint2* sm_q = reinterpret_cast<uint2*>(kb_smem + kKbWarps * kKbStages * kStage);    // [NT][kChunks][32]
  float* sm_fac = reinterpret_cast<float*>(sm_q + NT * kChunks * 32);                 // [NT * 8]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane >> 2, c = lane & 3;
  if (warp == 0) {
    const PlanStart p = plan_start<LOGT>(a, blockIdx.x, lane);
    if (lane == 0) sm_plan = p;
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  SegWalk w;
  w.init(sm_plan);
  const KvBlockView& kv = a.c;
  const int lb = kv.block_log2, bmask = (1 << lb) - 1;
  uint8_t* wptr = kb_smem + warp * kKbStages * kStage;
  const uint32_t wbuf = static_cast<uint32_t>(__cvta_generic_to_shared(wptr));

  // copy lanes: row cr (+ kRowsPerCopy i), piece cp
  const int cr = lane / kPieces, cp = lane % kPieces;
  // fragment reads
  const uint32_t k_frag = g * D + ((c ^ kb_swz<D>(g)) * 16);
  const uint32_t v_row = ((lane & 7) + 8 * ((lane >> 3) & 1)) * D;
  const int v_swz = kb_swz<D>(lane & 7), v_hi = lane >> 4;

  while (w.next<LOGT>(a)) {
    const Entry& t = w.t;
    const int64_t b = t.b;
    // ---- this warp's tiles: u0 + warp, u0 + warp + kKbWarps, ...
    const int ub = w.u0 + warp;
    const int nk = ub < w.u1 ? (w.u1 - ub + kKbWarps - 1) / kKbWarps : 0;
    const KeySpan span = t.span;
    const int hi = span.hi;
    const int32_t* trow = kv.table + b * kv.t_sb;
    const float* ksh = kv.ks + w.hk;
    const float* vsh = kv.vs + w.hk;
    // keys up to here, sinks apart, are outside every row's window
    const int hidden = a.window > 0 ? t.start + t.n_lo - a.window : -1;
    auto load_meta = [&](int batch, int& ph, float& ks, float& vs) {
      ph = 0;
      ks = vs = 0.f;
      const int kk = 16 * batch + (lane >> 1);
      if (kk < nk) {
        const int key = (span.tile(ub + kKbWarps * kk) << LOGT) + ((lane & 1) << 4);
        if (key < hi && (key + 15 > hidden || key < a.n_sink)) {
          int e = trow[key >> lb];
          if ((unsigned)e >= (unsigned)kv.n_blocks) {
            record_device_error(RCX_ERR_DEVICE_INDEX);
            e = 0;
          }
          ph = e;
          ks = ksh[(int64_t)e * kv.Hkv];
          vs = vsh[(int64_t)e * kv.Hkv];
          if (!(fabsf(vs) < INFINITY)) vs = __uint_as_float(0x7fffffffu);
        }
      }
    };
    const uint8_t* kb = kv.k + w.hk * kv.k_sh + cp * 16;
    const uint8_t* vb = kv.v + w.hk * kv.v_sh + cp * 16;
    int ph_a, ph_b = 0;
    float ks_a, vs_a, ks_b, vs_b;
    load_meta(0, ph_a, ks_a, vs_a);
    auto issue = [&](int kk, int batch, int st) {
      if (kk < nk) {
        const int src = (kk >> 4) == batch ? ph_a : ph_b;
        const int key0 = span.tile(ub + kKbWarps * kk) << LOGT;
        const int rem = hi - key0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ph = __shfl_sync(0xffffffffu, src, 2 * (kk & 15) + h);
          const int64_t tok = ((key0 + 16 * h) & bmask) + cr;
          const uint8_t* kp = kb + ph * kv.k_sb + tok * kv.k_sn;
          const uint8_t* vp = vb + ph * kv.v_sb + tok * kv.v_sn;
#pragma unroll
          for (int i = 0; i < 16 / kRowsPerCopy; ++i) {
            const int r = 16 * h + cr + kRowsPerCopy * i;
            const uint32_t dst = wbuf + st * kStage + r * D + ((cp ^ kb_swz<D>(r & 7)) * 16);
            const int bytes = r < rem ? 16 : 0;   // rows behind the keys: zeros, nothing read
            const int64_t step = bytes ? (int64_t)kRowsPerCopy * i : -(int64_t)cr;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(kp + step * kv.k_sn), "r"(bytes)
                         : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + kTile), "l"(vp + step * kv.v_sn),
                         "r"(bytes)
                         : "memory");
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kKbStages - 1; ++s) issue(s, 0, s);
    load_meta(1, ph_b, ks_b, vs_b);

    // the first tiles are on their way; now the queries
    // ---- Q^T operand: chunk i of lane (g, c) holds dims base + {0, 2}, base + {1, 3}
    // of row 8 nt + g, base = 16 c + 4 i (i < 4) or 64 + 16 c + 4 (i - 4)
    for (int nt = warp; nt < NT; nt += kKbWarps) {
      const int r = 8 * nt + g;
      float x[4 * kChunks];
      uint32_t mx = 0;
      if (r < t.rows) {
        const int n = (int)fast_div(t.r0 + r, a.div_g), h = t.r0 + r - n * a.G;
        const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q.ptr) + b * a.q.sb + (int64_t)n * a.q.sn +
                                  (int64_t)(w.hk * a.G + h) * a.q.sh + 16 * c;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint2 u = *reinterpret_cast<const uint2*>(qp + (i < 4 ? 4 * i : 64 + 4 * (i - 4)));
          const float2 lo = bf2_to_f2(u.x), hi = bf2_to_f2(u.y);
          x[4 * i] = lo.x; x[4 * i + 1] = lo.y; x[4 * i + 2] = hi.x; x[4 * i + 3] = hi.y;
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = max(mx, __float_as_uint(x[4 * i + e]) & 0x7fffffffu);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4 * kChunks; ++i) x[i] = 0.f;
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      float up, down;
      row_pow2(mx, up, down);
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        sm_q[(nt * kChunks + i) * 32 + lane] =
            make_uint2(f2_to_h2(x[4 * i] * up, x[4 * i + 2] * up), f2_to_h2(x[4 * i + 1] * up, x[4 * i + 3] * up));
      if (c == 0) sm_fac[r] = down * a.scale_log2 * (KIND == 1 ? kE4m3Unscale : 1.f);
    }
    __syncthreads();
    uint2 qf[kQRegs ? NT : 1][kChunks];
    if constexpr (kQRegs) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < kChunks; ++i) qf[nt][i] = sm_q[(nt * kChunks + i) * 32 + lane];
    }
    // per column (row of Q) 8 nt + 2 c + h: logit factor, token, running max, sum
    float fac[NT][2], m[NT][2], l[NT][2];
    int qi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * nt + 2 * c + h;
        fac[nt][h] = sm_fac[r];
        qi[nt][h] = r < t.rows ? t.start + (int)fast_div(t.r0 + r, a.div_g) : -1;
        m[nt][h] = -INFINITY;
        l[nt][h] = 0.f;
      }
    float o[kChunks][NT][4];
#pragma unroll
    for (int mt = 0; mt < kChunks; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    VRef vref = {0.f, 0.f, 0.f};
    bool uneven = false;                         // the reference moves tile by tile, or a scale is NaN
    uint32_t poison = 0;                         // rows 8 nt + 2 c + h (bit 2 nt + h) that saw one
    auto scale_o = [&](float f) {
#pragma unroll
      for (int mt = 0; mt < kChunks; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] *= f;
    };

    int st = 0;
    for (int kk = 0; kk < nk; ++kk) {
      const int batch = kk >> 4;
      if ((kk & 15) == 0 && kk > 0) {
        ph_a = ph_b;
        ks_a = ks_b;
        vs_a = vs_b;
        load_meta(batch + 1, ph_b, ks_b, vs_b);
      }
      if ((kk & 15) == 0) {                      // the reference for 16 tiles at once, if one can hold them all
        const uint32_t bits = vs_a > 0.f ? __float_as_uint(vs_a) : 0u;
        const float hi = __uint_as_float(__reduce_max_sync(0xffffffffu, bits));
        const float lo = __uint_as_float(__reduce_min_sync(0xffffffffu, bits ? bits : 0x7f7fffffu));
        uneven = (hi > 0.f && lo * 16.f < hi) || __any_sync(0xffffffffu, vs_a != vs_a);
        if (hi > 0.f && !uneven) {
          vref.begin(__shfl_sync(0xffffffffu, vs_a, __ffs(__ballot_sync(0xffffffffu, bits != 0u)) - 1));
          if (!vref.holds(lo, hi)) scale_o(vref.move(hi));
        }
      }
      issue(kk + kKbStages - 1, batch, st == 0 ? kKbStages - 1 : st - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kKbStages - 1) : "memory");
      __syncwarp();
      const uint8_t* sk = wptr + st * kStage;
      const int key0 = span.tile(ub + kKbWarps * kk) << LOGT;
      float ks[2], vs[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ks[u] = __shfl_sync(0xffffffffu, ks_a, 2 * (kk & 15) + u);
        vs[u] = __shfl_sync(0xffffffffu, vs_a, 2 * (kk & 15) + u);
      }
      // S^T per 16-key half u: element e is (key 16 u + g + 8 (e >> 1), row 8 nt + 2 c + (e & 1))
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
        float s2[NT <= 2 ? NT : 1][4];           // a second chain halves the latency of the dot products
#pragma unroll
        for (int nt = 0; nt < (NT <= 2 ? NT : 1); ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s2[nt][e] = 0.f;
        uint32_t kw[2][kChunks];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int hf = 0; hf < D / 64; ++hf) {
            const uint4 x = *reinterpret_cast<const uint4*>(sk + (16 * u + 8 * r) * D + (k_frag ^ (64 * hf)));
            kw[r][4 * hf] = x.x; kw[r][4 * hf + 1] = x.y; kw[r][4 * hf + 2] = x.z; kw[r][4 * hf + 3] = x.w;
          }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          uint32_t af[4];
          codes4_to_h2<KIND>(kw[0][i], af[0], af[2]);
          codes4_to_h2<KIND>(kw[1][i], af[1], af[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 q = kQRegs ? qf[kQRegs ? nt : 0][i] : sm_q[(nt * kChunks + i) * 32 + lane];
            mma_f16_16816(NT <= 2 && (i & 1) ? s2[NT <= 2 ? nt : 0] : s[u][nt], af, q.x, q.y);
          }
        }
        if constexpr (NT <= 2) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][nt][e] += s2[nt][e];
        }
      }
      // logits in log2 units; a tile cut by the mask or the keys' end element by element
      const bool full = key0 + kKbKeys <= t.start + 1 + t.n_lo &&
                        (a.window == 0 || key0 > t.start + t.n_hi - a.window || key0 + kKbKeys <= a.n_sink);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f0 = fac[nt][0] * ks[u], f1 = fac[nt][1] * ks[u];
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] *= e & 1 ? f1 : f0;
        }
      if (!full) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = key0 + 16 * u + g + 8 * (e >> 1), i = qi[nt][e & 1];
              if (!(j <= i && (a.window == 0 || j > i - a.window || j < a.n_sink))) s[u][nt][e] = -INFINITY;
            }
      }
      bool move = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          move |= fmaxf(fmaxf(s[0][nt][h], s[0][nt][h + 2]), fmaxf(s[1][nt][h], s[1][nt][h + 2])) > m[nt][h] + kKbLazy;
      float vratio[2] = {vs[0] * vref.inv, vs[1] * vref.inv}, unit1 = 1.f;     // unit1: of O before the second half
      if (uneven) {
        const float unit0 = vref.follow(vs[0]);
        vratio[0] = vs[0] * vref.inv;
        unit1 = vref.follow(vs[1]);
        vratio[1] = vs[1] * vref.inv;
        if (unit0 != 1.f) scale_o(unit0);
        // a block of scale NaN makes NaN of the rows that see it, however small their weight, and only of those
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (vs[u] != vs[u]) {
            vratio[u] = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (s[u][nt][e] != -INFINITY) poison |= 1u << (2 * nt + (e & 1));
          }
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float al[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(fmaxf(s[0][nt][h], s[0][nt][h + 2]), fmaxf(s[1][nt][h], s[1][nt][h + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            mx = fmaxf(mx, m[nt][h]);
            const float alpha = mx == m[nt][h] ? 1.f : dec_exp2(m[nt][h] - mx);   // 0 from m = -inf
            m[nt][h] = mx;
            l[nt][h] *= alpha;
            al[h] = alpha;
          }
#pragma unroll
          for (int mt = 0; mt < kChunks; ++mt) {
            o[mt][nt][0] *= al[0];
            o[mt][nt][1] *= al[1];
            o[mt][nt][2] *= al[0];
            o[mt][nt][3] *= al[1];
          }
        }
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mref[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) mref[h] = (m[nt][h] == -INFINITY ? 0.f : m[nt][h]) - kKbUp;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float ratio = vratio[u];
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = dec_exp2(s[u][nt][e] - mref[e & 1]);
            l[nt][e & 1] += p[e];
            p[e] *= ratio;
          }
          pb[u][nt][0] = movmatrix_t(f2_to_h2(p[0], p[1]));   // keys 2c, 2c + 1 of row 8 nt + g
          pb[u][nt][1] = movmatrix_t(f2_to_h2(p[2], p[3]));   // keys 2c + 8, 2c + 9
        }
      }
      // O^T += V^T P^T: MMA row g of m-tile mt is dim 16 mt + 2 g, row g + 8 is dim 16 mt + 2 g + 1
      const uint32_t sv = wbuf + st * kStage + kTile + v_row;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u == 1 && unit1 != 1.f) scale_o(unit1);
#pragma unroll
        for (int mp = 0; mp < D / 32; ++mp) {
          uint32_t rr[4];
          ldsm_x4_t(rr, sv + 16 * u * D + (((2 * mp + v_hi) ^ v_swz) * 16));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t af[4];
            codes4_to_h2<KIND>(rr[2 * h], af[0], af[1]);
            codes4_to_h2<KIND>(rr[2 * h + 1], af[2], af[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o[2 * mp + h][nt], af, pb[u][nt][0], pb[u][nt][1]);
          }
        }
      }
      __syncwarp();                              // the stage is refilled in the next iteration
      st = st == kKbStages - 1 ? 0 : st + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- merge the warps' states in shared memory (the stage buffers)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 4);
        l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 8);
        l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], 16);
        if (g == 0) {
          sm_m[warp][8 * nt + 2 * c + h] = m[nt][h];
          sm_l[warp][8 * nt + 2 * c + h] = l[nt][h];
        }
      }
#pragma unroll
    for (int i = 4; i < 32; i *= 2) poison |= __shfl_xor_sync(0xffffffffu, poison, i);
    __syncthreads();
    // [warps][8 NT][D + 4]: the pad spreads the rows of a store over the banks
    float* sm_o = reinterpret_cast<float*>(kb_smem);
    constexpr int kRow = D + 4;
    static_assert(kStage * kKbStages >= NT * 8 * kRow * 4, "merge area aliases the stage buffers");
    // each warp's own average: it cannot pass the largest value, whereas sums of values of 2^112 and more can pass fp32
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float av[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        av[h] = (poison >> (2 * nt + h)) & 1u ? __uint_as_float(0x7fffffffu) : l[nt][h] == 0.f ? 0.f : vref.v * (1.f / l[nt][h]);
#pragma unroll
      for (int mt = 0; mt < kChunks; ++mt) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = o[mt][nt][e] * av[e & 1] * (KIND == 1 ? kE4m3Unscale : 1.f);
        float* w0 = sm_o + (warp * NT * 8 + 8 * nt + 2 * c) * kRow + 16 * mt + 2 * g;
        *reinterpret_cast<float2*>(w0) = make_float2(y[0], y[2]);
        *reinterpret_cast<float2*>(w0 + kRow) = make_float2(y[1], y[3]);
      }
    }
    __syncthreads();
    const bool whole = w.whole();
    const int64_t prow = ((int64_t)blockIdx.x * 2 + w.slot()) * a.rows_item;
    for (int i = threadIdx.x; i < t.rows * (D / 4); i += kKbWarps * 32) {
      const int r = i / (D / 4), dd = (i % (D / 4)) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int x = 0; x < kKbWarps; ++x) mm = fmaxf(mm, sm_m[x][r]);
      const float mr = mm == -INFINITY ? 0.f : mm;
      float lt = 0.f, wl[kKbWarps];
      float4 ot = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kKbWarps; ++x) lt += wl[x] = dec_exp2(sm_m[x][r] - mr) * sm_l[x][r];
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
      for (int x = 0; x < kKbWarps; ++x) {
        const float wt = wl[x] * inv;
        const float4 y = *reinterpret_cast<const float4*>(sm_o + (x * NT * 8 + r) * kRow + dd);
        ot.x += wt * y.x; ot.y += wt * y.y; ot.z += wt * y.z; ot.w += wt * y.w;
      }
      const float lse = lt == 0.f ? -INFINITY : (mr - kKbUp + log2f(lt)) * 0.69314718055994530942f;
      if (whole) {
        const int n = (int)fast_div(t.r0 + r, a.div_g), hq = w.hk * a.G + t.r0 + r - n * a.G;
        store_o4(a, b * a.o.sb + (int64_t)n * a.o.sn + (int64_t)hq * a.o.sh + dd, ot);
        if (dd == 0 && a.lse) a.lse[b * a.lse_sb + hq * a.lse_sh + n] = lse;
      } else {
        *reinterpret_cast<float4*>(a.part_o + (prow + r) * D + dd) = ot;
        if (dd == 0) a.part_lse[prow + r] = lse;
      }
    }
    __syncthreads();                             // the buffers are free for the next segment
  }
  if (a.direct) empty_rows<D>(a, warp, kKbWarps, lane);
}

// Merge of items that several CTAs share, by the LSE rule of rcx_merge_partials,
// and zeros (LSE -inf) for the rows of tokens past a sequence's count.  One CTA
// per (entry, KV head) and slice of its rows; kWarpsPerRow warps share a row's
// partials.  A warp loads up to eight partials at once; of more, 32 LSE at once and
// then their rows with eight loads in flight: bound by the latency of that chain.
// x is the average so far, not the sum: averages stay within the values' range.
// It waits for the attention kernel's end on the device (programmatic dependent
// launch), so that its launch is hidden behind it.
template <int D, int kWarpsPerRow>
static __global__ void __launch_bounds__(256) attn_kv_block_merge_kernel(const KvAttnArgs a) {
  constexpr int kL = D / 4;                      // lanes that hold dims (d = 64: half a warp)
  __shared__ float sm_m[8], sm_l[8];
  __shared__ float4 sm_o[8][32];
  const int e = blockIdx.x, hk = blockIdx.y;
  const int bl = (int)fast_div(e, a.div_nrt), rt = e - bl * a.n_rt;
  const int64_t b = a.b0 + bl;
  const SeqRange s = seq_range(a.start, a.count, (int)b, a.N, a.c.cap);
  const int r0 = rt * a.rows_item;
  const int live = max(0, min(s.n * a.G - r0, a.rows_item));
  const int rows = min(a.N * a.G - r0, a.rows_item);
  // lengths were there before the attention kernel began; its tables and partials come now
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int T = a.prefix[a.B * a.n_rt], p0 = a.prefix[e];
  const int nt = (int)fast_div(a.prefix[e + 1] - p0, a.div_hkv);
  // CTAs c0 .. c1 hold pieces of the item; the first one's may be its range's last
  // segment (the line), all others are their CTA's first
  const int even = a.prefix[a.B * a.n_rt + 1];
  int c0 = 0, c1 = 0, first_slot = 0;
  if (nt > 0 && even > 0) {
    c0 = (e * a.c.Hkv + hk) * even;
    c1 = nt == 1 ? c0 : c0 + even - 1;       // a single tile is one whole piece
  } else if (nt > 0) {
    const int P = range_ctas(T, a), i0 = p0 + hk * nt;
    c0 = range_owner(T, i0, P);
    c1 = range_owner(T, i0 + nt - 1, P);
    first_slot = range_start(T, c0, P) == i0 ? 0 : 1;
  }
  if (live == rows && c0 == c1) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int team = warp / kWarpsPerRow, sub = warp % kWarpsPerRow;
  constexpr int kTeams = 8 / kWarpsPerRow;
  const int dd = 4 * (lane % kL);
  for (int rb = blockIdx.z * kTeams; rb < rows; rb += gridDim.z * kTeams) {
    const int r = rb + team;
    const bool row_ok = r < rows;
    const bool shared = row_ok && r < live && c0 != c1;
    float mm = -INFINITY, lsum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (shared && c1 - c0 < 8 * kWarpsPerRow) {
      // up to eight partials a warp, every lane on its own: all loads first
      float ls[8];
      float4 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = sub + kWarpsPerRow * i, c = c0 + j;
        const bool there = c <= c1 && (even == 0 || nt >= even || range_start(nt, j, even) < range_start(nt, j + 1, even));
        const int64_t pr = ((int64_t)c * 2 + (j == 0 ? first_slot : 0)) * a.rows_item + r;
        ls[i] = there ? a.part_lse[pr] : -INFINITY;
        y[i] = there ? *reinterpret_cast<const float4*>(a.part_o + pr * D + dd) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) mm = fmaxf(mm, ls[i]);                                // passes NaN over
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ls[i] = ls[i] == -INFINITY ? 0.f : expf(ls[i] - (mm == -INFINITY ? 0.f : mm));            // NaN stays here
        lsum += ls[i];
      }
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wi = ls[i] * inv;
        x.x += wi * y[i].x; x.y += wi * y[i].y; x.z += wi * y[i].z; x.w += wi * y[i].w;
      }
    } else if (shared) {
      for (int cb = c0 + sub; cb <= c1; cb += 32 * kWarpsPerRow) {
        const int c = cb + kWarpsPerRow * lane;
        const int n = min(32, (c1 - cb) / kWarpsPerRow + 1);
        const int64_t pr = ((int64_t)c * 2 + (c == c0 ? first_slot : 0)) * a.rows_item + r;
        // (even: an item with fewer tiles than pieces leaves some without any)
        const bool there = lane < n && (even == 0 || nt >= even || range_start(nt, c - c0, even) < range_start(nt, c - c0 + 1, even));
        const float ls = there ? a.part_lse[pr] : -INFINITY;
        const uint32_t some = __ballot_sync(0xffffffffu, ls != -INFINITY);       // partials with keys, however small
        float mn = ls;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));   // passes NaN over
        mn = fmaxf(mn, mm);
        float wt = ls == -INFINITY ? 0.f : expf(ls - (mn == -INFINITY ? 0.f : mn));              // NaN stays here
        const float f0 = mm == mn ? 1.f : expf(mm - mn);
        float ws = wt;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
        const float kept = lsum * f0;
        lsum = kept + ws;
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum, f1 = kept * inv;
        wt *= inv;
        x.x *= f1; x.y *= f1; x.z *= f1; x.w *= f1;
        mm = mn;
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
          const float wi = __shfl_sync(0xffffffffu, wt, i);
          const int64_t pi = __shfl_sync(0xffffffffu, pr, i);
          if (!((some >> i) & 1u)) continue;
          const float4 y = *reinterpret_cast<const float4*>(a.part_o + pi * D + dd);
          x.x += wi * y.x; x.y += wi * y.y; x.z += wi * y.z; x.w += wi * y.w;
        }
      }
    }
    if constexpr (kWarpsPerRow > 1) {
      if (lane == 0) {
        sm_m[warp] = mm;
        sm_l[warp] = lsum;
      }
      sm_o[warp][lane] = x;
      __syncthreads();
      if (sub == 0) {
        float mt = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarpsPerRow; ++i) mt = fmaxf(mt, sm_m[warp + i]);
        x = make_float4(0.f, 0.f, 0.f, 0.f);
        lsum = 0.f;
        float f[kWarpsPerRow];
#pragma unroll
        for (int i = 0; i < kWarpsPerRow; ++i) {
          f[i] = sm_l[warp + i] == 0.f ? 0.f : expf(sm_m[warp + i] - (mt == -INFINITY ? 0.f : mt)) * sm_l[warp + i];
          lsum += f[i];
        }
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
#pragma unroll
        for (int i = 0; i < kWarpsPerRow; ++i) {
          const float4 y = sm_o[warp + i][lane];
          const float wi = f[i] * inv;
          x.x += wi * y.x; x.y += wi * y.y; x.z += wi * y.z; x.w += wi * y.w;
        }
        mm = mt;
      }
      __syncthreads();
    }
    if (sub == 0 && row_ok && lane < kL && (shared || r >= live)) {
      const int n = (int)fast_div(r0 + r, a.div_g), hq = hk * a.G + (r0 + r) - n * a.G;
      store_o4(a, b * a.o.sb + (int64_t)n * a.o.sn + (int64_t)hq * a.o.sh + dd, x);
      if (lane == 0 && a.lse) a.lse[b * a.lse_sb + hq * a.lse_sh + n] = lsum == 0.f ? -INFINITY : mm + logf(lsum);
    }
  }
}

}  // namespace rcx
