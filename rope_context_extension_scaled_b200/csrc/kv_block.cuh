// Block-scaled 8-bit paged KV cache: quantisation of new tokens into the blocks
// they fall in, and reading tokens back.
//
// "Context window extension: 4K to 1M" section 6.1 keeps the KV cache in 8 bits
// instead of 16.  Here a block is 2^k tokens of one sequence and KV head with
// one fp32 scale for K and one for V; a table gives each sequence its blocks.
//   int8:  s = fl(amax / 127), at least 2^-120; code = rint(x * fl(1 / s)), the
//          product unrounded.  fma(x, inv, 1.5 * 2^23) rounds once, at the unit
//          place and ties to even (the constant is even), so its low byte is
//          the code; |x inv| <= 127 (1 + 2^-22), so no clamp is needed.
//   e4m3:  s = the smallest power of two with amax <= 448 s, from amax's
//          exponent and a comparison of its fraction with 0.75 (448 = 1.75 2^8);
//          x / s is exact, code = e4m3(x / s), ties to even.
// A block that already holds tokens keeps the larger of its scale and the new
// tokens'; when it grows, the old codes become rint(code * fl(s_old / s)) (or
// the e4m3 form of it).  Maxima are taken on bit patterns of |x|, where NaN >
// infinity > every number: a block given a non-finite value gets scale NaN and
// reads back as NaN.  e4m3's NaN codes are never written; the readers take
// their bits as +-480, so that no code can make a NaN.
#pragma once
#include <cuda_fp16.h>
#include "common.cuh"
#include "kv_block_args.h"

namespace rcx {

constexpr float kRoundMagic = 12582912.f;         // 1.5 * 2^23
constexpr float kE4m3Unscale = 256.f;             // codes4_to_h2<e4m3> gives value * 2^-8

// Start and number of new tokens of sequence b; a pair that does not fit the
// cache is reported in the device status word and counts as no tokens.
struct SeqRange {
  int start, n;
};

__device__ __forceinline__ SeqRange seq_range(const int64_t* start, const int64_t* count, int b, int N, int cap) {
  const int64_t s = start[b], n = count ? count[b] : N;
  SeqRange r{0, 0};
  if (s < 0 || n < 0 || n > N || s > cap || s + n > cap) {
    record_device_error(RCX_ERR_DEVICE_INDEX);
  } else {
    r.start = (int)s;
    r.n = (int)n;
  }
  return r;
}

// Physical block of a table entry; a bad entry is reported and gives -1.
__device__ __forceinline__ int checked_block(const KvBlockView& c, int b, int logical) {
  const int e = c.table[b * c.t_sb + logical];
  if ((unsigned)e >= (unsigned)c.n_blocks) {
    record_device_error(RCX_ERR_DEVICE_INDEX);
    return -1;
  }
  return e;
}

// Four codes -> fp16 pairs of bytes (0, 2) and (1, 3).
// int8 (exact): the byte with its sign flipped (u = code + 128) under the
// exponent of 1024 reads as 1024 + u; subtract 1152.
// e4m3 (value * 2^-8, exact, subnormals too): sign to bit 15, exponent and
// fraction to bits 13..7.
template <int KIND>
__device__ __forceinline__ void codes4_to_h2(uint32_t w, uint32_t& p02, uint32_t& p13) {
  if constexpr (KIND == 0) {
    const uint32_t x = w ^ 0x80808080u;
    const uint32_t h0 = __byte_perm(x, 0x64646464u, 0x4240), h1 = __byte_perm(x, 0x64646464u, 0x4341);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 r0 = __hsub2(*reinterpret_cast<const __half2*>(&h0), off);
    const __half2 r1 = __hsub2(*reinterpret_cast<const __half2*>(&h1), off);
    p02 = *reinterpret_cast<const uint32_t*>(&r0);
    p13 = *reinterpret_cast<const uint32_t*>(&r1);
  } else {
    p13 = ((w >> 1) & 0x3f803f80u) | (w & 0x80008000u);
    p02 = ((w << 7) & 0x3f803f80u) | ((w << 8) & 0x80008000u);
  }
}

__device__ __forceinline__ float2 h2_to_f2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// Four codes -> their values in fp32, in order.
template <int KIND>
__device__ __forceinline__ void codes4_to_f(uint32_t w, float* f) {
  uint32_t p02, p13;
  codes4_to_h2<KIND>(w, p02, p13);
  const float2 a = h2_to_f2(p02), b = h2_to_f2(p13);
  const float k = KIND == 0 ? 1.f : kE4m3Unscale;
  f[0] = a.x * k; f[1] = b.x * k; f[2] = a.y * k; f[3] = b.y * k;
}

// Four values y (already divided by the scale) -> packed codes.
template <int KIND>
__device__ __forceinline__ uint32_t codes4_of(float y0, float y1, float y2, float y3, float mul) {
  if constexpr (KIND == 0) {
    const uint32_t a = __float_as_uint(__fmaf_rn(y0, mul, kRoundMagic)), b = __float_as_uint(__fmaf_rn(y1, mul, kRoundMagic));
    const uint32_t c = __float_as_uint(__fmaf_rn(y2, mul, kRoundMagic)), d = __float_as_uint(__fmaf_rn(y3, mul, kRoundMagic));
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(__fmul_rn(y1, mul)), "f"(__fmul_rn(y0, mul)));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(__fmul_rn(y3, mul)), "f"(__fmul_rn(y2, mul)));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
}

// Scale of a block whose largest |x| has the fp32 bits `bits`.
template <int KIND>
__device__ __forceinline__ float block_scale(uint32_t bits) {
  if (bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);    // infinity or NaN inside
  if (bits == 0u) return 0.f;
  if constexpr (KIND == 0) {
    return fmaxf(__fdiv_rn(__uint_as_float(bits), 127.f), 0x1p-120f);
  } else {
    // amax = m 2^e, m in [0.5, 1): e = field - 126 (subnormals end at the clamp)
    int e = (int)(bits >> 23) - 126 - 9 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(-120, min(120, e));
    return __uint_as_float((uint32_t)(e + 127) << 23);
  }
}

// ---------------------------------------------------------------- append

template <typename T> struct Piece16;                       // 16 elements of a row
template <> struct Piece16<__nv_bfloat16> {
  uint4 u[2];
  __device__ __forceinline__ float at(int i) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
  // fp32 bits of the largest magnitude, two elements an instruction
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(u);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return max(m & 0xffff0000u, m << 16);
  }
};
template <> struct Piece16<float> {
  uint4 u[4];
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(reinterpret_cast<const uint32_t*>(u)[i]); }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(at(i)) & 0x7fffffffu);
    return m;
  }
};

// One CTA per (block touched, KV head, K or V, sequence), block * d / 32 threads,
// two 16-element pieces a thread: x is read once into registers, the maximum
// goes through warp reductions and shared memory, and the codes leave as
// 16-byte words.  Bound by HBM for prompts and by a chain of four dependent
// loads (start, table, x, old scale) for single tokens.
template <typename T, int KIND>
static __global__ void __launch_bounds__(512) kv_block_append_kernel(const KvAppendArgs a) {
  __shared__ uint32_t sm_max[16];
  const KvBlockView& c = a.c;
  const int tid = threadIdx.x, nt = blockDim.x;
  const unsigned g = blockIdx.x / (unsigned)c.Hkv, hk = blockIdx.x - g * (unsigned)c.Hkv;
  const int isv = g & 1, b = blockIdx.y + a.b0;
  const SeqRange s = seq_range(a.start, a.count, b, a.N, c.cap);
  const int blk = (s.start >> c.block_log2) + (int)(g >> 1);
  const int t0 = blk << c.block_log2;
  const int lo = max(s.start, t0), hi = min(s.start + s.n, t0 + (1 << c.block_log2));
  if (lo >= hi) return;
  const int phys = checked_block(c, b, blk);
  if (phys < 0) return;
  float* sp = (isv ? c.vs : c.ks) + (int64_t)phys * c.Hkv + hk;
  uint8_t* codes = isv ? c.v + phys * c.v_sb + hk * c.v_sh : c.k + phys * c.k_sb + hk * c.k_sh;
  const int64_t c_sn = isv ? c.v_sn : c.k_sn;
  const View4& xv = isv ? a.v : a.k;
  const T* x = static_cast<const T*>(xv.ptr) + b * xv.sb + hk * xv.sh;
  const bool has_old = t0 < s.start;
  const float s_old = has_old ? *sp : 0.f;

  const int ppr_log2 = a.d_log2 - 4;                       // 16-element pieces per row
  Piece16<T> p[2];
  int row[2], col[2];
  bool fresh[2];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int idx = i * nt + tid;
    row[i] = idx >> ppr_log2;
    col[i] = (idx & ((1 << ppr_log2) - 1)) * 16;
    const int tok = t0 + row[i];
    fresh[i] = tok >= lo && tok < hi;
    if (fresh[i]) {
      const uint4* src = reinterpret_cast<const uint4*>(x + (int64_t)(tok - s.start) * xv.sn + col[i]);
#pragma unroll
      for (int e = 0; e < (int)(sizeof(p[i].u) / 16); ++e) p[i].u[e] = __ldcs(src + e);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (fresh[i]) mx = max(mx, p[i].top());
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((tid & 31) == 0) sm_max[tid >> 5] = mx;
  __syncthreads();                                         // also: every thread has read the old scale
  for (int w = 0; w < nt / 32; ++w) mx = max(mx, sm_max[w]);
  const float s_new = block_scale<KIND>(mx);
  // scales are >= 0 or NaN: their bits order like the values, with NaN above all
  const uint32_t so = __float_as_uint(s_old) & 0x7fffffffu;
  const bool grown = __float_as_uint(s_new) > so;
  const float sc = grown ? s_new : s_old;
  const bool live = sc > 0.f && sc < INFINITY;
  const float inv = live ? __fdiv_rn(1.f, sc) : 0.f;
  if (tid == 0 && (grown || !has_old)) *sp = sc;
  const bool redo = has_old && grown && live;              // old tokens to the larger scale
  const float ratio = redo ? __fdiv_rn(s_old, sc) : 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4* dst = reinterpret_cast<uint4*>(codes + row[i] * c_sn + col[i]);
    if (fresh[i]) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = live ? codes4_of<KIND>(p[i].at(4 * e), p[i].at(4 * e + 1), p[i].at(4 * e + 2), p[i].at(4 * e + 3), inv)
                    : 0u;
      *dst = make_uint4(o[0], o[1], o[2], o[3]);
    } else if (redo && t0 + row[i] < s.start) {
      const uint4 w = *dst;
      uint32_t o[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f[4];
        codes4_to_f<KIND>(o[e], f);
        o[e] = codes4_of<KIND>(f[0], f[1], f[2], f[3], ratio);
      }
      *dst = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ------------------------------------------------------------------ read

constexpr int kKrThreads = 256;
constexpr int kKrPieces = 1;          // 16-code pieces of K and of V a thread takes (2, 4: no faster, longer for few tokens)

// 16 values of a row; wide: in 32-byte stores, which write whole sectors (a
// lane's neighbours are 32 or 64 bytes away).
template <typename T>
__device__ __forceinline__ void store16(T* dst, const float* f, bool wide);
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* dst, const float* f, bool wide) {
  uint32_t r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = f2_to_bf2(f[2 * e], f[2 * e + 1]);
  if (wide) {
    store_32b(dst, r);
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}
template <>
__device__ __forceinline__ void store16<float>(float* dst, const float* f, bool wide) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(f);
  if (wide) {
    store_32b(dst, r);
    store_32b(dst + 8, r + 8);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      reinterpret_cast<float4*>(dst)[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
  }
}

// x = code * scale (one fp32 product, rounded once to T) of tokens [0, len) of
// each sequence, zeros from len to the output's end.  A thread takes 16-code
// pieces in output order (d, head, token), so a CTA's 256 pieces are a few
// consecutive tokens of all heads: contiguous stores, and loads of whole rows
// of a block.  Bound by HBM.
template <typename T, int KIND>
static __global__ void __launch_bounds__(kKrThreads) kv_block_read_kernel(const KvReadArgs a) {
  const KvBlockView& c = a.c;
  const int b = blockIdx.y + a.b0;
  int64_t len = a.len[b];
  if (len < 0 || len > c.cap) {
    record_device_error(RCX_ERR_DEVICE_INDEX);
    len = 0;
  }
  const int ppr_log2 = a.d_log2 - 4;
  const uint32_t total = (uint32_t)a.n * (uint32_t)c.Hkv << ppr_log2;
  const uint32_t i0 = blockIdx.x * (kKrThreads * kKrPieces) + threadIdx.x;
  uint4 kw[kKrPieces], vw[kKrPieces];
  float ks[kKrPieces], vs[kKrPieces];
  int64_t ko[kKrPieces], vo[kKrPieces];
#pragma unroll
  for (int i = 0; i < kKrPieces; ++i) {
    const uint32_t idx = i0 + i * kKrThreads;
    kw[i] = vw[i] = make_uint4(0u, 0u, 0u, 0u);
    ks[i] = vs[i] = 0.f;
    if (idx < total) {
      const uint32_t rh = idx >> ppr_log2;
      const int col = (int)(idx & ((1u << ppr_log2) - 1)) * 16;
      const uint32_t t = rh / (uint32_t)c.Hkv, h = rh - t * (uint32_t)c.Hkv;
      ko[i] = b * a.k.sb + (int64_t)t * a.k.sn + h * a.k.sh + col;
      vo[i] = b * a.v.sb + (int64_t)t * a.v.sn + h * a.v.sh + col;
      if ((int64_t)t < len) {
        const int phys = checked_block(c, b, (int)(t >> c.block_log2));
        if (phys >= 0) {
          const int64_t r = t & ((1u << c.block_log2) - 1);
          kw[i] = __ldcs(reinterpret_cast<const uint4*>(c.k + phys * c.k_sb + r * c.k_sn + h * c.k_sh + col));
          vw[i] = __ldcs(reinterpret_cast<const uint4*>(c.v + phys * c.v_sb + r * c.v_sn + h * c.v_sh + col));
          ks[i] = c.ks[(int64_t)phys * c.Hkv + h];
          vs[i] = c.vs[(int64_t)phys * c.Hkv + h];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kKrPieces; ++i) {
    if (i0 + i * kKrThreads < total) {
      float f[16];
      const uint32_t k4[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w}, v4[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) codes4_to_f<KIND>(k4[e], f + 4 * e);
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] *= ks[i];
      store16<T>(static_cast<T*>(a.k.ptr) + ko[i], f, a.wide);
#pragma unroll
      for (int e = 0; e < 4; ++e) codes4_to_f<KIND>(v4[e], f + 4 * e);
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] *= vs[i];
      store16<T>(static_cast<T*>(a.v.ptr) + vo[i], f, a.wide);
    }
  }
}

}  // namespace rcx
