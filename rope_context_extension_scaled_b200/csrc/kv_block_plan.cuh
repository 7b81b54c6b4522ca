// Work split of the attention over a block-scaled KV cache: which key tiles of
// which item each CTA takes.  Lengths live on the device, so the split is made
// there, by the same arithmetic in every CTA.
//
// An item is (sequence, row tile, KV head); its rows are (token, query head of
// the group), row r = token r / G, head r % G.  Its key tiles are the window's
// tiles and the sink tiles before them.  All items' tiles, in the order
// sequence, row tile, head, form one line of T tiles; CTA i takes tiles
// [T i / P, T (i + 1) / P), so that ragged lengths, few rows and many rows all
// load the P CTAs evenly, and only items that a CTA border cuts need a merge.
// Heads are the fastest index: CTAs that run side by side on one sequence read
// the same head's keys.
//
// Beginning an item costs a CTA about start_tiles tiles (its queries, its first
// table entries and keys, its end), so two cases are dealt out otherwise:
//   even:    fewer items than CTAs: each item is cut into `even` equal pieces, one
//            a CTA, where these can be as small as min_tiles or, with items that
//            are alike, are within start_tiles of an even share;
//   direct:  items too short to be worth cutting (decided on the host, which
//            knows how long they can be): the line holds whole items, and there
//            is nothing to scan and nothing to merge.
#pragma once
#include "kv_block.cuh"

namespace rcx {

// One output row piece of 4 dims (16-byte aligned in fp32, 8-byte in bf16).
__device__ __forceinline__ void store_o4(const KvAttnArgs& a, int64_t off, float4 x) {
  if (a.o_bf16)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o.ptr) + off) = make_uint2(f2_to_bf2(x.x, x.y), f2_to_bf2(x.z, x.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(a.o.ptr) + off) = x;
}

// Key tiles (2^LOGT keys each) that rows of tokens n_lo .. n_hi may see.
struct KeySpan {
  int sink_tiles, first, n;         // tile u: u < sink_tiles ? u : first + u - sink_tiles
  int hi;                           // keys end here
  __device__ __forceinline__ int tile(int u) const { return u < sink_tiles ? u : first + u - sink_tiles; }
};

template <int LOGT>
__device__ __forceinline__ KeySpan key_span(int start, int n_lo, int n_hi, int window, int n_sink) {
  constexpr int T = 1 << LOGT;
  KeySpan s;
  s.hi = start + n_hi + 1;
  const int lo = window > 0 ? max(0, start + n_lo + 1 - window) : 0;
  s.first = lo >> LOGT;
  const int sinks = window > 0 ? min(n_sink, lo) : 0;
  s.sink_tiles = min((sinks + T - 1) >> LOGT, s.first);
  s.n = s.sink_tiles + ((s.hi + T - 1) >> LOGT) - s.first;
  return s;
}

// Entry e = (sequence, row tile).
struct Entry {
  int b, r0, rows;                  // first row of the tile, rows in it (0: nothing to do)
  int start, n_lo, n_hi;            // cached tokens before the call, tokens of the rows
  KeySpan span;
};

template <int LOGT>
__device__ __forceinline__ Entry entry_of(const KvAttnArgs& a, int e) {
  Entry t;
  const int bl = (int)fast_div(e, a.div_nrt), rt = e - bl * a.n_rt;
  t.b = a.b0 + bl;
  const SeqRange s = seq_range(a.start, a.count, t.b, a.N, a.c.cap);
  t.start = s.start;
  t.r0 = rt * a.rows_item;
  t.rows = min(s.n * a.G - t.r0, a.rows_item);
  if (t.rows <= 0) {
    t.rows = 0;
    t.n_lo = t.n_hi = 0;
    t.span.sink_tiles = t.span.first = t.span.n = t.span.hi = 0;
    return t;
  }
  t.n_lo = (int)fast_div(t.r0, a.div_g);
  t.n_hi = (int)fast_div(t.r0 + t.rows - 1, a.div_g);
  t.span = key_span<LOGT>(s.start, t.n_lo, t.n_hi, a.window, a.n_sink);
  return t;
}

// CTAs that T tiles go to: as many as there are, each with min_tiles at least.
__device__ __forceinline__ int range_ctas(int T, const KvAttnArgs& a) { return max(1, min(a.n_cta, T / a.min_tiles)); }
// First tile of CTA i.
__device__ __forceinline__ int range_start(int T, int i, int P) { return (int)((int64_t)T * i / P); }
// The CTA whose range holds tile x (the last i with range_start(i) <= x).
__device__ __forceinline__ int range_owner(int T, int x, int P) { return (int)((((int64_t)x + 1) * P - 1) / T); }

// Pieces of each item (0: the line is cut), from the T tiles of `items` items of
// at most `most` tiles each: as small as min_tiles allows where there are CTAs
// for that.
__device__ __forceinline__ int even_pieces(const KvAttnArgs& a, int T, int items, int most) {
  const int ctas = a.n_cta / items, s = max(1, most / a.min_tiles);
  if (ctas >= s) return s;
  return ctas >= 1 && (most + ctas - 1) / ctas <= T / a.n_cta + a.start_tiles ? ctas : 0;
}

// Where a CTA begins: entry e, tile `off` of its Hkv * span.n tiles, and the
// CTA's range [x0, x1) (direct: of items).  even: entry e, head off, piece x0 of x1.
struct PlanStart {
  int e, off, x0, x1, even;
};

// Run by one whole warp; CTA 0 also writes the prefix table for the merge.
template <int LOGT>
__device__ __forceinline__ PlanStart plan_start(const KvAttnArgs& a, int cta, int lane) {
  const int E = a.B * a.n_rt, Hkv = a.c.Hkv;
  PlanStart p;
  p.even = 0;
  if (a.direct) {
    p.e = p.off = 0;
    const bool one = E * Hkv == a.n_cta;        // an item each: no 64-bit divisions on the way
    p.x0 = one ? cta : range_start(E * Hkv, cta, a.n_cta);
    p.x1 = one ? cta + 1 : range_start(E * Hkv, cta + 1, a.n_cta);
    return p;
  }
  int carry = 0, incl = 0, mine = 0, most = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    mine = e < E ? entry_of<LOGT>(a, e).span.n : 0;
    most = max(most, __reduce_max_sync(0xffffffffu, mine));
    mine *= Hkv;
    incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += y;
    }
    if (cta == 0 && e < E) a.prefix[e] = carry + incl - mine;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  const int T = carry;
  const int s = even_pieces(a, T, E * Hkv, most);
  if (cta == 0 && lane == 0) {
    a.prefix[E] = T;
    a.prefix[E + 1] = s;
  }
  if (s > 0) {
    const int item = cta / s;
    p.even = 1;
    p.e = (int)fast_div(item, a.div_hkv);
    p.off = item - p.e * Hkv;
    p.x0 = cta - item * s;
    p.x1 = s;
    return p;
  }
  const int P = range_ctas(T, a);
  p.x0 = range_start(T, min(cta, P), P);
  p.x1 = range_start(T, min(cta + 1, P), P);
  p.e = 0;
  p.off = 0;
  if (p.x0 >= p.x1) return p;
  carry = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    if (E > 32) {
      const int e = e0 + lane;
      mine = e < E ? entry_of<LOGT>(a, e).span.n * Hkv : 0;
      incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
    }
    const uint32_t past = __ballot_sync(0xffffffffu, carry + incl > p.x0);
    if (past) {
      const int l = __ffs(past) - 1;
      p.e = e0 + l;
      p.off = p.x0 - (carry + __shfl_sync(0xffffffffu, incl - mine, l));
      break;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  return p;
}

// Walk over the CTA's segments: parts [u0, u1) of one item's tiles.
struct SegWalk {
  int e, off, x, x0, x1, even;
  Entry t;
  int hk, u0, u1;
  bool fresh;                       // t is entry e
  __device__ __forceinline__ void init(const PlanStart& p) {
    e = p.e;
    off = p.off;
    x = x0 = p.x0;
    x1 = p.x1;
    even = p.even;
    fresh = false;
  }
  template <int LOGT>
  __device__ __forceinline__ bool next(const KvAttnArgs& a) {
    if (a.direct) {
      while (x < x1) {
        const int i = x++;
        e = (int)fast_div(i, a.div_hkv);
        hk = i - e * a.c.Hkv;
        t = entry_of<LOGT>(a, e);
        u0 = 0;
        u1 = t.span.n;
        if (u1 > 0) return true;
      }
      return false;
    }
    const int E = a.B * a.n_rt;
    if (even) {
      if (x >= x1 || e >= E) return false;
      t = entry_of<LOGT>(a, e);
      hk = off;
      u0 = range_start(t.span.n, x, x1);
      u1 = range_start(t.span.n, x + 1, x1);
      x = x1;                       // one piece
      return u1 > u0;
    }
    while (x < x1 && e < E) {
      if (!fresh) {
        t = entry_of<LOGT>(a, e);
        fresh = true;
      }
      if (off >= t.span.n * a.c.Hkv) {
        off -= t.span.n * a.c.Hkv;
        ++e;
        fresh = false;
        continue;
      }
      hk = off / t.span.n;
      u0 = off - hk * t.span.n;
      u1 = min(t.span.n, u0 + (x1 - x));
      off += u1 - u0;
      x += u1 - u0;
      return true;
    }
    return false;
  }
  // the segment's place among the CTA's partials: 0 if it opens the range, else 1
  __device__ __forceinline__ int slot() const { return even || x - (u1 - u0) == x0 ? 0 : 1; }
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == t.span.n; }
};

// O = 0 and LSE = -inf for the rows of tokens past a sequence's count (direct
// launches; the merge writes them otherwise).  A warp per token.
template <int D>
__device__ __forceinline__ void empty_rows(const KvAttnArgs& a, int warp, int n_warps, int lane) {
  for (unsigned i = blockIdx.x * n_warps + warp; i < (unsigned)(a.B * a.N); i += gridDim.x * n_warps) {
    const int bl = (int)fast_div(i, a.div_n);
    const int64_t b = a.b0 + bl, n = i - bl * a.N;
    if (n < seq_range(a.start, a.count, (int)b, a.N, a.c.cap).n) continue;
    const int H = (int)a.q.H;
    for (int x = lane; x < H * (D / 4); x += 32) {
      const int h = x / (D / 4), dd = 4 * (x % (D / 4));
      store_o4(a, b * a.o.sb + n * a.o.sn + h * a.o.sh + dd, make_float4(0.f, 0.f, 0.f, 0.f));
      if (dd == 0 && a.lse) a.lse[b * a.lse_sb + h * a.lse_sh + n] = -INFINITY;
    }
  }
}

}  // namespace rcx
