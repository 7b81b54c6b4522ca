// rope_axes_apply: rotate Q and K by positions on several axes -- memory-bound
// elementwise kernel.
//
// Pair i of a head turns by phi_i = pos[axis_i][b][n] * theta_i: one position
// per axis (time, height, width, ...) and token, and a map from pairs to axes.
// With one axis this is R(m) of the "Context Extension" concept page,
// Technical principles.  The pair is (i, i + d/2) (halves) or (2i, 2i + 1).
// R is orthogonal, so the gradient of the rotation is the rotation by -phi
// (inverse): dx = R(phi)^T dy.
//
// Bound by HBM: one read and one write of every element.  A thread owns a unit
// of kPairs = 16 bytes' worth of pairs (two 16-byte vectors: the two halves of
// the pairs, or adjacent vectors) of one token, computes their angles once
// (float64 product and reduction, see rope_cos_sin) and applies them to its
// share of the heads, kRaGroup heads' loads in flight at a time.  With many
// tokens a thread takes all heads, so that an angle is paid once per
// Hq + Hkv vectors; with fewer the heads are dealt over gridDim.y until the GPU
// has several waves of CTAs (16,384 tokens x 40 heads in fp32: 75 us as one wave
// and a seventh, 4.5 TB/s), and with few (decoding) because the call is bound by
// the latency of a thread's loop over the heads, where repeated angles are free.
#pragma once
#include "rope_apply.cuh"

namespace rcx {

struct RopeAxesArgs {
  View4 q_in, q_out, k_in, k_out;   // ptr == nullptr: operand skipped
  const int64_t* positions;         // [axes, B, N], strides pos_sa, pos_sb, 1
  int64_t pos_sa, pos_sb;
  int64_t n_tok;                    // B * N
  int64_t N;
  int units;                        // units per head: d / 2 / pairs per unit
  int heads_per_y;                  // heads each blockIdx.y takes
  int halves, inverse;
  int wide;                         // adjacent pairs in 32-byte aligned rows: both vectors at once
  Freqs f;
  uint8_t axis[kMaxPairs];
};

constexpr int kRaThreads = 128;
constexpr int kRaGroup = 4;         // heads in flight: two 16-byte vectors each
constexpr int kRaCtasPerSm = 16;    // CTAs an SM gets at least, where heads can be dealt out for it

template <typename T>
__device__ __forceinline__ void rope_unit(uint4& u, uint4& w, const float2* cs, bool halves);

// 8 pairs: halves -> (u[p], w[p]); adjacent -> u holds pairs 0..3, w pairs 4..7
template <>
__device__ __forceinline__ void rope_unit<__nv_bfloat16>(uint4& u, uint4& w, const float2* cs, bool halves) {
  uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 x = bf2_to_f2(a[p]), y = bf2_to_f2(b[p]);
    if (halves) {
      const float2 c0 = cs[2 * p], c1 = cs[2 * p + 1];
      a[p] = f2_to_bf2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
      b[p] = f2_to_bf2(x.x * c0.y + y.x * c0.x, x.y * c1.y + y.y * c1.x);
    } else {
      const float2 c0 = cs[p], c1 = cs[4 + p];
      a[p] = f2_to_bf2(x.x * c0.x - x.y * c0.y, x.x * c0.y + x.y * c0.x);
      b[p] = f2_to_bf2(y.x * c1.x - y.y * c1.y, y.x * c1.y + y.y * c1.x);
    }
  }
  u = make_uint4(a[0], a[1], a[2], a[3]);
  w = make_uint4(b[0], b[1], b[2], b[3]);
}

// 4 pairs: halves -> (u[p], w[p]); adjacent -> u holds pairs 0, 1, w pairs 2, 3
template <>
__device__ __forceinline__ void rope_unit<float>(uint4& u, uint4& w, const float2* cs, bool halves) {
  float a[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
  float b[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
  if (halves) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float x = a[p], y = b[p];
      a[p] = x * cs[p].x - y * cs[p].y;
      b[p] = x * cs[p].y + y * cs[p].x;
    }
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float* v = p < 2 ? a + 2 * p : b + 2 * (p - 2);
      const float x = v[0], y = v[1];
      v[0] = x * cs[p].x - y * cs[p].y;
      v[1] = x * cs[p].y + y * cs[p].x;
    }
  }
  u = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3]));
  w = make_uint4(__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]), __float_as_uint(b[3]));
}

template <typename T>
__global__ void __launch_bounds__(kRaThreads) rope_axes_kernel(const RopeAxesArgs a) {
  constexpr int kPairs = 16 / sizeof(T);        // pairs per unit = elements per vector
  const int units = a.units;
  const int tpb = blockDim.x / units;           // tokens per CTA pass
  const int j = threadIdx.x % units;            // this thread's unit of a head, fixed
  const int e0 = a.halves ? j * kPairs : 2 * j * kPairs;             // first vector
  const int e1 = a.halves ? (units + j) * kPairs : e0 + kPairs;      // second vector
  const int hq = a.q_in.ptr ? (int)a.q_in.H : 0;
  const int H = hq + (a.k_in.ptr ? (int)a.k_in.H : 0);
  const int h_lo = blockIdx.y * a.heads_per_y, h_hi = min(H, h_lo + a.heads_per_y);
  const T* qi = static_cast<const T*>(a.q_in.ptr);
  const T* ki = static_cast<const T*>(a.k_in.ptr);
  T* qo = static_cast<T*>(a.q_out.ptr);
  T* ko = static_cast<T*>(a.k_out.ptr);
  const int64_t n = (int64_t)blockIdx.x * tpb + threadIdx.x / units;
  if (n < a.n_tok) {
    const int64_t b = a.N == a.n_tok ? 0 : n / a.N;
    const int64_t nn = n - b * a.N;
    const int64_t qin0 = b * a.q_in.sb + nn * a.q_in.sn, qout0 = b * a.q_out.sb + nn * a.q_out.sn;
    const int64_t kin0 = b * a.k_in.sb + nn * a.k_in.sn, kout0 = b * a.k_out.sb + nn * a.k_out.sn;
    const int64_t* pos = a.positions + b * a.pos_sb + nn;
    float2 cs[kPairs];
    for (int h0 = h_lo; h0 < h_hi; h0 += kRaGroup) {
      uint4 u[kRaGroup], w[kRaGroup];
#pragma unroll
      for (int g = 0; g < kRaGroup; ++g) {
        const int h = h0 + g;
        if (h < h_hi) {
          const T* src = h < hq ? qi + qin0 + h * a.q_in.sh : ki + kin0 + (h - hq) * a.k_in.sh;
          if (a.wide) {
            uint32_t r[8];
            load_32b(r, src + e0);
            u[g] = make_uint4(r[0], r[1], r[2], r[3]);
            w[g] = make_uint4(r[4], r[5], r[6], r[7]);
          } else {
            u[g] = __ldcs(reinterpret_cast<const uint4*>(src + e0));
            w[g] = __ldcs(reinterpret_cast<const uint4*>(src + e1));
          }
        }
      }
      if (h0 == h_lo) {                         // angles while the first loads are in flight
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
          const int i = j * kPairs + p;
          rope_cos_sin(pos[a.axis[i] * a.pos_sa], a.f.theta[i], cs[p].x, cs[p].y);
          if (a.inverse) cs[p].y = -cs[p].y;
        }
      }
#pragma unroll
      for (int g = 0; g < kRaGroup; ++g) {
        const int h = h0 + g;
        if (h < h_hi) {
          rope_unit<T>(u[g], w[g], cs, a.halves);
          T* dst = h < hq ? qo + qout0 + h * a.q_out.sh : ko + kout0 + (h - hq) * a.k_out.sh;
          if (a.wide) {
            const uint32_t r[8] = {u[g].x, u[g].y, u[g].z, u[g].w, w[g].x, w[g].y, w[g].z, w[g].w};
            store_32b(dst + e0, r);
          } else {
            *reinterpret_cast<uint4*>(dst + e0) = u[g];
            *reinterpret_cast<uint4*>(dst + e1) = w[g];
          }
        }
      }
    }
  }
}

}  // namespace rcx
