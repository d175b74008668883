// Modified attention scores: which keys a row sees, the soft cap and the
// distance bias, shared by the decode and key-weight kernels.
//
// In the decode kernels a modifier costs arithmetic on scores already in
// registers and no traffic, so HBM stays the bound where it was (32 sequences
// of 2048 to 32768 keys, 8 heads, 32 rows: 185 us in a graph with a distance
// bias, 187 without, 6.3 TB/s).  Short spans are bound by what a CTA costs besides its
// tiles: 64 sequences, 8 heads, a window of 1024 keys under a cap are 512 CTAs
// of 9 tiles, two of them an SM, in two waves of 17 us, about 5 of each the
// start and the end (34 us for 132 MB; three CTAs an SM with two stages 39,
// every CTA's tiles cut in two or three 44 to 46).
#pragma once

#include <vector_types.h>
#include <vector_functions.h>

#include <cstdint>

#include "mj_device.cuh"

namespace mj {

// Keys a query token sees: j < pfx or lo <= j <= hi.
struct RowRange {
  int lo, hi, pfx;
};

// Query token qi of sequence b (L keys in the cache).  Host and device: the
// host form of the spans follows the same rule.
__host__ __device__ __forceinline__ RowRange row_range(const ScoreModDev& m, int causal, int q_len, int b, int L,
                                                       int qi) {
  const int pos = L - q_len + qi;
  RowRange r;
  r.hi = causal && pos < L - 1 ? pos : L - 1;
  r.lo = 0;
  if (m.window > 0) {
    const int w = pos - m.window + 1;  // window <= 2^30: no overflow
    r.lo = w > 0 ? w : 0;
  }
  if (m.key_begin) {
    const int k = m.key_begin[static_cast<int64_t>(b) * q_len + qi];
    r.lo = k > r.lo ? k : r.lo;
  }
  if (m.key_end) {
    const int k = m.key_end[static_cast<int64_t>(b) * q_len + qi];
    const int last = (k > 0 ? k : 0) - 1;
    r.hi = last < r.hi ? last : r.hi;
  }
  r.pfx = 0;
  if (m.prefix) {
    const int p = m.prefix[b];
    r.pfx = p < 0 ? 0 : (p > L ? L : p);
  }
  return r;
}

// The span of a sequence whose rows see keys [first, last] between them
// (last < first: none) and [0, pfx), and the length to plan with: its tiles
// are the prefix's, then those from first / 128 to the end.
__host__ __device__ __forceinline__ int4 make_span(int first, int last, int pfx, int32_t* plan_len) {
  int begin = pfx, end = pfx;
  if (first <= last) {
    begin = first > pfx ? first : pfx;
    end = last + 1 > pfx ? last + 1 : pfx;
    begin = begin < end ? begin : end;
  }
  const int jump = begin / 128 - (pfx + 127) / 128;  // tiles between them
  *plan_len = jump > 0 ? end - 128 * jump : end;
  return make_int4(pfx, begin, end, 0);
}

// tanh(t) to about fp32 precision.  Below 0.6 an odd polynomial (degree 11,
// relative error 1e-7 after rounding; coefficients fitted for this file by
// minimax over [0, 0.6]); above, (1 - e) / (1 + e) with e = exp(-2|t|) <= 0.31,
// whose subtraction no longer cancels.  (tanh.approx is good to 2^-11 only: a
// cap of 50 would make that 0.02 in a logit.)
__device__ __forceinline__ float tanh_small(float t) {
  const float u = t * t;
  float p = -5.852168662e-03f;
  p = fmaf(p, u, 2.075362916e-02f);
  p = fmaf(p, u, -5.376870490e-02f);
  p = fmaf(p, u, 1.333168896e-01f);
  p = fmaf(p, u, -3.333328326e-01f);
  p = fmaf(p, u, 9.999999975e-01f);
  return t * p;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// scale tanh(t) / t of two values of u = t^2: the same polynomial with its
// coefficients times `scale` (one rounding each; a multiplication a pair less
// than scaling the result)
struct TanhRatio {
  float c[6];
  __device__ __forceinline__ explicit TanhRatio(float scale)
      : c{-5.852168662e-03f * scale, 2.075362916e-02f * scale, -5.376870490e-02f * scale,
          1.333168896e-01f * scale,  -3.333328326e-01f * scale, 9.999999975e-01f * scale} {}
  __device__ __forceinline__ float2 operator()(float2 u) const {
    float2 p = make_float2(c[0], c[0]);
#pragma unroll
    for (int i = 1; i < 6; ++i) p = fma2(p, u, make_float2(c[i], c[i]));
    return p;
  }
};
constexpr float kTanhSmall = 0.6f;
__device__ __forceinline__ float tanh_any(float t) {
  const float at = fabsf(t);
  const float e = fast_exp2(at * (-2.f * kLog2e));
  const float big = copysignf((1.f - e) * rcp_approx(1.f + e), t);
  return at < kTanhSmall ? tanh_small(t) : big;
}

// Scores s[0..N) (N even) over the cap, t = s c1, -> cap2 tanh(t) + b, where
// b(e) gives the addend of score e.  Scores small against the cap (most, in
// practice) take the polynomial, two a time; a warp with others takes the
// exponential form for all of them.
template <int N, typename Bias>
__device__ __forceinline__ void cap_scores(float* s, float c1, float cap2, Bias b) {
  const float2 c12 = make_float2(c1, c1);
  float2 sq[N / 2];
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    const float2 t = mul2(make_float2(s[2 * e], s[2 * e + 1]), c12);
    sq[e] = mul2(t, t);
    top = fmax3(top, sq[e].x, sq[e].y);
    s[2 * e] = t.x;
    s[2 * e + 1] = t.y;
  }
  if (__all_sync(0xffffffffu, top < kTanhSmall * kTanhSmall)) {
    const TanhRatio ratio(cap2);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float2 o = fma2(make_float2(s[2 * e], s[2 * e + 1]), ratio(sq[e]), make_float2(b(2 * e), b(2 * e + 1)));
      s[2 * e] = o.x;
      s[2 * e + 1] = o.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = fmaf(tanh_any(s[e]), cap2, b(e));
  }
}

// Raw scores r[0..N) (fp32 bits) of one row at keys j0 .. j0 + N - 1 -> logits
// in log2 units, in place.
//   c1: raw score -> t = z / softcap, or (no cap) -> log2 units
//   cap2: softcap in log2 units (0: no cap)
//   slope2, pos_minus_j0: the row's bias in log2 units per position (0: none)
template <int N>
__device__ __forceinline__ void modify_scores(uint32_t* r, float c1, float cap2, bool bias, float slope2,
                                              float pos_minus_j0) {
  float s[N];
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = __uint_as_float(r[e]);
  if (!bias) {
    if (cap2 > 0.f) {
      cap_scores<N>(s, c1, cap2, [](int) { return 0.f; });
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] *= c1;
    }
  } else if (__all_sync(0xffffffffu, pos_minus_j0 >= static_cast<float>(N - 1))) {
    // no key past its row (a warp's usual case): -slope (pos - j0 - e) is
    // linear in e, one fma a score
    const float base = -slope2 * pos_minus_j0;
    auto linear = [&](int e) { return fmaf(slope2, static_cast<float>(e), base); };
    if (cap2 > 0.f) {
      cap_scores<N>(s, c1, cap2, linear);
    } else {  // four running pairs of addends
      const float2 c12 = make_float2(c1, c1), step = make_float2(8.f * slope2, 8.f * slope2);
      float2 b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = make_float2(linear(2 * i), linear(2 * i + 1));
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float2 o = fma2(make_float2(s[2 * e], s[2 * e + 1]), c12, b[e & 3]);
        b[e & 3] = add2(b[e & 3], step);
        s[2 * e] = o.x;
        s[2 * e + 1] = o.y;
      }
    }
  } else {
    if (cap2 > 0.f) {
      cap_scores<N>(s, c1, cap2, [](int) { return 0.f; });
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] *= c1;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = fmaf(-slope2, fabsf(pos_minus_j0 - static_cast<float>(e)), s[e]);
  }
#pragma unroll
  for (int e = 0; e < N; ++e) r[e] = __float_as_uint(s[e]);
}

// The same for one key and N rows: s[c] is row c's score of the key at
// position `key`, the rows' slopes (log2 units) and positions in shared memory.
// Key and rows count from one position near the rows (whole positions past
// 2^24 share fp32 values: the bias would be of a neighbouring distance).
template <int N>
__device__ __forceinline__ void modify_columns(float* s, float c1, float cap2, bool bias, const float* slope2,
                                               const float* pos, float key) {
  if (cap2 > 0.f) {
    cap_scores<N>(s, c1, cap2, [](int) { return 0.f; });
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] *= c1;
  }
  if (bias) {
#pragma unroll
    for (int c = 0; c < N; ++c) s[c] = fmaf(-slope2[c], fabsf(pos[c] - key), s[c]);
  }
}

}  // namespace mj
