// qk_row.hpp -- one query, key or value head of one token in a group of
// lanes: which lane holds which values, the RMS norm and the position
// rotation.  Shared by the norm-and-rotation kernels (qk_rope.hip) and the
// cache's write and read (kv_cache.hip).
#pragma once

#include <type_traits>

#include "kv.hpp"

namespace nvfp4 {

constexpr int kRowThreads = 256;

// Lanes of a head: D / 8 rounded up to a power of two; each holds two groups
// of four consecutive values, at e0 and e1.  Both members of every rotated
// pair are in one lane (halves: value i of group 0 pairs with value i of
// group 1; neighbours: inside a group), so the rotation moves nothing between
// lanes, and four consecutive lanes hold a 16-value block in each group, as
// rot and D are multiples of 32.
template <int LPH>
struct RowMap {
  int e0, e1;   // first value of each group
  int j0, j1;   // pair of the first angle of each group (rotated lanes)
  bool active;  // the lane holds values (D / 8 need not be a power of two)
  bool rotated;
  __device__ __forceinline__ RowMap(int D, int rot, int pairs) {
    const int u = (int)(threadIdx.x & (LPH - 1));
    active = u < D / 8;
    rotated = u < rot / 8;
    if (rotated) {
      e0 = 4 * u;
      e1 = rot / 2 + 4 * u;
      j0 = pairs == NVFP4_PAIRS_HALVES ? 4 * u : 2 * u;
      j1 = pairs == NVFP4_PAIRS_HALVES ? 4 * u : rot / 4 + 2 * u;
    } else {
      const int v = u - rot / 8;
      e0 = rot + 4 * v;
      e1 = rot + (D - rot) / 2 + 4 * v;
      j0 = j1 = 0;
    }
  }
};

template <int LPH>
__device__ __forceinline__ void row_load(const uint16_t* p, const RowMap<LPH>& m, float (&x)[8]) {
  uint2 a = make_uint2(0, 0), b = make_uint2(0, 0);
  if (m.active) {
    a = *reinterpret_cast<const uint2*>(p + m.e0);
    b = *reinterpret_cast<const uint2*>(p + m.e1);
  }
  x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
  x[4] = bf16_lo(b.x); x[5] = bf16_hi(b.x); x[6] = bf16_lo(b.y); x[7] = bf16_hi(b.y);
}

template <int LPH>
__device__ __forceinline__ void row_store(uint16_t* p, const RowMap<LPH>& m, const uint2& a,
                                          const uint2& b) {
  if (m.active) {
    *reinterpret_cast<uint2*>(p + m.e0) = a;
    *reinterpret_cast<uint2*>(p + m.e1) = b;
  }
}

// cos and sin of the lane's four pairs: pairs i of (group 0, group 1) for
// halves; pairs 0, 1 of group 0 and 2, 3 of group 1 for neighbours.  A
// position outside the table gives NaN.
struct RowAngles {
  float c[4], s[4];
};
template <int LPH>
__device__ __forceinline__ RowAngles row_angles(const nvfp4_qk_args& a, const RowMap<LPH>& m,
                                                int64_t token) {
  RowAngles r;
  if (!m.rotated || !m.active) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { r.c[i] = 1.0f; r.s[i] = 0.0f; }
    return r;
  }
  const int64_t pos = a.positions[token];
  if (pos < 0 || pos >= a.max_pos) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.c[i] = r.s[i] = __builtin_nanf("");
    return r;
  }
  const int64_t base = pos * (a.rot_dim / 2);
  // halves: j1 == j0, so j0 + 2 .. j0 + 3 follow; neighbours: j1, j1 + 1
  const int64_t second = a.pairs == NVFP4_PAIRS_HALVES ? m.j0 + 2 : m.j1;
  const float2 c0 = *reinterpret_cast<const float2*>(a.cos + base + m.j0);
  const float2 c1 = *reinterpret_cast<const float2*>(a.cos + base + second);
  const float2 s0 = *reinterpret_cast<const float2*>(a.sin + base + m.j0);
  const float2 s1 = *reinterpret_cast<const float2*>(a.sin + base + second);
  r.c[0] = c0.x; r.c[1] = c0.y; r.c[2] = c1.x; r.c[3] = c1.y;
  r.s[0] = s0.x; r.s[1] = s0.y; r.s[2] = s1.x; r.s[3] = s1.y;
  return r;
}

// The pair i of a lane: values (pair_a(i), pair_b(i)).
__device__ __forceinline__ constexpr int pair_a(int pairs, int i) {
  return pairs == NVFP4_PAIRS_HALVES ? i : 2 * i;
}
__device__ __forceinline__ constexpr int pair_b(int pairs, int i) {
  return pairs == NVFP4_PAIRS_HALVES ? i + 4 : 2 * i + 1;
}

// Rotation of the lane's pairs by the angles, or back by them (DIR = -1).
template <int PAIRS, int DIR, typename R>
__device__ __forceinline__ void row_rotate(R (&y)[8], const RowAngles& g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const R a = y[pair_a(PAIRS, i)], b = y[pair_b(PAIRS, i)];
    const R c = (R)g.c[i], s = DIR > 0 ? (R)g.s[i] : -(R)g.s[i];
    y[pair_a(PAIRS, i)] = a * c - b * s;
    y[pair_b(PAIRS, i)] = b * c + a * s;
  }
}

// Sum over the lanes of a head, in every lane, in a fixed order.
template <int LPH, typename R>
__device__ __forceinline__ R row_sum(R v) {
  auto step = [&](R x, auto d) {
    constexpr int D = decltype(d)::value;
    if constexpr (sizeof(R) == 8) {
      const uint64_t u = __builtin_bit_cast(uint64_t, x);
      const uint32_t lo = xor_lane_u32<D>((uint32_t)u), hi = xor_lane_u32<D>((uint32_t)(u >> 32));
      return x + __builtin_bit_cast(R, ((uint64_t)hi << 32) | lo);
    } else {
      return x + __builtin_bit_cast(R, xor_lane_u32<D>(__builtin_bit_cast(uint32_t, x)));
    }
  };
  v = step(v, std::integral_constant<int, 1>{});
  v = step(v, std::integral_constant<int, 2>{});
  if constexpr (LPH >= 8) v = step(v, std::integral_constant<int, 4>{});
  if constexpr (LPH >= 16) v = step(v, std::integral_constant<int, 8>{});
  if constexpr (LPH >= 32) v = v + __shfl_xor(v, 16);
  return v;
}

// (a)^-1/2 in binary64: the hardware's approximation and two Newton steps
// (each squares the relative error, which is below 2^-14 at the start).  An
// infinite a gives 0.
__device__ __forceinline__ double rsqrt64(double a) {
  double y = __builtin_amdgcn_rsq(a);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double h = 0.5 * a * y;
    y = __builtin_fma(y, __builtin_fma(-h, y, 0.5), y);
  }
  return __builtin_isinf(a) ? 0.0 : y;
}

// Norm (w not null) and rotation of the lane's values: bf16 patterns of
// group 0 and group 1.  binary64 throughout: the result is the formula's
// rounded once (up to 2^-50 before the rounding), whatever the sum's order,
// so that a key lands on the formula's side of the 4-bit borders behind it.
template <int LPH, int PAIRS>
__device__ __forceinline__ void row_norm_rope(const float (&x)[8], const RowMap<LPH>& m,
                                              const uint16_t* w, double eps, double inv_d,
                                              const RowAngles& g, uint2& o0, uint2& o1) {
  double y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = (double)x[i];
  if (w) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fma(y[i], y[i], ss);
    const double r = rsqrt64(row_sum<LPH>(ss) * inv_d + eps);
    float wf[8];
    row_load(w, m, wf);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * r * (double)wf[i];
  }
  if (m.rotated) row_rotate<PAIRS, 1>(y, g);
  o0 = make_uint2(bf16_pair((float)y[0], (float)y[1]), bf16_pair((float)y[2], (float)y[3]));
  o1 = make_uint2(bf16_pair((float)y[4], (float)y[5]), bf16_pair((float)y[6], (float)y[7]));
}

// The wavefront's task: a token and the first of 64 / LPH consecutive heads.
struct RowTask {
  int64_t token;
  int head;
};
template <int LPH>
__device__ __forceinline__ RowTask row_task(int64_t wave, int per_token) {
  RowTask t;
  uint32_t part;
  if ((uint64_t)wave >> 32) {
    t.token = wave / per_token;
    part = (uint32_t)(wave - t.token * per_token);
  } else {
    t.token = (uint32_t)wave / (uint32_t)per_token;
    part = (uint32_t)wave - (uint32_t)t.token * (uint32_t)per_token;
  }
  t.head = (int)part * (64 / LPH) + (int)((threadIdx.x & 63) / LPH);
  return t;
}

inline int lanes_per_head(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Workgroups for `tasks` wavefront tasks, four a workgroup; the kernels loop
// where there are more than the grid holds.
inline unsigned row_grid(int64_t tasks) {
  const int64_t g = (tasks + 3) / 4, cap = (int64_t)1 << 30;
  return (unsigned)(g < cap ? g : cap);
}

}  // namespace nvfp4
