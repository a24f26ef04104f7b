// qk_row.hpp -- one query, key or value head of one token in a group of
// lanes: which lane holds which values, the RMS norm and the position
// rotation.  Shared by the norm-and-rotation kernels (qk_rope.hip) and the
// cache's write and read (kv_cache.hip).
#pragma once

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
    const int u = (int)(threadIdx.x & (LPH - 1)), v = u - rot / 8;
    const bool halves = pairs == NVFP4_PAIRS_HALVES;
    active = u < D / 8;
    rotated = u < rot / 8;
    // a lane without values reads value 0 and uses none of it
    e0 = !active ? 0 : rotated ? 4 * u : rot + 4 * v;
    e1 = !active ? 0 : rotated ? rot / 2 + 4 * u : rot + (D - rot) / 2 + 4 * v;
    j0 = !rotated ? 0 : halves ? 4 * u : 2 * u;
    j1 = !rotated ? 0 : halves ? 4 * u : rot / 4 + 2 * u;
  }
};

// The lane's eight values as bf16 patterns: group 0 and group 1.
struct Row8 {
  uint2 a, b;
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
    x[4] = bf16_lo(b.x); x[5] = bf16_hi(b.x); x[6] = bf16_lo(b.y); x[7] = bf16_hi(b.y);
  }
  __device__ __forceinline__ Row8 or_zero(bool keep) const {
    return Row8{make_uint2(keep ? a.x : 0u, keep ? a.y : 0u), make_uint2(keep ? b.x : 0u, keep ? b.y : 0u)};
  }
};

// Without a branch: a load that some lanes skip makes the wait for an older
// one wait for this one too.
template <int LPH>
__device__ __forceinline__ Row8 row_load(const uint16_t* p, const RowMap<LPH>& m) {
  return Row8{*reinterpret_cast<const uint2*>(p + m.e0), *reinterpret_cast<const uint2*>(p + m.e1)};
}

template <int LPH>
__device__ __forceinline__ void row_store(uint16_t* p, const RowMap<LPH>& m, const Row8& r) {
  *reinterpret_cast<uint2*>(p + m.e0) = r.a;
  *reinterpret_cast<uint2*>(p + m.e1) = r.b;
}

// Walks the head groups [g0, g1) of one token's heads at x: f(head, values)
// for each, with the next group's values in flight.  Heads past the last one
// repeat it; f is told by its head number.
template <int LPH, class F>
__device__ __forceinline__ void row_walk(const uint16_t* x, int heads, int D, int g0, int g1,
                                         const RowMap<LPH>& m, const F& f) {
  constexpr int N = 64 / LPH;
  if (g0 >= g1) return;
  const int sub = (int)(threadIdx.x & 63) / LPH;
  const auto load = [&](int g) {
    const int h = g * N + sub;
    return row_load(x + (h < heads ? h : heads - 1) * D, m);
  };
  Row8 v = load(g0);
  for (int g = g0; g < g1; ++g) {
    const Row8 next = load(g + 1 < g1 ? g + 1 : g);
    f(g * N + sub, v);
    v = next;
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
    if constexpr (sizeof(R) == 8) {
      y[pair_a(PAIRS, i)] = __builtin_fma(a, c, -(b * s));
      y[pair_b(PAIRS, i)] = __builtin_fma(b, c, a * s);
    } else {
      y[pair_a(PAIRS, i)] = __builtin_fmaf(a, c, -(b * s));
      y[pair_b(PAIRS, i)] = __builtin_fmaf(b, c, a * s);
    }
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

// Norm (with a weight) and rotation of the lane's values: bf16 patterns of
// group 0 and group 1.  binary64 throughout: the result is the formula's
// rounded once (up to 2^-50 before the rounding), whatever the sum's order,
// so that a key lands on the formula's side of the 4-bit borders behind it.
// gfx950 runs binary64 fused multiply-adds at the rate of unpacked binary32
// ones, so the pass stays bound by memory.
template <int LPH, int PAIRS>
__device__ __forceinline__ Row8 row_norm_rope(const Row8& in, const RowMap<LPH>& m, bool norm,
                                              const Row8& weight, double eps, double inv_d,
                                              const RowAngles& g) {
  float x[8];
  in.or_zero(m.active).unpack(x);
  double y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = (double)x[i];
  if (norm) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fma(y[i], y[i], ss);
    const double r = rsqrt64(row_sum<LPH>(ss) * inv_d + eps);
    weight.unpack(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] * r * (double)x[i];
  }
  if (m.rotated) row_rotate<PAIRS, 1>(y, g);
  return Row8{make_uint2(bf16_pair((float)y[0], (float)y[1]), bf16_pair((float)y[2], (float)y[3])),
              make_uint2(bf16_pair((float)y[4], (float)y[5]), bf16_pair((float)y[6], (float)y[7]))};
}

// The lane's part of a weight; zeros without one.
template <int LPH>
__device__ __forceinline__ Row8 weight_load(const uint16_t* w, const RowMap<LPH>& m) {
  return w ? row_load(w, m) : Row8{make_uint2(0, 0), make_uint2(0, 0)};
}

// A wavefront takes one token and a run of its head groups (64 / LPH heads
// each; the groups of queries, then of keys, then of values, so that a group
// is of one kind).  Its angles and weights are loaded once and stay in
// registers.
struct RowGrid {
  int q_groups, k_groups, v_groups;
  int per_wave;  // groups a wavefront takes
  int parts;     // wavefronts a token takes
  int64_t waves;
};
// Enough wavefronts to fill the card (256 CUs x 32) come first, long runs
// second: a token is cut up only where there are few tokens.
inline RowGrid row_grid_of(int64_t tokens, int lph, int q_heads, int k_heads, int v_heads) {
  const int n = 64 / lph;
  RowGrid g = {(q_heads + n - 1) / n, (k_heads + n - 1) / n, (v_heads + n - 1) / n, 1, 1, 0};
  const int groups = g.q_groups + g.k_groups + g.v_groups;
  const int64_t want = (int64_t)device_cu_count() * 32;
  int64_t parts = tokens > 0 ? (want + tokens - 1) / tokens : 1;
  parts = parts < groups ? parts : groups;
  g.per_wave = (int)((groups + parts - 1) / parts);
  g.parts = (groups + g.per_wave - 1) / g.per_wave;
  g.waves = tokens * g.parts;
  return g;
}
inline unsigned row_blocks(const RowGrid& g) {
  // threads of one launch stay in 32 bits; more work makes the workgroups walk
  const int64_t n = (g.waves + 3) / 4, cap = (int64_t)1 << 23;
  return (unsigned)(n < cap ? n : cap);
}

struct RowTask {
  int64_t token;
  int first, last;  // groups [first, last)
};
// A token is cut up only where there are fewer tokens than wavefronts on the
// card, so the division is one of 32 bits.
__device__ __forceinline__ RowTask row_task(int64_t wave, const RowGrid& g) {
  const uint32_t cut = g.parts == 1 ? 0u : (uint32_t)wave / (uint32_t)g.parts;
  const int part = g.parts == 1 ? 0 : (int)((uint32_t)wave - cut * (uint32_t)g.parts);
  const int groups = g.q_groups + g.k_groups + g.v_groups;
  const int first = part * g.per_wave, end = first + g.per_wave;
  return RowTask{g.parts == 1 ? wave : (int64_t)cut, first, end < groups ? end : groups};
}

// The part of a task's groups that lies in [from, from + n), counted from `from`.
struct RowPart {
  int g0, g1;
};
__device__ __forceinline__ RowPart part_of(const RowTask& t, int from, int n) {
  const int a = t.first - from, b = t.last - from;
  return RowPart{a > 0 ? a : 0, b < n ? b : n};
}

inline int lanes_per_head(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

}  // namespace nvfp4
