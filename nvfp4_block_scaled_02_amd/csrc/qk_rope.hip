// qk_rope.hip -- RMS norm of each query and key head with the position
// rotation in the same pass, and its gradient.

#include "qk_row.hpp"

namespace nvfp4 {

// A lane reads 16 bytes of a head and writes 16; the next group's bytes are in
// flight while one is computed.  Each value is read and written once: 8192
// tokens of 32 + 8 heads of 128 values move 172 MB in 30 us (5.7 TB/s, partly
// from the last-level cache; a copy of the query view alone by the library
// takes 28).  The arithmetic in 64 bits keeps the vector units 77 % busy.
template <int LPH, int PAIRS>
__global__ void __launch_bounds__(kRowThreads)
qk_norm_rope_kernel(nvfp4_qk_args a, RowGrid grid) {
  const int D = a.head_dim;
  const RowMap<LPH> m(D, a.rot_dim, PAIRS);
  const Row8 wq = weight_load(a.q_weight, m), wk = weight_load(a.k_weight, m);
  const double inv_d = 1.0 / D, eps = a.eps;
  for (int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       wave < grid.waves; wave += (int64_t)gridDim.x * 4) {
    const RowTask t = row_task(wave, grid);
    const RowAngles ang = row_angles(a, m, t.token);
    const auto side = [&](const uint16_t* x, uint16_t* out, int heads, const RowPart& p, bool norm, const Row8& w) {
      row_walk(x, heads, D, p.g0, p.g1, m, [&](int h, const Row8& v) {
        const Row8 y = row_norm_rope<LPH, PAIRS>(v, m, norm, w, eps, inv_d, ang);
        if (m.active && h < heads) row_store(out + h * D, m, y);
      });
    };
    side(a.q + t.token * a.q_stride, a.q_out + t.token * a.q_out_stride, a.q_heads,
         part_of(t, 0, grid.q_groups), a.q_weight != nullptr, wq);
    side(a.k + t.token * a.k_stride, a.k_out + t.token * a.k_out_stride, a.k_heads,
         part_of(t, grid.q_groups, grid.k_groups), a.k_weight != nullptr, wk);
  }
}

template <int LPH>
static hipError_t launch_fwd(const nvfp4_qk_args& a, hipStream_t s) {
  const RowGrid g = row_grid_of(a.tokens, LPH, a.q_heads, a.k_heads, 0);
  if (a.pairs == NVFP4_PAIRS_HALVES)
    hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, NVFP4_PAIRS_HALVES>), dim3(row_blocks(g)),
                       dim3(kRowThreads), 0, s, a, g);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, NVFP4_PAIRS_NEIGHBOURS>), dim3(row_blocks(g)),
                       dim3(kRowThreads), 0, s, a, g);
  return hipGetLastError();
}

hipError_t launch_qk_norm_rope(const nvfp4_qk_args& a, hipStream_t s) {
  switch (lanes_per_head(a.head_dim)) {
    case 4: return launch_fwd<4>(a, s);
    case 8: return launch_fwd<8>(a, s);
    case 16: return launch_fwd<16>(a, s);
    default: return launch_fwd<32>(a, s);
  }
}

// ---------------------------------------------------------------- gradient
// Workspace: arrival counters of the teams and of the whole launch (each on a
// 128-byte line), then one partial (dq_weight, dk_weight) of D doubles each
// per workgroup and one per team.
constexpr int kBwdGroups = 1024;
constexpr int kBwdTeams = 32;
constexpr size_t kBwdHead = 128 * (kBwdTeams + 1);

size_t qk_norm_rope_bwd_workspace(int head_dim) {
  return kBwdHead + (size_t)(kBwdGroups + kBwdTeams) * 2 * head_dim * sizeof(double);
}

struct BwdArgs {
  nvfp4_qk_args a;
  const uint16_t *gq, *gk;
  int64_t gq_stride, gk_stride;
  float *dqw, *dkw;
  uint8_t* ws;
  RowGrid grid;
};

// One head's gradient in the lane; g n is added to dw.  A lane that is not on
// holds zeros, and its r is 0 (not 0^-1/2, where eps is 0): it adds nothing.
template <int LPH, int PAIRS>
__device__ __forceinline__ Row8 row_bwd(const Row8& in, const Row8& grad, const RowMap<LPH>& m, bool on, bool norm,
                                        const Row8& weight, float eps, float inv_d,
                                        const RowAngles& ang, float (&dw)[8]) {
  float g[8];
  grad.unpack(g);
  if (m.rotated) row_rotate<PAIRS, -1>(g, ang);
  if (norm) {
    float x[8], w[8], ss = 0.0f;
    in.unpack(x);
    weight.unpack(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(x[i], x[i], ss);
    const float v = row_sum<LPH>(ss) * inv_d + eps;
    float r = on ? 1.0f / __builtin_sqrtf(v) : 0.0f;
    // r = r 2^up of a head whose squares leave binary32 (a bf16 value's do
    // beyond 2^64 and below 2^-75): from binary64, as in the forward call
    int up = 0;
    const bool far = on && !(v > 0x1p-100f && v < 0x1p100f), any_far = __any(far);
    if (any_far) {
      double ss64 = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss64 = __builtin_fma((double)x[i], (double)x[i], ss64);
      const double r64 = rsqrt64(row_sum<LPH>(ss64) * (double)inv_d + (double)eps);
      if (far) {
        r = (float)__builtin_amdgcn_frexp_mant(r64);
        up = __builtin_amdgcn_frexp_exp(r64);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_ldexpf(x[i], up);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= r;  // n
      dw[i] = __builtin_fmaf(g[i], x[i], dw[i]);
      g[i] *= w[i];
      dot = __builtin_fmaf(g[i], x[i], dot);
    }
    dot = row_sum<LPH>(dot) * inv_d;
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = r * __builtin_fmaf(-x[i], dot, g[i]);
    if (any_far) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = __builtin_ldexpf(g[i], up);
    }
  }
  return Row8{make_uint2(bf16_pair(g[0], g[1]), bf16_pair(g[2], g[3])),
              make_uint2(bf16_pair(g[4], g[5]), bf16_pair(g[6], g[7]))};
}

__device__ __forceinline__ void put64(double* p, double v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get64(const double* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Sum of slots first, first + step, ... < last of n doubles each, in the
// threads e < n, in order (eight loads in flight).
__device__ __forceinline__ double sum_slots(const double* slots, int n, int e, int first, int last, int step) {
  double v = 0.0;
  int i = first;
  for (; i + 7 * step < last; i += 8 * step) {
    double x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = get64(slots + (size_t)(i + k * step) * n + e);
#pragma unroll
    for (int k = 0; k < 8; ++k) v += x[k];
  }
  for (; i < last; i += step) v += get64(slots + (size_t)i * n + e);
  return v;
}

// A wavefront walks tokens; over one token's heads the sums of dw stay in
// binary32 (at most 1024 terms of one lane's column), over tokens in
// binary64.  A workgroup's sums go to its slot; the last workgroup of each of
// 32 teams adds the team's slots in order, the last team the teams' sums: no
// atomic addition, the same bits on every run.  Slots are written and read at
// the level that the whole GPU sees, so no cache is written back.
// Bound by its bytes: 261 MB (254 without the partial sums) in 51 us at 8192
// tokens of 32 + 8 heads of 128, 5.1 TB/s with the vector units 75 % busy;
// 1023 tokens of 12 + 4 heads of 64 take 12.6 us, most of it latency: of the
// loads, and of the two levels that join up to 1024 workgroups' sums.
template <int LPH, int PAIRS>
__global__ void __launch_bounds__(kRowThreads, 4)
qk_norm_rope_bwd_kernel(BwdArgs b) {
  constexpr int N = 64 / LPH;
  __shared__ double part[4][2 * 256];
  __shared__ bool last;
  const nvfp4_qk_args& a = b.a;
  const RowGrid& grid = b.grid;
  const int D = a.head_dim, sub = (int)(threadIdx.x & 63) / LPH, wv = threadIdx.x >> 6;
  const RowMap<LPH> m(D, a.rot_dim, PAIRS);
  const float inv_d = 1.0f / (float)D, eps = a.eps;
  const bool sums = b.dqw || b.dkw;
  // all of the wavefront's query heads, then its key heads: one set of sums in
  // registers at a time
  const auto side = [&](const uint16_t* x0, int64_t xs, const uint16_t* y0, int64_t ys, uint16_t* d0, int64_t ds,
                        int heads, int kind, const uint16_t* w, int column0) {
    const bool norm = w != nullptr;
    const Row8 weight = weight_load(w, m);
    double sum[8] = {};
    for (int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(wv); wave < grid.waves;
         wave += (int64_t)gridDim.x * 4) {
      const RowTask t = row_task(wave, grid);
      const RowPart p = kind == 0 ? part_of(t, 0, grid.q_groups) : part_of(t, grid.q_groups, grid.k_groups);
      if (p.g0 >= p.g1) continue;
      const RowAngles ang = row_angles(a, m, t.token);
      const uint16_t* x = x0 + t.token * xs;
      const uint16_t* y = y0 + t.token * ys;
      uint16_t* d = d0 + t.token * ds;
      const auto head_of = [&](int g) { return g * N + sub; };
      const auto load = [&](const uint16_t* s, int g) {
        const int h = head_of(g);
        return row_load(s + (h < heads ? h : heads - 1) * D, m);
      };
      float dw[8] = {};
      Row8 xv = load(x, p.g0), yv = load(y, p.g0);
      for (int g = p.g0; g < p.g1; ++g) {
        const int gn = g + 1 < p.g1 ? g + 1 : g;
        const Row8 xn = load(x, gn), yn = load(y, gn);
        // lanes without values, and heads past the last one, add nothing
        const bool on = m.active && head_of(g) < heads;
        const Row8 r = row_bwd<LPH, PAIRS>(xv.or_zero(on), yv.or_zero(on), m, on, norm, weight, eps, inv_d, ang,
                                               dw);
        if (on) row_store(d + head_of(g) * D, m, r);
        xv = xn;
        yv = yn;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += dw[i];
    }
    if (!sums) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      for (int k = LPH; k < 64; k <<= 1) sum[i] += __shfl_xor(sum[i], k);
    if ((threadIdx.x & 63) < LPH && m.active) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part[wv][column0 + m.e0 + i] = sum[i];
        part[wv][column0 + m.e1 + i] = sum[4 + i];
      }
    }
  };
  side(a.q, a.q_stride, b.gq, b.gq_stride, a.q_out, a.q_out_stride, a.q_heads, 0, a.q_weight, 0);
  side(a.k, a.k_stride, b.gk, b.gk_stride, a.k_out, a.k_out_stride, a.k_heads, 1, a.k_weight, D);
  if (!sums) return;
  __syncthreads();
  const int n = 2 * D, G = gridDim.x;
  double* slots = reinterpret_cast<double*>(b.ws + kBwdHead);
  double* team_slots = slots + (size_t)kBwdGroups * n;
  for (int e = threadIdx.x; e < n; e += kRowThreads)
    put64(slots + (size_t)blockIdx.x * n + e, (part[0][e] + part[1][e]) + (part[2][e] + part[3][e]));
  // arrive once the slot has reached the level that all see
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  const int teams = G < kBwdTeams ? G : kBwdTeams, team = blockIdx.x % teams;
  const uint32_t members = (uint32_t)((G - team + teams - 1) / teams);
  if (threadIdx.x == 0) {
    uint32_t* c = reinterpret_cast<uint32_t*>(b.ws + 128 * (1 + team));
    last = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == members - 1;
    if (last) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  for (int e = threadIdx.x; e < n; e += kRowThreads)
    put64(team_slots + (size_t)team * n + e, sum_slots(slots, n, e, team, G, teams));
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t* c = reinterpret_cast<uint32_t*>(b.ws);
    last = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)teams - 1;
    if (last) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  for (int e = threadIdx.x; e < n; e += kRowThreads) {
    float* out = e < D ? b.dqw : b.dkw;
    if (out) out[e < D ? e : e - D] = (float)sum_slots(team_slots, n, e, 0, teams, 1);
  }
}

template <int LPH>
static hipError_t launch_bwd(BwdArgs b, hipStream_t s) {
  b.grid = row_grid_of(b.a.tokens, LPH, b.a.q_heads, b.a.k_heads, 0);
  // with no tokens one workgroup writes the zero gradients of the weights
  int64_t blocks = (b.grid.waves + 3) / 4;
  blocks = blocks < 1 ? 1 : blocks < kBwdGroups ? blocks : kBwdGroups;
  if (b.a.pairs == NVFP4_PAIRS_HALVES)
    hipLaunchKernelGGL((qk_norm_rope_bwd_kernel<LPH, NVFP4_PAIRS_HALVES>), dim3((unsigned)blocks),
                       dim3(kRowThreads), 0, s, b);
  else
    hipLaunchKernelGGL((qk_norm_rope_bwd_kernel<LPH, NVFP4_PAIRS_NEIGHBOURS>), dim3((unsigned)blocks),
                       dim3(kRowThreads), 0, s, b);
  return hipGetLastError();
}

hipError_t launch_qk_norm_rope_bwd(const nvfp4_qk_args& a, const uint16_t* gq, int64_t gq_stride,
                                   const uint16_t* gk, int64_t gk_stride, float* dqw, float* dkw,
                                   uint8_t* ws, hipStream_t s) {
  BwdArgs b = {};
  b.a = a;
  b.gq = gq; b.gk = gk; b.gq_stride = gq_stride; b.gk_stride = gk_stride;
  b.dqw = dqw; b.dkw = dkw; b.ws = ws;
  switch (lanes_per_head(a.head_dim)) {
    case 4: return launch_bwd<4>(b, s);
    case 8: return launch_bwd<8>(b, s);
    case 16: return launch_bwd<16>(b, s);
    default: return launch_bwd<32>(b, s);
  }
}

}  // namespace nvfp4
