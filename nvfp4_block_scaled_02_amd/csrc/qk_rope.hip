// qk_rope.hip -- RMS norm of each query and key head with the position
// rotation in the same pass, and its gradient.

#include "qk_row.hpp"

namespace nvfp4 {

// One wavefront per 64 / LPH heads of a token: a lane reads 16 bytes and
// writes 16.
template <int LPH, int PAIRS>
__global__ void __launch_bounds__(kRowThreads)
qk_norm_rope_kernel(nvfp4_qk_args a, int64_t tasks, int per_token) {
  const RowMap<LPH> m(a.head_dim, a.rot_dim, PAIRS);
  const int heads = a.q_heads + a.k_heads;
  const double inv_d = 1.0 / a.head_dim;
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < tasks; w += (int64_t)gridDim.x * 4) {
    const RowTask t = row_task<LPH>(w, per_token);
    const bool on = t.head < heads;
    const bool isq = t.head < a.q_heads;
    const int h = isq ? t.head : t.head - a.q_heads;
    RowMap<LPH> mm = m;
    mm.active = m.active && on;
    const RowAngles g = row_angles(a, mm, t.token);
    float x[8];
    row_load(isq ? a.q + t.token * a.q_stride + (int64_t)h * a.head_dim
                 : a.k + t.token * a.k_stride + (int64_t)h * a.head_dim, mm, x);
    uint2 o0, o1;
    row_norm_rope<LPH, PAIRS>(x, mm, isq ? a.q_weight : a.k_weight, a.eps, inv_d, g, o0, o1);
    row_store(isq ? a.q_out + t.token * a.q_out_stride + (int64_t)h * a.head_dim
                  : a.k_out + t.token * a.k_out_stride + (int64_t)h * a.head_dim, mm, o0, o1);
  }
}

template <int LPH>
static hipError_t launch_fwd(const nvfp4_qk_args& a, hipStream_t s) {
  const int per_token = (a.q_heads + a.k_heads + 64 / LPH - 1) / (64 / LPH);
  const int64_t tasks = a.tokens * per_token;
  if (a.pairs == NVFP4_PAIRS_HALVES)
    hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, NVFP4_PAIRS_HALVES>), dim3(row_grid(tasks)),
                       dim3(kRowThreads), 0, s, a, tasks, per_token);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<LPH, NVFP4_PAIRS_NEIGHBOURS>), dim3(row_grid(tasks)),
                       dim3(kRowThreads), 0, s, a, tasks, per_token);
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
// Workspace: a counter, then one partial dw of D doubles per workgroup.
constexpr int kBwdGroups = 1024;
constexpr size_t kBwdHead = 256;

size_t qk_norm_rope_bwd_workspace(int head_dim) {
  return kBwdHead + (size_t)kBwdGroups * head_dim * sizeof(double);
}

struct BwdArgs {
  nvfp4_qk_args a;
  const uint16_t *gq, *gk;
  int64_t gq_stride, gk_stride;
  float *dqw, *dkw;
  uint8_t* ws;
  int64_t q_tasks, k_tasks;
  int q_per_token, k_per_token;
  int q_groups, groups;  // workgroups [0, q_groups) take queries, the rest keys
};

// Each workgroup takes query heads or key heads only, so that a lane keeps
// one set of dw sums, in binary64, over all its rows; a workgroup's sums go
// to its slot of the workspace and the last workgroup adds the slots in
// order.
template <int LPH, int PAIRS>
__global__ void __launch_bounds__(kRowThreads)
qk_norm_rope_bwd_kernel(BwdArgs b) {
  __shared__ double part[4][256];
  __shared__ bool last;
  const nvfp4_qk_args& a = b.a;
  const int D = a.head_dim;
  const RowMap<LPH> m(D, a.rot_dim, PAIRS);
  const bool isq = (int)blockIdx.x < b.q_groups;
  const int group = isq ? blockIdx.x : blockIdx.x - b.q_groups;
  const int groups = isq ? b.q_groups : b.groups - b.q_groups;
  const int64_t tasks = isq ? b.q_tasks : b.k_tasks;
  const int per_token = isq ? b.q_per_token : b.k_per_token;
  const int heads = isq ? a.q_heads : a.k_heads;
  const uint16_t* x = isq ? a.q : a.k;
  const uint16_t* gy = isq ? b.gq : b.gk;
  uint16_t* dx = isq ? a.q_out : a.k_out;
  const int64_t xs = isq ? a.q_stride : a.k_stride, gs = isq ? b.gq_stride : b.gk_stride;
  const int64_t ds = isq ? a.q_out_stride : a.k_out_stride;
  const uint16_t* w = isq ? a.q_weight : a.k_weight;
  const float inv_d = 1.0f / (float)D, eps = a.eps;
  float wf[8];
  if (w) row_load(w, m, wf);
  double dw[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int64_t t0 = (int64_t)group * 4 + (threadIdx.x >> 6); t0 < tasks; t0 += (int64_t)groups * 4) {
    const RowTask t = row_task<LPH>(t0, per_token);
    RowMap<LPH> mm = m;
    mm.active = m.active && t.head < heads;
    const RowAngles g = row_angles(a, mm, t.token);
    float xv[8], gv[8];
    row_load(x + t.token * xs + (int64_t)t.head * D, mm, xv);
    row_load(gy + t.token * gs + (int64_t)t.head * D, mm, gv);
    if (mm.rotated) row_rotate<PAIRS, -1>(gv, g);
    if (w) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(xv[i], xv[i], ss);
      const float v = row_sum<LPH>(ss) * inv_d + eps;
      const float r = __builtin_isinf(v) ? 0.0f : 1.0f / __builtin_sqrtf(v);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xv[i] *= r;  // n
        if (mm.active) dw[i] += (double)(gv[i] * xv[i]);
        gv[i] *= wf[i];
        dot = __builtin_fmaf(gv[i], xv[i], dot);
      }
      dot = row_sum<LPH>(dot) * inv_d;
#pragma unroll
      for (int i = 0; i < 8; ++i) gv[i] = r * __builtin_fmaf(-xv[i], dot, gv[i]);
    }
    row_store(dx + t.token * ds + (int64_t)t.head * D, mm,
              make_uint2(bf16_pair(gv[0], gv[1]), bf16_pair(gv[2], gv[3])),
              make_uint2(bf16_pair(gv[4], gv[5]), bf16_pair(gv[6], gv[7])));
  }
  if (!b.dqw && !b.dkw) return;
  // the wavefront's heads, then the workgroup's wavefronts
#pragma unroll
  for (int i = 0; i < 8; ++i)
    for (int d = LPH; d < 64; d <<= 1) dw[i] += __shfl_xor(dw[i], d);
  if ((threadIdx.x & 63) < LPH && m.active) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      part[threadIdx.x >> 6][m.e0 + i] = dw[i];
      part[threadIdx.x >> 6][m.e1 + i] = dw[4 + i];
    }
  }
  __syncthreads();
  double* slots = reinterpret_cast<double*>(b.ws + kBwdHead);
  uint32_t* counter = reinterpret_cast<uint32_t*>(b.ws);
  if ((int)threadIdx.x < D) {
    const int e = threadIdx.x;
    const double v = (part[0][e] + part[1][e]) + (part[2][e] + part[3][e]);
    __hip_atomic_store(&slots[(size_t)blockIdx.x * D + e], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // the slot has reached the coherent level before the workgroup arrives
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           (uint32_t)b.groups - 1;
  __syncthreads();
  if (!last) return;
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if ((int)threadIdx.x < D) {
    for (int kind = 0; kind < 2; ++kind) {
      float* out = kind == 0 ? b.dqw : b.dkw;
      if (!out) continue;
      double v = 0.0;
      for (int i = kind == 0 ? 0 : b.q_groups; i < (kind == 0 ? b.q_groups : b.groups); ++i)
        v += __hip_atomic_load(&slots[(size_t)i * D + threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      out[threadIdx.x] = (float)v;
    }
  }
}

template <int LPH>
static hipError_t launch_bwd(BwdArgs b, hipStream_t s) {
  const int per = 64 / LPH;
  b.q_per_token = (b.a.q_heads + per - 1) / per;
  b.k_per_token = (b.a.k_heads + per - 1) / per;
  b.q_tasks = b.a.tokens * b.q_per_token;
  b.k_tasks = b.a.tokens * b.k_per_token;
  // workgroups in proportion to the tasks, at least one for each side that
  // has heads, at most the workspace's slots
  auto wgs = [](int64_t tasks, int64_t cap) {
    const int64_t g = (tasks + 3) / 4;
    return (int)(g < cap ? g : cap);
  };
  const int64_t all = b.q_tasks + b.k_tasks;
  int64_t qcap = all ? (int64_t)((double)kBwdGroups * (double)b.q_tasks / (double)all) : 0;
  qcap = qcap < 1 ? 1 : qcap > kBwdGroups - 1 ? kBwdGroups - 1 : qcap;
  b.q_groups = b.a.q_heads ? (b.q_tasks ? wgs(b.q_tasks, qcap) : 1) : 0;
  b.groups = b.q_groups + (b.a.k_heads ? (b.k_tasks ? wgs(b.k_tasks, kBwdGroups - qcap) : 1) : 0);
  if (b.a.pairs == NVFP4_PAIRS_HALVES)
    hipLaunchKernelGGL((qk_norm_rope_bwd_kernel<LPH, NVFP4_PAIRS_HALVES>), dim3((unsigned)b.groups),
                       dim3(kRowThreads), 0, s, b);
  else
    hipLaunchKernelGGL((qk_norm_rope_bwd_kernel<LPH, NVFP4_PAIRS_NEIGHBOURS>),
                       dim3((unsigned)b.groups), dim3(kRowThreads), 0, s, b);
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
