// kv_cache.hip -- writing a step's keys and values into the paged NVFP4 cache
// (with the norm and rotation of queries and keys in the same pass), and
// reading them back.
#include "qk_row.hpp"

namespace nvfp4 {

// Value of lane i of the quad (a compile-time i).
template <int I>
__device__ __forceinline__ float quad_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), I * 0x55, 0xF, 0xF, false));
}

// Encodes the 16-value blocks that a quad of lanes holds, one per group (x[0
// .. 3] group 0, x[4 .. 7] group 1): bits 0 .. 15 of codes[g] are the lane's
// four nibbles, scale[g] the block's byte.  The steps are those of
// nvfp4_quantize in their order (fmaf chain per four values, then (P0 + P1) +
// (P2 + P3): lane pairs add in that order).  The effective scale and its
// correctly rounded reciprocal of the block's candidates (two groups x max->6,
// max->4) are computed once a quad, one candidate a lane.  All lanes of the
// quad call it.
template <int SELECT>
__device__ __forceinline__ void quad_quantize(const float (&x)[8], const TensorScale& ts,
                                              uint32_t (&codes)[2], uint32_t (&scale)[2]) {
  uint32_t cand[2];
  bool nan[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float* v = x + 4 * g;
    float a = __builtin_elementwise_maximum(
        __builtin_elementwise_maximum(__builtin_fabsf(v[0]), __builtin_fabsf(v[1])),
        __builtin_elementwise_maximum(__builtin_fabsf(v[2]), __builtin_fabsf(v[3])));
    a = __builtin_elementwise_maximum(a, __uint_as_float(xor1_u32(__float_as_uint(a))));
    a = __builtin_elementwise_maximum(a, __uint_as_float(xor2_u32(__float_as_uint(a))));
    nan[g] = ts.nan || a != a;
    cand[g] = SELECT == SELECT_6 ? e4m3_encode_pair(a * ts.k6, 0.0f) : e4m3_encode_pair(a * ts.k6, a * ts.k4);
  }
  // lane i of the quad: group i / 2, max->6 (i even) or max->4
  const uint32_t pair = (threadIdx.x & 2) ? cand[1] : cand[0];
  const f32x2 e = scale_entry(FMT_E4M3, (threadIdx.x & 1) ? pair >> 8 : pair & 0xFFu, ts.alpha);
  auto block = [&](int g, f32x2 t6, f32x2 t4) {
    const float* v = x + 4 * g;
    auto encode = [&](const f32x2& t) {
      uint32_t w = NVFP4_CVT_PK_FP4(0u, v[0] * t[1], v[1] * t[1], 0);
      return NVFP4_CVT_PK_FP4(w, v[2] * t[1], v[3] * t[1], 1) & 0xFFFFu;
    };
    const uint32_t w6 = encode(t6);
    if constexpr (SELECT == SELECT_6) {
      codes[g] = w6;
      scale[g] = cand[g] & 0xFFu;
    } else {
      const uint32_t w4 = encode(t4);
      auto error = [&](uint32_t w, float S) {
        const f32x2 q0 = NVFP4_DEC_PK_FP4(w, 0), q1 = NVFP4_DEC_PK_FP4(w, 1);
        float d = __builtin_fmaf(-q0[0], S, v[0]), p = __builtin_fmaf(d, d, 0.0f);
        d = __builtin_fmaf(-q0[1], S, v[1]); p = __builtin_fmaf(d, d, p);
        d = __builtin_fmaf(-q1[0], S, v[2]); p = __builtin_fmaf(d, d, p);
        d = __builtin_fmaf(-q1[1], S, v[3]); p = __builtin_fmaf(d, d, p);
        p = p + __uint_as_float(xor1_u32(__float_as_uint(p)));
        return p + __uint_as_float(xor2_u32(__float_as_uint(p)));
      };
      const bool four = error(w4, t4[0]) < error(w6, t6[0]);
      codes[g] = four ? w4 : w6;
      scale[g] = four ? cand[g] >> 8 : cand[g] & 0xFFu;
    }
    if (nan[g]) {
      codes[g] = 0;
      scale[g] = 0x7Fu;
    }
  };
  block(0, f32x2{quad_lane<0>(e[0]), quad_lane<0>(e[1])}, f32x2{quad_lane<1>(e[0]), quad_lane<1>(e[1])});
  block(1, f32x2{quad_lane<2>(e[0]), quad_lane<2>(e[1])}, f32x2{quad_lane<3>(e[0]), quad_lane<3>(e[1])});
}

// Heads of a token: queries (normed, rotated, returned), keys (normed,
// rotated, quantized), values (quantized).  A value's bytes lie eight tokens
// apart, so its stores are single bytes that meet in the L2.  Bound by the
// vector units (81 % busy with 4/6, where max->6 and max->4 are both encoded
// and compared, 74 with max->6) and by bytes: 8192 tokens of 32 + 8 + 8 heads of
// 128 move 187 MB in 44 us, in a loop of launches in 42.4 and, with max->6,
// 41.1; the keys' and values' part alone takes 23.0 and 20.0.  64 single tokens
// 5.0 us.
template <int LPH, int PAIRS, int SELECT>
__global__ void __launch_bounds__(kRowThreads)
kv_append_kernel(nvfp4_kv_append_args p, RowGrid grid) {
  const nvfp4_qk_args& a = p.qk;
  const nvfp4_kv_cache& c = p.cache;
  const int D = a.head_dim, heads = a.k_heads;
  // the outer scales of the heads' keys and values, worked out once a workgroup
  extern __shared__ float4 outer[];  // [2][heads]: alpha, K6, K4, whether it is unusable
  for (int i = threadIdx.x; i < 2 * heads; i += kRowThreads) {
    const TensorScale ts = tensor_scale(i < heads ? c.k_amax[i] : c.v_amax[i - heads], c.global_fp8_max);
    outer[i] = make_float4(ts.alpha, ts.k6, ts.k4, ts.nan ? 1.0f : 0.0f);
  }
  __syncthreads();
  const RowMap<LPH> m(D, a.rot_dim, PAIRS);
  const Row8 wq = weight_load(a.q_weight, m), wk = weight_load(a.k_weight, m);
  const double inv_d = 1.0 / D, eps = a.eps;
  const int64_t slots_end = c.num_pages * c.page_size;
  const int shift = __builtin_ctz((unsigned)c.page_size);
  for (int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       wave < grid.waves; wave += (int64_t)gridDim.x * 4) {
    const RowTask t = row_task(wave, grid);
    const int64_t slot = p.slots[t.token];
    const bool stored = slot >= 0 && slot < slots_end;
    const RowAngles ang = row_angles(a, m, t.token);
    const RowPart pq = part_of(t, 0, grid.q_groups);
    row_walk(a.q + t.token * a.q_stride, a.q_heads, D, pq.g0, pq.g1, m, [&](int h, const Row8& v) {
      const Row8 y = row_norm_rope<LPH, PAIRS>(v, m, a.q_weight != nullptr, wq, eps, inv_d, ang);
      if (m.active && h < a.q_heads) row_store(a.q_out + t.token * a.q_out_stride + h * D, m, y);
    });
    if (!stored) continue;  // the wavefront together
    // where head 0 of the token lies; a head further is page_size tokens on
    // (below 2^28 bytes for all of them)
    const int64_t page_tokens = (slot >> shift) * heads << shift;
    const int off = (int)(slot & (c.page_size - 1));
    const int64_t kt = page_tokens + off, vt = page_tokens + (off & ~7);
    uint8_t* kc = c.k_codes + kt * (D / 2);
    uint8_t* ks = c.k_scales + kt * (D / 16);
    uint8_t* vc = c.v_codes + vt * (D / 2) + (off & 7);
    uint8_t* vs = c.v_scales + vt * (D / 16) + (off & 7);
    const auto quantize = [&](int h, const Row8& v, int kind, uint32_t (&codes)[2], uint32_t (&scale)[2]) {
      float x[8];
      v.unpack(x);
      const float4 o = outer[kind * heads + (h < heads ? h : heads - 1)];
      quad_quantize<SELECT>(x, TensorScale{o.x, o.y, o.z, o.w != 0.0f}, codes, scale);
    };
    const RowPart pk = part_of(t, grid.q_groups, grid.k_groups);
    row_walk(a.k + t.token * a.k_stride, heads, D, pk.g0, pk.g1, m, [&](int h, const Row8& v) {
      uint32_t codes[2], scale[2];
      quantize(h, row_norm_rope<LPH, PAIRS>(v, m, a.k_weight != nullptr, wk, eps, inv_d, ang), 0, codes, scale);
      if (!m.active || h >= heads) return;
      const uint32_t at = ((uint32_t)h << shift) * (uint32_t)(D / 2), sat = ((uint32_t)h << shift) * (uint32_t)(D / 16);
      *reinterpret_cast<uint16_t*>(kc + at + m.e0 / 2) = (uint16_t)codes[0];
      *reinterpret_cast<uint16_t*>(kc + at + m.e1 / 2) = (uint16_t)codes[1];
      if ((threadIdx.x & 3) == 0) {
        ks[sat + m.e0 / 16] = (uint8_t)scale[0];
        ks[sat + m.e1 / 16] = (uint8_t)scale[1];
      }
    });
    const RowPart pv = part_of(t, grid.q_groups + grid.k_groups, grid.v_groups);
    row_walk(p.v + t.token * p.v_stride, heads, D, pv.g0, pv.g1, m, [&](int h, const Row8& v) {
      uint32_t codes[2], scale[2];
      quantize(h, v.or_zero(m.active), 1, codes, scale);
      if (!m.active || h >= heads) return;
      const uint32_t at = ((uint32_t)h << shift) * (uint32_t)(D / 2), sat = ((uint32_t)h << shift) * (uint32_t)(D / 16);
      vc[at + 4 * m.e0] = (uint8_t)codes[0];
      vc[at + 4 * m.e0 + 8] = (uint8_t)(codes[0] >> 8);
      vc[at + 4 * m.e1] = (uint8_t)codes[1];
      vc[at + 4 * m.e1 + 8] = (uint8_t)(codes[1] >> 8);
      if ((threadIdx.x & 3) == 0) {
        vs[sat + m.e0 / 2] = (uint8_t)scale[0];
        vs[sat + m.e1 / 2] = (uint8_t)scale[1];
      }
    });
  }
}

template <int LPH, int PAIRS>
static hipError_t launch_append2(const nvfp4_kv_append_args& a, hipStream_t s) {
  const RowGrid g = row_grid_of(a.qk.tokens, LPH, a.qk.q_heads, a.qk.k_heads, a.qk.k_heads);
  const size_t lds = 2 * (size_t)a.qk.k_heads * sizeof(float4);  // at most 32 KB
  if (a.select == NVFP4_SELECT_6)
    hipLaunchKernelGGL((kv_append_kernel<LPH, PAIRS, SELECT_6>), dim3(row_blocks(g)), dim3(kRowThreads),
                       lds, s, a, g);
  else
    hipLaunchKernelGGL((kv_append_kernel<LPH, PAIRS, SELECT_4OVER6>), dim3(row_blocks(g)),
                       dim3(kRowThreads), lds, s, a, g);
  return hipGetLastError();
}

template <int LPH>
static hipError_t launch_append(const nvfp4_kv_append_args& a, hipStream_t s) {
  return a.qk.pairs == NVFP4_PAIRS_HALVES ? launch_append2<LPH, NVFP4_PAIRS_HALVES>(a, s)
                                          : launch_append2<LPH, NVFP4_PAIRS_NEIGHBOURS>(a, s);
}

hipError_t launch_kv_append(const nvfp4_kv_append_args& a, hipStream_t s) {
  switch (lanes_per_head(a.qk.head_dim)) {
    case 8: return launch_append<8>(a, s);
    case 16: return launch_append<16>(a, s);
    default: return launch_append<32>(a, s);
  }
}

// ---------------------------------------------------------------- read
// 8192 tokens of 8 heads of 128 keys and values (51 MB, 34 of them written):
// 12.4 us; 64 tokens 3.6 us.
template <int LPH>
__global__ void __launch_bounds__(kRowThreads)
kv_read_kernel(nvfp4_kv_cache c, const int64_t* slots, RowGrid grid, uint16_t* k_out, uint16_t* v_out) {
  constexpr int N = 64 / LPH;
  const int D = c.head_dim, sub = (int)(threadIdx.x & 63) / LPH;
  extern __shared__ float alphas[];  // [2][heads], worked out once a workgroup
  for (int i = threadIdx.x; i < 2 * c.kv_heads; i += kRowThreads)
    alphas[i] = outer_alpha(i < c.kv_heads ? c.k_amax[i] : c.v_amax[i - c.kv_heads], c.global_fp8_max);
  __syncthreads();
  const RowMap<LPH> m(D, D, NVFP4_PAIRS_HALVES);
  const int64_t slots_end = c.num_pages * c.page_size;
  const int shift = __builtin_ctz((unsigned)c.page_size);
  for (int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       wave < grid.waves; wave += (int64_t)gridDim.x * 4) {
    const RowTask t = row_task(wave, grid);
    int64_t slot = slots[t.token];
    const bool there = slot >= 0 && slot < slots_end;
    slot = there ? slot : 0;  // page 0 is always there to read
#pragma unroll 2
    for (int g = t.first; g < t.last; ++g) {
      const bool isv = g >= grid.k_groups;
      const int h = (isv ? g - grid.k_groups : g) * N + sub;
      if (!m.active || h >= c.kv_heads) continue;
      uint32_t w0, w1, s0, s1;
      const KvAddr k = {(slot >> shift) * c.kv_heads + h, (int)(slot & (c.page_size - 1)), c.page_size, D};
      if (!isv) {
        const uint8_t* kc = c.k_codes + k.k_code();
        const uint8_t* ks = c.k_scales + k.k_scale();
        w0 = *reinterpret_cast<const uint16_t*>(kc + m.e0 / 2);
        w1 = *reinterpret_cast<const uint16_t*>(kc + m.e1 / 2);
        s0 = ks[m.e0 / 16];
        s1 = ks[m.e1 / 16];
      } else {
        const uint8_t* vc = c.v_codes + k.v_code();
        const uint8_t* vs = c.v_scales + k.v_scale();
        w0 = vc[8 * (m.e0 / 2)] | (uint32_t)vc[8 * (m.e0 / 2 + 1)] << 8;
        w1 = vc[8 * (m.e1 / 2)] | (uint32_t)vc[8 * (m.e1 / 2 + 1)] << 8;
        s0 = vs[8 * (m.e0 / 16)];
        s1 = vs[8 * (m.e1 / 16)];
      }
      const float alpha = alphas[isv ? c.kv_heads + h : h];
      // E2M1 x E4M3 is exact in binary32; times alpha rounds once
      const float f0 = decode_scale(FMT_E4M3, s0), f1 = decode_scale(FMT_E4M3, s1);
      const f32x2 a0 = NVFP4_DEC_PK_FP4(w0, 0), a1 = NVFP4_DEC_PK_FP4(w0, 1);
      const f32x2 b0 = NVFP4_DEC_PK_FP4(w1, 0), b1 = NVFP4_DEC_PK_FP4(w1, 1);
      Row8 y = {make_uint2(bf16_pair(a0[0] * f0 * alpha, a0[1] * f0 * alpha),
                           bf16_pair(a1[0] * f0 * alpha, a1[1] * f0 * alpha)),
                make_uint2(bf16_pair(b0[0] * f1 * alpha, b0[1] * f1 * alpha),
                           bf16_pair(b1[0] * f1 * alpha, b1[1] * f1 * alpha))};
      if (!there) y.a = y.b = make_uint2(0, 0);  // also under an unusable amax
      row_store((isv ? v_out : k_out) + (t.token * c.kv_heads + h) * D, m, y);
    }
  }
}

template <int LPH>
static hipError_t launch_read(const nvfp4_kv_cache& c, const int64_t* slots, int64_t tokens,
                              uint16_t* k_out, uint16_t* v_out, hipStream_t s) {
  const RowGrid g = row_grid_of(tokens, LPH, 0, k_out ? c.kv_heads : 0, v_out ? c.kv_heads : 0);
  const unsigned lds = 2 * (unsigned)c.kv_heads * sizeof(float);
  hipLaunchKernelGGL((kv_read_kernel<LPH>), dim3(row_blocks(g)), dim3(kRowThreads), lds, s, c, slots,
                     g, k_out, v_out);
  return hipGetLastError();
}

hipError_t launch_kv_read(const nvfp4_kv_cache& c, const int64_t* slots, int64_t tokens,
                          uint16_t* k_out, uint16_t* v_out, hipStream_t s) {
  switch (lanes_per_head(c.head_dim)) {
    case 8: return launch_read<8>(c, slots, tokens, k_out, v_out, s);
    case 16: return launch_read<16>(c, slots, tokens, k_out, v_out, s);
    default: return launch_read<32>(c, slots, tokens, k_out, v_out, s);
  }
}

}  // namespace nvfp4
